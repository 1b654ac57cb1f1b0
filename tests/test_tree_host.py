"""Host-side checks of the operators around a tree of drafted tokens that need no GPU: refusals come
before any device work, and tensors or a stream of another device never reach the library."""
import ctypes

import pytest

from sparse_attention_lightning_indexer_gb300 import build, ds4idx

from .test_devices_host import BF16, F32, I32, I64, U8, Tensor, lib as devices  # noqa: F401
from .test_devices_host import test_one_device_and_the_current_one as one_device
from . import test_devices_host

P = 1 << 20          # an aligned address that no call may touch
BIG = (1 << 63) - 1


@pytest.fixture(scope="module")
def library():
    build.build()
    return ds4idx.load()


def test_latents_fp8_refusals(library):
    w = lambda x=P, dt=0, n=4, slots=None, off=0, c=P, s=P, R=8: (  # noqa: E731
        library.ds4idx_quantize_latents_fp8(x, dt, n, slots, off, c, s, R, None))
    for bad in (dict(x=None), dict(x=P + 8), dict(dt=1), dict(n=-1), dict(slots=P + 4), dict(off=5),
                dict(off=-1), dict(off=BIG), dict(c=None), dict(c=P + 16), dict(R=-1), dict(s=None),
                dict(s=P + 2)):
        assert w(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert w(n=0) == ds4idx.OK
    r = lambda c=P, s=P, R=8, rows=None, start=0, n=4, out=P, dt=0: (  # noqa: E731
        library.ds4idx_read_latents_fp8(c, s, R, rows, start, n, out, dt, None))
    for bad in (dict(c=None), dict(c=P + 16), dict(s=None), dict(s=P + 1), dict(rows=P + 4),
                dict(start=5), dict(start=-1), dict(start=BIG), dict(n=-1), dict(out=None),
                dict(out=P + 8), dict(dt=1)):
        assert r(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert r(n=0) == ds4idx.OK


def _where(**kw):
    w = ds4idx.Placement()
    for k, v in kw.items():
        setattr(w, k, v)
    return ctypes.addressof(w), w


def test_tree_attention_refusals(library):
    def call(q=P, fmt=1, cache=P, scale=P, R=100, lens=P, mask=P, where=None, B=2, N=4, H=16, dqk=576,
             dv=512, most=64, sm=1.0, out=P, lse=P, ws=None, ws_bytes=0):
        return library.ds4idx_tree_attention(q, fmt, cache, scale, R, lens, mask, where, B, N, H, dqk,
                                             dv, most, sm, out, lse, ws, ws_bytes, None)
    for bad in (dict(q=None), dict(q=P + 8), dict(fmt=-1), dict(fmt=3), dict(fmt=0), dict(fmt=2),
                dict(scale=None), dict(scale=P + 2), dict(cache=None), dict(cache=P + 16), dict(R=0),
                dict(R=1 << 31), dict(lens=None), dict(lens=P + 2), dict(mask=None), dict(mask=P + 4),
                dict(B=-1), dict(B=1 << 30), dict(N=0), dict(N=65), dict(H=0), dict(H=129),
                dict(most=-1), dict(most=1 << 31), dict(sm=0.0), dict(sm=-1.0), dict(sm=float("nan")),
                dict(sm=float("inf")), dict(out=None), dict(out=P + 8), dict(lse=P + 2)):
        assert call(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert call(dqk=512) == ds4idx.ERR_UNSUPPORTED and call(dv=576) == ds4idx.ERR_UNSUPPORTED
    assert call(B=0) == ds4idx.OK
    for kw in (dict(kv_row0=P + 4), dict(token_seq=P), dict(kv_row0=P, page_table=P),
               dict(page_table=P, page_size=0, pages_per_seq=2, n_seqs=2),
               dict(page_table=P, page_size=4, pages_per_seq=0, n_seqs=2),
               dict(page_table=P, page_size=4, pages_per_seq=2, n_seqs=1),
               dict(page_table=P + 2, page_size=4, pages_per_seq=2, n_seqs=2)):
        at, keep = _where(**kw)
        assert call(where=at) == ds4idx.ERR_INVALID_ARG, kw
    n = ctypes.c_int64(-7)
    ws = lambda *a: library.ds4idx_tree_attention_workspace(*a, ctypes.addressof(n))  # noqa: E731
    for bad in ((-1, 4, 16, 64), (2, 0, 16, 64), (2, 65, 16, 64), (2, 4, 0, 64), (2, 4, 129, 64),
                (2, 4, 16, -1), (2, 4, 16, 1 << 31), (1 << 30, 64, 128, 64)):
        assert ws(*bad) == ds4idx.ERR_INVALID_ARG, bad
    assert n.value == -7
    assert library.ds4idx_tree_attention_workspace(2, 4, 16, 64, None) == ds4idx.ERR_INVALID_ARG


def _arrays(*rows):
    return ctypes.cast((ds4idx.RowArray * max(1, len(rows)))(*[
        ds4idx.RowArray(src=r.get("src", P), dst=r.get("dst", r.get("src", P)), src_rows=r.get("n", 100),
                        dst_rows=r.get("m", r.get("n", 100)), row_bytes=r.get("bytes", 16)) for r in rows]),
        ctypes.c_void_p)


def test_tree_commit_refusals(library):
    L = 1 << 30          # the small tensors, far from the arrays

    def call(lens=L, path=L + 4096, count=L + 8192, new=L + 16384, where=None, B=2, N=4, R=100,
             arrays=(dict(),), n=None, given=True):
        return library.ds4idx_tree_commit(lens, path, count, new, where, B, N, R,
                                          len(arrays) if n is None else n,
                                          _arrays(*arrays) if given else None, None)
    for bad in (dict(lens=None), dict(lens=L + 2), dict(path=None), dict(path=L + 1), dict(count=None),
                dict(count=L + 8194), dict(new=None), dict(new=L + 16386), dict(B=-1),
                dict(B=(1 << 20) + 1), dict(N=0), dict(N=65), dict(R=0), dict(R=1 << 31), dict(n=-1),
                dict(n=9), dict(given=False), dict(arrays=(dict(src=None, dst=None),)),
                dict(arrays=(dict(dst=P + 16),)), dict(arrays=(dict(n=99),)),
                dict(arrays=(dict(m=99),)), dict(arrays=(dict(bytes=0),)),
                dict(arrays=(dict(bytes=65537),)),
                # overlaps: two arrays, an array with what is read, the new lengths with it
                dict(arrays=(dict(), dict(src=P + 1599))), dict(arrays=(dict(src=L - 1599),)),
                dict(arrays=(dict(src=L + 4096 + 31),)), dict(new=L + 4), dict(new=L + 4096 + 28),
                dict(new=L + 8188), dict(arrays=(dict(src=L + 16384 - 1596),))):
        assert call(**bad) == ds4idx.ERR_INVALID_ARG, bad
    at, keep = _where(kv_row0=P + 1592)
    assert call(where=at) == ds4idx.ERR_INVALID_ARG
    at, keep = _where(page_table=P + 1596, page_size=8, pages_per_seq=3, n_seqs=2)
    assert call(where=at) == ds4idx.ERR_INVALID_ARG
    assert call(B=0) == ds4idx.OK


CALLS = {
    "ds4idx_quantize_latents_fp8": (
        lambda x, c, a, s, **k: ds4idx.quantize_latents_fp8(x, c, a, slots=s, **k),
        [((4, 576), BF16), ((9, 640), U8), ((9,), F32), ((4,), I64)]),
    "ds4idx_read_latents_fp8": (
        lambda c, a, r, o, **k: ds4idx.read_latents_fp8(c, a, rows=r, out=o, **k),
        [((9, 640), U8), ((9,), F32), ((4,), I64), ((4, 576), F32)]),
    "ds4idx_tree_attention": (
        lambda q, c, a, n, m, t, s, o, l, w, **k: ds4idx.tree_attention(
            q, c, n, m, 1.0, scale=a, page_table=t, page_size=8, token_seq=s, out=o, lse=l,
            workspace=w, **k),
        [((4, 2, 16, 576), BF16), ((9, 640), U8), ((9,), F32), ((4,), I32), ((4, 2), I64),
         ((3, 2), I32), ((4,), I32), ((4, 2, 16, 512), BF16), ((4, 2, 16), F32), ((64,), U8)]),
    "ds4idx_tree_commit": (
        lambda a, b, n, p, c, r, o, **k: ds4idx.tree_commit([a, b], n, p, c, kv_row0=r, new_lens=o, **k),
        [((9, 640), U8), ((9,), F32), ((4,), I32), ((4, 2), I32), ((4,), I32), ((4,), I64), ((4,), I32)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_tree_calls_on_one_device(devices, monkeypatch, name):  # noqa: F811
    class Library:
        def __init__(self):
            self.calls = []

        def __getattr__(self, entry):
            if entry.endswith("_workspace"):
                return lambda *a: ds4idx.OK
            return lambda *a: self.calls.append((entry, a[-1])) or ds4idx.OK

    library = Library()
    monkeypatch.setattr(ds4idx, "load", lambda: library)
    monkeypatch.setitem(test_devices_host.CALLS, name, CALLS[name])
    one_device(library, name)


def test_cache_formats(devices):  # noqa: F811
    scale = Tensor((9,), F32)
    fmt = ds4idx._cache_format
    assert fmt(Tensor((9, 576), BF16), None, 0) == (ds4idx.CACHE_BF16, 9)
    assert fmt(Tensor((9, 640), U8), scale, 0) == (ds4idx.CACHE_FP8, 9)
    assert fmt(Tensor((9, 416), U8), None, 0) == (ds4idx.CACHE_Q4, 9)
    for c, s in ((Tensor((9, 576), BF16), scale), (Tensor((9, 416), U8), scale),
                 (Tensor((9, 640), U8), None), (Tensor((9, 640), U8), Tensor((8,), F32)),
                 (Tensor((9, 512), U8), None), (Tensor((9, 640), BF16), None)):
        with pytest.raises(ValueError):
            fmt(c, s, 0)


def test_tree_attention_output_is_32_byte_aligned(library):
    assert library.ds4idx_tree_attention(P, 1, P, P, 100, P, P, None, 2, 4, 16, 576, 512, 64, 1.0,
                                         P + 16, P, None, 0, None) == ds4idx.ERR_INVALID_ARG
