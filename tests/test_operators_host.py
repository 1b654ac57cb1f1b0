"""Host-side checks of the operators around the 4-bit latent cache that need no GPU: refusals come
before any device work, and the rotary frequencies are the formula's."""
import ctypes

import numpy as np
import pytest

from sparse_attention_lightning_indexer_gb300 import build, ds4idx

from . import latent_reference as ref

P = 1 << 20          # an aligned address that no call may touch


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ds4idx.load()


def _vp(x):
    return ctypes.cast(x, ctypes.c_void_p)


@pytest.mark.parametrize("rot,base,scaling,factor", [(2, 10000.0, "none", 1.0),
                                                     (64, 10000.0, "yarn", 40.0),
                                                     (256, 500000.0, "linear", 8.0),
                                                     (64, 1e6, "yarn", 1.0)])
def test_rotary_freqs(lib, rot, base, scaling, factor):
    fr = ds4idx.rotary_freqs(rot, base, scaling=scaling, factor=factor)
    f, m = ref.rotary_frequencies(rot, base, scaling, factor)
    turns = np.array([int(x) / 2.0 ** 64 for x in fr.freqs])
    # a frequency is held in steps of 2^-64 turn
    np.testing.assert_allclose(turns * 2 * np.pi, f, rtol=4e-15, atol=2 * np.pi * 2.0 ** -64)
    assert abs(fr.scale - m) <= 2.0 ** -24 * m


def test_rotary_freqs_refusals(lib):
    f, s = (ctypes.c_uint64 * 128)(), ctypes.c_float()
    call = lambda rot=64, base=1e4, kind=2, factor=2.0, orig=4096, bf=32.0, bs=1.0, o=_vp(f): (  # noqa: E731
        lib.ds4idx_rotary_freqs(rot, base, kind, factor, orig, bf, bs, o,
                                _vp(ctypes.byref(s))))
    assert call() == ds4idx.OK
    for bad in (dict(rot=0), dict(rot=63), dict(rot=258), dict(base=1.0), dict(base=float("nan")),
                dict(kind=3), dict(kind=-1), dict(factor=0.5), dict(factor=float("inf")),
                dict(orig=0), dict(bs=0.0), dict(bf=0.5), dict(o=None)):
        assert call(**bad) == ds4idx.ERR_INVALID_ARG, bad


def _rot(**kw):
    d = dict(x=P, out=P, dtype=0, interleaved=1, n_heads=2, reserved=0, x_stride_t=128,
             x_stride_h=64, out_stride_t=128, out_stride_h=64)
    d.update(kw)
    return (ds4idx.RotaryTensor * 1)(ds4idx.RotaryTensor(**d))


def test_rotary_refusals(lib):
    f = (ctypes.c_uint64 * 128)()
    call = lambda n=1, t=None, T=4, rot=64, pos=P, fr=_vp(f), scale=1.0: lib.ds4idx_rotary(  # noqa: E731
        n, _vp(t if t is not None else _rot()), T, rot, pos, fr, scale, 0, None)
    for bad in (dict(n=0), dict(n=5), dict(T=-1), dict(rot=1), dict(rot=258), dict(pos=None),
                dict(pos=P + 4), dict(fr=None), dict(scale=0.0), dict(scale=float("inf")),
                dict(t=_rot(dtype=1)), dict(t=_rot(n_heads=0)), dict(t=_rot(x=None)),
                dict(t=_rot(x=P + 1)), dict(t=_rot(out=P + 1))):
        assert call(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert lib.ds4idx_rotary(1, None, 4, 64, P, _vp(f), 1.0, 0, None) == ds4idx.ERR_INVALID_ARG
    assert call(T=0) == ds4idx.OK


def test_latent_refusals(lib):
    w = lambda x=P, dt=0, n=4, slots=None, off=0, c=P, R=8: (  # noqa: E731
        lib.ds4idx_quantize_latents(x, dt, n, slots, off, c, R, None))
    for bad in (dict(x=None), dict(x=P + 8), dict(dt=1), dict(n=-1), dict(slots=P + 4), dict(off=5),
                dict(off=-1), dict(off=(1 << 63) - 1), dict(c=None), dict(c=P + 16), dict(R=-1)):
        assert w(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert w(n=0) == ds4idx.OK
    r = lambda c=P, R=8, rows=None, start=0, n=4, out=P, dt=0: (  # noqa: E731
        lib.ds4idx_read_latents(c, R, rows, start, n, out, dt, None))
    for bad in (dict(c=None), dict(c=P + 16), dict(rows=P + 4), dict(start=5), dict(start=-1),
                dict(n=-1), dict(out=None), dict(out=P + 8), dict(dt=1)):
        assert r(**bad) == ds4idx.ERR_INVALID_ARG, bad


def _place(**kw):
    d = dict(kv_row0=None, page_table=P, token_seq=P, page_size=64, pages_per_seq=2, n_seqs=3)
    d.update(kw)
    return ctypes.byref(ds4idx.Placement(**d))


BAD_PLACES = [dict(kv_row0=P), dict(page_size=0), dict(pages_per_seq=0), dict(n_seqs=0),
              dict(page_table=P + 2), dict(token_seq=P + 1), dict(token_seq=None),
              dict(page_table=None), dict(page_table=None, token_seq=None, kv_row0=P + 4)]


def test_attention_refusals(lib):
    def call(q=P, c=P, R=100, idx=P, place=None, T=4, H=128, dqk=576, dv=512, n=512, s=1.0, out=P,
             lse=None, w=None):
        return lib.ds4idx_sparse_attention_q4(q, c, R, idx, place, T, H, dqk, dv, n, s, out, lse, w,
                                              None)
    for bad in (dict(q=None), dict(q=P + 8), dict(c=None), dict(c=P + 16), dict(R=0),
                dict(R=1 << 31), dict(idx=None), dict(idx=P + 2), dict(T=-1), dict(T=1 << 25),
                dict(H=0), dict(H=129), dict(n=0), dict(n=513), dict(s=0.0), dict(s=-1.0),
                dict(s=float("nan")), dict(s=float("inf")), dict(out=None), dict(out=P + 16),
                dict(lse=P + 2), dict(w=P + 1), *[dict(place=_place(**b)) for b in BAD_PLACES]):
        assert call(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert call(dqk=512) == ds4idx.ERR_UNSUPPORTED and call(dv=576) == ds4idx.ERR_UNSUPPORTED
    assert call(T=0) == ds4idx.OK


def test_evict_refusals(lib):
    def acc(t=P, R=100, w=P, idx=P, place=None, T=4, n=512):
        return lib.ds4idx_evict_accumulate(t, R, w, idx, place, T, n, None)
    for bad in (dict(t=None), dict(t=P + 4), dict(R=0), dict(w=None), dict(idx=None), dict(T=-1),
                dict(n=0), *[dict(place=_place(**b)) for b in BAD_PLACES]):
        assert acc(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert acc(T=0) == ds4idx.OK

    i64 = lambda *v: _vp((ctypes.c_int64 * len(v))(*v))  # noqa: E731

    def sel(t=P, R=100, B=1, st=(0,), n=(50,), k=(10,), sink=0, rec=0, kept=P, width=10):
        return lib.ds4idx_evict_select(t, R, B, i64(*st), i64(*n), i64(*k), sink, rec, kept, width,
                                       None)
    for bad in (dict(t=None), dict(B=0), dict(B=65), dict(st=(-1,)), dict(st=(51,)), dict(n=(-1,)),
                dict(n=(101,)), dict(k=(-1,)), dict(sink=6, rec=5), dict(sink=-1), dict(rec=-1),
                dict(kept=None), dict(kept=P + 2), dict(width=9), dict(t=P + 4)):
        assert sel(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert sel(width=0, n=(0,)) == ds4idx.OK

    def mov(kept=P, width=10, ss=(0,), sl=(50,), ds=(0,), c=(10,), n=1, **a):
        d = dict(src=P, dst=P + (1 << 16), src_rows=50, dst_rows=10, row_bytes=16, reserved=0)
        d.update(a)
        return lib.ds4idx_evict_compact(kept, width, 1, i64(*ss), i64(*sl), i64(*ds), i64(*c), n,
                                        _vp((ds4idx.RowArray * 1)(ds4idx.RowArray(**d))), None)
    for bad in (dict(kept=None), dict(width=9), dict(ss=(1,)), dict(sl=(9,)), dict(ds=(1,)),
                dict(c=(11,)), dict(c=(-1,)), dict(n=0), dict(n=9), dict(src=None), dict(dst=None),
                dict(row_bytes=0), dict(row_bytes=65537), dict(dst=P + 16 * 49), dict(dst=P - 16)):
        assert mov(**bad) == ds4idx.ERR_INVALID_ARG, bad
    assert mov(c=(0,)) == ds4idx.OK
