"""The calls around the 4-bit latent cache launch on the current device: tensors of another device, of
two devices, or a stream of another device are refused before the library is reached. No GPU: the
tensors are stand-ins that report a device."""
import types

import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

BF16, F32, I64, I32, U8 = torch.bfloat16, torch.float32, torch.int64, torch.int32, torch.uint8


class Tensor:
    def __init__(self, shape, dtype, dev=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        self.is_cuda, self.device, self.requires_grad = dev >= 0, "meta", False
        self.nbytes = self.shape.numel() * dtype.itemsize

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 1 << 20

    def element_size(self):
        return self.dtype.itemsize


class Library:
    """Records the entry points that are reached; each succeeds."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a[-1])) or ds4idx.OK


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(ds4idx, "load", lambda: lib)
    monkeypatch.setattr(ds4idx, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(ds4idx, "_raw_stream", lambda dev: 1000 + dev)
    return lib


def _freqs():
    return types.SimpleNamespace(rot_dim=64, address=0, scale=1.0)


# entry point -> (call of its tensors, the tensors)
CALLS = {
    "ds4idx_rotary": (lambda x, o, p, **k: ds4idx.rotary([x], p, _freqs(), outs=[o], **k),
                      [((4, 2, 64), BF16), ((4, 2, 64), BF16), ((4,), I64)]),
    "ds4idx_quantize_latents": (lambda x, c, s, **k: ds4idx.quantize_latents(x, c, slots=s, **k),
                                [((4, 576), BF16), ((9, 416), U8), ((4,), I64)]),
    "ds4idx_read_latents": (lambda c, r, o, **k: ds4idx.read_latents(c, rows=r, out=o, **k),
                            [((9, 416), U8), ((4,), I64), ((4, 576), F32)]),
    "ds4idx_sparse_attention_q4": (
        lambda q, c, i, o, l, w, t, s, **k: ds4idx.sparse_attention_q4(
            q, c, i, 1.0, page_table=t, page_size=8, token_seq=s, out=o, lse=l, weights=w, **k),
        [((4, 16, 576), BF16), ((9, 416), U8), ((4, 70), I32), ((4, 16, 512), BF16), ((4, 16), F32),
         ((4, 70), F32), ((3, 2), I32), ((4,), I32)]),
    "ds4idx_evict_accumulate": (
        lambda t, w, i, r, **k: ds4idx.evict_accumulate(t, w, i, kv_row0=r, **k),
        [((9,), I64), ((4, 70), F32), ((4, 70), I32), ((4,), I64)]),
    "ds4idx_evict_select": (lambda t, k, **kw: ds4idx.evict_select(t, [0], [9], [5], kept=k, **kw),
                            [((9,), I64), ((1, 5), I32)]),
    "ds4idx_evict_compact": (
        lambda k, a, b, c, d, **kw: ds4idx.evict_compact(k, [9], [5], [0], [0], [a, b], [c, d], **kw),
        [((1, 5), I32), ((9, 416), U8), ((9,), F32), ((5, 416), U8), ((5,), F32)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_one_device_and_the_current_one(lib, name):
    call, specs = CALLS[name]
    call(*[Tensor(*s) for s in specs])
    assert lib.calls == [(name, 1000)]                  # the current stream of the tensors' device
    own = types.SimpleNamespace(cuda_stream=77, device_index=0)
    call(*[Tensor(*s) for s in specs], stream=own)
    assert lib.calls.pop() == (name, 77) and len(lib.calls) == 1
    for odd in range(len(specs)):                       # one tensor elsewhere, or on the host
        for dev in (1, -1):
            with pytest.raises(ValueError):
                call(*[Tensor(*s, dev=dev if i == odd else 0) for i, s in enumerate(specs)])
    with pytest.raises(ValueError):                     # all on a device that is not current
        call(*[Tensor(*s, dev=1) for s in specs])
    with pytest.raises(ValueError):                     # a stream of another device
        call(*[Tensor(*s) for s in specs],
             stream=types.SimpleNamespace(cuda_stream=77, device_index=1))
    assert len(lib.calls) == 1


def test_missing_tensors_are_named(lib):
    x = Tensor((4, 2, 64), BF16)
    with pytest.raises(ValueError, match="positions"):
        ds4idx.rotary([x], None, _freqs(), outs=[x])
    assert not lib.calls


def test_row_start_of_another_device(lib):
    t = [Tensor((4, 16, 576), BF16), Tensor((9, 416), U8), Tensor((4, 70), I32)]
    outs = dict(out=Tensor((4, 16, 512), BF16), lse=Tensor((4, 16), F32))
    ds4idx.sparse_attention_q4(*t, 1.0, kv_row0=Tensor((4,), I64), **outs)
    with pytest.raises(ValueError):
        ds4idx.sparse_attention_q4(*t, 1.0, kv_row0=Tensor((4,), I64, 1), **outs)
    assert len(lib.calls) == 1
