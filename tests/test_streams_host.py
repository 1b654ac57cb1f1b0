"""Outputs that a call allocates for a given stream come from that stream's memory, and the current
stream is recorded as their user. No GPU: stand-ins for tensors, streams and the allocator."""
import contextlib

import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from .test_devices_host import BF16, F32, I32, I64, U8, Library, Tensor, _freqs

DEVICE = "cuda:0"


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device_index = handle, 0


class CudaTensor(Tensor):
    def __init__(self, shape, dtype, made_on=None):
        super().__init__(shape, dtype)
        self.device, self.made_on, self.users = DEVICE, made_on, []

    def record_stream(self, s):
        self.users.append(s.cuda_stream)


@pytest.fixture
def gpu(monkeypatch):
    """The library, and the list of (allocating stream, recorded users) of what calls allocate."""
    lib, current, made, empty = Library(), [Stream(1000)], [], torch.empty

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def allocate(shape, dtype=None, device=None, **k):
        if device != DEVICE:
            return empty(shape, dtype=dtype, device=device, **k)
        made.append(CudaTensor(shape, dtype, current[-1].cuda_stream))
        return made[-1]

    monkeypatch.setattr(ds4idx, "load", lambda: lib)
    monkeypatch.setattr(ds4idx, "_current_device", lambda: 0)
    monkeypatch.setattr(ds4idx, "_raw_stream", lambda dev: current[-1].cuda_stream)
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    return lib, made


def _indexer(lib):
    ix = object.__new__(ds4idx.Indexer)
    ix._lib, ix._h, ix.dtype, ix.topk = lib, None, ds4idx.BF16, 512
    return ix


T = CudaTensor
CALLS = {
    "rotary": (lambda lib, **k: ds4idx.rotary([T((4, 2, 64), BF16)], T((4,), I64), _freqs(), **k), 1),
    "read_latents": (lambda lib, **k: ds4idx.read_latents(T((9, 416), U8), **k), 1),
    "sparse_attention_q4": (lambda lib, **k: ds4idx.sparse_attention_q4(
        T((4, 16, 576), BF16), T((9, 416), U8), T((4, 70), I32), 1.0, want_weights=True, **k), 3),
    "evict_select": (lambda lib, **k: ds4idx.evict_select(T((9,), I64), [0], [9], [5], **k), 1),
    "quantize_queries": (lambda lib, **k: ds4idx.quantize_queries(
        T((4, 64, 128), BF16), T((4, 64), F32), **k), 3),
    "merge_topk": (lambda lib, **k: ds4idx.merge_topk(
        T((2, 4, 512), I32), T((2, 4, 512), F32), [0, 9], **k), 2),
    "sparse_attention": (lambda lib, **k: ds4idx.sparse_attention(
        T((4, 128, 576), BF16), T((9, 576), BF16), T((4, 512), I32), 1.0, **k), 2),
    "score_topk": (lambda lib, **k: _indexer(lib).score_topk(
        T((4, 64, 128), BF16), T((4, 64), F32), T((9, 128), BF16), **k), 2),
    "score_topk_batched": (lambda lib, **k: _indexer(lib).score_topk_batched(
        T((2, 4, 64, 128), BF16), T((2, 4, 64), F32), T((2, 9, 128), BF16), None, [0, 0], **k), 2),
    "score_topk_varlen": (lambda lib, **k: _indexer(lib).score_topk_varlen(
        T((4, 64, 128), BF16), T((4, 64), F32), [0, 4], T((9, 128), BF16), None, [9], [0], **k), 2),
    "score_dense_debug": (lambda lib, **k: _indexer(lib).score_dense_debug(
        T((4, 64, 128), BF16), T((4, 64), F32), T((9, 128), BF16), **k), 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_belong_to_the_stream_of_the_call(gpu, name):
    lib, made = gpu
    call, n = CALLS[name]
    call(lib)
    assert [(t.made_on, t.users) for t in made] == [(1000, [])] * n
    assert lib.calls.pop()[1] == 1000
    made.clear()
    call(lib, stream=Stream(77))
    assert [(t.made_on, t.users) for t in made] == [(77, [1000])] * n
    assert lib.calls.pop()[1] == 77
