"""Rotary outputs in the layouts that a program uses: slices of one projection in place, one half of a
buffer into the other, broadcast inputs, transposed storage. Tolerances as in test_gpu_rotary."""
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref
from .test_gpu_rotary import _check

pytestmark = pytest.mark.gpu

ROT = 64


def _setup(T, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 100000, (T,), generator=g)
    f, m = ref.rotary_frequencies(ROT, 10000.0)
    return g, pos, ds4idx.rotary_freqs(ROT), f, m


@pytest.mark.parametrize("T", [1, 2, 41])
def test_slices_of_one_projection_in_place(T):
    g, pos, fr, f, m = _setup(T, 1)
    H, I = 6, 5
    width = H * 192 + 576 + I * 128 + 128          # query, latent, index query, index key
    buf = torch.randn(T, width, generator=g).to(torch.bfloat16).cuda()
    before = buf.clone()

    def views(b):
        q = b[:, :H * 192].view(T, H, 192)[..., 128:]
        kv = b[:, H * 192:H * 192 + 576][:, 512:]
        iq = b[:, H * 192 + 576:-128].view(T, I, 128)[..., :ROT]
        return [q, kv, iq, b[:, -128:][:, :ROT]]
    layouts = [True, True, False, False]
    ds4idx.rotary(views(buf), pos.cuda(), fr, interleaved=layouts, outs=views(buf))
    for y, x, il in zip(views(buf), views(before), layouts):
        _check(y, x, pos, f, m, il, False)
    for b in (buf, before):
        for v in views(b):
            v.zero_()
    assert torch.equal(buf, before)                 # the rest is not touched


@pytest.mark.parametrize("T,H", [(1, 1), (1, 9), (23, 1), (23, 9)])
def test_one_half_into_the_other(T, H):
    g, pos, fr, f, m = _setup(T, 2)
    buf = torch.randn(T, H, 2 * ROT, generator=g).cuda()
    x = buf[..., :ROT].clone()
    ds4idx.rotary(buf[..., :ROT], pos.cuda(), fr, outs=buf[..., ROT:])
    _check(buf[..., ROT:], x, pos, f, m, True, False)
    assert torch.equal(buf[..., :ROT], x)


def test_broadcast_inputs_and_transposed_storage():
    T, H = 19, 4
    g, pos, fr, f, m = _setup(T, 3)
    one = torch.randn(T, 1, ROT, generator=g).cuda().expand(T, H, ROT)
    _check(ds4idx.rotary(one, pos.cuda(), fr), one, pos, f, m, True, False)
    same = torch.randn(1, H, ROT, generator=g).cuda().expand(T, H, ROT)
    _check(ds4idx.rotary(same, pos.cuda(), fr), same, pos, f, m, True, False)
    x = torch.randn(H, T, ROT, generator=g).cuda()
    a, b = ds4idx.rotary([x.transpose(0, 1)] * 2, pos.cuda(), fr, interleaved=[True, False])
    y = x.clone()
    ds4idx.rotary(y.transpose(0, 1), pos.cuda(), fr, outs=y.transpose(0, 1))
    assert torch.equal(y.transpose(0, 1), a)
    _check(b, x.transpose(0, 1), pos, f, m, False, False)


def test_overlapping_outs_are_refused():
    T, H = 5, 3
    _, pos, fr, _, _ = _setup(T, 4)
    pos = pos.cuda()
    x = torch.zeros(T, H, ROT, device="cuda")
    buf = torch.zeros(T, H, ROT + 8, device="cuda")
    for xs, outs in ((x, torch.zeros(T, 1, ROT, device="cuda").expand(T, H, ROT)),
                     (x[:, :1].expand(T, H, ROT), x[:, :1].expand(T, H, ROT)),
                     (buf[..., :ROT], buf[..., 8:]), ([x, x], [x, torch.zeros_like(x)])):
        with pytest.raises(ds4idx.Ds4IdxError):
            ds4idx.rotary(xs, pos, fr, outs=outs)
