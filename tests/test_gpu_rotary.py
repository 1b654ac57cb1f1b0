"""Rotary positions against the formula in 64 bits.

Tolerance. The fp32 cosine and sine are off by at most 4 * 2^-24 (conversion of the angle within an
eighth of a turn, sincospi, the product with the scale), the two products and the sum by 2^-24 of
their size each: 8 * 2^-24 * m * (|a| + |b|) in all; a bf16 output adds half a step, 2^-8 |y|."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref

pytestmark = pytest.mark.gpu


def _check(y, x, pos, f, m, interleaved, inverse):
    xf = x.double().cpu().numpy()
    want = ref.rotate(xf, pos.cpu().numpy(), f, m, interleaved, inverse)
    h = xf.shape[-1] // 2
    a = np.abs(xf)
    if interleaved:
        size = np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1)
    else:
        size = np.concatenate([a[..., :h] + a[..., h:]] * 2, axis=-1)
    bound = 8 * 2.0 ** -24 * m * size
    if y.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= bound + 1e-37), float((err - bound).max())


SCALINGS = [("none", {}), ("linear", dict(factor=8.0)),
            ("yarn", dict(factor=40.0, original_max_position=4096))]


def _reference(rot, base, scaling, kw):
    return ref.rotary_frequencies(rot, base, scaling, kw.get("factor", 1.0),
                                  kw.get("original_max_position", 4096))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,rot,scaling", [(1, 1, 2, 0), (1, 128, 64, 2), (7, 3, 64, 2),
                                             (33, 5, 30, 1), (300, 16, 128, 2), (5, 2, 256, 0),
                                             (700, 130, 32, 1)])
def test_rotary_matches_formula(T, H, rot, scaling, interleaved, dtype):
    name, kw = SCALINGS[scaling]
    g = torch.Generator().manual_seed(T * 1000 + rot)
    x = torch.randn(T, H, rot, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    pos[0] = (1 << 20) - 1
    if T > 2:
        pos[1], pos[2] = 0, 1 << 30
    fr = ds4idx.rotary_freqs(rot, 10000.0, scaling=name, **kw)
    f, m = _reference(rot, 10000.0, name, kw)
    for inverse in (False, True):
        y = ds4idx.rotary(x, pos.cuda(), fr, interleaved=interleaved, inverse=inverse)
        _check(y, x, pos, f, m, interleaved, inverse)


def test_four_tensors_part_of_the_head_in_place_and_strided():
    T, rot = 37, 64
    g = torch.Generator().manual_seed(3)
    q = torch.randn(T, 128, 576, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(T, 576, generator=g).to(torch.bfloat16).cuda()
    iq = torch.randn(T, 64, 128, generator=g).cuda()
    odd = torch.randn(T, 3, 67, generator=g).to(torch.bfloat16).cuda()[..., 1:65]  # unaligned
    pos = torch.randint(0, 262144, (T,), generator=g)
    fr = ds4idx.rotary_freqs(rot, 10000.0, scaling="yarn", factor=40.0)
    f, m = ref.rotary_frequencies(rot, 10000.0, "yarn", 40.0)
    before = [t.clone() for t in (q, kv, iq, odd)]
    views = [q[..., 512:], kv[:, 512:], iq[..., :64], odd]
    layouts = [True, True, False, False]
    ds4idx.rotary(views, pos.cuda(), fr, interleaved=layouts, outs=views)
    olds = [before[0][..., 512:], before[1][:, 512:], before[2][..., :64], before[3]]
    for v, o, il in zip(views, olds, layouts):
        _check(v, o, pos, f, m, il, False)
    assert torch.equal(q[..., :512], before[0][..., :512])     # the rest is not touched
    assert torch.equal(kv[:, :512], before[1][:, :512])
    assert torch.equal(iq[..., 64:], before[2][..., 64:])
    # a transposed view, [H, T, rot] storage, into another layout of strides
    x = torch.randn(9, T, rot, generator=g).cuda().transpose(0, 1)
    out = torch.empty(T, 9, 80, device="cuda")[..., 8:72]
    ds4idx.rotary(x, pos.cuda(), fr, interleaved=False, outs=out)
    _check(out, x, pos, f, m, False, False)


def test_negative_positions_and_inverse_undo_each_other():
    T, rot = 64, 64
    x = torch.randn(T, 2, rot, device="cuda")
    pos = torch.arange(-32, 32, device="cuda")
    fr = ds4idx.rotary_freqs(rot)
    a = ds4idx.rotary(x, pos, fr)
    b = ds4idx.rotary(x, -pos, fr, inverse=True)
    assert torch.equal(a, b)


def test_gradient_is_the_transpose_and_agrees_with_differences():
    T, H, rot = 5, 2, 16
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, rot, generator=g).cuda().requires_grad_()
    k = torch.randn(T, rot, generator=g).cuda().requires_grad_()
    pos = torch.randint(0, 100000, (T,), generator=g).cuda()
    fr = ds4idx.rotary_freqs(rot, scaling="yarn", factor=4.0)
    f, m = ref.rotary_frequencies(rot, 10000.0, "yarn", 4.0)
    y, z = ds4idx.rotary_autograd([x, k], pos, fr, interleaved=[True, False])
    gy = torch.randn(T, H, rot, generator=g).cuda()
    gz = torch.randn(T, 1, generator=g).cuda().expand(T, rot)   # stride 0: a broadcast gradient
    dx, dk = torch.autograd.grad([y, z], [x, k], [gy, gz])
    _check(dx, gy, pos, f, m, True, True)
    _check(dk, gz, pos, f, m, False, True)
    # the operator is linear: (F(x + h d) - F(x - h d)) / 2h = F(d), and <g, F(d)> = <F'(g), d>
    d = torch.randn(T, H, rot, generator=g).cuda()
    h = 2.0 ** -3
    diff = (ds4idx.rotary(x.detach() + h * d, pos, fr) - ds4idx.rotary(x.detach() - h * d, pos, fr))
    lhs = float((gy.double() * diff.double()).sum() / (2 * h))
    rhs = float((dx.double() * d.double()).sum())
    # each rotated value is off by 8 * 2^-24 * m * (|a| + |b|) <= 2^-20 * 8; divided by 2h
    assert abs(lhs - rhs) <= float(gy.abs().sum()) * 2.0 ** -20 * 8 / (2 * h)


def test_side_stream_graph_and_empty():
    T, rot = 16, 64
    x = torch.randn(T, 4, rot, device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, device="cuda") * 1000
    fr = ds4idx.rotary_freqs(rot)
    want = ds4idx.rotary(x, pos, fr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    ds4idx.rotary(x, pos, fr, outs=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ds4idx.rotary(x, pos, fr, outs=out)
    out.zero_()
    x.copy_(x.flip(0))
    gr.replay()
    assert torch.equal(out, ds4idx.rotary(x, pos, fr))
    assert ds4idx.rotary(x[:0], pos[:0], fr).shape == (0, 4, rot)


def test_refusals():
    x = torch.zeros(4, 2, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    fr = ds4idx.rotary_freqs(64)
    with pytest.raises(ValueError):
        ds4idx.rotary(x[..., :32], pos, fr)
    with pytest.raises(ValueError):
        ds4idx.rotary(x.transpose(1, 2), pos, fr)
    with pytest.raises(ValueError):
        ds4idx.rotary(x, pos[:3], fr)
    with pytest.raises(TypeError):
        ds4idx.rotary(x.half(), pos, fr)
    with pytest.raises(TypeError):
        ds4idx.rotary(x, pos.int(), fr)
    with pytest.raises(ValueError):
        ds4idx.rotary([x] * 5, pos, fr)
    with pytest.raises(ValueError):
        ds4idx.rotary(x, pos, fr, outs=torch.zeros(4, 2, 64, device="cuda").bfloat16())
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.rotary_freqs(63)
    with pytest.raises(ValueError):
        ds4idx.rotary_freqs(64, scaling="other")
