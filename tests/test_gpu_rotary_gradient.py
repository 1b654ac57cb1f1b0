"""``rotary`` itself records gradients: they are the inverse rotation, for any stream and direction, and
nothing that requires them is silently cut off."""
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

pytestmark = pytest.mark.gpu


def _setup(T=21):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, 3, 64, generator=g).cuda()
    k = torch.randn(T, 64, generator=g).cuda()
    gy, gz = torch.randn(T, 3, 64, generator=g).cuda(), torch.randn(T, 64, generator=g).cuda()
    pos = torch.randint(0, 9999, (T,), generator=g).cuda()
    return x, k, gy, gz, pos, ds4idx.rotary_freqs(64, scaling="yarn", factor=4.0)


@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_is_the_other_direction(inverse):
    x, k, gy, gz, pos, fr = _setup()
    want = ds4idx.rotary([x, k], pos, fr, [True, False], inverse)
    back = ds4idx.rotary([gy, gz], pos, fr, [True, False], not inverse)
    for stream in (None, torch.cuda.Stream()):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        a, b = x.clone().requires_grad_(), k.clone()
        torch.cuda.synchronize()
        y, z = ds4idx.rotary([a, b], pos, fr, [True, False], inverse, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
        (da,) = torch.autograd.grad([y, z], [a], [gy, gz])
        torch.cuda.synchronize()
        assert torch.equal(da, back[0])
    one = x.clone().requires_grad_()
    y = ds4idx.rotary(one, pos, fr, True, inverse)
    y.backward(gy)
    assert torch.equal(one.grad, back[0])


def test_outs_are_refused_where_a_gradient_would_be_lost():
    x, _, _, _, pos, fr = _setup()
    x.requires_grad_()
    with pytest.raises(ValueError):
        ds4idx.rotary(x, pos, fr, outs=torch.empty_like(x))
    with pytest.raises(ValueError):
        ds4idx.rotary([x[:, :2] * 1.0], pos, fr, outs=[torch.empty(21, 2, 64, device="cuda")])
    with torch.no_grad():
        y = ds4idx.rotary(x, pos, fr)
        out = ds4idx.rotary(x, pos, fr, outs=torch.empty_like(x))
    assert not y.requires_grad and torch.equal(y, out)
    assert not ds4idx.rotary(x.detach(), pos, fr).requires_grad
