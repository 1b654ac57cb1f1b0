"""The 4-bit latent cache's writer and reader: bytes and values equal to the definition, exactly."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref

pytestmark = pytest.mark.gpu


def _bytes(x):
    rope = x[:, 512:].to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return ref.quantize(x.double().numpy(), rope)


def _rows(n, dtype, seed):
    """Rows with wide ranges, zeros, exact ties of integers and of scales, and tiny or huge groups."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 576, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    if n > 4:
        x[1] = 0
        x[2, :512] = 0.5 * torch.randint(-15, 16, (512,), generator=g)   # ties at s = 1 and others
        x[2, 0:512:16] = 7.0
        x[3, :512] *= 2.0 ** -24
        x[4, :512] *= 2.0 ** 15
        # absmax / 7 halfway between two scales: 7 * (1 + (2k + 1) / 16)
        for k in range(8):
            x[0, 16 * k:16 * k + 16] = 7.0 * (1 + (2 * k + 1) / 16) * 2.0 ** (k - 4)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 2, 9, 1000])
def test_write_and_read_are_exact(n, dtype):
    x = _rows(n, dtype, n)
    R = n + 5
    cache = torch.full((R, 416), 0xA5, dtype=torch.uint8, device="cuda")
    ds4idx.quantize_latents(x.cuda(), cache, dst_offset=3)
    got = cache.cpu().numpy()
    want = _bytes(x)
    bad = np.argwhere(got[3:3 + n] != want)
    assert bad.size == 0, (bad[:4], got[3:3 + n][tuple(bad[0])], want[tuple(bad[0])])
    assert np.all(got[:3] == 0xA5) and np.all(got[3 + n:] == 0xA5)
    vals = ref.dequantize(want)
    for out in (torch.bfloat16, torch.float32):
        v = ds4idx.read_latents(cache, start=3, n=n, dtype=out)
        assert np.array_equal(v.double().cpu().numpy(), vals)


def test_fp32_values_next_to_ties():
    # x / s one step of fp32 from k + 1/2, and absmax / 7 one step from a scale's border
    s = 1.875
    x = torch.zeros(4, 576)
    x[:, 0] = 7 * s
    t = (torch.arange(1, 16) % 7 + 0.5) * s
    x[0, 1:16] = torch.nextafter(t, torch.full_like(t, 100.0))
    x[1, 1:16] = torch.nextafter(t, torch.zeros_like(t))
    x[2, 1:16] = t
    for k in range(8):
        a = torch.tensor(7.0 * (1 + (2 * k + 1) / 16))
        x[3, 16 * k] = torch.nextafter(a, torch.tensor(100.0 if k % 2 else 0.0))
    cache = torch.zeros(4, 416, dtype=torch.uint8, device="cuda")
    ds4idx.quantize_latents(x.cuda(), cache)
    assert np.array_equal(cache.cpu().numpy(), _bytes(x))


def test_past_the_largest_scale():
    # the largest scale is 3840: 7.5 of it is a tie that must clamp to 7, far values saturate
    x = torch.zeros(3, 576)
    for k in range(32):
        v = 3840.0 * torch.tensor([7.5, 7.25, 7.4375, 6.5, 5.5, 100.0, 3e38, 1.0])
        x[0, 16 * k:16 * k + 8] = v * (1 if k % 2 else -1)
        x[1, 16 * k:16 * k + 5] = v[:5]
        x[2, 16 * k] = v[0]
    cache = torch.zeros(3, 416, dtype=torch.uint8, device="cuda")
    ds4idx.quantize_latents(x.cuda(), cache)
    assert np.array_equal(cache.cpu().numpy(), _bytes(x))


def test_slots_and_reading_by_rows():
    n, R = 200, 333
    x = _rows(n, torch.bfloat16, 7)
    g = torch.Generator().manual_seed(2)
    slots = torch.randperm(R, generator=g)[:n]
    slots[::9] = -1
    slots[5] = R            # outside: skipped
    cache = torch.zeros(R, 416, dtype=torch.uint8, device="cuda")
    ds4idx.quantize_latents(x.cuda(), cache, slots=slots.cuda())
    want = np.zeros((R, 416), np.uint8)
    b = _bytes(x)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < R:
            want[s] = b[i]
    assert np.array_equal(cache.cpu().numpy(), want)
    v = ds4idx.read_latents(cache, rows=slots.cuda()).double().cpu().numpy()
    ok = ((slots >= 0) & (slots < R)).numpy()
    assert np.array_equal(v[ok], ref.dequantize(b)[ok]) and np.all(v[~ok] == 0)


def test_refusals_and_empty():
    cache = torch.zeros(8, 416, dtype=torch.uint8, device="cuda")
    x = torch.zeros(4, 576, device="cuda")
    assert ds4idx.quantize_latents(x[:0], cache) is cache
    assert ds4idx.read_latents(cache, start=8).shape == (0, 576)
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.quantize_latents(x, cache, dst_offset=5)
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.read_latents(cache, start=6, n=3)
    with pytest.raises(TypeError):
        ds4idx.quantize_latents(x.half(), cache)
    with pytest.raises(ValueError):
        ds4idx.quantize_latents(x, cache[:, :400])
    with pytest.raises(ValueError):
        ds4idx.quantize_latents(x[:, :512], cache)
    shifted = torch.zeros(8 * 416 + 16, dtype=torch.uint8, device="cuda")[16:].view(8, 416)
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.quantize_latents(x, shifted)
