"""The 8-bit latent cache's writer and reader: bytes and values equal to the definition, exactly."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import tree_reference as ref

pytestmark = pytest.mark.gpu


def _want(x):
    rope = x[:, 512:].to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return ref.quantize_f8(x.double().numpy(), rope)


def _rows(n, dtype, seed):
    """Rows with wide ranges, zeros of both signs, exact ties, maxima at a scale's border, rows below the
    least and above the largest scale."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 576, generator=g) * torch.exp(2 * torch.randn(n, 1, generator=g))
    x[0, :512] = 2.0 ** torch.arange(512).remainder(20).float() * (torch.arange(512) % 17 - 8)
    if n > 8:
        x[1] = 0
        x[2] = -0.0
        # ties: halfway between two codes at scale 1, subnormal ones among them
        c = torch.arange(512) % 126
        t = torch.from_numpy((ref.E4M3[1:] + ref.E4M3[:-1]) / 2)
        x[3, :512] = t[c].float() * (1 - 2 * (torch.arange(512) % 2))
        x[3, 0] = 448.0
        x[4, :512] = 448.0 * 2.0 ** -3         # the border: the smaller scale holds it
        x[5, :512] = 450.0 * 2.0 ** -3         # just past it (bf16 holds 450)
        x[6, :512] *= 2.0 ** -30
        x[7, :512] *= 2.0 ** 16
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 2, 9, 1000])
def test_write_and_read_are_exact(n, dtype):
    x = _rows(n, dtype, n)
    R = n + 5
    cache = torch.full((R, 640), 0xA5, dtype=torch.uint8, device="cuda")
    scale = torch.full((R,), 7.0, device="cuda")
    ds4idx.quantize_latents_fp8(x.cuda(), cache, scale, dst_offset=3)
    got, s = cache.cpu().numpy(), scale.cpu().numpy()
    want, ws = _want(x)
    assert np.array_equal(s[3:3 + n], ws)
    bad = np.argwhere(got[3:3 + n] != want)
    assert bad.size == 0, (bad[:4], got[3:3 + n][tuple(bad[0])], want[tuple(bad[0])])
    assert np.all(got[:3] == 0xA5) and np.all(got[3 + n:] == 0xA5)
    assert np.all(s[:3] == 7) and np.all(s[3 + n:] == 7)
    vals = ref.dequantize_f8(want, ws)
    for out in (torch.bfloat16, torch.float32):
        v = ds4idx.read_latents_fp8(cache, scale, start=3, n=n, dtype=out)
        assert np.array_equal(v.double().cpu().numpy(), vals)


def test_fp32_values_next_to_ties_and_borders():
    t = torch.from_numpy((ref.E4M3[1:] + ref.E4M3[:-1]) / 2).float()
    x = torch.zeros(5, 576)
    x[:3, 0] = 448.0
    x[0, 1:127] = torch.nextafter(t, torch.full_like(t, 500.0))
    x[1, 1:127] = torch.nextafter(t, torch.zeros_like(t))
    x[2, 1:127] = -t
    x[3, 7] = torch.nextafter(torch.tensor(448.0), torch.tensor(500.0))
    x[4, 7] = torch.nextafter(torch.tensor(448.0), torch.tensor(0.0))
    x[:, 512:] = torch.linspace(-3, 3, 64)[None]
    cache = torch.zeros(5, 640, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(5, device="cuda")
    ds4idx.quantize_latents_fp8(x.cuda(), cache, scale)
    want, ws = _want(x)
    assert np.array_equal(scale.cpu().numpy(), ws)
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("n", [1, 5, 333])
def test_slots_and_gathered_rows(n):
    R = 400
    x = _rows(n, torch.bfloat16, 3)
    slots = torch.randperm(R, generator=torch.Generator().manual_seed(n))[:n]
    slots[2::5] = -1
    slots[4::11] = R
    cache = torch.full((R, 640), 0x11, dtype=torch.uint8, device="cuda")
    scale = torch.full((R,), 3.0, device="cuda")
    ds4idx.quantize_latents_fp8(x.cuda(), cache, scale, slots=slots.cuda())
    rows, s = _want(x)
    want, ws = np.full((R, 640), 0x11, np.uint8), np.full(R, 3.0)
    for i, at in enumerate(slots.tolist()):
        if 0 <= at < R:
            want[at], ws[at] = rows[i], s[i]
    assert np.array_equal(cache.cpu().numpy(), want) and np.array_equal(scale.cpu().numpy(), ws)
    v = ds4idx.read_latents_fp8(cache, scale, rows=slots.cuda(), dtype=torch.float32)
    vals = ref.dequantize_f8(rows, s)
    vals[[not 0 <= at < R for at in slots.tolist()]] = 0
    assert np.array_equal(v.double().cpu().numpy(), vals)


def test_every_code_is_read_and_agrees_with_torch():
    codes = torch.arange(512, dtype=torch.int32).to(torch.uint8)
    codes[codes & 127 == 127] = 0           # NaN codes: the writer makes none
    cache = torch.zeros(32, 640, dtype=torch.uint8, device="cuda")
    cache[:, :512] = codes.cuda()
    scale = torch.tensor([2.0 ** e for e in range(-24, 8)], device="cuda")
    v = ds4idx.read_latents_fp8(cache, scale)
    want = codes.view(torch.float8_e4m3fn).double()[None] * scale.cpu().double()[:, None]
    assert torch.equal(v[:, :512].double().cpu(), want)


def test_no_rows_and_other_streams():
    cache = torch.zeros(4, 640, dtype=torch.uint8, device="cuda")
    scale = torch.ones(4, device="cuda")
    ds4idx.quantize_latents_fp8(torch.zeros(0, 576, device="cuda"), cache, scale)
    assert ds4idx.read_latents_fp8(cache, scale, n=0).shape == (0, 576)
    x = _rows(4, torch.float32, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ds4idx.quantize_latents_fp8(x.cuda(), cache, scale, stream=s)
    v = ds4idx.read_latents_fp8(cache, scale, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert np.array_equal(v.double().cpu().numpy(), ref.dequantize_f8(*_want(x)))
