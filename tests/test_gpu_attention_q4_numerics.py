"""Attention over the 4-bit cache at scores of any size."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from .test_gpu_sparse_attn_q4 import _cache, _lists, _q

pytestmark = pytest.mark.gpu


def _run(q, rows, idx, scale):
    out, lse, w = ds4idx.sparse_attention_q4(q.cuda(), torch.from_numpy(rows).cuda(),
                                             torch.from_numpy(idx).cuda(), scale, want_weights=True)
    ds4idx.sparse_attention_status()
    return out, lse, w


@pytest.mark.parametrize("T", [4, 30, 60, 300])      # clusters of 8, 4 and 2 CTAs a token, and one
@pytest.mark.parametrize("H", [1, 5, 128])
@pytest.mark.parametrize("kind", ["spread", "close"])
def test_weights_of_a_token_sum_to_the_number_of_heads(T, H, kind):
    """A head's weights are the terms of its sum l, each times 1 / l. l is a chain of at most 64 sums
    of two terms a thread, then of 4 threads and of up to 8 CTAs at 16 terms a thread: at most 67
    roundings of 2^-24 relative. 1 / l and the product add one each, the sum over the heads 5 + 2:
    76, and 80 with the products of these. What underflows is below 2^-126 an entry."""
    R = 900
    rows = _cache(R, 21)
    q = _q(T, H, 22 + H, scale=200.0)                # scores of several hundred, one key dominates
    if kind == "close":                              # every score near +-1280, many keys matter
        q = _q(T, H, 22 + H, scale=1.0)
        q[:, :, 512:] = torch.where(torch.arange(T)[:, None, None] % 2 == 0, 20.0, -20.0)
        rope = np.full((R, 64), 0x41A0, np.uint16)   # 20 in bf16
        rows[:, 288:] = rope.view(np.uint8)
    idx = _lists(T, 512, R, 23, [512, 300, 77, 1])
    _, lse, w = _run(q, rows, idx, 0.05)
    assert float(lse.abs().max()) > 500
    off = np.abs(w.double().cpu().numpy().sum(axis=1) - H)
    assert np.all(off <= 80 * 2.0 ** -24 * H + 512 * H * 2.0 ** -126), off.max() / H
