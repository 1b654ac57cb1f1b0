"""Attention over the 4-bit cache at scores of any size, NaN and infinities among them."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref
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


def _definition(q, kv, pool, scale):
    """lse, out and weights in 64 bits, infinities and NaN as the formulas give them."""
    T, H, _ = q.shape
    lse, out = np.full((T, H), -np.inf), np.zeros((T, H, 512))
    w = np.zeros(pool.shape)
    with np.errstate(all="ignore"):
        for t in range(T):
            use = np.flatnonzero(pool[t] >= 0)
            if use.size:
                k = kv[pool[t][use]]
                s = scale * (q[t][:, None, :] * k[None]).sum(axis=2)
                lse[t] = np.logaddexp.reduce(s, axis=1)
                p = np.exp(s - lse[t][:, None])
                out[t] = (p[:, :, None] * k[None, :, :512]).sum(axis=1)
                w[t, use] = p.sum(axis=0)
    return lse, out, w


def _class(x):
    return np.select([np.isnan(x), np.isposinf(x), np.isneginf(x)], [0, 1, 2], 3)


@pytest.mark.parametrize("T", [8, 30, 60, 300])      # clusters of 8, 4 and 2 CTAs a token, and one
def test_nan_and_infinite_scores_follow_the_formulas(T):
    H, R, n_sel = 7, 300, 130
    rows = _cache(R, 31)
    rope = rows[:, 288:].copy().view(np.uint16)
    rope[7, 3] = 0x7FC0                              # NaN
    rope[8, 10] = 0x7F80                             # +infinity: scores of both signs over the heads
    rows[:, 288:] = rope.view(np.uint8)
    q = _q(T, H, 32)
    idx = _lists(T, n_sel, R - 50, 33, [n_sel, 70, 9])
    idx = np.where(idx >= 0, idx + 50, idx)          # none of rows 0..49 yet
    clean_q, clean_idx = q.clone(), idx.copy()
    for t in range(T):
        kind = t % 8
        if kind == 1:
            q[t, 3, 5] = float("nan")
        if kind in (2, 6):
            idx[t, 64] = 7
        if kind in (3, 6):
            idx[t, 0] = 8
        if kind == 4:                                # one key, of infinite score, is the whole list
            idx[t] = -1
            idx[t, 99] = 8
        if kind == 5:                                # an empty list and a NaN query
            idx[t] = -1
            q[t, 0] = float("nan")
        if kind == 7:
            q[t, 2, 530] = float("inf")
        clean_idx[t] = np.where(idx[t] >= 50, idx[t], -1)
    out, lse, w = (x.double().cpu().numpy() for x in _run(q, rows, idx, 0.04))
    out2, lse2, _ = (x.double().cpu().numpy() for x in _run(clean_q, rows, clean_idx, 0.04))
    want = _definition(q.double().numpy(), ref.dequantize(rows), idx.astype(np.int64), 0.04)
    assert set(np.unique(_class(want[0]))) == {0, 1, 2, 3}
    assert np.array_equal(_class(lse), _class(want[0]))
    assert np.array_equal(_class(out), _class(want[1]))
    assert np.array_equal(_class(w), _class(want[2]))
    assert np.all(out[5::8] == 0) and np.all(w[5::8] == 0)
    fine = np.isfinite(want[0])                      # a key of score -infinity counts for nothing
    assert np.array_equal(lse[fine], lse2[fine]) and np.array_equal(out[fine], out2[fine])
