"""Sparse attention over bf16 rows: lse and out of lists with a NaN or infinite score follow the
formulas, so that joining shards by lse does not take such a list for an empty one."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from .test_gpu_sparse_attn import H, _inputs

pytestmark = pytest.mark.gpu


def test_nan_and_infinite_scores_follow_the_formulas():
    T, R = 12, 900
    q, kv, idx = _inputs(T, R - 50, seed=3, n_valid=[512, 200, 9])
    idx = np.where(idx >= 0, idx + 50, idx)             # none of rows 0..49
    kv[7, 520] = float("nan")
    kv[8, 530] = float("inf")                           # scores of both signs over the heads
    clean_q, clean_idx = q.clone(), idx.copy()
    q[1, 3, 5] = float("nan")
    idx[2, 64] = 7
    idx[3, 0] = 8
    idx[4] = -1                                         # one key, of infinite score
    idx[4, 99] = 8
    idx[5] = -1                                         # an empty list
    q[5, 0] = float("nan")
    clean_idx[4] = clean_idx[5] = -1
    clean_idx[3, 0] = -1                                # the slot that the infinite key takes
    call = lambda q, i: [x.float().cpu().numpy() for x in ds4idx.sparse_attention(  # noqa: E731
        q.cuda(), kv.cuda(), torch.from_numpy(i).cuda(), 0.04)]
    out, lse = call(q, idx)
    ds4idx.sparse_attention_status()
    out2, lse2 = call(clean_q, clean_idx)
    assert np.isnan(lse[1, 3]) and np.isnan(out[1, 3]).all()
    assert np.isnan(lse[2]).all() and np.isnan(out[2]).all()
    up = q[3, :, 530].float().numpy() > 0
    assert 0 < up.sum() < H
    assert np.isposinf(lse[3, up]).all() and np.isnan(out[3, up]).all()
    up = q[4, :, 530].float().numpy() > 0
    assert np.isposinf(lse[4, up]).all() and np.isneginf(lse[4, ~up]).all() and np.isnan(out[4]).all()
    assert np.isneginf(lse[5]).all() and np.all(out[5] == 0)
    fine = np.isfinite(lse)                             # a key of score -infinity counts for nothing
    fine_want = np.isfinite(lse2)
    fine_want[1, 3] = False
    fine_want[2] = False
    fine_want[3] &= ~(q[3, :, 530].float().numpy() > 0)
    assert np.array_equal(fine, fine_want)
    assert np.array_equal(lse[fine], lse2[fine]) and np.array_equal(out[fine], out2[fine])
