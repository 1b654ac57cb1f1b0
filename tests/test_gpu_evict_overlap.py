"""Moves that touch but do not overlap: several arrays in one buffer, shared sources, a pool's other
half."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

pytestmark = pytest.mark.gpu


def test_neighbouring_ranges_are_moved():
    lens, keep, starts, dst = [40, 30, 25], [10, 30, 25], [0, 40, 45], [10, 20, 50]
    counts = [10, 30, 25]
    n_src, n_dst = 70, 75
    rng = np.random.default_rng(4)
    buf = torch.from_numpy(rng.integers(0, 256, (4 * 100, 16))).to(torch.uint8).cuda()
    # every written range begins where another range ends
    srcs = [buf[0:n_src], buf[170:170 + n_src]]
    dsts = [buf[60:60 + n_dst], buf[230:230 + n_dst]]
    before = buf.cpu().numpy().copy()
    total = torch.from_numpy(rng.integers(0, 9, n_src)).cuda()
    kept = ds4idx.evict_select(total, starts, lens, keep)
    ds4idx.evict_compact(kept, lens, keep, starts, dst, srcs, dsts)
    want, k = before.copy(), kept.cpu().numpy()
    for s, d in ((0, 60), (170, 230)):
        for b in range(3):
            rows = s + starts[b] + k[b, :counts[b]]
            want[d + dst[b]:d + dst[b] + counts[b]] = before[rows]
    assert np.array_equal(buf.cpu().numpy(), want)
    with pytest.raises(ds4idx.Ds4IdxError):          # one row earlier: over the first array's source
        ds4idx.evict_compact(kept, lens, keep, starts, [9, 20, 50], srcs, dsts)
    assert np.array_equal(buf.cpu().numpy(), want)
