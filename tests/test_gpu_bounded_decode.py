"""The decode loop of examples/bounded_decode.py: after several evictions every row of every cache is
the one written for its position, the totals are the sums of the weights, and a step's attention is
the definition's over the selected rows (tolerances as in test_gpu_sparse_attn_q4)."""
import numpy as np
import pytest
import torch

from examples import bounded_decode
from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref
from .test_gpu_sparse_attn_q4 import _check

pytestmark = pytest.mark.gpu


def test_rows_totals_and_attention_stay_right():
    written, totals, kept_sizes = {}, {}, []

    def on_step(step, cache, q, idx, out, lse, weights):
        s, n = cache.start, cache.rows
        pos = cache.position[s:s + n].cpu().numpy()
        rows = cache.latents[s:s + n].cpu().numpy()
        keys = cache.keys[s:s + n].cpu().numpy()
        assert np.all(np.diff(pos) > 0)
        for p, r, k in zip(pos.tolist(), rows, keys):
            have = written.setdefault(p, (r.copy(), k.copy()))
            assert np.array_equal(have[0], r) and np.array_equal(have[1], k), (step, p)
        i, w = idx[0].cpu().numpy(), weights[0].cpu().numpy()
        for j in np.flatnonzero(i >= 0):
            p = int(pos[i[j]])
            totals[p] = totals.get(p, 0) + int(np.rint(np.float64(w[j]) * 2.0 ** 32))
        got = cache.totals[s:s + n].cpu().numpy()
        assert got.tolist() == [totals.get(p, 0) for p in pos.tolist()]
        assert abs(float(w.sum()) - 128) < 1e-2
        if step % 40 == 7:
            pool = np.where(i >= 0, i, -1).astype(np.int64)[None]
            _check(q.cpu(), rows, pool, 576 ** -0.5, out, lse, weights)
        kept_sizes.append(n)

    cache = bounded_decode.run(prefill=700, steps=200, budget=600, slack=30, on_step=on_step)
    assert max(kept_sizes) <= cache.half and kept_sizes.count(601) >= 2    # evicted twice or more
    pos = cache.position[cache.start:cache.start + cache.rows].tolist()
    assert pos[:4] == [0, 1, 2, 3] and pos[-1] == 899                     # sinks, and the last token
    assert ref.ROW_BYTES == ds4idx.Q4_ROW_BYTES
    torch.cuda.synchronize()
