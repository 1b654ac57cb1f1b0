"""Decode with a bounded cache: rotary positions, the 4-bit latent cache, the indexer, sparse
attention over the selected rows, accumulated attention weight and eviction, in the order of use.

One sequence with synthetic projections. Each step rotates the new token's queries and keys, writes
its latent row (4 bits) and its index key (FP8), selects up to 512 rows, attends over them and adds
the weight that every row received to its total. When the cache holds ``budget + slack`` rows it is
cut to ``budget``: the first ``sink``, the last ``recent`` and the rows with the largest totals.
The kept rows move to the other half of the pool.

    python examples/bounded_decode.py [--prefill 1500] [--steps 400] [--budget 1024]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_attention_lightning_indexer_gb300 import ds4idx  # noqa: E402

HEADS, LATENT, ROPE, INDEX = 128, 512, 64, 128


class BoundedCache:
    """The rows of one sequence in one half of a pool: 4-bit latents, FP8 index keys and scales,
    attention totals, and each row's position in the text."""

    def __init__(self, budget: int, slack: int, sink: int = 4, recent: int = 64):
        self.budget, self.sink, self.recent = budget, sink, recent
        self.half = budget + slack
        r, dev = 2 * self.half, "cuda"
        self.latents = torch.zeros(r, ds4idx.Q4_ROW_BYTES, dtype=torch.uint8, device=dev)
        self.keys = torch.zeros(r, INDEX, dtype=torch.uint8, device=dev)
        self.scales = torch.zeros(r, device=dev)
        self.totals = torch.zeros(r, dtype=torch.int64, device=dev)
        self.position = torch.full((r,), -1, dtype=torch.int64, device=dev)
        self.start, self.rows, self.text = 0, 0, 0    # text: tokens seen

    def append(self, latents, index_keys):
        n = latents.shape[0]
        if self.rows + n > self.half:
            raise ValueError("the cache is full: evict first")
        at = self.start + self.rows
        ds4idx.quantize_latents(latents, self.latents, dst_offset=at)
        ds4idx.quantize_keys(index_keys, self.keys, self.scales, dst_offset=at)
        self.totals[at:at + n] = 0
        self.position[at:at + n] = torch.arange(self.text, self.text + n, device="cuda")
        self.rows += n
        self.text += n

    def evict(self):
        if self.rows <= self.budget:
            return
        kept = ds4idx.evict_select(self.totals, [self.start], [self.rows], [self.budget],
                                   n_sink=self.sink, n_recent=self.recent)
        arrays = [self.latents, self.keys, self.scales, self.totals, self.position]
        other = self.half - self.start        # 0 <-> half
        ds4idx.evict_compact(kept, [self.rows], [self.budget], [self.start], [other], arrays, arrays)
        self.start, self.rows = other, self.budget


def project(n: int, g: torch.Generator):
    """Synthetic projections of n tokens: attention query, latent row, index query, weights, key."""
    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    return (r(n, HEADS, LATENT + ROPE).to(torch.bfloat16), r(n, LATENT + ROPE).to(torch.bfloat16),
            r(n, ds4idx.H_I, INDEX), r(n, ds4idx.H_I) / ds4idx.H_I, r(n, INDEX))


def run(prefill: int, steps: int, budget: int, slack: int = 64, seed: int = 0, on_step=None):
    """Returns the cache after ``steps`` decode steps. on_step(step, cache, q, idx, out, lse, weights)
    is called after each one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    freqs = ds4idx.rotary_freqs(ROPE, 10000.0, scaling="yarn", factor=40.0)
    cache = BoundedCache(budget, max(slack, prefill - budget))
    scale = (LATENT + ROPE) ** -0.5

    def rotate(q, latent, iq, ik, first):
        """The rotated slices in place: interleaved pairs for the attention, halves for the
        indexer."""
        pos = torch.arange(first, first + latent.shape[0], device="cuda")
        views = [q[..., LATENT:], latent[:, LATENT:], iq[..., :ROPE], ik[:, :ROPE]]
        ds4idx.rotary(views, pos, freqs, interleaved=[True, True, False, False], outs=views)

    q, latent, iq, _, ik = project(prefill, g)
    rotate(q, latent, iq, ik, 0)
    cache.append(latent, ik)
    with ds4idx.Indexer(ds4idx.FP8_E4M3, max_T=1, max_S=cache.half) as indexer:
        for step in range(steps):
            if cache.rows == cache.half:
                cache.evict()
            q, latent, iq, iw, ik = project(1, g)
            rotate(q, latent, iq, ik, cache.text)
            cache.append(latent, ik)
            s, n = cache.start, cache.rows
            qc, w, _ = ds4idx.quantize_queries(iq, iw)
            idx, _ = indexer.score_topk(qc, w, cache.keys[s:s + n], cache.scales[s:s + n],
                                        pos_offset=n - 1)
            row0 = torch.full((1,), s, dtype=torch.int64, device="cuda")
            out, lse, weights = ds4idx.sparse_attention_q4(q, cache.latents, idx, scale,
                                                           kv_row0=row0, want_weights=True)
            ds4idx.evict_accumulate(cache.totals, weights, idx, kv_row0=row0)
            if on_step is not None:
                on_step(step, cache, q, idx, out, lse, weights)
        indexer.sync_status()
    ds4idx.sparse_attention_status()
    return cache


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--prefill", type=int, default=1500)
    ap.add_argument("--steps", type=int, default=400)
    ap.add_argument("--budget", type=int, default=1024)
    a = ap.parse_args()
    from sparse_attention_lightning_indexer_gb300 import build
    build.build()
    cache = run(a.prefill, a.steps, a.budget)
    pos = cache.position[cache.start:cache.start + cache.rows]
    print(f"{cache.text} tokens seen, {cache.rows} rows kept "
          f"({cache.rows * (ds4idx.Q4_ROW_BYTES + INDEX + 4) / 1e3:.0f} kB), of them "
          f"{int((pos < a.prefill).sum())} from the prefill")


if __name__ == "__main__":
    main()
