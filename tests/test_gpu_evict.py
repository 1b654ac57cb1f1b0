"""Accumulated attention weight and eviction by it: whole numbers, equal to the definition."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,n_sel,R", [(1, 1, 1), (3, 300, 50), (64, 512, 900), (700, 33, 40)])
def test_accumulate_is_exact_with_collisions(T, n_sel, R):
    rng = np.random.default_rng(T)
    w = (rng.random((T, n_sel)) * 128).astype(np.float32)
    w.flat[::7] = 2.0 ** -33                   # a tie of the rounding: to even, 0
    w.flat[::11] *= -1
    idx = rng.integers(-3, R + 3, (T, n_sel)).astype(np.int32)
    row0 = rng.integers(0, 4, T).astype(np.int64)
    w[0, 0] = np.nan if T > 1 else w[0, 0]     # adds nothing
    if n_sel > 5:
        w[0, 1], w[0, 2], w[0, 3] = np.inf, 2.0 ** 30, 2.0 ** 30 - 64
    total = rng.integers(-(1 << 50), 1 << 50, R).astype(np.int64)
    want = total.copy()
    for t in range(T):
        for j in range(n_sel):
            r = int(idx[t, j]) + int(row0[t])
            if idx[t, j] >= 0 and r < R and abs(w[t, j]) < 2.0 ** 30:
                want[r] += int(np.rint(np.float64(w[t, j]) * 2.0 ** 32))
    got = torch.from_numpy(total).cuda()
    ds4idx.evict_accumulate(got, torch.from_numpy(w).cuda(), torch.from_numpy(idx).cuda(),
                            kv_row0=torch.from_numpy(row0).cuda())
    assert np.array_equal(got.cpu().numpy(), want)


def test_accumulate_through_a_page_table():
    T, page, n_seqs, pages = 10, 7, 3, 9
    rng = np.random.default_rng(0)
    table = rng.permutation(40)[:27].reshape(n_seqs, pages).astype(np.int32)
    seq = rng.integers(0, n_seqs, T).astype(np.int32)
    idx = rng.integers(-1, page * pages + 2, (T, 20)).astype(np.int32)
    w = rng.random((T, 20)).astype(np.float32)
    want = np.zeros(280, np.int64)
    for t in range(T):
        for j in range(20):
            s = int(idx[t, j])
            if 0 <= s < page * pages:
                want[table[seq[t], s // page] * page + s % page] += int(np.rint(float(w[t, j]) * 2 ** 32))
    got = torch.zeros(280, dtype=torch.int64, device="cuda")
    ds4idx.evict_accumulate(got, torch.from_numpy(w).cuda(), torch.from_numpy(idx).cuda(),
                            page_table=torch.from_numpy(table).cuda(), page_size=page,
                            token_seq=torch.from_numpy(seq).cuda())
    assert np.array_equal(got.cpu().numpy(), want)


def _totals(kind, R, rng):
    if kind == "wide":
        return rng.integers(-(1 << 62), 1 << 62, R).astype(np.int64)
    if kind == "extremes":
        return rng.choice(np.array([-(1 << 63), (1 << 63) - 1, 0, -1, 1], np.int64), R)
    if kind == "zeros":
        return np.zeros(R, np.int64)
    if kind == "mostly zeros":
        return np.where(rng.random(R) < 0.9, 0, rng.integers(0, 1 << 40, R)).astype(np.int64)
    if kind == "few":
        return rng.integers(5, 9, R).astype(np.int64)
    return np.exp(rng.random(R) * 25).astype(np.int64)


@pytest.mark.parametrize("kind", ["wide", "extremes", "zeros", "mostly zeros", "few", "log"])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([10], [3], 0, 0), ([10], [1], 1, 0), ([10], [9], 4, 5), ([5, 0, 7], [5, 2, 9], 1, 1),
    ([300, 4096, 1], [150, 4095, 1], 0, 1), ([4097, 100], [2000, 99], 4, 60),
    ([40001, 9000, 20000], [31000, 100, 20000], 3, 77),
    # every cluster size, and past what stays on chip
    ([16384], [16383], 0, 0), ([16385, 17], [9000, 16], 0, 3), ([70000], [1], 0, 0),
    ([140001, 5], [70000, 13], 4, 9), ([262150], [131000], 4, 64),
])
def test_select_matches_definition(lens, keep, sink, recent, kind):
    rng = np.random.default_rng(len(lens) + lens[0])
    starts, R = [], 3
    for n in lens:
        starts.append(R)
        R += n + 2
    total = _totals(kind, R, rng)
    kept = ds4idx.evict_select(torch.from_numpy(total).cuda(), starts, lens, keep, n_sink=sink,
                               n_recent=recent).cpu().numpy()
    for b, (s, n, k) in enumerate(zip(starts, lens, keep)):
        want = ref.evict_select(total, s, n, k, sink, recent)
        assert kept[b, :len(want)].tolist() == want, (b, kind)
        assert np.all(kept[b, len(want):] == -1)


@pytest.mark.parametrize("row_shapes", [[(416,), (128,), (), (3,)], [(1,), (7,), (2, 5)], [(40000,)]])
def test_compact_moves_whole_rows(row_shapes):
    rng = np.random.default_rng(5)
    lens, keep = [700, 0, 33, 1500], [300, 4, 40, 1499]
    starts = [5, 705, 705, 800]
    R = 2400
    total = rng.integers(0, 50, R).astype(np.int64)
    kept = ds4idx.evict_select(torch.from_numpy(total).cuda(), starts, lens, keep, 2, 2)
    counts = [min(a, b) for a, b in zip(keep, lens)]
    dst = [10, 320, 330, 400]
    dtypes = [torch.uint8, torch.uint8, torch.float32, torch.int64]
    srcs, dsts = [], []
    for sh, dt in zip(row_shapes, dtypes):
        src = torch.from_numpy(rng.integers(0, 200, (R, *sh))).to(dt).cuda()
        srcs.append(src)
        dsts.append(torch.full((1950, *sh), 77, dtype=dt, device="cuda"))
    ds4idx.evict_compact(kept, lens, keep, starts, dst, srcs, dsts)
    k = kept.cpu().numpy()
    for s, d in zip(srcs, dsts):
        want = np.full(tuple(d.shape), 77, d.cpu().numpy().dtype)
        for b, n in enumerate(counts):
            want[dst[b]:dst[b] + n] = s.cpu().numpy()[starts[b] + k[b, :n]]
        assert np.array_equal(d.cpu().numpy(), want)


def test_compact_within_one_pool_and_refused_overlap():
    pool = torch.arange(100, dtype=torch.int64, device="cuda")
    total = pool.clone()
    kept = ds4idx.evict_select(total, [0], [40], [10])
    ds4idx.evict_compact(kept, [40], [10], [0], [60], [pool], [pool])
    assert pool[60:70].tolist() == list(range(30, 40))
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.evict_compact(kept, [40], [10], [0], [35], [pool], [pool])


def test_select_graph_and_refusals():
    total = torch.arange(9000, dtype=torch.int64, device="cuda")
    kept = torch.empty(1, 100, dtype=torch.int32, device="cuda")
    ds4idx.evict_select(total, [0], [9000], [100], kept=kept)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ds4idx.evict_select(total, [0], [9000], [100], kept=kept)
    total.neg_()
    g.replay()
    assert kept[0].tolist() == list(range(100))
    bad = [dict(starts=[1], seq_lens=[9000], keep=[5]), dict(starts=[0], seq_lens=[-1], keep=[5]),
           dict(starts=[0], seq_lens=[10], keep=[3], n_sink=2, n_recent=2),
           dict(starts=[0], seq_lens=[10], keep=[-1]),
           dict(starts=[0], seq_lens=[10], keep=[7], kept=kept[:, :5].contiguous()),
           dict(starts=[0] * 65, seq_lens=[1] * 65, keep=[1] * 65)]
    for a in bad:
        with pytest.raises(ds4idx.Ds4IdxError):
            ds4idx.evict_select(total, **a)
    with pytest.raises(TypeError):
        ds4idx.evict_select(total.int(), [0], [10], [5])
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.evict_compact(kept, [9000], [100], [0], [9950], [total], [torch.zeros_like(total)])
