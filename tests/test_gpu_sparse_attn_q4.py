"""Attention over the selected rows of a 4-bit latent cache against the definition in 64 bits.

Tolerance. A score is 576 products added in fp32 in 36 steps of 16, each step off by at most
2^-22 of A = sm_scale * sum |q_i k_i| (also with truncating adders): d = 36 * 2^-22 * A. Its
product with log2 e, the subtraction of the maximum and the exponential add 2^-20 (1 + |s|), with
|s| <= A. A probability is off by 2 (d + 2^-20 (1 + A)) relative (itself and the sum), plus half a bf16 step,
2^-8, before the value product; the output by half a bf16 step more. Probabilities below 2^-126, the
least normal fp32 and bf16 number, may count as zero. lse: d + 2^-20 (1 + A)."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as ref

pytestmark = pytest.mark.gpu


def _cache(R, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, 576, generator=g) * torch.exp(0.5 * torch.randn(R, 1, generator=g)))
    x = x.to(torch.bfloat16)
    rope = x[:, 512:].contiguous().view(torch.int16).numpy().view(np.uint16)
    return ref.quantize(x.double().numpy(), rope)


def _lists(T, n_sel, R, seed, counts):
    rng = np.random.default_rng(seed)
    idx = np.full((T, n_sel), -1, np.int32)
    for t in range(T):
        n = min(counts[t % len(counts)], n_sel, R)
        idx[t, rng.choice(n_sel, n, replace=False)] = rng.choice(R, n, replace=False)
    return idx


def _q(T, H, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(T, H, 576, generator=g)).to(torch.bfloat16)


def _check(q, rows_bytes, pool, scale, out, lse, w):
    qd = q.double().numpy()
    o_ref, l_ref, w_ref, av, big = ref.attention(qd, ref.dequantize(rows_bytes), pool, scale)
    d = 36 * 2.0 ** -22 * big + 2.0 ** -20 * (1 + big)      # [T, H]
    o = out.double().cpu().numpy()
    under = 512 * 2.0 ** -126 * np.abs(ref.dequantize(rows_bytes)).max()
    bound = (2.0 ** -8 + 2 * d[:, :, None]) * av
    bound = bound + 2.0 ** -8 * (np.abs(o_ref) + bound) + under
    err = np.abs(o - o_ref)
    bad = np.argwhere(~(err <= bound))
    assert bad.size == 0, (bad[:3], err[tuple(bad[0])], bound[tuple(bad[0])])
    ll = lse.double().cpu().numpy()
    none = np.isneginf(l_ref)
    assert np.array_equal(np.isneginf(ll), none)
    assert np.all(np.abs(ll[~none] - l_ref[~none]) <= d[~none])
    if w is not None:
        ww = w.double().cpu().numpy()
        rel = 2 * d.max(axis=1)[:, None] + 2.0 ** -20
        assert np.all(np.abs(ww - w_ref) <= rel * w_ref + 1e-30)
        assert np.all(ww[pool < 0] == 0)


# one case for every cluster size and both sides of its borders; ragged and empty lists
@pytest.mark.parametrize("T,H,n_sel,counts", [
    (1, 128, 512, [512]), (1, 1, 1, [1]), (2, 128, 1, [1, 0]), (3, 37, 65, [65, 1, 0]),
    (16, 128, 512, [512, 0, 1, 63, 64, 65, 300, 511]), (17, 16, 512, [512, 130, 0, 7]),
    (32, 128, 200, [200, 128, 129, 1]), (33, 128, 512, [512, 256, 257, 0, 31]),
    (76, 64, 512, [512, 100]), (77, 128, 512, [512, 255, 1, 0, 257]),
    (15, 128, 512, [512, 449]), (36, 128, 300, [300, 0, 200]), (37, 128, 512, [512, 9]),
    (160, 128, 512, [512, 500, 32]), (90, 5, 33, [33, 0, 9]),
    # several tokens a CTA, empty ones first, last and in a row
    (470, 16, 512, [0, 0, 512, 3, 0, 300, 257]), (460, 128, 512, [512, 511, 64, 1, 129]),
])
def test_matches_definition(T, H, n_sel, counts):
    R = 3001
    rows = _cache(R, 11)
    idx = _lists(T, n_sel, R, T + n_sel, counts)
    q = _q(T, H, T)
    scale = 576 ** -0.5
    args = (q.cuda(), torch.from_numpy(rows).cuda(), torch.from_numpy(idx).cuda(), scale)
    out, lse, w = ds4idx.sparse_attention_q4(*args, want_weights=True)
    ds4idx.sparse_attention_status()
    _check(q, rows, idx.astype(np.int64), scale, out, lse, w)
    # without the weights, and again: the same bits
    out2, lse2, w2 = ds4idx.sparse_attention_q4(*args)
    assert w2 is None and torch.equal(out, out2) and torch.equal(lse, lse2)
    _, _, w3 = ds4idx.sparse_attention_q4(*args, want_weights=True)
    assert torch.equal(w, w3)


@pytest.mark.parametrize("T", [4, 20, 50, 100])
def test_large_scores_and_one_dominant_key(T):
    R = 700
    rows = _cache(R, 5)
    idx = _lists(T, 512, R, 3, [512, 400])
    q = _q(T, 128, 9, scale=60.0)
    out, lse, w = ds4idx.sparse_attention_q4(q.cuda(), torch.from_numpy(rows).cuda(),
                                             torch.from_numpy(idx).cuda(), 0.05, want_weights=True)
    ds4idx.sparse_attention_status()
    _check(q, rows, idx.astype(np.int64), 0.05, out, lse, w)


@pytest.mark.parametrize("T", [5, 24, 40, 90])
def test_empty_entries_read_nothing(T):
    # rows that no list names hold NaN and infinity in their rotary dims, row 0 among them
    R = 600
    rows = _cache(R, 6)
    rope = rows[:, 288:].copy().view(np.uint16)
    rope[0, :] = 0x7FC0
    rope[300:, ::2] = 0xFF80
    rows[:, 288:] = rope.view(np.uint8)
    idx = _lists(T, 512, 298, 4, [250, 0, 3])
    idx = np.where(idx >= 0, idx + 1, idx)
    idx[0, 0] = R + 5          # outside the pool: empty
    q = _q(T, 128, 2)
    out, lse, w = ds4idx.sparse_attention_q4(q.cuda(), torch.from_numpy(rows).cuda(),
                                             torch.from_numpy(idx).cuda(), 0.04, want_weights=True)
    ds4idx.sparse_attention_status()
    pool = np.where(idx < R, idx, -1).astype(np.int64)
    clean = rows.copy()
    clean[0] = clean[1]
    clean[300:] = clean[1]
    _check(q, clean, pool, 0.04, out, lse, w)


@pytest.mark.parametrize("T,page", [(9, 48), (30, 1), (81, 64)])
def test_paged_pool_with_bad_pages(T, page):
    n_seqs, S = 4, 500
    pages = -(-S // page)
    rng = np.random.default_rng(page)
    n_pages = n_seqs * pages + 3
    rows = _cache(n_pages * page, 8)
    table = rng.permutation(n_pages)[:n_seqs * pages].reshape(n_seqs, pages).astype(np.int32)
    table[1, 2] = -1
    table[2, 0] = n_pages + 7
    seq = rng.integers(0, n_seqs, T).astype(np.int32)
    seq[0] = n_seqs            # no such table row: all entries empty
    if T > 4:
        seq[3] = -2
    idx = _lists(T, 512, S, 2, [400, 17])
    idx[5 % T, 0] = pages * page + 1     # past the table row
    q = _q(T, 32, 3)
    out, lse, w = ds4idx.sparse_attention_q4(
        q.cuda(), torch.from_numpy(rows).cuda(), torch.from_numpy(idx).cuda(), 0.04,
        page_table=torch.from_numpy(table).cuda(), page_size=page,
        token_seq=torch.from_numpy(seq).cuda(), want_weights=True)
    ds4idx.sparse_attention_status()
    pool = np.full(idx.shape, -1, np.int64)
    for t in range(T):
        for j, s in enumerate(idx[t]):
            if s >= 0 and 0 <= seq[t] < n_seqs and s // page < pages:
                pg = int(table[seq[t], s // page])
                r = pg * page + s % page
                if pg >= 0 and r < rows.shape[0]:
                    pool[t, j] = r
    _check(q, rows, pool, 0.04, out, lse, w)


def test_rows_past_32_bit_offsets():
    # 5.3 M rows: byte offsets beyond 2^31
    R = 5_300_000
    rows = _cache(600, 12)
    cache = torch.zeros(R, 416, dtype=torch.uint8, device="cuda")
    cache[R - 600:] = torch.from_numpy(rows).cuda()
    for T in (2, 80):
        idx = _lists(T, 512, 600, 5, [512, 30])
        q = _q(T, 128, 4)
        row0 = torch.full((T,), R - 600, dtype=torch.int64, device="cuda")
        out, lse, w = ds4idx.sparse_attention_q4(q.cuda(), cache, torch.from_numpy(idx).cuda(), 0.04,
                                                 kv_row0=row0, want_weights=True)
        ds4idx.sparse_attention_status()
        _check(q, rows, idx.astype(np.int64), 0.04, out, lse, w)


def test_side_stream_and_graph():
    for T in (4, 90):
        rows = _cache(700, 1)
        cache = torch.from_numpy(rows).cuda()
        idx = torch.from_numpy(_lists(T, 512, 700, 6, [512])).cuda()
        q = _q(T, 128, 5).cuda()
        want, lse, _ = ds4idx.sparse_attention_q4(q, cache, idx, 0.04)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out, l2 = torch.empty_like(want), torch.empty_like(lse)
        ds4idx.sparse_attention_q4(q, cache, idx, 0.04, out=out, lse=l2, stream=s)
        ds4idx.sparse_attention_status(s)
        assert torch.equal(out, want) and torch.equal(l2, lse)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ds4idx.sparse_attention_q4(q, cache, idx, 0.04, out=out, lse=l2)
        out.zero_()
        g.replay()
        ds4idx.sparse_attention_status()
        assert torch.equal(out, want)


def test_refusals_and_empty_call():
    q = torch.zeros(2, 128, 576, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(10, 416, dtype=torch.uint8, device="cuda")
    idx = torch.zeros(2, 512, dtype=torch.int32, device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    f = ds4idx.sparse_attention_q4
    out, lse, _ = f(q[:0], cache, idx[:0], 1.0)
    assert out.shape == (0, 128, 512)
    for bad in (dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(q=q.repeat(1, 2, 1)),
                dict(idx=idx.repeat(1, 2)), dict(page_table=table, page_size=5)):
        a = dict(q=q, cache=cache, idx=idx, sm_scale=1.0)
        a.update(bad)
        with pytest.raises(ds4idx.Ds4IdxError):
            f(**a)
    with pytest.raises(ds4idx.Ds4IdxError):
        f(q, cache, idx, 1.0, page_table=table, page_size=0, token_seq=seq)
    with pytest.raises(ValueError):
        f(q, cache, idx, 1.0, token_seq=seq)
    with pytest.raises(ValueError):
        f(q, cache, idx, 1.0, kv_row0=torch.zeros(2, dtype=torch.int64, device="cuda"),
          page_table=table, page_size=5)
    with pytest.raises(TypeError):
        f(q.float(), cache, idx, 1.0)
    with pytest.raises(ValueError):
        f(q[:, :, :512], cache, idx, 1.0)
