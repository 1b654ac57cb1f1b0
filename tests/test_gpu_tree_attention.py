"""Attention of drafted trees over a latent cache against the definition in 64 bits.

Tolerance. A score is 576 products added in fp32 in 36 steps of 16, each step off by at most 2^-22 of
A = sm_scale * sum |q_i k_i| (also with truncating adders), and once more where two halves are joined:
37 * 2^-22 * A. Its product with log2 e, the subtraction of a maximum and the exponential add
2^-20 (1 + |s|), |s| <= A: together d. A sum over n rows is taken in steps of at least one row, with
corrections of its scale every 64 rows and a join of parts: at most n 2^-23 + 2^-20 of the sum of
magnitudes, t. A probability is off by 2 d + t relative (itself and the sum), plus half a bf16 step, 2^-8,
before the value product, whose sum adds t. The products are divided by the sum of the rounded terms, whose
mean error is at most another half step: together 2^-7, and the product of two such factors, 2^-16. The
output is off by half a bf16 step more. Probabilities
below 2^-126, the least normal fp32 and bf16 number, may count as zero. lse: d + t."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import latent_reference as q4ref
from . import tree_reference as ref

pytestmark = pytest.mark.gpu


def _cache(kind, R, seed):
    """(cache, scale or None, values float64 on the GPU)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, 576, generator=g) * torch.exp(0.5 * torch.randn(R, 1, generator=g))
    x = x.to(torch.bfloat16)
    if kind == "bf16":
        return x.cuda(), None, x.double().cuda()
    rope = x[:, 512:].contiguous().view(torch.int16).numpy().view(np.uint16)
    if kind == "q4":
        rows = q4ref.quantize(x.double().numpy(), rope)
        return torch.from_numpy(rows).cuda(), None, torch.from_numpy(q4ref.dequantize(rows)).cuda()
    rows, s = ref.quantize_f8(x.double().numpy(), rope)
    return (torch.from_numpy(rows).cuda(), torch.from_numpy(s).float().cuda(),
            torch.from_numpy(ref.dequantize_f8(rows, s)).cuda())


def _masks(B, N, seed, padding=False):
    """Random trees: chains, bushes and several roots; with padding every third node is none."""
    rng = np.random.default_rng(seed)
    res = []
    for b in range(B):
        up = []
        for i in range(N):
            real = [j for j in range(i) if up[j] is not None]
            if padding and (i + b) % 3 == 2:
                up.append(None)
            else:
                up.append(int(rng.choice(real)) if real and rng.random() < 0.8 else -1)
        res.append(ref.tree_masks(up))
    return res


def _q(B, N, H, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(B, N, H, 576, generator=g)).to(torch.bfloat16).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


def _check(q, kv, rows, lens, masks, scale, out, lse):
    o_ref, l_ref, av, big, seen = ref.attention(q.double(), kv, rows, lens, masks, scale)
    d = 37 * 2.0 ** -22 * big + 2.0 ** -20 * (1 + big)
    t = seen * 2.0 ** -23 + 2.0 ** -20
    under = seen[..., None] * 2.0 ** -126 * kv.abs().nan_to_num(0, 0, 0).max()
    bound = (2.0 ** -7 + 2.0 ** -15 + 2 * (d + t)[..., None]) * av
    bound = bound + 2.0 ** -8 * (o_ref.abs() + bound) + under
    err = (out.double() - o_ref).abs()
    bad = (~(err <= bound)).nonzero()
    assert bad.numel() == 0, (bad[:3], err[tuple(bad[0])], bound[tuple(bad[0])])
    none = torch.isneginf(l_ref)
    assert torch.equal(torch.isneginf(lse), none)
    assert bool(((lse.double() - l_ref).abs() <= d + t)[~none].all())
    assert bool((out[none] == 0).all())


def _contiguous(lens, N, gap=3):
    starts, at = [], 2
    for n in lens:
        starts.append(at)
        at += n + N + gap
    rows = [list(range(s, s + n + N)) for s, n in zip(starts, lens)]
    return starts, at, rows


@pytest.mark.parametrize("kind", ["fp8", "bf16", "q4"])
@pytest.mark.parametrize("N,H,lens", [
    (1, 128, [0]), (1, 1, [1]), (1, 128, [63]), (2, 128, [62, 64, 65]), (5, 16, [0, 1, 130, 59]),
    (64, 2, [100, 0, 64]), (64, 16, [777]), (3, 37, [500, 126, 127, 128]), (7, 128, [1300, 3]),
    (13, 128, [4001]), (1, 128, [9000]), (33, 5, [63, 31, 95]),
])
def test_matches_definition(kind, N, H, lens):
    starts, R, rows = _contiguous(lens, N)
    cache, scale, kv = _cache(kind, R, N + H)
    masks = _masks(len(lens), N, N)
    q = _q(len(lens), N, H, H)
    args = (q, cache, _i32(lens), _i64(masks), 576 ** -0.5)
    out, lse = ds4idx.tree_attention(*args, scale=scale, kv_row0=_i64(starts), max_kv_len=max(lens))
    ds4idx.sparse_attention_status()
    _check(q, kv, rows, lens, masks, 576 ** -0.5, out, lse)
    # again, the same bits; and laid out for another length, which is off by no more
    out2, lse2 = ds4idx.tree_attention(*args, scale=scale, kv_row0=_i64(starts), max_kv_len=max(lens))
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for most in (0, None, 100000):
        out2, lse2 = ds4idx.tree_attention(*args, scale=scale, kv_row0=_i64(starts), max_kv_len=most)
        _check(q, kv, rows, lens, masks, 576 ** -0.5, out2, lse2)
    ds4idx.sparse_attention_status()


def test_many_sequences_and_long_ones():
    for lens, N, H in (([700 + 37 * b for b in range(40)], 3, 64), ([20000, 10, 7777], 2, 128)):
        starts, R, rows = _contiguous(lens, N)
        cache, scale, kv = _cache("fp8", R, 5)
        masks = _masks(len(lens), N, 8)
        q = _q(len(lens), N, H, 2)
        out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                         kv_row0=_i64(starts))
        ds4idx.sparse_attention_status()
        _check(q, kv, rows, lens, masks, 0.04, out, lse)


@pytest.mark.parametrize("kind", ["fp8", "bf16", "q4"])
def test_large_scores_and_rising_maxima(kind):
    # every row's score is far above those before it, and the other way round
    lens, N = [900, 900], 4
    starts, R, rows = _contiguous(lens, N)
    cache, scale, kv = _cache(kind, R, 5)
    masks = _masks(2, N, 1)
    q = _q(2, N, 128, 9, scale=60.0)
    out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.05, scale=scale,
                                     kv_row0=_i64(starts))
    ds4idx.sparse_attention_status()
    _check(q, kv, rows, lens, masks, 0.05, out, lse)
    if kind == "bf16":
        g = torch.Generator().manual_seed(3)
        base = torch.randn(576, generator=g)
        ramp = torch.linspace(-4, 4, lens[0] + N)[:, None] * base
        cache[starts[0]:starts[0] + lens[0] + N] = ramp.to(torch.bfloat16).cuda()
        cache[starts[1]:starts[1] + lens[1] + N] = ramp.flip(0).to(torch.bfloat16).cuda()
        q = (q * 0.02 + base.cuda()).to(torch.bfloat16)
        out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.05, kv_row0=_i64(starts))
        _check(q, cache.double(), rows, lens, masks, 0.05, out, lse)


@pytest.mark.parametrize("kind", ["fp8", "bf16", "q4"])
def test_padding_and_unseen_rows_reach_nothing(kind):
    # rows of padding nodes, before and behind the sequences hold NaN and infinity
    lens, N, H = [130, 5, 64], 9, 128
    starts, R, rows = _contiguous(lens, N)
    cache, scale, kv = _cache(kind, R, 6)
    masks = _masks(3, N, 4, padding=True)
    masks[1] = [0] * N
    used = set()
    for b, n in enumerate(lens):
        if any(masks[b]):
            used |= set(rows[b][:n])
        used |= {rows[b][n + j] for j in range(N) if any(m >> j & 1 for m in masks[b])}
    junk = [r for r in range(R) if r not in used]
    assert 0 in junk and R - 1 in junk
    if kind == "bf16":
        cache[junk] = float("nan")
        cache[junk[::2]] = float("inf")
    else:
        at = 512 if kind == "fp8" else 288
        cache[junk, at:] = 0xFF
        if kind == "fp8":
            cache[junk, :512] = 0x7F
            scale[junk] = float("inf")
    kv[junk] = 0
    q = _q(3, N, H, 2)
    out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                     kv_row0=_i64(starts))
    ds4idx.sparse_attention_status()
    _check(q, kv, rows, lens, masks, 0.04, out, lse)


@pytest.mark.parametrize("kind,page", [("fp8", 48), ("q4", 1), ("bf16", 64), ("fp8", 7)])
def test_paged_pool_with_bad_pages(kind, page):
    N, lens = 6, [300, 299, 0, 64 * 3, 250]
    B, n_seqs = len(lens), 7
    pages = -(-(max(lens) + N) // page)
    rng = np.random.default_rng(page)
    n_pages = n_seqs * pages + 3
    cache, scale, kv = _cache(kind, n_pages * page, 8)
    table = rng.permutation(n_pages)[:n_seqs * pages].reshape(n_seqs, pages).astype(np.int32)
    table[1, 2 % pages] = -1
    table[2, 0] = n_pages + 7
    seq = [1, 4, 2, n_seqs, 0]          # the fourth has no such table row
    rows = []
    for b, n in enumerate(lens):
        r = []
        for s in range(n + N):
            id_ = int(table[seq[b], s // page]) if seq[b] < n_seqs else -1
            r.append(id_ * page + s % page if 0 <= id_ < n_pages else -1)
        rows.append(r)
    masks = _masks(B, N, 3)
    q = _q(B, N, 128, 4)
    out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                     page_table=torch.from_numpy(table).cuda(), page_size=page,
                                     token_seq=_i32(seq))
    ds4idx.sparse_attention_status()
    _check(q, kv, rows, lens, masks, 0.04, out, lse)


def test_lengths_past_the_pool_and_odd_starts():
    # what is not there is not seen: a length past the pool or its table row, a start outside it, a
    # negative length
    N, R = 3, 400
    cache, scale, kv = _cache("fp8", R, 2)
    lens, starts = [500, 2 ** 31 - 1, 10, 10, -5, 398], [100, 390, -1, R + 50, 20, 0]
    rows = [[s + i if s >= 0 and s + i < R else -1 for i in range(max(0, min(n, 600)) + N)]
            for n, s in zip(lens, starts)]
    short = [max(0, min(n, 600)) for n in lens]
    masks = _masks(len(lens), N, 3)
    q = _q(len(lens), N, 128, 4)
    out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                     kv_row0=_i64(starts))
    ds4idx.sparse_attention_status()
    _check(q, kv, rows, short, masks, 0.04, out, lse)


def test_masks_of_any_bits():
    # bits of later nodes and the sign bit are only bits; bits past the last node name nothing
    N, lens = 64, [70]
    starts, R, rows = _contiguous(lens, N)
    cache, scale, kv = _cache("fp8", R, 3)
    rng = np.random.default_rng(1)
    masks = [[ref.signed(int(rng.integers(0, 2 ** 64, dtype=np.uint64))) for _ in range(N)]]
    masks[0][5], masks[0][6] = ref.signed(1 << 63), 2
    q = _q(1, N, 16, 4)
    out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                     kv_row0=_i64(starts))
    _check(q, kv, rows, lens, masks, 0.04, out, lse)
    few = 5
    q5 = q[:, :few].contiguous()
    m5 = [[ref.signed((1 << 40) | (1 << i)) for i in range(few)]]
    out, lse = ds4idx.tree_attention(q5, cache, _i32(lens), _i64(m5), 0.04, scale=scale,
                                     kv_row0=_i64(starts))
    _check(q5, kv, [rows[0][:lens[0] + few]], lens, m5, 0.04, out, lse)
    ds4idx.sparse_attention_status()


@pytest.mark.parametrize("n", [40, 300])
def test_scores_that_are_not_finite(n):
    # NaN gives lse, out NaN; +infinity lse +infinity, out NaN; -infinity alone lse -infinity, out NaN
    N, H = 3, 128
    cache = torch.randn(n + N, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    inf = float("inf")

    def run(c, q):
        out, lse = ds4idx.tree_attention(q, c.cuda(), _i32([n]), _i64([[1, 2, 4]]), 0.04)
        ds4idx.sparse_attention_status()
        return out[0], lse[0]

    q = torch.ones(1, N, H, 576, dtype=torch.bfloat16, device="cuda")
    c = cache.clone()
    c[n // 2, 550] = float("nan")
    out, lse = run(c, q)
    assert bool(lse.isnan().all()) and bool(out.isnan().all())
    c = cache.clone()
    c[n // 2, 550] = inf
    out, lse = run(c, q)
    assert bool((lse == inf).all()) and bool(out.isnan().all())
    c = cache.clone()
    c[:, 550] = -inf
    out, lse = run(c, q)
    assert bool((lse == -inf).all()) and bool(out.isnan().all())
    c = cache.clone()
    c[n + 1, 550] = float("nan")           # a drafted row that node 1 alone sees
    out, lse = run(c, q)
    assert bool(lse[1].isnan().all()) and bool(out[1].isnan().all())
    assert bool(lse[[0, 2]].isfinite().all()) and bool(out[[0, 2]].isfinite().all())
    c = cache.clone()
    c[n // 3, 550] = -inf                  # one row out of many: probability 0
    out, lse = run(c, q)
    assert bool(lse.isfinite().all()) and bool(out.isfinite().all())


def test_no_sequence_other_stream_given_outputs_and_workspace():
    cache, scale, kv = _cache("fp8", 3000, 3)
    e = ds4idx.tree_attention(_q(0, 4, 16, 1), cache, _i32([]), torch.zeros(0, 4, dtype=torch.int64,
                                                                           device="cuda"),
                              0.04, scale=scale)
    assert e[0].shape == (0, 4, 16, 512)
    lens, masks = [2500], _masks(1, 4, 2)
    q = _q(1, 4, 16, 1)
    args = (q, cache, _i32(lens), _i64(masks), 0.04)
    want = ds4idx.tree_attention(*args, scale=scale)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ds4idx.tree_attention(*args, scale=scale, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    need = ds4idx.tree_attention_workspace(1, 4, 16, 3000)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    ds4idx.tree_attention(*args, scale=scale, max_kv_len=3000, out=out, lse=lse, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    if need:
        with pytest.raises(ds4idx.Ds4IdxError):
            ds4idx.tree_attention(*args, scale=scale, max_kv_len=3000, workspace=ws[:need - 16])


def test_captured_and_replayed_with_other_lengths():
    # lengths, masks and queries are read on the device: one graph serves a growing sequence
    N, H = 5, 128
    cache, scale, kv = _cache("fp8", 2000, 3)
    q, ln, mk = _q(2, N, H, 1), _i32([0, 0]), torch.zeros(2, N, dtype=torch.int64, device="cuda")
    starts = _i64([0, 1000])
    call = lambda: ds4idx.tree_attention(q, cache, ln, mk, 0.04, scale=scale, kv_row0=starts,  # noqa: E731
                                         max_kv_len=500)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call()
    for lens in ([3, 500], [64, 0], [990, 127]):
        masks = _masks(2, N, sum(lens), padding=True)
        ln.copy_(_i32(lens))
        mk.copy_(_i64(masks))
        q.copy_(_q(2, N, H, lens[0]))
        g.replay()
        rows = [list(range(lens[0] + N)), list(range(1000, 1000 + lens[1] + N))]
        _check(q, kv, rows, lens, masks, 0.04, out, lse)
    ds4idx.sparse_attention_status()
