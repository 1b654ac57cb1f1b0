"""Tree attention and commit at the limits of their arguments, and the bounds that the choices in it give.
Tolerances: those of test_gpu_tree_attention and test_gpu_tree_edges where nothing else is said."""
import math

import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import tree_reference as ref
from .test_gpu_tree_attention import _cache, _check, _contiguous, _i32, _i64, _masks, _q

pytestmark = pytest.mark.gpu
KINDS = ["fp8", "bf16", "q4"]


def _fp8_rows(x):
    """(cache, scale, values in 64 bits) of bf16 rows x."""
    rope = x[:, 512:].contiguous().view(torch.int16).numpy().view(np.uint16)
    rows, s = ref.quantize_f8(x.double().numpy(), rope)
    return (torch.from_numpy(rows).cuda(), torch.from_numpy(s).float().cuda(),
            torch.from_numpy(ref.dequantize_f8(rows, s)).cuda())


# The query's error beside 8-bit rows, 2^-21 of the largest value of its row or of 2^-119, enters the scores'.
def _check_ends(q, kv, rows, lens, masks, sm, out, lse, f8):
    o_ref, l_ref, av, big, seen = ref.attention(q.double(), kv, rows, lens, masks, sm)
    qe = torch.zeros_like(big)
    if f8:
        top = q.double().abs().amax(dim=-1).clamp_min(2.0 ** -119)
        qe = 2.0 ** -21 * sm * top * kv[:, :512].abs().sum(dim=1).max()
    d = 37 * 2.0 ** -22 * (big + qe) + 2.0 ** -20 * (1 + big + qe) + qe
    t = seen * 2.0 ** -23 + 2.0 ** -20
    bound = (2.0 ** -7 + 2.0 ** -15 + 2 * (d + t)[..., None]) * av
    bound = bound + 2.0 ** -8 * (o_ref.abs() + bound) + seen[..., None] * 2.0 ** -126 * kv.abs().max()
    assert bool(((out.double() - o_ref).abs() <= bound).all())
    assert bool(((lse.double() - l_ref).abs() <= d + t).all())


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("size,sm,rows_up", [
    (2.0 ** 110, 0.04 * 2.0 ** -110, 0), (2.0 ** 118, 0.04 * 2.0 ** -118, 0),
    (2.0 ** 122, 0.04 * 2.0 ** -118, -4), (2.0 ** 125, 0.04 * 2.0 ** -118, -7), (2.0 ** -105, 2.0 ** 99, 2),
    (2.0 ** -112, 2.0 ** 99, 9), (2.0 ** -118, 2.0 ** 99, 13), (2.0 ** -124, 2.0 ** 99, 13)])
def test_queries_at_the_ends_of_their_range(kind, size, sm, rows_up):
    n, N = 200, 2
    g = torch.Generator().manual_seed(7)
    x = (torch.randn(n + N, 576, generator=g) * 2.0 ** rows_up).to(torch.bfloat16)
    cache, scale, kv = _fp8_rows(x) if kind == "fp8" else (x.cuda(), None, x.double().cuda())
    q = (torch.randn(1, N, 128, 576, generator=g).clamp(-4, 4).double() * size).to(torch.bfloat16).cuda()
    assert bool(q.isfinite().all())
    sm = float(np.float32(sm))                    # (products stay below 2^128; more than 2^99 is refused)
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64([[1, 3]]), sm, scale=scale)
    ds4idx.sparse_attention_status()
    _check_ends(q, kv, [list(range(n + N))], [n], [[1, 3]], sm, out, lse, kind == "fp8")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("at", [5, 550])
def test_queries_that_are_not_finite_make_nan_of_their_rows_alone(kind, at):
    n, N, H = 130, 2, 16
    cache, scale, kv = _cache(kind, n + N, 3)
    q = _q(1, N, H, 3)
    q[0, 0, 3, at] = float("inf")
    q[0, 1, 0, at] = -float("inf")
    q[0, 1, 7, at] = float("nan")
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64([[1, 3]]), 0.04, scale=scale)
    ds4idx.sparse_attention_status()
    bad = torch.zeros(N, H, dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[1, 0] = bad[1, 7] = True
    assert bool(out[0][bad].isnan().all()) and not bool(lse[0][bad].isfinite().any())
    clean = q.clone()
    clean[0][bad] = 0
    want, l_want = ds4idx.tree_attention(clean, cache, _i32([n]), _i64([[1, 3]]), 0.04, scale=scale)
    assert torch.equal(out[0][~bad], want[0][~bad]) and torch.equal(lse[0][~bad], l_want[0][~bad])


# The least normal fp32 number is 2^-126.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sm", [2.0 ** -125, 2.0 ** -126, 2.0 ** -127, 0.7 * 2.0 ** -129])
def test_scales_of_scores_below_the_least_normal_number(kind, sm):
    n, N = 200, 2
    g = torch.Generator().manual_seed(5)
    cache, scale, kv = _cache(kind, n + N, 5)
    q = torch.randn(1, N, 128, 576, generator=g).clamp(-3, 3).double() * 2.0 ** 116
    q = q.to(torch.bfloat16).cuda()
    if kind != "fp8":                   # (products stay below 2^128)
        assert float(q.double().norm(dim=-1).max() * kv.norm(dim=-1).max()) < 2.0 ** 128
    sm = float(np.float32(sm))
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64([[1, 3]]), sm, scale=scale)
    ds4idx.sparse_attention_status()
    _check_ends(q, kv, [list(range(n + N))], [n], [[1, 3]], sm, out, lse, kind == "fp8")


# Beside 8-bit rows the products may pass 2^128 before they are scaled.
@pytest.mark.parametrize("sm", [0.04 * 2.0 ** -125, 2.0 ** -133, 3 * 2.0 ** -149])
def test_subnormal_scales_beside_large_8_bit_rows(sm):
    n, N = 200, 2
    g = torch.Generator().manual_seed(6)
    up = 1.0 if sm > 2.0 ** -131 else 2.0 ** 10
    cache, scale, kv = _fp8_rows((torch.randn(n + N, 576, generator=g) * up).to(torch.bfloat16))
    q = (torch.randn(1, N, 128, 576, generator=g).clamp(-3, 3).double() * 2.0 ** 125).to(torch.bfloat16).cuda()
    sm = float(np.float32(sm))
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64([[1, 3]]), sm, scale=scale)
    ds4idx.sparse_attention_status()
    _check_ends(q, kv, [list(range(n + N))], [n], [[1, 3]], sm, out, lse, True)


# log2 of the scores of the rows behind the first tile, by a rotary dim alone; values next to 2^80 / rows, of one sign
# in a dim, so that a maximum left where it was would give sums past 2^128 (max_kv_len 0: one range)
@pytest.mark.parametrize("above", [20.0, 47.0, 49.0, 60.0, 63.0, 66.0])
def test_values_up_to_2_to_the_80_over_the_rows(above):
    n, N, H = 700, 1, 16
    g = torch.Generator().manual_seed(2)
    sign = torch.where(torch.rand(512, generator=g) < 0.5, -1.0, 1.0)
    x = torch.zeros(n + N, 576)
    x[:, :512] = sign * (0.75 + 0.24 * torch.rand(n + N, 512, generator=g)) * (2.0 ** 80 / (n + N))
    x[64:, 550] = above
    x = x.to(torch.bfloat16)
    assert bool((x.abs() < 2.0 ** 80 / (n + N)).all())
    q = torch.zeros(1, N, H, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 550] = 1
    sm = float(np.float32(math.log(2)))
    out, lse = ds4idx.tree_attention(q, x.cuda(), _i32([n]), _i64([[1]]), sm, max_kv_len=0)
    ds4idx.sparse_attention_status()
    _check(q, x.double().cuda(), [list(range(n + N))], [n], [[1]], sm, out, lse)


@pytest.mark.parametrize("factor", [1.5, 1 + 2.0 ** -23, 1 - 2.0 ** -24, -1.0])
def test_a_scale_that_is_no_power_of_two_makes_nan_of_the_nodes_that_see_its_row(factor):
    n, N, H = 200, 3, 16
    for row in (30, 150, n + 1):
        cache, scale, kv = _cache("fp8", n + N, 5)
        scale[row] *= factor
        out, lse = ds4idx.tree_attention(_q(1, N, H, 1), cache, _i32([n]), _i64([[1, 3, 5]]), 0.04, scale=scale)
        ds4idx.sparse_attention_status()
        seen = [0, 1, 2] if row < n else [1]
        rest = [i for i in range(N) if i not in seen]
        assert bool(out[0, seen].isnan().all()) and bool(lse[0, seen].isnan().all())
        assert bool(out[0, rest].isfinite().all()) and bool(lse[0, rest].isfinite().all())


def test_new_lengths_end_at_the_largest_int32():
    top = 2 ** 31 - 1
    new = ds4idx.tree_commit([], _i32([top, top - 2, top - 3, 5, -1]), _i32([[0, 1, 2]] * 5), _i32([3] * 5))
    assert new.tolist() == [top, top, top, 8, 2]


def _parts_written(N, H, n, bound):
    """How many ranges of a sequence of n rows leave a partial output when the work is laid out for `bound`."""
    R = n + N
    cache = torch.randn(R, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q = _q(1, N, H, 2)
    masks = [[1 << i for i in range(N)]]
    ws = torch.zeros(ds4idx.tree_attention_workspace(1, N, H, bound), dtype=torch.uint8, device="cuda")
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64(masks), 0.04, max_kv_len=bound, workspace=ws)
    ds4idx.sparse_attention_status()
    _check(q, cache.double(), [list(range(R))], [n], masks, 0.04, out, lse)
    part = 128 * 512 * 4
    return int((ws[:ws.numel() // part * part].view(-1, part).view(torch.int64) != 0).any(dim=1).sum())


@pytest.mark.parametrize("N,H,n", [(1, 128, 8192), (1, 128, 1500), (7, 16, 8192), (3, 128, 6000)])
def test_a_loose_bound_leaves_the_work_spread(N, H, n):
    exact = _parts_written(N, H, n, n)
    assert exact > 8
    for bound in (2 * n, 262144, 1 << 20):
        assert _parts_written(N, H, n, bound) >= 0.8 * exact, bound


@pytest.mark.parametrize("B,N,H,bounds", [
    (4, 64, 128, (11968, 12032, 16384, 100000)), (32, 4, 128, (2000, 37056, 37120, 50000)),
    (1, 5, 128, (64, 640, 896, 960, 5000)), (8, 7, 128, (100, 5000, 30000, 262144)),
    (1, 1, 16, (10, 4096, 70000, 1 << 20)), (2, 9, 64, (500, 3000, 20000, 20100))])
def test_a_workspace_for_a_bound_serves_every_shorter_one(B, N, H, bounds):
    lens = [70 + b % 3 for b in range(B)]
    starts, R, rows = _contiguous(lens, N)
    cache, scale, kv = _cache("fp8", R, 3)
    masks = [[1] + [0] * (N - 2) + [1 << N - 1] if N > 1 else [1]] * B
    masks = [[ref.signed(m) for m in row] for row in masks]
    q = _q(B, N, H, 2)
    need = [ds4idx.tree_attention_workspace(B, N, H, n) for n in bounds]
    assert need == sorted(need)
    ws = torch.empty(max(16, need[-1]), dtype=torch.uint8, device="cuda")
    for n in bounds:
        out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                         kv_row0=_i64(starts), max_kv_len=n, workspace=ws)
        ds4idx.sparse_attention_status()
        _check(q, kv, rows, lens, masks, 0.04, out, lse)


# The products are divided by the sum of the rounded terms: with e of a term its rounding, at most u = 2^-8, and
# twice the error d of its score, out - o = sum p (1 + e) (v - o) / sum p (1 + e), which is at most
# e / (1 - e) sum p |v - o|, and goes to 0 where one key outweighs the others. Besides: the output's own
# rounding, t of sum p |v| for the sums in fp32, and the terms that are less than 2^-126 of the largest: there
# exp2 gives 0 where the term is below the least normal number, and the maximum that terms are taken against is a
# score of the row, so that what is lost of an output is less than 2^-126 |v| for each row seen. (It shows in 4-bit
# rows, where a value of exactly 0 in the one row that counts leaves outputs of 1e-44.)

# One key outweighs the rest (of one range: max_kv_len 0). Its term, 2^12 times 1.0037 above the maximum it is taken
# against, loses 0.95 of half a bf16 step by its rounding. Divided by the exact sum the output would be 0.95 u off,
# which rounds to the next bf16 number wherever the value's significand is above 1.06.
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [100, 1000])
def test_a_key_that_outweighs_the_others_keeps_its_value(kind, n):
    N, H, at = 1, 128, 90
    cache, scale, kv = _cache(kind, n + N, 4)
    rope = torch.zeros(n + N, 64, dtype=torch.bfloat16, device="cuda")
    rope[at, 38] = 16
    if kind == "bf16":
        cache[:, 512:] = rope
    else:
        cache[:, -128:] = rope.view(torch.uint8)
    kv[:, 512:] = rope.double()
    q = torch.zeros(1, N, H, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 550] = 1
    sm = float(np.float32(math.log(2) * (12 + math.log2(1.0037)) / 16))
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64([[1]]), sm, scale=scale, max_kv_len=0)
    ds4idx.sparse_attention_status()
    p = torch.softmax(sm * 16 * (torch.arange(n + N, device="cuda") == at).double(), 0)
    v = kv[:, :512]
    o = p @ v
    u = 2.0 ** -8
    spread = p @ (v - o).abs()
    half = torch.exp2(torch.floor(torch.log2(o.abs())) - 8)
    t = 2 * ((n + N) * 2.0 ** -23 + 2.0 ** -18) * (p @ v.abs())
    assert bool(((out[0, 0].double() - o).abs() <= half + (u / (1 - u) + 2.0 ** -15) * spread + t).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,size", [(13, 2.0), (200, 2.0), (200, 12.0), (3000, 1.0), (3000, 30.0)])
def test_outputs_divided_by_the_sum_of_the_rounded_terms(kind, n, size):
    N, H, sm = 3, 128, 0.04
    cache, scale, kv = _cache(kind, n + N, 9)
    q, masks = _q(1, N, H, 5, scale=size), [[1, 3, 5]]
    rows = [list(range(n + N))]
    out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64(masks), sm, scale=scale, max_kv_len=n // 4)
    ds4idx.sparse_attention_status()
    o, _, av, big, seen = ref.attention(q.double(), kv, rows, [n], masks, sm)
    d = 37 * 2.0 ** -22 * big + 2.0 ** -20 * (1 + big)
    if kind == "fp8":
        d = d + 2.0 ** -21 * sm * q.double().abs().amax(dim=-1) * kv[:, :512].abs().sum(dim=1).max()
    t = seen * 2.0 ** -23 + 2.0 ** -20
    spread = torch.zeros_like(o)
    for i in range(N):
        at = torch.tensor(list(range(n)) + [n + j for j in range(N) if masks[0][i] >> j & 1], device="cuda")
        p = torch.softmax(sm * q[0, i].double() @ kv[at].t(), dim=1)
        for h in range(H):
            spread[0, i, h] = p[h] @ (kv[at, :512] - o[0, i, h]).abs()
    e = (2.0 ** -8 + 2 * d + 2.0 ** -15)[..., None]
    bound = e / (1 - e) * spread + 2 * t[..., None] * av
    bound = bound + 2.0 ** -8 * (o.abs() + bound) + seen[..., None] * 2.0 ** -126 * kv.abs().max()
    assert bool(((out.double() - o).abs() <= bound).all())
