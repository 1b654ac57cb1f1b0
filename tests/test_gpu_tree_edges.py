"""Trees of drafted tokens where they can go wrong: rows that only some nodes see, extremes of the scales,
offsets past 32 bits, calls at once; and the operators one after another, as a decode step uses them.
Tolerances: those of test_gpu_tree_attention, and beside 8-bit rows 2^-21 of a query's largest value for
each of its latent dims (the kernel holds them as two 8-bit numbers)."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

from . import tree_reference as ref
from .test_gpu_tree_attention import _cache, _check, _contiguous, _i32, _i64, _masks, _q

pytestmark = pytest.mark.gpu
KINDS = ["fp8", "bf16", "q4"]
ROW = {"fp8": 640, "bf16": 1152, "q4": 416}


def _bytes(cache):
    return cache.view(torch.uint8).reshape(cache.shape[0], -1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,H", [(100, 16), (0, 16), (62, 5)])
def test_drafted_rows_not_finite_reach_only_nodes_that_see_them(kind, n, H):
    # all nodes share a tile of 128 rows; nodes 3 and 5 see the bad row
    N, bad = 8, 3
    starts, R, rows = _contiguous([n], N)
    masks = [[1 << i for i in range(N)]]
    masks[0][5] |= 1 << bad
    q = _q(1, N, H, 2)
    for what in ((float("nan"), float("inf"), -float("inf")) if kind == "bf16" else (float("nan"),)):
        cache, scale, kv = _cache(kind, R, 6)
        at = rows[0][n + bad]
        if kind == "bf16":
            cache[at] = what
        else:
            cache[at, ROW[kind] - 128:] = 0xFF
            if kind == "fp8":
                cache[at, :512] = 0x7F
                scale[at] = float("inf")
        kv[at] = 0
        out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64(masks), 0.04, scale=scale,
                                         kv_row0=_i64(starts))
        ds4idx.sparse_attention_status()
        assert bool(out[:, [3, 5]].isnan().all())
        out[:, [3, 5]], lse[:, [3, 5]] = 0, -float("inf")
        rest = [[0 if i in (3, 5) else m for i, m in enumerate(masks[0])]]
        _check(q, kv, rows, [n], rest, 0.04, out, lse)


def _check_f8(q, kv, rows, lens, masks, sm, out, lse):
    """As _check, with the queries' error added to the scores'."""
    o_ref, l_ref, av, big, seen = ref.attention(q.double(), kv, rows, lens, masks, sm)
    top = q.double().abs().amax(dim=-1)
    qe = 2.0 ** -21 * sm * top * kv[:, :512].abs().sum(dim=1).max()
    d = 37 * 2.0 ** -22 * (big + qe) + 2.0 ** -20 * (1 + big + qe) + qe
    t = seen * 2.0 ** -23 + 2.0 ** -20
    bound = (2.0 ** -7 + 2.0 ** -15 + 2 * (d + t)[..., None]) * av
    bound = bound + 2.0 ** -8 * (o_ref.abs() + bound) + seen[..., None] * 2.0 ** -126 * kv.abs().max()
    assert bool(((out.double() - o_ref).abs() <= bound).all())
    assert bool(((lse.double() - l_ref).abs() <= d + t).all())


def test_every_code_and_every_scale():
    # codes of all values, subnormal ones among them, and scales of 2^-24 .. 2^7 side by side
    n, N = 400, 3
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 254, (n + N, 512))
    rows8 = np.zeros((n + N, 640), np.uint8)
    rows8[:, :512] = np.where(codes >= 127, codes + 1, codes)
    rows8[::3, :512] &= 0x87                                      # subnormal alone
    rows8[:, 512:] = torch.randn(n + N, 64).to(torch.bfloat16).view(torch.uint8).numpy()
    scale = 2.0 ** rng.integers(-24, 8, n + N)
    kv = torch.from_numpy(ref.dequantize_f8(rows8, scale)).cuda()
    for sm in (1e-4, 1.0):
        q = (torch.randn(1, N, 128, 576, generator=torch.Generator().manual_seed(1)) * 1e-3)
        q = q.to(torch.bfloat16).cuda()
        masks = [[1, 3, 5]]
        out, lse = ds4idx.tree_attention(q, torch.from_numpy(rows8).cuda(), _i32([n]), _i64(masks), sm,
                                         scale=torch.from_numpy(scale).float().cuda())
        ds4idx.sparse_attention_status()
        _check_f8(q, kv, [list(range(n + N))], [n], masks, sm, out, lse)


@pytest.mark.parametrize("high", [2.0 ** 5, 2.0 ** 14, 2.0 ** 40, 2.0 ** -100])
def test_queries_with_one_large_dim(high):
    # the dim meets values of 0 in most rows, so that the others count there
    n, N = 200, 2
    g = torch.Generator().manual_seed(7)
    x = torch.randn(n + N, 576, generator=g)
    x[:, 5] = 0
    x = x.to(torch.bfloat16)
    rows8, s = ref.quantize_f8(x.double().numpy(),
                               x[:, 512:].contiguous().view(torch.int16).numpy().view(np.uint16))
    kv = torch.from_numpy(ref.dequantize_f8(rows8, s)).cuda()
    q = torch.randn(1, N, 128, 576, generator=g)
    if high < 1:
        q *= high
    else:
        q[..., 5] = high
    q = q.to(torch.bfloat16).cuda()
    sm = 0.04 if high >= 1 else 2.0 ** 90
    out, lse = ds4idx.tree_attention(q, torch.from_numpy(rows8).cuda(), _i32([n]), _i64([[1, 3]]), sm,
                                     scale=torch.from_numpy(s).float().cuda())
    ds4idx.sparse_attention_status()
    _check_f8(q, kv, [list(range(n + N))], [n], [[1, 3]], sm, out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_scales_of_scores_at_the_ends(kind):
    # scores that are all next to 0, or that only one row exceeds; masked rows stay masked
    n, N = 70, 3
    starts, R, rows = _contiguous([n], N)
    cache, scale, kv = _cache(kind, R, 6)
    masks = [[1, 2, 4]]
    for size, sm in ((2.0 ** -120, 1e-30), (2.0 ** -100, 1e-38), (0.0, 1e29)):
        q = (torch.ones(1, N, 16, 576) * size).to(torch.bfloat16).cuda()
        out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64(masks), sm, scale=scale,
                                         kv_row0=_i64(starts))
        ds4idx.sparse_attention_status()
        _check(q, kv, rows, [n], masks, sm, out, lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [0, 1, 4096])
def test_rows_past_32_bit_offsets(kind, page):
    n, N = 300, 4
    small, scale_s, kv = _cache(kind, n + N, 5)
    R = (1 << 32) // ROW[kind] + 20000
    R -= R % 4096
    cache = torch.zeros(R, ROW[kind], dtype=torch.uint8, device="cuda")
    scale = torch.zeros(R, device="cuda") if scale_s is not None else None
    if page:
        pages = -(-(n + N) // page)
        table = R // page - 1 - torch.arange(pages, dtype=torch.int32)
        at = torch.tensor([int(table[s // page]) * page + s % page for s in range(n + N)])
        where = dict(page_table=table[None].cuda(), page_size=page)
    else:
        at = torch.arange(R - n - N, R)
        where = dict(kv_row0=_i64([R - n - N]))
    assert int(at.min()) * ROW[kind] > 1 << 32
    cache[at.cuda()] = _bytes(small)
    if scale is not None:
        scale[at.cuda()] = scale_s
    pool = cache.view(torch.bfloat16).reshape(R, 576) if kind == "bf16" else cache
    q, masks = _q(1, N, 64, 3), [[1, 3, 5, 9]]
    out, lse = ds4idx.tree_attention(q, pool, _i32([n]), _i64(masks), 0.04, scale=scale,
                                     max_kv_len=n, **where)
    ds4idx.sparse_attention_status()
    _check(q, kv, [list(range(n + N))], [n], masks, 0.04, out, lse)
    # and the accepted rows are moved there
    arrays = [cache] + ([scale] if scale is not None else [])
    new = ds4idx.tree_commit(arrays, _i32([n]), _i32([[0, 3, 0, 0]]), _i32([2]), **where)
    assert new.tolist() == [n + 2]
    assert torch.equal(cache[at[n + 1]], _bytes(small)[n + 3])
    assert torch.equal(cache[at[n + 2]], _bytes(small)[n + 2])


def test_a_page_of_half_the_positions_and_many_short_sequences():
    N, n = 2, 130
    cache, scale, kv = _cache("fp8", 200, 5)
    q, masks = _q(1, N, 128, 3), [[1, 3]]
    for page in (1 << 30, 2 ** 31 - 1):
        out, lse = ds4idx.tree_attention(q, cache, _i32([n]), _i64(masks), 0.04, scale=scale,
                                         page_table=_i32([[0, 7]]), page_size=page, max_kv_len=n)
        _check(q, kv, [list(range(n + N))], [n], masks, 0.04, out, lse)
    B = 1500
    lens = [b % 5 for b in range(B)]
    starts, R, rows = _contiguous(lens, 1, gap=0)
    cache, scale, kv = _cache("fp8", R, 5)
    q, masks = _q(B, 1, 2, 3), [[1 if b % 7 else 0] for b in range(B)]
    out, lse = ds4idx.tree_attention(q, cache, _i32(lens), _i64(masks), 0.04, scale=scale,
                                     kv_row0=_i64(starts))
    ds4idx.sparse_attention_status()
    _check(q, kv, rows, lens, masks, 0.04, out, lse)


def test_two_calls_at_once():
    # on two streams, each with its workspace: the same bits as one after the other
    N, lens = 7, [2000]
    starts, R, rows = _contiguous(lens, N)
    cases = []
    for kind, H in (("fp8", 128), ("q4", 100), ("bf16", 128)):
        cache, scale, _ = _cache(kind, R, 4)
        args = (_q(1, N, H, 3), cache, _i32(lens), _i64(_masks(1, N, 2)), 0.04)
        kw = dict(scale=scale, kv_row0=_i64(starts), max_kv_len=2000)
        ws = torch.empty(ds4idx.tree_attention_workspace(1, N, H, 2000) + 16, dtype=torch.uint8,
                         device="cuda")
        cases.append((args, dict(kw, workspace=ws), ds4idx.tree_attention(*args, **kw)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for s, (args, kw, _) in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(ds4idx.tree_attention(*args, **kw))
        torch.cuda.synchronize()
        for g, (_, _, want) in zip(got, cases):
            assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])
    ds4idx.sparse_attention_status()


@pytest.mark.parametrize("kind,paged", [("fp8", True), ("fp8", False), ("q4", True), ("bf16", False)])
def test_steps_of_speculative_decoding(kind, paged):
    # Drafted rows are rotated and written behind their sequences, the nodes attend, the accepted path is
    # kept: four steps as one graph that is replayed, against sequences grown row by row.
    B, N, H, page, room = 3, 6, 32, 16, 256
    g = torch.Generator().manual_seed(3)
    R = B * room
    if paged:
        table = torch.randperm(R // page, generator=g).reshape(B, -1).int()
        row_of = lambda b, s: int(table[b, s // page]) * page + s % page  # noqa: E731
        where = dict(page_table=table.cuda(), page_size=page)
    else:
        row_of = lambda b, s: b * room + s  # noqa: E731
        where = dict(kv_row0=_i64([b * room for b in range(B)]))
    flat = torch.tensor([[row_of(b, s) for s in range(room)] for b in range(B)]).cuda()
    pool = torch.zeros(R, ROW[kind], dtype=torch.uint8, device="cuda")
    if kind == "bf16":
        pool = pool.view(torch.bfloat16).reshape(R, 576)
    scale = torch.zeros(R, device="cuda") if kind == "fp8" else None
    arrays = [pool] + ([scale] if kind == "fp8" else [])
    freqs = ds4idx.rotary_freqs(64)

    def write(x, slots):
        if kind == "fp8":
            ds4idx.quantize_latents_fp8(x, pool, scale, slots=slots)
        elif kind == "q4":
            ds4idx.quantize_latents(x, pool, slots=slots)
        else:
            pool[slots] = x

    def read():
        if kind == "fp8":
            return ds4idx.read_latents_fp8(pool, scale).double()
        return ds4idx.read_latents(pool).double() if kind == "q4" else pool.double()

    lens = _i32([37, 0, 64])
    depth = _i32([0, 1, 1, 2, 2, 3])
    masks = ref.tree_masks([-1, 0, 0, 1, 2, 4])
    mask = _i64([masks] * B)
    x, q = torch.zeros(B * N, 576, dtype=torch.bfloat16, device="cuda"), _q(B, N, H, 1)
    path, count = torch.zeros(B, N, dtype=torch.int32, device="cuda"), _i32([0] * B)
    prefix = torch.randn(B, 64, 576, generator=g).to(torch.bfloat16).cuda()
    for b in range(B):
        n = int(lens[b])
        if n:
            write(prefix[b, :n].contiguous(), flat[b, :n].contiguous())

    def step():
        pos = (lens[:, None] + depth).reshape(-1).long()
        r = x.clone()
        ds4idx.rotary([r[:, 512:]], pos, freqs, outs=[r[:, 512:]])
        slots = flat.gather(1, (lens[:, None] + torch.arange(N, device="cuda")).long()).reshape(-1)
        write(r, slots)
        out, lse = ds4idx.tree_attention(q, pool, lens, mask, 0.04, scale=scale, max_kv_len=100, **where)
        before = read()
        new = ds4idx.tree_commit(arrays, lens, path, count, **where)
        return out, lse, before, lens.clone(), new

    keep_pool, keep_scale = pool.clone(), None if scale is None else scale.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, before, was, new = step()
    pool.copy_(keep_pool)
    if scale is not None:
        scale.copy_(keep_scale)
    grown = [read()[flat[b, :int(lens[b])]] for b in range(B)]
    for k, (p, c) in enumerate([([0, 2, 4, 5], [4, 1, 0]), ([0, 1, 3, 0], [3, 3, 2]),
                                ([0, 2, 4, 5], [2, 4, 4]), ([0, 1, 3, 0], [1, 0, 3])]):
        x.copy_(torch.randn(B * N, 576, generator=g).to(torch.bfloat16))
        q.copy_(_q(B, N, H, 10 + k))
        path.copy_(_i32([p + [0, 0]] * B))
        count.copy_(_i32(c))
        graph.replay()
        torch.cuda.synchronize()
        n = was.tolist()
        assert n == [len(v) for v in grown]
        rows = flat.tolist()
        _check(q, before, rows, n, [masks] * B, 0.04, out, lse)
        for b in range(B):
            assert torch.equal(before[flat[b, :n[b]]], grown[b])
            new_rows = before[flat[b, [n[b] + i for i in p[:c[b]]]]]
            grown[b] = torch.cat([grown[b], new_rows])
            assert torch.equal(read()[flat[b, :n[b] + c[b]]], grown[b])
        assert new.tolist() == [v + i for v, i in zip(n, c)]
        lens.copy_(new)
    ds4idx.sparse_attention_status()
