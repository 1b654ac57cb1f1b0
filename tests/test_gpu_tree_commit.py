"""Keeping the accepted path of drafted trees: rows moved in place, exactly, and nothing else touched."""
import numpy as np
import pytest
import torch

from sparse_attention_lightning_indexer_gb300 import ds4idx

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _arrays(R, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = dict(generator=g, device="cuda", dtype=torch.uint8)
    return [torch.randint(0, 256, (R, 640), **byte), torch.rand(R, generator=g, device="cuda"),
            torch.randint(0, 256, (R, 128), **byte),
            torch.randint(0, 1 << 40, (R,), generator=g, device="cuda"),
            torch.randint(0, 256, (R, 3), **byte), torch.randint(0, 256, (R, 416), **byte),
            torch.randn(R, 576, generator=g, device="cuda").to(torch.bfloat16),
            torch.randn(R, 7, 50, generator=g, device="cuda").to(torch.bfloat16)]


def _want(arrays, row, lens, path, count):
    """row(b, position) -> pool row or -1."""
    res = [a.clone() for a in arrays]
    N = path.shape[1]
    for b, n in enumerate(lens):
        for j in range(max(0, min(N, count[b]))):
            k = int(path[b, j])
            if not 0 <= k < N:
                continue
            src, dst = row(b, n + k), row(b, n + j)
            if src < 0 or dst < 0:
                continue
            for a, r in zip(arrays, res):
                r[dst] = a[src]
    return res


@pytest.mark.parametrize("B,N", [(1, 1), (1, 8), (3, 64), (17, 5)])
def test_contiguous(B, N):
    rng = np.random.default_rng(B * N)
    lens = rng.integers(0, 50, B)
    starts = np.cumsum([0] + [int(n) + N + 2 for n in lens])
    R = int(starts[-1]) + 4
    arrays = _arrays(R, B)
    count = rng.integers(0, N + 1, B)
    count[0] = N
    path = np.full((B, N), -1)
    for b in range(B):
        path[b, :count[b]] = np.sort(rng.choice(N, count[b], replace=False))
    want = _want(arrays, lambda b, s: int(starts[b]) + s, lens, path, count)
    new = ds4idx.tree_commit(arrays, _i32(lens), _i32(path), _i32(count),
                             kv_row0=torch.tensor(starts[:B], device="cuda"))
    assert new.tolist() == (lens + count).tolist()
    for a, w in zip(arrays, want):
        assert torch.equal(a, w)


def test_any_order_the_same_node_twice_and_entries_of_no_node():
    N, lens, count = 64, [10, 100, 200, 300], [64, 64, 99, -3]
    rng = np.random.default_rng(3)
    path = np.stack([rng.permutation(N), rng.integers(0, N, N), rng.integers(-2, N + 2, N),
                     rng.permutation(N)])
    arrays = _arrays(500, 2)
    want = _want(arrays, lambda b, s: s, lens, path, count)
    new = ds4idx.tree_commit(arrays, _i32(lens), _i32(path), _i32(count))
    assert new.tolist() == [74, 164, 264, 300]
    for a, w in zip(arrays, want):
        assert torch.equal(a, w)


@pytest.mark.parametrize("page", [1, 7, 64])
def test_paged_with_bad_pages(page):
    B, N, n_seqs = 5, 9, 6
    lens = [0, 60, 33, 20, 5]
    pages = -(-(max(lens) + N) // page)
    rng = np.random.default_rng(page)
    n_pages = n_seqs * pages + 2
    table = rng.permutation(n_pages)[:n_seqs * pages].reshape(n_seqs, pages).astype(np.int32)
    table[1, (lens[2] + 3) // page] = -1
    table[2, (lens[3] + 1) // page] = n_pages + 5
    seq = [0, 5, 1, 2, n_seqs]
    R = n_pages * page

    def row(b, s):
        if seq[b] >= n_seqs or s // page >= pages:
            return -1
        i = int(table[seq[b], s // page])
        return i * page + s % page if 0 <= i < n_pages else -1

    count = [9, 3, 5, 8, 4]
    path = np.stack([np.sort(rng.permutation(N)[:N]) for _ in range(B)])
    for b in range(B):
        path[b, :count[b]] = np.sort(rng.choice(N, count[b], replace=False))
    arrays = _arrays(R, 4)
    want = _want(arrays, row, lens, path, count)
    new = ds4idx.tree_commit(arrays, _i32(lens), _i32(path), _i32(count),
                             page_table=torch.from_numpy(table).cuda(), page_size=page,
                             token_seq=_i32(seq))
    assert new.tolist() == [n + c for n, c in zip(lens, count)]
    for a, w in zip(arrays, want):
        assert torch.equal(a, w)


def test_lengths_alone_no_sequence_and_rows_past_the_pool():
    new = ds4idx.tree_commit([], _i32([5, 6]), _i32([[0, 1], [1, 0]]), _i32([2, 1]))
    assert new.tolist() == [7, 7]
    assert ds4idx.tree_commit([], _i32([]), torch.zeros(0, 3, dtype=torch.int32, device="cuda"),
                              _i32([])).shape == (0,)
    a = _arrays(20, 1)
    lens, path, count = [17, -4, 2 ** 31 - 70], np.array([[1, 2, 4, 0, 3]] * 3), [4, 2, 1]
    want = _want(a, lambda b, s: s if 0 <= s < 20 and lens[b] >= 0 else -1, lens, path, count)
    ds4idx.tree_commit(a, _i32(lens), _i32(path), _i32(count))
    for x, w in zip(a, want):
        assert torch.equal(x, w)


def test_overlaps_are_refused():
    pool = torch.arange(4000, dtype=torch.int32, device="cuda")
    before = pool.clone()
    lens, path, count = pool[:2], pool[100:106].view(2, 3), pool[200:202]
    big = pool.view(1000, 4)
    bad = [dict(arrays=[big]),                                   # the array holds the lengths
           dict(arrays=[], new_lens=lens), dict(arrays=[], new_lens=pool[105:107]),
           dict(arrays=[], new_lens=count)]
    for kw in bad:
        with pytest.raises(ds4idx.Ds4IdxError):
            ds4idx.tree_commit(kv_lens=lens, path=path, n_accepted=count, **kw)
    x = torch.zeros(100, 8, dtype=torch.uint8, device="cuda")
    args = (_i32([4, 9]), _i32([[0, 1, 2]] * 2), _i32([3, 2]))
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.tree_commit([x, x], *args)
    with pytest.raises(ds4idx.Ds4IdxError):
        ds4idx.tree_commit([x, x.view(-1)[1:601].view(100, 6)], *args)
    with pytest.raises(ValueError):
        ds4idx.tree_commit([x, x[:50].clone()], *args)
    with pytest.raises(ValueError):
        ds4idx.tree_commit([x.clone() for _ in range(9)], *args)
    torch.cuda.synchronize()
    assert torch.equal(pool, before)


def test_other_stream_and_graph():
    arrays = _arrays(300, 9)
    lens, path, count = _i32([100]), _i32([[2, 5, 6, -1, -1, -1, -1]]), _i32([3])
    want = _want(arrays, lambda b, s: s, [100], np.array([[2, 5, 6, -1, -1, -1, -1]]), [3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    new = ds4idx.tree_commit(arrays, lens, path, count, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert new.tolist() == [103]
    for a, w in zip(arrays, want):
        assert torch.equal(a, w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new = ds4idx.tree_commit(arrays, lens, path, count)
    for k in range(2):
        lens.fill_(50 + 20 * k)
        path.copy_(_i32([[1 + k, 4, 6, 2, -1, -1, -1]]))
        count.fill_(4 - k)
        want = _want(arrays, lambda b, s: s, [50 + 20 * k], path.cpu().numpy(), [4 - k])
        g.replay()
        assert new.tolist() == [50 + 20 * k + 4 - k]
        for a, w in zip(arrays, want):
            assert torch.equal(a, w)
