"""The operators around the 4-bit latent cache from their definitions, in numpy at 64 bits. Shares
no code with the library: scales and integers are found by comparison with all candidates."""
import math

import numpy as np

LATENT, ROPE, GROUP, ROW_BYTES = 512, 64, 16, 416
SCALES = np.array([2.0 ** (c // 8 - 20) * (1 + (c % 8) / 8) for c in range(256)])


def rotary_frequencies(rot, base, scaling="none", factor=1.0, original=4096, beta_fast=32.0,
                       beta_slow=1.0):
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), rot - 1)
        r = np.clip((np.arange(rot // 2) - low) / max(high - low, 0.001), 0, 1)
        return f * (1 - r) + f / factor * r, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, positions, f, m, interleaved, inverse=False):
    """x [T, ..., rot] float64."""
    a = np.outer(positions.astype(np.float64), f) * (-1.0 if inverse else 1.0)
    c, s = m * np.cos(a), m * np.sin(a)
    if x.ndim == 3:
        c, s = c[:, None], s[:, None]
    h = x.shape[-1] // 2
    y = np.empty_like(x)
    i0, i1 = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, h), slice(h, None))
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i0] * s + x[..., i1] * c
    return y


def _nearest_even(t, grid):
    """Index of the grid value nearest to each t >= 0 (ascending grid), ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, t, side="left"), np.searchsorted(mid, t, side="right")
    return np.where(lo == hi, lo, lo + lo % 2)


def quantize(x, rope_bf16):
    """Latent rows x [n, 576] float64 and their rotary dims as uint16 bf16 bits -> bytes [n, 416]."""
    n = x.shape[0]
    g = x[:, :LATENT].reshape(n, LATENT // GROUP, GROUP)
    code = _nearest_even(np.abs(g).max(axis=2) / 7.0, SCALES)
    k = _nearest_even(np.abs(g) / SCALES[code][:, :, None], np.arange(0, 9, dtype=np.float64))
    k = np.minimum(k, 7) * np.sign(g).astype(np.int64)
    rows = np.zeros((n, ROW_BYTES), np.uint8)
    u = (k.reshape(n, LATENT) + 8).astype(np.uint32)
    for d in range(LATENT):
        nib = (d % 8) // 2 + 4 * (d % 2)
        rows[:, (d // 8) * 4 + nib // 2] |= (u[:, d] << (4 * (nib % 2))).astype(np.uint8)
    rows[:, 256:288] = code
    rows[:, 288:] = rope_bf16.view(np.uint8).reshape(n, 128)
    return rows


def dequantize(rows):
    n = rows.shape[0]
    v = np.zeros((n, LATENT + ROPE))
    for d in range(LATENT):
        nib = (d % 8) // 2 + 4 * (d % 2)
        b = (rows[:, (d // 8) * 4 + nib // 2] >> (4 * (nib % 2))) & 15
        v[:, d] = (b.astype(np.float64) - 8) * SCALES[rows[:, 256 + d // GROUP]]
    rope = np.ascontiguousarray(rows[:, 288:]).view(np.uint16).astype(np.uint32) << 16
    v[:, LATENT:] = rope.view(np.float32)
    return v


def attention(q, kv, pool_rows, scale):
    """q [T, H, 576] float64, kv [R, 576] float64, pool_rows [T, n] (-1 empty) ->
    out [T, H, 512], lse [T, H], weights [T, n], and for tolerances sum_j p_j |v_j| [T, H, 512] and
    the largest sum_i |q_i k_i| * scale of a row [T, H]."""
    T, H, _ = q.shape
    n = pool_rows.shape[1]
    out, av = np.zeros((T, H, LATENT)), np.zeros((T, H, LATENT))
    lse, w, big = np.full((T, H), -np.inf), np.zeros((T, n)), np.zeros((T, H))
    for t in range(T):
        use = np.flatnonzero(pool_rows[t] >= 0)
        if use.size == 0:
            continue
        k = kv[pool_rows[t][use]]
        s = scale * q[t] @ k.T
        m = s.max(axis=1, keepdims=True)
        e = np.exp(s - m)
        l = e.sum(axis=1, keepdims=True)
        p = e / l
        out[t], av[t] = p @ k[:, :LATENT], p @ np.abs(k[:, :LATENT])
        lse[t] = (m + np.log(l))[:, 0]
        w[t, use] = p.sum(axis=0)
        big[t] = (scale * np.abs(q[t]) @ np.abs(k).T).max(axis=1)
    return out, lse, w, av, big


def evict_select(total, start, n, keep, sink, recent):
    if keep >= n:
        return list(range(n))
    mid = [(-int(total[start + i]), i) for i in range(sink, n - recent)]
    best = sorted(mid)[:keep - sink - recent]
    return sorted(list(range(sink)) + [i for _, i in best] + list(range(n - recent, n)))
