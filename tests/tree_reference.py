"""The operators around a tree of drafted tokens from their definitions at 64 bits. Shares no code with
the library: E4M3 codes are found by comparison with every one of them."""
import math

import numpy as np
import torch

LATENT, ROPE, F8_ROW = 512, 64, 640
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (1 + (c % 8) / 8) * 2.0 ** (c // 8 - 7)
                 for c in range(127)])
POWERS = np.array([2.0 ** e for e in range(-24, 8)])


def quantize_f8(x, rope_bf16):
    """Latent rows x [n, 576] float64 and their rotary dims as uint16 bf16 bits -> (bytes [n, 640],
    scale [n])."""
    n = x.shape[0]
    v = x[:, :LATENT]
    at = np.searchsorted(448.0 * POWERS[:-1], np.abs(v).max(axis=1), side="left")
    s = POWERS[at]
    y = np.abs(v) / s[:, None]
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
    code = np.where(lo == hi, lo, lo + lo % 2) | (np.signbit(v).astype(np.int64) << 7)
    rows = np.zeros((n, F8_ROW), np.uint8)
    rows[:, :LATENT] = code
    rows[:, LATENT:] = rope_bf16.view(np.uint8).reshape(n, 2 * ROPE)
    return rows, s


def dequantize_f8(rows, scale):
    c = rows[:, :LATENT].astype(np.int64)
    v = np.zeros((rows.shape[0], LATENT + ROPE))
    with np.errstate(invalid="ignore"):
        v[:, :LATENT] = np.append(E4M3, np.nan)[c & 127] * (1 - 2 * (c >> 7)) * scale[:, None]
    rope = np.ascontiguousarray(rows[:, LATENT:]).view(np.uint16).astype(np.uint32) << 16
    v[:, LATENT:] = rope.view(np.float32)
    return v


def signed(mask):
    """An unsigned 64-bit mask as the int64 of the same bits."""
    return mask - (1 << 64) if mask >= 1 << 63 else mask


def tree_masks(parents):
    """Masks of a tree from its nodes' parents (-1: a root; None: padding)."""
    bits = []
    for i, up in enumerate(parents):
        if up is None:
            bits.append(0)
        else:
            assert up < i
            bits.append((bits[up] if up >= 0 else 0) | 1 << i)
    return [signed(b) for b in bits]


def attention(q, kv, rows, lens, masks, scale):
    """q [B, N, H, 576], kv [R, 576] (float64, one device), rows[b]: the pool row of each position of
    sequence b (-1: not there), lens, masks: ints -> out, lse, and for tolerances sum_j p_j |v_j|, the
    largest sum_i |q_i k_i| * scale of a row, and the rows that a node sees."""
    B, N, H, _ = q.shape
    out = torch.zeros(B, N, H, LATENT, dtype=torch.float64, device=q.device)
    av = torch.zeros_like(out)
    lse = torch.full((B, N, H), -math.inf, dtype=torch.float64, device=q.device)
    big, seen = torch.zeros_like(lse), torch.zeros(B, N, 1, dtype=torch.float64, device=q.device)
    for b in range(B):
        for i in range(N):
            if masks[b][i] == 0:
                continue
            at = list(range(lens[b])) + [lens[b] + j for j in range(N) if masks[b][i] >> j & 1]
            r = [rows[b][a] for a in at if a < len(rows[b]) and rows[b][a] >= 0]
            if not r:
                continue
            k = kv[torch.tensor(r, device=q.device)]
            s = scale * q[b, i] @ k.t()
            m = s.amax(dim=1, keepdim=True)
            e = torch.exp(s - m)
            l = e.sum(dim=1, keepdim=True)
            p = e / l
            out[b, i], av[b, i] = p @ k[:, :LATENT], p @ k[:, :LATENT].abs()
            lse[b, i] = (m + torch.log(l))[:, 0]
            big[b, i] = (scale * q[b, i].abs() @ k.abs().t()).amax(dim=1)
            seen[b, i] = len(r)
    return out, lse, av, big, seen
