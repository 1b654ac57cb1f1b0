"""Cases, inputs and plain forms of the operators around a bounded 4-bit latent cache.

The operators run in this order in a decode step or a prefill chunk of sparse attention:
rotary positions on queries and keys; latent rows written to (and read back from) a cache in
4 bits; attention over the selected rows of that cache; each row's received attention weight
accumulated; and, when the cache is over its budget, eviction of the rows that received least.

``run`` computes a case in plain torch operations when ``own`` is false and calls the framework
when it is true. Everything a case needs is made by ``prepare`` from the case and a seed.
"""
from __future__ import annotations

import math

import torch

own = False

D_LATENT, D_ROPE = 512, 64       # the latent row: 512 dims that are also the value, 64 rotary
D_ROW = D_LATENT + D_ROPE
GROUP = 16                       # latent dims that share a scale
ROW_BYTES = D_LATENT // 2 + D_LATENT // GROUP + 2 * D_ROPE   # 416
D_INDEX = 128                    # width of an index key or query
NOPE = 128                       # un-rotated head dims before the rotary ones in a projection
BASE, FACTOR, ORIGINAL, BETA_FAST, BETA_SLOW = 10000.0, 40.0, 4096, 32.0, 1.0


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # A decode step of eight sequences near the end of a 262144-key context: the attention
        # query and key, and the indexer's query and key, in one call. Latency.
        dict(name="rotary_decode_8", op="rotary", T=8, heads=128, index_heads=64, rot=64,
             interleaved=True, dtype="bf16", max_pos=262144, scaling="yarn", inverse=False),
        # An odd-sized prefill chunk of the same tensors.
        dict(name="rotary_chunk_4095", op="rotary", T=4095, heads=128, index_heads=64, rot=64,
             interleaved=True, dtype="bf16", max_pos=262144, scaling="yarn", inverse=False),
        # The gradient of fp32 training in the half layout: rotation by the opposite angle.
        dict(name="rotary_gradient_f32_2048", op="rotary", T=2048, heads=64, index_heads=0, rot=64,
             interleaved=False, dtype="f32", max_pos=65536, scaling="none", inverse=True),
        # One new row for each of eight decode sequences.
        dict(name="latent_write_8", op="latents", n=8, rows=65536, dtype="bf16", slots=True),
        # The rows of a 64k prefill, written and read back.
        dict(name="latent_write_65536", op="latents", n=65536, rows=65536, dtype="bf16",
             slots=False),
        # A single decode token of a 262144-row context: latency.
        dict(name="attention_decode_1", op="attention", T=1, S=262144, seqs=1, heads=128, n_sel=512,
             page=0, weights=False, holes=False),
        # A batch of decode tokens, each of its own sequence in a paged pool, with key weights.
        dict(name="attention_decode_37_paged", op="attention", T=37, S=5000, seqs=37, heads=128,
             n_sel=512, page=64, weights=True, holes=True),
        # A prefill chunk of 4096 tokens at the end of a 64k context.
        dict(name="attention_chunk_4096", op="attention", T=4096, S=65536, seqs=1, heads=128,
             n_sel=512, page=0, weights=False, holes=False),
        # The key weights of a decode batch and of a prefill chunk, added to the rows' totals.
        dict(name="accumulate_decode_8", op="accumulate", T=8, S=8192, seqs=8, n_sel=512),
        dict(name="accumulate_chunk_2048", op="accumulate", T=2048, S=65536, seqs=1, n_sel=512),
        # Three short ragged sequences over their budget, with many equal totals.
        dict(name="evict_3x3000", op="evict", B=3, S=3000, keep=2048, sink=4, recent=128,
             ragged=True, ties=True),
        # Eight long contexts halved: selection over 262144 rows each, then the move.
        dict(name="evict_8x262144", op="evict", B=8, S=262144, keep=131072, sink=4, recent=1024,
             ragged=False, ties=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "latents", "attention", "attention", "accumulate", "evict"])
    if op == "rotary":
        return dict(op=op, T=_log_int(rng, 1, 4095), heads=_log_int(rng, 1, 128),
                    index_heads=rng.choice([0, 64]), rot=rng.choice([32, 64, 64, 128]),
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    max_pos=_log_int(rng, 1024, 1 << 20),
                    scaling=rng.choice(["none", "linear", "yarn"]), inverse=rng.random() < 0.4)
    if op == "latents":
        n = _log_int(rng, 1, 65536)
        return dict(op=op, n=n, rows=n + _log_int(rng, 1, 4096),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), slots=rng.random() < 0.5)
    if op == "attention":
        T = _log_int(rng, 1, 4096)
        seqs = 1 if T > 128 else rng.choice([1, T])
        S = _log_int(rng, max(64, -(-T // seqs)), 262144 // seqs if seqs > 1 else 262144)
        return dict(op=op, T=T, S=S, seqs=seqs, heads=rng.choice([128, 128, 64, 16, 37]),
                    n_sel=rng.choice([512, 512, _log_int(rng, 1, 512)]),
                    page=rng.choice([0, 64, 48]), weights=rng.random() < 0.4,
                    holes=rng.random() < 0.5)
    if op == "accumulate":
        T = _log_int(rng, 1, 2048)
        seqs = 1 if T > 128 else rng.choice([1, T])
        S = _log_int(rng, max(64, -(-T // seqs)), 65536 // seqs if seqs > 1 else 65536)
        return dict(op=op, T=T, S=S, seqs=seqs, n_sel=rng.choice([512, _log_int(rng, 1, 512)]))
    B = rng.randint(1, 8)
    S = _log_int(rng, 300, 262144)
    sink, recent = rng.randint(0, 16), rng.randint(0, 128)
    return dict(op=op, B=B, S=S, keep=rng.randint(sink + recent + 1, max(S, sink + recent + 1)),
                sink=sink, recent=recent, ragged=rng.random() < 0.7, ties=rng.random() < 0.4)


def _shapes(case):
    """(heads or 0 for no head axis, width, start of the rotated dims, index tensor?) of each."""
    rot = case["rot"]
    t = [(case["heads"], NOPE + rot, NOPE, False), (0, D_LATENT + rot, D_LATENT, False)]
    if case["index_heads"]:
        t += [(case["index_heads"], D_INDEX, 0, True), (0, D_INDEX, 0, True)]
    return t


def _seq_lens(case):
    S, B = case["S"], case["B"]
    return [S - (b * 37) % max(1, S // 4) if case["ragged"] else S for b in range(B)]


def work(case):
    op = case["op"]
    if op == "rotary":
        n = sum(max(1, h) for h, _, _, _ in _shapes(case)) * case["T"] * case["rot"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * size + 8 * case["T"], "flops": 3 * n}
    if op == "latents":
        n = case["n"]
        size = 2 if case["dtype"] == "bf16" else 4
        # rows in, the cache written, the cache read back as bf16 rows
        return {"bytes": n * (D_ROW * size + 2 * ROW_BYTES + 2 * D_ROW),
                "flops": 4 * n * D_LATENT}
    if op == "attention":
        T, H = case["T"], case["heads"]
        n = min(case["n_sel"], case["S"])
        touched = min(T * n, case["S"] * case["seqs"])
        b = T * H * (D_ROW + D_LATENT) * 2 + T * H * 4 + T * case["n_sel"] * 4
        b += touched * ROW_BYTES + (T * case["n_sel"] * 4 if case["weights"] else 0)
        return {"bytes": b, "flops": 2 * T * H * n * (D_ROW + D_LATENT)}
    if op == "accumulate":
        T, n = case["T"], case["n_sel"]
        return {"bytes": T * n * 8 + 16 * case["S"] * case["seqs"],
                "flops": T * n}
    lens = _seq_lens(case)
    kept = sum(min(s, case["keep"]) for s in lens)
    return {"bytes": 8 * sum(lens) + kept * (4 + 2 * (ROW_BYTES + D_INDEX + 4 + 8)),
            "flops": sum(lens)}


# ----------------------------------------------------------------------- what a user has in hand

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * (int(seed) + 1))
    return g


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _latents(n, g, dtype):
    """Normalised latent rows with a few large channels, and some rows of zeros."""
    x = torch.randn(n, D_ROW, generator=g, device="cuda")
    x[:, ::97] *= 6.0
    x *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
    x[5::1009] = 0.0
    return x.to(dtype)


def _lists(T, n_sel, last, g, holes):
    """Distinct positions 0..last[t] in no order, -1 after them; with holes, some slots and one
    row in eleven are empty."""
    dev = "cuda"
    j = torch.arange(n_sel, device=dev)[None, :]
    vis = last[:, None] + 1
    lo = (j * vis) // n_sel
    hi = ((j + 1) * vis) // n_sel
    u = torch.rand(T, n_sel, generator=g, device=dev, dtype=torch.float64)
    pos = lo + ((hi - lo) * u).long().clamp_(max=(hi - lo - 1).clamp(min=0))
    pos = torch.where(hi > lo, pos, torch.full_like(pos, -1))
    order = torch.argsort(torch.rand(T, n_sel, generator=g, device=dev) +
                          2.0 * (pos < 0), dim=1)
    pos = torch.gather(pos, 1, order)
    if holes:
        pos[torch.rand(T, n_sel, generator=g, device=dev) < 0.1] = -1
        pos[7::11] = -1
    return pos.to(torch.int32)


def _placing(case, g):
    """Where the tokens' sequences lie in the pool: rows, kv_row0 or page_table and token_seq."""
    T, S, seqs, page = case["T"], case["S"], case["seqs"], case.get("page", 0)
    t = torch.arange(T, device="cuda")
    seq = (t * seqs) // T
    per = -(-T // seqs)
    last = (S - 1 - torch.clamp(per - 1 - (t % per if seqs > 1 else t), min=0)).clamp(min=0)
    if page:
        per_seq = -(-S // page)
        table = torch.randperm(seqs * per_seq, generator=g, device="cuda").to(torch.int32)
        return dict(rows=seqs * per_seq * page, last=last, row0=None,
                    table=table.view(seqs, per_seq), seq=seq.to(torch.int32), page=page)
    return dict(rows=seqs * S, last=last, row0=(seq * S).to(torch.int64), table=None, seq=None,
                page=0)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "rotary":
        T, dt = case["T"], _dtype(case["dtype"])
        pos = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda")
        pos[-1] = case["max_pos"] - 1
        xs, outs, layouts = [], [], []
        for heads, width, start, index in _shapes(case):
            shape = (T, heads, width) if heads else (T, width)
            x = torch.randn(shape, generator=g, device="cuda").to(dt)
            # the rotated query goes behind the latent dims of the attention query
            owidth = D_LATENT + case["rot"] if start == NOPE else width
            ostart = D_LATENT if start == NOPE else start
            o = torch.zeros((T, heads, owidth) if heads else (T, owidth), dtype=dt, device="cuda")
            xs.append(x[..., start:start + case["rot"]])
            outs.append(o[..., ostart:ostart + case["rot"]])
            layouts.append(case["interleaved"] != index)
        st.update(xs=xs, outs=outs, layouts=layouts, pos=pos)
        if own:
            from sparse_attention_lightning_indexer_gb300 import ds4idx
            st["freqs"] = ds4idx.rotary_freqs(case["rot"], BASE, scaling=case["scaling"],
                                              factor=FACTOR, original_max_position=ORIGINAL,
                                              beta_fast=BETA_FAST, beta_slow=BETA_SLOW)
    elif op == "latents":
        n, R = case["n"], case["rows"]
        st.update(x=_latents(n, g, _dtype(case["dtype"])),
                  cache=torch.zeros(R, ROW_BYTES, dtype=torch.uint8, device="cuda"))
        if case["slots"]:
            s = torch.randperm(R, generator=g, device="cuda")[:n]
            s[3::17] = -1      # padding tokens
            st["slots"] = s
        else:
            st["slots"] = None
            st["dst"] = R - n
    elif op == "attention":
        T = case["T"]
        pl = _placing(case, g)
        cache = torch.empty(pl["rows"], ROW_BYTES, dtype=torch.uint8, device="cuda")
        for a in range(0, pl["rows"], 65536):
            b = min(pl["rows"], a + 65536)
            cache[a:b] = _pack(*_quantize(_latents(b - a, g, torch.bfloat16)))
        q = 2.0 * torch.randn(T, case["heads"], D_ROW, generator=g, device="cuda")
        st.update(pl, cache=cache, q=q.to(torch.bfloat16), scale=D_ROW ** -0.5,
                  idx=_lists(T, case["n_sel"], pl["last"], g, case["holes"]))
    elif op == "accumulate":
        pl = _placing(case, g)
        idx = _lists(case["T"], case["n_sel"], pl["last"], g, False)
        w = torch.randn(case["T"], case["n_sel"], generator=g, device="cuda") * 2.0
        w = torch.softmax(w.masked_fill(idx < 0, -math.inf), dim=1) * 128.0
        acc = torch.randint(0, 1 << 40, (pl["rows"],), generator=g, device="cuda")
        st.update(pl, idx=idx, w=w, acc=acc)
    else:
        lens = _seq_lens(case)
        start = [case["S"] * b for b in range(case["B"])]
        R = case["S"] * case["B"]
        acc = torch.exp(8.0 * torch.rand(R, generator=g, device="cuda", dtype=torch.float64) + 18)
        acc = (acc.long() >> 24) if case["ties"] else acc.long()
        byte = dict(generator=g, device="cuda", dtype=torch.uint8)
        keep = [case["keep"]] * case["B"]
        counts = [min(k, s) for k, s in zip(keep, lens)]
        dst = [sum(counts[:b]) for b in range(case["B"])]
        arrays = [torch.randint(0, 256, (R, ROW_BYTES), **byte),
                  torch.randint(0, 256, (R, D_INDEX), **byte),
                  torch.rand(R, generator=g, device="cuda"), acc]
        outs = [torch.zeros((sum(counts), *a.shape[1:]), dtype=a.dtype, device="cuda")
                for a in arrays]
        st.update(lens=lens, start=start, keep=keep, dst=dst, arrays=arrays, outs=outs, acc=acc)
    return st


# ------------------------------------------------------------------------------- the plain forms

def _angles(case, pos):
    """(cos, sin) [T, rot/2], fp32 from angles in 64 bits: position * frequency."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=pos.device)
    f = torch.pow(torch.tensor(BASE, dtype=torch.float64, device=pos.device), -2.0 * i / rot)
    m = 1.0
    if case["scaling"] == "linear":
        f = f / FACTOR
    elif case["scaling"] == "yarn":
        def dim(turns):
            return rot * math.log(ORIGINAL / (2.0 * math.pi * turns)) / (2.0 * math.log(BASE))
        low, high = max(math.floor(dim(BETA_FAST)), 0), min(math.ceil(dim(BETA_SLOW)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / FACTOR * ramp
        m = 0.1 * math.log(FACTOR) + 1.0
    a = pos.double()[:, None] * f[None, :]
    return (torch.cos(a) * m).float(), (torch.sin(a) * m).float()


def _rotate(x, cos, sin, interleaved, inverse):
    x = x.float()
    if x.dim() == 3:
        cos, sin = cos[:, None, :], sin[:, None, :]
    if inverse:
        sin = -sin
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)


def _quantize(x):
    """(integers [n, 512] in -7..7, scale codes [n, 32], rope bf16 [n, 64]) of latent rows.

    A scale code c stands for 2^(c // 8 - 20) * (1 + (c % 8) / 8), the representable number
    nearest to the group's absmax / 7 (ties to the even code); an integer is x / scale to the
    nearest, ties to even. In 64 bits: both roundings have values next to their borders."""
    g = x[:, :D_LATENT].double().view(x.shape[0], D_LATENT // GROUP, GROUP)
    m, e = torch.frexp(g.abs().amax(dim=2) / 7.0)      # m in [1/2, 1)
    code = (e.long() - 1 + 20) * 8 + torch.round((2.0 * m - 1.0) * 8.0).long()
    code = torch.where(m > 0, code, torch.zeros_like(code)).clamp(0, 255)
    scale = _scale(code)
    n = torch.round(g / scale[:, :, None]).clamp(-7, 7)
    return n.flatten(1).long(), code, x[:, D_LATENT:].to(torch.bfloat16)


def _scale(code):
    code = code.long()
    return torch.ldexp(1.0 + (code % 8).double() / 8.0, (code // 8 - 20).double())


def _pack(n, code, rope):
    """Rows of bytes: of each eight integers, stored as n + 8, element 2p stands in nibble p of
    a little-endian word and element 2p + 1 in nibble p + 4; then the scales; then the rope."""
    u = (n + 8).view(n.shape[0], -1, 4, 2).transpose(2, 3).reshape(n.shape[0], -1, 2)
    codes = (u[:, :, 0] | (u[:, :, 1] << 4)).to(torch.uint8)
    return torch.cat([codes, code.to(torch.uint8), rope.contiguous().view(torch.uint8)], dim=1)


def _unpack(rows):
    """[..., 416] bytes -> fp32 rows [..., 576]; the product of integer and scale is exact."""
    c = rows[..., :D_LATENT // 2]
    u = torch.stack([c & 15, c >> 4], dim=-1).unflatten(-2, (D_LATENT // 8, 4)).flatten(-2)
    u = u.unflatten(-1, (2, 4)).transpose(-1, -2).flatten(-3)
    s = _scale(rows[..., D_LATENT // 2:D_LATENT // 2 + D_LATENT // GROUP]).float()
    v = (u.float() - 8.0) * s.repeat_interleave(GROUP, dim=-1)
    rope = rows[..., ROW_BYTES - 2 * D_ROPE:].contiguous().view(torch.bfloat16).float()
    return torch.cat([v, rope], dim=-1)


def _rows_of(st, idx, a, b):
    """Pool rows of tokens a..b's list entries (0 where empty) and which entries are used."""
    p = idx[a:b].long()
    ok = p >= 0
    p = p.clamp(min=0)
    if st["table"] is not None:
        page = st["page"]
        tab = st["table"].long()[st["seq"][a:b].long()]
        return torch.gather(tab, 1, p // page) * page + p % page, ok
    return p + st["row0"][a:b, None], ok


def _plain_attention(st):
    case, q, idx = st["case"], st["q"], st["idx"]
    outs, lses, ws = [], [], []
    for a in range(0, case["T"], 512):
        b = min(case["T"], a + 512)
        rows, ok = _rows_of(st, idx, a, b)
        kv = _unpack(st["cache"][rows])
        s = torch.bmm(q[a:b].float(), kv.transpose(1, 2)) * st["scale"]
        s = s.masked_fill(~ok[:, None, :], -math.inf)
        m = s.amax(dim=2, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        e = torch.exp(s - m)
        l = e.sum(dim=2, keepdim=True)
        p = torch.where(l > 0, e / l, torch.zeros_like(e))
        outs.append(torch.bmm(p, kv[:, :, :D_LATENT]).to(torch.bfloat16))
        lses.append((m + torch.log(l)).squeeze(2))
        ws.append(p.sum(dim=1))
    r = dict(out=torch.cat(outs), lse=torch.cat(lses))
    if case["weights"]:
        r["weights"] = torch.cat(ws)
    return r


def _plain_evict(st):
    case = st["case"]
    sink, recent = case["sink"], case["recent"]
    kept_all, rows = [], []
    width = max(min(k, s) for k, s in zip(st["keep"], st["lens"]))
    for b, (s0, n, keep) in enumerate(zip(st["start"], st["lens"], st["keep"])):
        if keep >= n:
            kept = torch.arange(n, device="cuda")
        else:
            mid = st["acc"][s0 + sink:s0 + n - recent]
            best = torch.sort(mid, descending=True, stable=True).indices[:keep - sink - recent]
            kept = torch.cat([torch.arange(sink, device="cuda"), best + sink,
                              torch.arange(n - recent, n, device="cuda")]).sort().values
        rows.append(kept + s0)
        kept_all.append(torch.nn.functional.pad(kept.to(torch.int32), (0, width - kept.numel()),
                                                value=-1))
    rows = torch.cat(rows)
    return dict(kept=torch.stack(kept_all), arrays=[a[rows] for a in st["arrays"]])


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rotary":
        cos, sin = _angles(case, st["pos"])
        return [_rotate(x, cos, sin, il, case["inverse"]).to(x.dtype)
                for x, il in zip(st["xs"], st["layouts"])]
    if op == "latents":
        n, code, rope = _quantize(st["x"])
        v = n.double() * _scale(code).repeat_interleave(GROUP, dim=1)
        v = torch.cat([v.to(torch.bfloat16), rope], dim=1)
        if st["slots"] is not None:
            v = torch.where(st["slots"][:, None] >= 0, v, torch.zeros_like(v))
        return v
    if op == "attention":
        return _plain_attention(st)
    if op == "accumulate":
        rows, ok = _rows_of(st, st["idx"], 0, case["T"])
        add = torch.round(st["w"].double() * 2.0 ** 32).long()
        add = torch.where(ok, add, torch.zeros_like(add))
        return st["acc"].clone().index_add_(0, rows.flatten(), add.flatten())
    return _plain_evict(st)


# --------------------------------------------------------------------------- the framework's calls

def _framework(st):
    from sparse_attention_lightning_indexer_gb300 import ds4idx
    case = st["case"]
    op = case["op"]
    if op == "rotary":
        return ds4idx.rotary(st["xs"], st["pos"], st["freqs"], interleaved=st["layouts"],
                             inverse=case["inverse"], outs=st["outs"])
    if op == "latents":
        if st["slots"] is not None:
            ds4idx.quantize_latents(st["x"], st["cache"], slots=st["slots"])
            return ds4idx.read_latents(st["cache"], rows=st["slots"])
        ds4idx.quantize_latents(st["x"], st["cache"], dst_offset=st["dst"])
        return ds4idx.read_latents(st["cache"], start=st["dst"], n=case["n"])
    place = {}
    if op in ("attention", "accumulate"):
        if st["table"] is not None:
            place = dict(page_table=st["table"], page_size=st["page"], token_seq=st["seq"])
        else:
            place = dict(kv_row0=st["row0"])
    if op == "attention":
        out, lse, w = ds4idx.sparse_attention_q4(st["q"], st["cache"], st["idx"], st["scale"],
                                                 want_weights=case["weights"], **place)
        return dict(out=out, lse=lse, weights=w) if case["weights"] else dict(out=out, lse=lse)
    if op == "accumulate":
        acc = st["acc"].clone()
        ds4idx.evict_accumulate(acc, st["w"], st["idx"], **place)
        return acc
    kept = ds4idx.evict_select(st["acc"], st["start"], st["lens"], st["keep"],
                               n_sink=case["sink"], n_recent=case["recent"])
    ds4idx.evict_compact(kept, st["lens"], st["keep"], st["start"], st["dst"], st["arrays"],
                         st["outs"])
    return dict(kept=kept, arrays=st["outs"])


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------- the definitions, in 64 bits

def _exact_rows(rows):
    """Bytes [m, 416] -> fp64 rows [m, 576], one element's nibble and scale looked up at a time."""
    dev = rows.device
    i = torch.arange(D_LATENT, device=dev)
    word, e = i // 8, i % 8
    nibble = e // 2 + 4 * (e % 2)
    by = rows[:, word * 4 + nibble // 2].long()
    n = ((by >> (4 * (nibble % 2))) & 15) - 8
    codes = torch.arange(256, device=dev, dtype=torch.float64)
    table = 2.0 ** (torch.floor(codes / 8) - 20) * (1 + torch.remainder(codes, 8) / 8)
    s = table[rows[:, D_LATENT // 2 + i // GROUP].long()]
    lo = rows[:, ROW_BYTES - 2 * D_ROPE::2].long()
    hi = rows[:, ROW_BYTES - 2 * D_ROPE + 1::2].long()
    rope = ((hi << 24) | (lo << 16)).to(torch.int32).view(torch.float32).double()
    return torch.cat([n.double() * s, rope], dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        rot = case["rot"]
        f, m = [], 1.0
        for i in range(rot // 2):
            x = BASE ** (-2.0 * i / rot)
            if case["scaling"] == "linear":
                x /= FACTOR
            elif case["scaling"] == "yarn":
                m = 0.1 * math.log(FACTOR) + 1.0
                lo = rot * math.log(ORIGINAL / (2 * math.pi * BETA_FAST)) / (2 * math.log(BASE))
                hi = rot * math.log(ORIGINAL / (2 * math.pi * BETA_SLOW)) / (2 * math.log(BASE))
                lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
                r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
                x = x * (1 - r) + x / FACTOR * r
            f.append(x)
        a = torch.outer(st["pos"].double(), torch.tensor(f, dtype=torch.float64, device="cuda"))
        z = torch.polar(torch.full_like(a, m), -a if case["inverse"] else a)
        res = []
        for x, il in zip(st["xs"], st["layouts"]):
            x = x.double()
            c = torch.view_as_complex((x.unflatten(-1, (rot // 2, 2)) if il else
                                       x.unflatten(-1, (2, rot // 2)).transpose(-1, -2))
                                      .contiguous())
            y = torch.view_as_real(c * (z[:, None] if x.dim() == 3 else z))
            res.append((y if il else y.transpose(-1, -2)).flatten(-2))
        return res
    if op == "latents":
        # the representable scale and integer nearest to each quotient, by comparison with all
        x = st["x"].double()
        table = torch.tensor([2.0 ** (c // 8 - 20) * (1 + (c % 8) / 8) for c in range(256)],
                             dtype=torch.float64, device="cuda")
        mid = (table[1:] + table[:-1]) / 2
        grp = x[:, :D_LATENT].reshape(-1, GROUP)
        t = grp.abs().amax(dim=1) / 7.0
        lo = torch.bucketize(t, mid, right=False)     # midpoints below t
        hi = torch.bucketize(t, mid, right=True)      # midpoints at or below t
        s = table[torch.where(lo == hi, lo, lo + lo % 2)][:, None]
        v = (torch.sign(grp) * torch.clamp(torch.round(grp.abs() / s), max=7.0) * s)
        v = torch.cat([v.view(x.shape[0], D_LATENT), st["x"][:, D_LATENT:].to(torch.bfloat16)
                       .double()], dim=1)
        if st["slots"] is not None:
            v[st["slots"] < 0] = 0.0
        return v
    if op == "attention":
        T = case["T"]
        res = dict(out=[], lse=[], weights=[])
        for a in range(0, T, 256):
            b = min(T, a + 256)
            rows, ok = _rows_of(st, st["idx"], a, b)
            uniq, inv = torch.unique(rows, return_inverse=True)
            kv = _exact_rows(st["cache"][uniq])[inv]
            s = st["scale"] * torch.einsum("thd,tnd->thn", st["q"][a:b].double(), kv)
            s = torch.where(ok[:, None, :], s, torch.full_like(s, -math.inf))
            lse = torch.logsumexp(s, dim=2)
            p = torch.where(ok[:, None, :], torch.exp(s - lse[:, :, None]), torch.zeros_like(s))
            res["out"].append(torch.einsum("thn,tnd->thd", p, kv[:, :, :D_LATENT]))
            res["lse"].append(lse)
            res["weights"].append(p.sum(dim=1))
        if not case["weights"]:
            del res["weights"]
        return {k: torch.cat(v) for k, v in res.items()}
    return None      # accumulate and evict: whole numbers
