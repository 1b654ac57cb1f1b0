"""Python binding of the ds4idx C ABI (include/ds4idx.h): argument marshalling only.

Every step of the indexer runs in the CUDA kernels of ``libds4idx.so``; this module checks
tensor shapes, dtypes and devices, passes raw device pointers and the current CUDA stream, and
turns status codes into exceptions. PyTorch provides device memory and streams. There is no
CPU fallback: if the library is missing or the device is not sm_103, calls raise.
"""
from __future__ import annotations

import array
import ctypes
import math
import os
import struct
import threading

import torch

from . import build as _build

BF16 = 0
FP8_E4M3 = 1
F32 = 2
H_I = 64
D_I = 128
TOPK = 512

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_ALLOC = -3
ERR_LAUNCH = -4
ERR_DEVICE_TIMEOUT = -5
ERR_CUDA = -6
ERR_SCRATCH_LIMIT = -7

EXPORTS = ("ds4idx_create", "ds4idx_score_topk", "ds4idx_score_topk_batched",
           "ds4idx_score_dense_debug", "ds4idx_sync_status", "ds4idx_destroy",
           "ds4idx_status_string", "ds4idx_version", "ds4idx_score_topk_batched_noalloc",
           "ds4idx_kernels_launched", "ds4idx_debug_wait_test", "ds4idx_plan_query",
           "ds4idx_quantize_keys", "ds4idx_quantize_queries", "ds4idx_score_topk_varlen",
           "ds4idx_merge_topk", "ds4idx_sparse_attention", "ds4idx_sparse_attention_status",
           "ds4idx_rotary_freqs", "ds4idx_rotary", "ds4idx_quantize_latents",
           "ds4idx_read_latents", "ds4idx_sparse_attention_q4", "ds4idx_evict_accumulate",
           "ds4idx_evict_select", "ds4idx_evict_compact", "ds4idx_quantize_latents_fp8",
           "ds4idx_read_latents_fp8", "ds4idx_tree_attention", "ds4idx_tree_attention_workspace",
           "ds4idx_tree_commit")

_lock = threading.Lock()
_lib = None


class Ds4IdxError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("max_T", ctypes.c_int64), ("max_S", ctypes.c_int64),
                ("max_batch", ctypes.c_int64)]


class RotaryTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_stride_t", ctypes.c_int64),
                ("x_stride_h", ctypes.c_int64), ("out_stride_t", ctypes.c_int64),
                ("out_stride_h", ctypes.c_int64)]


class Placement(ctypes.Structure):
    _fields_ = [("kv_row0", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("token_seq", ctypes.c_void_p), ("page_size", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("n_seqs", ctypes.c_int64)]


class RowArray(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_rows", ctypes.c_int64),
                ("dst_rows", ctypes.c_int64), ("row_bytes", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Loads libds4idx.so (built in-tree by ``build.build()``). Raises if it is absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or library_path()
        if not os.path.exists(p):
            raise RuntimeError(f"ds4idx library not built: {p} is missing (run build())")
        lib = ctypes.CDLL(p)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        lib.ds4idx_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(Config)]
        lib.ds4idx_create.restype = ctypes.c_int
        lib.ds4idx_score_topk.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, vp, vp]
        lib.ds4idx_score_topk.restype = ctypes.c_int
        lib.ds4idx_score_topk_batched.argtypes = [vp, i32, vp, vp, vp, vp, i64, i64, vp, i32, vp,
                                                  vp, vp]
        lib.ds4idx_score_topk_batched.restype = ctypes.c_int
        lib.ds4idx_score_dense_debug.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
        lib.ds4idx_score_dense_debug.restype = ctypes.c_int
        lib.ds4idx_sync_status.argtypes = [vp, vp]
        lib.ds4idx_sync_status.restype = ctypes.c_int
        lib.ds4idx_destroy.argtypes = [vp]
        lib.ds4idx_destroy.restype = ctypes.c_int
        lib.ds4idx_status_string.argtypes = [ctypes.c_int]
        lib.ds4idx_status_string.restype = ctypes.c_char_p
        lib.ds4idx_version.argtypes = []
        lib.ds4idx_version.restype = ctypes.c_int
        lib.ds4idx_score_topk_batched_noalloc.argtypes = [i32, i32, vp, vp, vp, vp, i64, i64, vp,
                                                          i32, vp, vp, vp]
        lib.ds4idx_score_topk_batched_noalloc.restype = ctypes.c_int
        lib.ds4idx_kernels_launched.argtypes = []
        lib.ds4idx_kernels_launched.restype = ctypes.c_uint64
        lib.ds4idx_debug_wait_test.argtypes = [vp, ctypes.c_uint64, i32]
        lib.ds4idx_debug_wait_test.restype = ctypes.c_int
        lib.ds4idx_plan_query.argtypes = [i32, i32, i64, i64, vp, i32, vp]
        lib.ds4idx_plan_query.restype = ctypes.c_int
        lib.ds4idx_score_topk_varlen.argtypes = [vp, i32, vp, vp, vp, vp, vp, i64, vp, vp, i32,
                                                 i32, vp, vp, i32, vp, vp, vp]
        lib.ds4idx_score_topk_varlen.restype = ctypes.c_int
        lib.ds4idx_sparse_attention.argtypes = [vp, vp, i64, vp, vp, i64, i32, i32, i32, i32,
                                                ctypes.c_float, vp, vp, vp]
        lib.ds4idx_sparse_attention.restype = ctypes.c_int
        lib.ds4idx_sparse_attention_status.argtypes = [vp]
        lib.ds4idx_sparse_attention_status.restype = ctypes.c_int
        lib.ds4idx_merge_topk.argtypes = [i32, i64, vp, vp, vp, vp, i32, vp, vp, vp]
        lib.ds4idx_merge_topk.restype = ctypes.c_int
        lib.ds4idx_quantize_keys.argtypes = [vp, i32, i64, vp, i64, vp, vp, i64, vp]
        lib.ds4idx_quantize_keys.restype = ctypes.c_int
        lib.ds4idx_quantize_queries.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp]
        lib.ds4idx_quantize_queries.restype = ctypes.c_int
        f32, f64 = ctypes.c_float, ctypes.c_double
        lib.ds4idx_rotary_freqs.argtypes = [i32, f64, i32, f64, i64, f64, f64, vp, vp]
        lib.ds4idx_rotary.argtypes = [i32, vp, i64, i32, vp, vp, f32, i32, vp]
        lib.ds4idx_quantize_latents.argtypes = [vp, i32, i64, vp, i64, vp, i64, vp]
        lib.ds4idx_read_latents.argtypes = [vp, i64, vp, i64, i64, vp, i32, vp]
        lib.ds4idx_sparse_attention_q4.argtypes = [vp, vp, i64, vp, vp, i64, i32, i32, i32, i32,
                                                   f32, vp, vp, vp, vp]
        lib.ds4idx_evict_accumulate.argtypes = [vp, i64, vp, vp, vp, i64, i32, vp]
        lib.ds4idx_evict_select.argtypes = [vp, i64, i32, vp, vp, vp, i64, i64, vp, i64, vp]
        lib.ds4idx_evict_compact.argtypes = [vp, i64, i32, vp, vp, vp, vp, i32, vp, vp]
        lib.ds4idx_quantize_latents_fp8.argtypes = [vp, i32, i64, vp, i64, vp, vp, i64, vp]
        lib.ds4idx_read_latents_fp8.argtypes = [vp, vp, i64, vp, i64, i64, vp, i32, vp]
        lib.ds4idx_tree_attention.argtypes = [vp, i32, vp, vp, i64, vp, vp, vp, i32, i32, i32, i32,
                                              i32, i64, f32, vp, vp, vp, i64, vp]
        lib.ds4idx_tree_attention_workspace.argtypes = [i32, i32, i32, i64, vp]
        lib.ds4idx_tree_commit.argtypes = [vp, vp, vp, vp, vp, i32, i32, i64, i32, vp, vp]
        for name in ("rotary_freqs", "rotary", "quantize_latents", "read_latents",
                     "sparse_attention_q4", "quantize_latents_fp8", "read_latents_fp8",
                     "tree_attention", "tree_attention_workspace", "tree_commit",
                     "evict_accumulate", "evict_select", "evict_compact"):
            getattr(lib, "ds4idx_" + name).restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def kernels_launched() -> int:
    """Kernels the library has enqueued in this process (its own count, for benchmarks)."""
    return int(load().ds4idx_kernels_launched())


PLAN_FIELDS = ("queries_per_cta", "query_blocks", "splits", "tiles_per_split", "grid",
               "list_words", "tickets")


def plan_query(num_sms: int, B: int, T: int, S: int, pos_offsets, fixed_scratch: bool = False):
    """The work decomposition of a call (host computation only): a dict of PLAN_FIELDS."""
    pos = (ctypes.c_int64 * B)(*[int(x) for x in pos_offsets])
    out = (ctypes.c_int64 * len(PLAN_FIELDS))()
    _check(load().ds4idx_plan_query(num_sms, B, T, S, ctypes.cast(pos, ctypes.c_void_p),
                                    1 if fixed_scratch else 0, ctypes.cast(out, ctypes.c_void_p)),
           "ds4idx_plan_query")
    return dict(zip(PLAN_FIELDS, list(out)))


_IN_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _in_dtype(t: torch.Tensor, name: str) -> int:
    code = _IN_DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return code


def quantize_keys(k, kcache, kscale, dst_offset: int = 0, slots=None, stream=None):
    """Writes k [n, 128] (fp32/bf16) as E4M3 codes + scales into kcache [R, 128] uint8 /
    kscale [R] fp32, at rows dst_offset.. or at slots [n] (int64, -1 skips a row)."""
    n = k.shape[0]
    _need(k, (n, D_I), "k")
    R = kcache.shape[0]
    _need(kcache, (R, D_I), "kcache", torch.uint8)
    _need(kscale, (R,), "kscale", torch.float32)
    if slots is not None:
        _need(slots, (n,), "slots", torch.int64)
    _check(load().ds4idx_quantize_keys(_ptr(k), _in_dtype(k, "k"), n, _ptr(slots),
                                       int(dst_offset), _ptr(kcache), _ptr(kscale), R,
                                       _stream_ptr(stream)), "ds4idx_quantize_keys")
    return kcache, kscale


def quantize_queries(q, w, q_codes=None, w_out=None, qscale=None, stream=None):
    """q [T, 64, 128] (fp32/bf16), w [T, 64] -> (E4M3 codes [T, 64, 128] uint8, w' [T, 64],
    qscale [T])."""
    T = q.shape[0]
    _need(q, (T, H_I, D_I), "q")
    _need(w, (T, H_I), "w", torch.float32)
    dev = q.device
    if q_codes is None:
        q_codes = _new((T, H_I, D_I), torch.uint8, dev, stream)
    if w_out is None:
        w_out = _new((T, H_I), torch.float32, dev, stream)
    if qscale is None:
        qscale = _new((T,), torch.float32, dev, stream)
    _need(q_codes, (T, H_I, D_I), "q_codes", torch.uint8)
    _need(w_out, (T, H_I), "w_out", torch.float32)
    _need(qscale, (T,), "qscale", torch.float32)
    _check(load().ds4idx_quantize_queries(_ptr(q), _in_dtype(q, "q"), T, _ptr(w), _ptr(q_codes),
                                          _ptr(w_out), _ptr(qscale), _stream_ptr(stream)),
           "ds4idx_quantize_queries")
    return q_codes, w_out, qscale


def merge_topk(in_idx, in_score, idx_offsets, row0=None, out_idx=None, out_score=None,
               stream=None):
    """Merges key-sharded Top-512 lists: in_idx / in_score [L, rows, 512] (shard-local indices,
    -1 empty), idx_offsets: L host ints (each shard's first key), row0: L host ints or None.
    Returns (out_idx [rows, 512], out_score [rows, 512])."""
    L, rows = in_idx.shape[0], in_idx.shape[1]
    _need(in_idx, (L, rows, TOPK), "in_idx", torch.int32)
    _need(in_score, (L, rows, TOPK), "in_score", torch.float32)
    dev = in_idx.device
    if out_idx is None:
        out_idx = _new((rows, TOPK), torch.int32, dev, stream)
    if out_score is None:
        out_score = _new((rows, TOPK), torch.float32, dev, stream)
    _need(out_idx, (rows, TOPK), "out_idx", torch.int32)
    _need(out_score, (rows, TOPK), "out_score", torch.float32)
    if len(idx_offsets) != L or (row0 is not None and len(row0) != L):
        raise ValueError("idx_offsets and row0 need one entry per list")
    offs = (ctypes.c_int64 * L)(*[int(x) for x in idx_offsets])
    r0 = None if row0 is None else (ctypes.c_int64 * L)(*[int(x) for x in row0])
    vp = ctypes.c_void_p
    _check(load().ds4idx_merge_topk(L, rows, _ptr(in_idx), _ptr(in_score), ctypes.cast(offs, vp),
                                    None if r0 is None else ctypes.cast(r0, vp), TOPK,
                                    _ptr(out_idx), _ptr(out_score), _stream_ptr(stream)),
           "ds4idx_merge_topk")
    return out_idx, out_score


SA_HEADS, SA_DQK, SA_DV = 128, 576, 512


def sparse_attention(q, kv, idx, sm_scale: float, kv_row0=None, out=None, lse=None, stream=None):
    """Attention of q [T, 128, 576] (bf16) over the selected rows of kv [R, 576] (bf16):
    idx [T, 512] int32 positions (-1 empty), kv_row0 [T] int64 or None.
    Returns (out [T, 128, 512] bf16, lse [T, 128] fp32)."""
    T, R = q.shape[0], kv.shape[0]
    _need(q, (T, SA_HEADS, SA_DQK), "q", torch.bfloat16)
    _need(kv, (R, SA_DQK), "kv", torch.bfloat16)
    _need(idx, (T, TOPK), "idx", torch.int32)
    if kv_row0 is not None:
        _need(kv_row0, (T,), "kv_row0", torch.int64)
    if out is None:
        out = _new((T, SA_HEADS, SA_DV), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _new((T, SA_HEADS), torch.float32, q.device, stream)
    _need(out, (T, SA_HEADS, SA_DV), "out", torch.bfloat16)
    _need(lse, (T, SA_HEADS), "lse", torch.float32)
    _check(load().ds4idx_sparse_attention(_ptr(q), _ptr(kv), R, _ptr(idx), _ptr(kv_row0), T,
                                          SA_HEADS, SA_DQK, SA_DV, TOPK, float(sm_scale),
                                          _ptr(out), _ptr(lse), _stream_ptr(stream)),
           "ds4idx_sparse_attention")
    return out, lse


def sparse_attention_status(stream=None):
    _check(load().ds4idx_sparse_attention_status(_stream_ptr(stream)), "ds4idx_sparse_attention")


# ---- rotary positions

# RotaryTensor, 1 to 4 of them, without its field-by-field cost
_ROTARY_TENSORS = [struct.Struct("=" + "QQiiiiqqqq" * n) for n in range(5)]
ROTARY_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}


class RotaryFreqs:
    """Frequencies of a rotary embedding: 64-bit fractions of a turn per position, and the scale of
    the cosines and sines. Made on the host by ``rotary_freqs``."""

    def __init__(self, rot_dim: int, freqs, scale: float):
        self.rot_dim = rot_dim
        self.freqs = freqs          # ctypes uint64 [rot_dim / 2]
        self.address = ctypes.addressof(freqs)
        self.scale = scale


def rotary_freqs(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_max_position: int = 4096, beta_fast: float = 32.0,
                 beta_slow: float = 1.0) -> RotaryFreqs:
    """Plain, linearly scaled or YaRN frequencies (see include/ds4idx.h). The scale of the cosines and
    sines is 1, with YaRN 0.1 ln(factor) + 1; ``scale`` of the result may be set to a model's own."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALINGS)}")
    f = (ctypes.c_uint64 * max(1, int(rot_dim) // 2))()
    scale = ctypes.c_float()
    _check(load().ds4idx_rotary_freqs(int(rot_dim), float(base), ROTARY_SCALINGS[scaling],
                                      float(factor), int(original_max_position), float(beta_fast),
                                      float(beta_slow), ctypes.addressof(f),
                                      ctypes.addressof(scale)), "ds4idx_rotary_freqs")
    return RotaryFreqs(int(rot_dim), f, scale.value)


def rotary(xs, positions, freqs: RotaryFreqs, interleaved=True, inverse: bool = False, outs=None,
           stream=None):
    """Rotates one tensor or up to four (of the same tokens) in one launch.

    Each is the rotated slice of a projection, [T, H, rot_dim] or [T, rot_dim] (bf16 or fp32, any
    strides, the last dim adjacent). positions [T] int64. interleaved: one bool, or one for each
    tensor (False = halves). inverse: the transposed rotation, which is the gradient. outs: tensors
    of the same shapes to write, which may be the inputs themselves but not overlap otherwise; None
    allocates dense ones. Where gradients are recorded for an input, the results carry them (the inverse
    rotation); outs cannot, and are refused then.
    """
    single = isinstance(xs, torch.Tensor)
    xs = [xs] if single else list(xs)
    n = len(xs)
    if not 1 <= n <= 4:
        raise ValueError("rotary takes 1 to 4 tensors")
    layouts = [interleaved] * n if isinstance(interleaved, bool) else list(interleaved)
    for x in xs:
        if x.requires_grad and torch.is_grad_enabled():
            if outs is not None:
                raise ValueError("outs carry no gradient: leave them out, or call under torch.no_grad()")
            ys = _rotary_recorded(xs, positions, freqs, layouts, inverse, stream)
            return ys[0] if single else list(ys)
    if outs is None:
        outs = [_new(x.shape, x.dtype, x.device, stream) for x in xs]
    else:
        outs = [outs] if isinstance(outs, torch.Tensor) else list(outs)
    if len(layouts) != n or len(outs) != n:
        raise ValueError("interleaved and outs need one entry per tensor")
    T = xs[0].shape[0]
    dev = _device(positions, "positions")
    _need(positions, (T,), "positions", torch.int64, dev)
    rot = freqs.rot_dim
    fields = []
    for k, (x, o, il) in enumerate(zip(xs, outs, layouts)):
        shape, st, so = x.shape, x.stride(), o.stride()
        dims = len(shape)
        if dims not in (2, 3) or shape[0] != T or shape[-1] != rot:
            raise ValueError(f"tensor {k} has shape {tuple(shape)}, expected [{T}, H, {rot}] or "
                             f"[{T}, {rot}]")
        dtype = x.dtype
        if o.shape != shape or o.dtype != dtype:
            raise ValueError(f"out {k} must have the shape and dtype of tensor {k}")
        if x.get_device() != dev or o.get_device() != dev:
            raise ValueError(f"tensor {k} and its out must be on the device of positions, cuda:{dev}")
        if st[-1] != 1 or so[-1] != 1:
            raise ValueError(f"the rotated dim of tensor {k} must be adjacent")
        heads, xh, oh = (shape[1], st[1], so[1]) if dims == 3 else (1, 0, 0)
        if heads < 1:
            raise ValueError(f"tensor {k} has no head")
        code = _IN_DTYPES.get(dtype)
        if code is None:
            raise TypeError(f"tensor {k} must be float32 or bfloat16")
        fields += (x.data_ptr(), o.data_ptr(), code, 1 if il else 0, heads, 0, st[0], xh, so[0], oh)
    _check(load().ds4idx_rotary(n, _ROTARY_TENSORS[n].pack(*fields), T, rot, positions.data_ptr(),
                                freqs.address, freqs.scale, 1 if inverse else 0,
                                _stream_ptr(stream, dev)), "ds4idx_rotary")
    return outs[0] if single else outs


class _RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, positions, freqs, layouts, inverse, *xs):
        ctx.save_for_backward(positions)
        ctx.args = (freqs, layouts, inverse)
        return tuple(rotary(list(xs), positions, freqs, layouts, inverse))

    @staticmethod
    def backward(ctx, *grads):
        freqs, layouts, inverse = ctx.args
        grads = [g if g.stride(-1) == 1 else g.contiguous() for g in grads]
        back = _RotaryFunction.apply(ctx.saved_tensors[0], freqs, layouts, not inverse, *grads)
        return (None, None, None, None, *back)


def _rotary_recorded(xs, positions, freqs, layouts, inverse, stream):
    """The rotation in the autograd graph. The backward pass runs on the stream that is current here."""
    if stream is None:
        return _RotaryFunction.apply(positions, freqs, layouts, inverse, *xs)
    current = torch.cuda.current_stream(positions.device)
    with torch.cuda.stream(stream):
        ys = _RotaryFunction.apply(positions, freqs, layouts, inverse, *xs)
    for y in ys:
        y.record_stream(current)
    return ys


def rotary_autograd(xs, positions, freqs: RotaryFreqs, interleaved=True):
    """``rotary`` for training: new tensors whose gradients are the inverse rotation."""
    return rotary(xs, positions, freqs, interleaved)


# ---- the 4-bit latent cache

Q4_ROW_BYTES = 416


def _cache_rows(cache, dev) -> int:
    rows = cache.shape[0]
    _need(cache, (rows, Q4_ROW_BYTES), "cache", torch.uint8, dev)
    return rows


def quantize_latents(x, cache, dst_offset: int = 0, slots=None, stream=None):
    """Writes latent rows x [n, 576] (fp32/bf16) in 4 bits into cache [R, 416] uint8, at rows
    dst_offset.. or at slots [n] (int64, -1 skips a row)."""
    n = x.shape[0]
    dev = _device(cache, "cache")
    _need(x, (n, SA_DQK), "x", None, dev)
    R = _cache_rows(cache, dev)
    if slots is not None:
        _need(slots, (n,), "slots", torch.int64, dev)
    _check(load().ds4idx_quantize_latents(_ptr(x), _in_dtype(x, "x"), n, _ptr(slots),
                                          int(dst_offset), _ptr(cache), R,
                                          _stream_ptr(stream, dev)),
           "ds4idx_quantize_latents")
    return cache


def read_latents(cache, rows=None, start: int = 0, n: int | None = None, out=None,
                 dtype=torch.bfloat16, stream=None):
    """The values of cache rows ``rows`` [n] (int64; rows outside the cache give zeros) or of rows
    start .. start + n - 1 (n None: to the end), as [n, 576] bf16 or fp32."""
    dev = _device(cache, "cache")
    R = _cache_rows(cache, dev)
    if rows is not None:
        n = rows.shape[0]
        _need(rows, (n,), "rows", torch.int64, dev)
    elif n is None:
        n = R - int(start)
    if out is None:
        out = _new((n, SA_DQK), dtype, cache.device, stream)
    _need(out, (n, SA_DQK), "out", None, dev)
    _check(load().ds4idx_read_latents(_ptr(cache), R, _ptr(rows), int(start), n, _ptr(out),
                                      _in_dtype(out, "out"), _stream_ptr(stream, dev)),
           "ds4idx_read_latents")
    return out


def _placement(T, kv_row0, page_table, page_size, token_seq, dev):
    """The ds4idx_placement of a call, or None (row = position)."""
    if kv_row0 is None and page_table is None:
        if token_seq is not None:
            raise ValueError("token_seq needs a page_table")
        return None
    w = Placement()
    if kv_row0 is not None:
        if page_table is not None or token_seq is not None:
            raise ValueError("kv_row0 and page_table exclude each other")
        _need(kv_row0, (T,), "kv_row0", torch.int64, dev)
        w.kv_row0 = kv_row0.data_ptr()
        return w
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seqs, pages_per_seq]")
    _need(page_table, tuple(page_table.shape), "page_table", torch.int32, dev)
    w.page_table = page_table.data_ptr()
    w.n_seqs, w.pages_per_seq, w.page_size = page_table.shape[0], page_table.shape[1], int(page_size)
    if token_seq is not None:
        _need(token_seq, (T,), "token_seq", torch.int32, dev)
        w.token_seq = token_seq.data_ptr()
    return w


def _ref(w):
    return None if w is None else ctypes.addressof(w)


def sparse_attention_q4(q, cache, idx, sm_scale: float, kv_row0=None, page_table=None,
                        page_size: int = 0, token_seq=None, out=None, lse=None, weights=None,
                        want_weights: bool = False, stream=None):
    """Attention of q [T, H, 576] (bf16, 1 <= H <= 128) over the selected rows of a 4-bit latent
    cache [R, 416]: idx [T, n_sel] int32 positions (negative = empty, n_sel <= 512). Position s of
    token t is cache row kv_row0[t] + s, or is found through page_table [n_seqs, pages] int32 with
    page_size positions a page and token_seq [T] int32 (None: row t).
    Returns (out [T, H, 512] bf16, lse [T, H] fp32, weights [T, n_sel] fp32 or None): weights is
    each entry's probability summed over the heads."""
    T, H, n_sel = q.shape[0], q.shape[1], idx.shape[1]
    dev = _device(q, "q")
    R = _cache_rows(cache, dev)
    _need(q, (T, H, SA_DQK), "q", torch.bfloat16, dev)
    _need(idx, (T, n_sel), "idx", torch.int32, dev)
    where = _placement(T, kv_row0, page_table, page_size, token_seq, dev)
    if out is None:
        out = _new((T, H, SA_DV), torch.bfloat16, q.device, stream)
    if lse is None:
        lse = _new((T, H), torch.float32, q.device, stream)
    if weights is None and want_weights:
        weights = _new((T, n_sel), torch.float32, q.device, stream)
    _need(out, (T, H, SA_DV), "out", torch.bfloat16, dev)
    _need(lse, (T, H), "lse", torch.float32, dev)
    if weights is not None:
        _need(weights, (T, n_sel), "weights", torch.float32, dev)
    _check(load().ds4idx_sparse_attention_q4(_ptr(q), _ptr(cache), R, _ptr(idx), _ref(where), T, H,
                                             SA_DQK, SA_DV, n_sel, float(sm_scale), _ptr(out),
                                             _ptr(lse), _ptr(weights), _stream_ptr(stream, dev)),
           "ds4idx_sparse_attention_q4")
    return out, lse, weights


# ---- the 8-bit latent cache

F8_ROW_BYTES = 640


def _cache_f8_rows(cache, scale, dev) -> int:
    rows = cache.shape[0]
    _need(cache, (rows, F8_ROW_BYTES), "cache", torch.uint8, dev)
    _need(scale, (rows,), "scale", torch.float32, dev)
    return rows


def quantize_latents_fp8(x, cache, scale, dst_offset: int = 0, slots=None, stream=None):
    """Writes latent rows x [n, 576] (fp32/bf16) as E4M3 codes and bf16 rotary dims into cache [R, 640]
    uint8 and their scales, powers of two, into scale [R] fp32, at rows dst_offset.. or at slots [n]
    (int64, -1 skips a row)."""
    n = x.shape[0]
    dev = _device(cache, "cache")
    _need(x, (n, SA_DQK), "x", None, dev)
    R = _cache_f8_rows(cache, scale, dev)
    if slots is not None:
        _need(slots, (n,), "slots", torch.int64, dev)
    _check(load().ds4idx_quantize_latents_fp8(_ptr(x), _in_dtype(x, "x"), n, _ptr(slots),
                                              int(dst_offset), _ptr(cache), _ptr(scale), R,
                                              _stream_ptr(stream, dev)),
           "ds4idx_quantize_latents_fp8")
    return cache, scale


def read_latents_fp8(cache, scale, rows=None, start: int = 0, n: int | None = None, out=None,
                     dtype=torch.bfloat16, stream=None):
    """The values of 8-bit cache rows ``rows`` [n] (int64; rows outside the cache give zeros) or of rows
    start .. start + n - 1 (n None: to the end), as [n, 576] bf16 or fp32."""
    dev = _device(cache, "cache")
    R = _cache_f8_rows(cache, scale, dev)
    if rows is not None:
        n = rows.shape[0]
        _need(rows, (n,), "rows", torch.int64, dev)
    elif n is None:
        n = R - int(start)
    if out is None:
        out = _new((n, SA_DQK), dtype, cache.device, stream)
    else:
        _need(out, (n, SA_DQK), "out", None, dev)
    _check(load().ds4idx_read_latents_fp8(_ptr(cache), _ptr(scale), R, _ptr(rows), int(start), n,
                                          _ptr(out), _in_dtype(out, "out"), _stream_ptr(stream, dev)),
           "ds4idx_read_latents_fp8")
    return out


# ---- trees of drafted tokens

CACHE_BF16, CACHE_FP8, CACHE_Q4 = 0, 1, 2
TREE_NODES = 64


def _cache_format(cache, scale, dev):
    """(ds4idx_cache_format, rows) of a latent cache."""
    rows = cache.shape[0]
    if cache.dtype == torch.bfloat16:
        _need(cache, (rows, SA_DQK), "cache", torch.bfloat16, dev)
        fmt = CACHE_BF16
    elif cache.shape[-1] == F8_ROW_BYTES:
        return CACHE_FP8, _cache_f8_rows(cache, scale, dev)
    else:
        fmt = CACHE_Q4
        _cache_rows(cache, dev)
    if scale is not None:
        raise ValueError("scale belongs to an 8-bit cache")
    return fmt, rows


def tree_attention(q, cache, kv_lens, mask, sm_scale: float, scale=None, kv_row0=None,
                   page_table=None, page_size: int = 0, token_seq=None,
                   max_kv_len: int | None = None, out=None, lse=None, workspace=None, stream=None):
    """Attention of the nodes of B drafted trees, q [B, N, H, 576] (bf16, N <= 64, H <= 128), over all
    rows of their sequences and the drafted rows that each node sees (see include/ds4idx.h).

    cache: bf16 [R, 576], or uint8 [R, 640] with its ``scale`` [R] (the powers of two that
    ``quantize_latents_fp8`` writes; others make NaN), or the 4-bit uint8 [R, 416]. The drafted rows
    stand behind the kv_lens [B] (int32) rows of their sequence; bit j of mask [B, N] (int64) says that
    a node sees drafted row j (itself among them; 0: padding). Position s of sequence b is row
    kv_row0[b] + s, or is found through page_table as in ``sparse_attention_q4`` (token_seq: the table
    row of each sequence). max_kv_len: a bound of kv_lens that the work is laid out for (None: what the
    pool or a table row holds). Returns (out [B, N, H, 512] bf16, lse [B, N, H] fp32)."""
    B, N, H = q.shape[0], q.shape[1], q.shape[2]
    dev = _device(q, "q")
    _need(q, (B, N, H, SA_DQK), "q", torch.bfloat16, dev)
    fmt, R = _cache_format(cache, scale, dev)
    _need(kv_lens, (B,), "kv_lens", torch.int32, dev)
    _need(mask, (B, N), "mask", torch.int64, dev)
    where = _placement(B, kv_row0, page_table, page_size, token_seq, dev)
    if max_kv_len is None:
        max_kv_len = R if page_table is None else min(R, page_table.shape[1] * int(page_size))
    if out is None:
        out = _new((B, N, H, SA_DV), torch.bfloat16, q.device, stream)
    else:
        _need(out, (B, N, H, SA_DV), "out", torch.bfloat16, dev)
    if lse is None:
        lse = _new((B, N, H), torch.float32, q.device, stream)
    else:
        _need(lse, (B, N, H), "lse", torch.float32, dev)
    if workspace is None:
        have = tree_attention_workspace(B, N, H, max_kv_len)
        if have:
            workspace = _new((have,), torch.uint8, q.device, stream)
    else:
        have = workspace.shape[0]
        _need(workspace, (have,), "workspace", torch.uint8, dev)
    _check(load().ds4idx_tree_attention(_ptr(q), fmt, _ptr(cache), _ptr(scale), R, _ptr(kv_lens),
                                        _ptr(mask), _ref(where), B, N, H, SA_DQK, SA_DV,
                                        int(max_kv_len), float(sm_scale), _ptr(out), _ptr(lse),
                                        _ptr(workspace), have, _stream_ptr(stream, dev)),
           "ds4idx_tree_attention")
    return out, lse


def tree_attention_workspace(B: int, N: int, H: int, max_kv_len: int) -> int:
    """Bytes of a ``workspace`` that tree_attention calls of these sizes, and of any ``max_kv_len`` up to
    this one, may share (on one stream)."""
    n = ctypes.c_int64()
    _check(load().ds4idx_tree_attention_workspace(B, N, H, int(max_kv_len), ctypes.addressof(n)),
           "ds4idx_tree_attention_workspace")
    return n.value


def tree_commit(arrays, kv_lens, path, n_accepted, kv_row0=None, page_table=None, page_size: int = 0,
                token_seq=None, new_lens=None, stream=None):
    """Keeps the accepted path of each drafted tree, in place in up to 8 per-row arrays of one pool: the
    row of position kv_lens[b] + j becomes that of kv_lens[b] + path[b, j], j < n_accepted[b]. kv_lens,
    n_accepted [B] and path [B, N] int32 on the device; the placement as in ``tree_attention``. Returns
    the new lengths, kv_lens + n_accepted."""
    B, N = path.shape[0], path.shape[1]
    arrays = list(arrays)
    dev = _device(path, "path")
    _need(path, (B, N), "path", torch.int32, dev)
    _need(kv_lens, (B,), "kv_lens", torch.int32, dev)
    _need(n_accepted, (B,), "n_accepted", torch.int32, dev)
    where = _placement(B, kv_row0, page_table, page_size, token_seq, dev)
    n = len(arrays)
    if n > 8:
        raise ValueError("at most 8 arrays")
    rows = arrays[0].shape[0] if n else 1
    d = ctypes.create_string_buffer(max(1, n) * _ROW_ARRAY.size)
    for k, a in enumerate(arrays):
        if a is None or a.get_device() != dev or a.shape[0] != rows or not a.is_contiguous():
            _need(a, (rows,) if a is None else (rows, *a.shape[1:]), f"arrays[{k}]", None, dev)
        at = a.data_ptr()
        row = a.element_size() * math.prod(a.shape[1:])
        _ROW_ARRAY.pack_into(d, k * _ROW_ARRAY.size, at, at, rows, rows, row, 0)
    if new_lens is None:
        new_lens = _new((B,), torch.int32, path.device, stream)
    else:
        _need(new_lens, (B,), "new_lens", torch.int32, dev)
    _check(load().ds4idx_tree_commit(_ptr(kv_lens), _ptr(path), _ptr(n_accepted), _ptr(new_lens),
                                     _ref(where), B, N, rows, n, ctypes.addressof(d),
                                     _stream_ptr(stream, dev)), "ds4idx_tree_commit")
    return new_lens


# ---- eviction by accumulated attention weight

_ROW_ARRAY = struct.Struct("=QQqqii")            # RowArray


def evict_accumulate(total, weights, idx, kv_row0=None, page_table=None, page_size: int = 0,
                     token_seq=None, stream=None):
    """total [R] int64 (units of 2^-32) += weights [T, n_sel] of the rows of idx [T, n_sel]; the
    placement as in ``sparse_attention_q4``."""
    T, n_sel = idx.shape[0], idx.shape[1]
    R = total.shape[0]
    dev = _device(total, "total")
    _need(total, (R,), "total", torch.int64, dev)
    _need(weights, (T, n_sel), "weights", torch.float32, dev)
    _need(idx, (T, n_sel), "idx", torch.int32, dev)
    where = _placement(T, kv_row0, page_table, page_size, token_seq, dev)
    _check(load().ds4idx_evict_accumulate(_ptr(total), R, _ptr(weights), _ptr(idx), _ref(where), T,
                                          n_sel, _stream_ptr(stream, dev)), "ds4idx_evict_accumulate")
    return total


def _i64(values):
    return array.array("q", values)


def _i64_address(a):
    return a.buffer_info()[0]


def evict_select(total, starts, seq_lens, keep, n_sink: int = 0, n_recent: int = 0, kept=None,
                 stream=None):
    """The positions that sequences keep (see include/ds4idx.h): starts, seq_lens, keep: B host ints
    each. Returns kept [B, max count] int32, ascending, then -1."""
    B = len(seq_lens)
    if len(starts) != B or len(keep) != B:
        raise ValueError("starts, seq_lens and keep need one entry per sequence")
    R = total.shape[0]
    dev = _device(total, "total")
    _need(total, (R,), "total", torch.int64, dev)
    if kept is None:
        width = max(map(min, keep, seq_lens), default=0)
        kept = _new((B, max(width, 0)), torch.int32, total.device, stream)
    _need(kept, (B, kept.shape[1]), "kept", torch.int32, dev)
    host = _i64([*starts, *seq_lens, *keep])
    at = _i64_address(host)
    _check(load().ds4idx_evict_select(_ptr(total), R, B, at, at + 8 * B, at + 16 * B, int(n_sink),
                                      int(n_recent), _ptr(kept), kept.shape[1],
                                      _stream_ptr(stream, dev)), "ds4idx_evict_select")
    return kept


def evict_compact(kept, seq_lens, keep, src_starts, dst_starts, srcs, dsts, stream=None):
    """Moves the kept rows (``evict_select`` of the same seq_lens and keep) of up to 8 per-row
    arrays: dsts[k][dst_starts[b] + i] = srcs[k][src_starts[b] + kept[b, i]]. Written rows must not
    overlap other written rows or any sequence's source rows, in any of the arrays."""
    B = len(seq_lens)
    if any(len(v) != B for v in (keep, src_starts, dst_starts)):
        raise ValueError("keep, src_starts and dst_starts need one entry per sequence")
    if len(srcs) != len(dsts):
        raise ValueError("srcs and dsts need the same number of arrays")
    dev = _device(kept, "kept")
    _need(kept, (B, kept.shape[1]), "kept", torch.int32, dev)
    n = len(srcs)
    if n > 8:
        raise ValueError("at most 8 arrays")
    d = ctypes.create_string_buffer(max(1, n) * _ROW_ARRAY.size)
    for k, (src, dst) in enumerate(zip(srcs, dsts)):
        shape, dshape = src.shape, dst.shape
        if not (src.get_device() == dev and dst.get_device() == dev and src.is_contiguous()
                and dst.is_contiguous() and src.dtype == dst.dtype and shape[1:] == dshape[1:]):
            _need(src, tuple(shape), f"srcs[{k}]", None, dev)
            _need(dst, (dshape[0], *shape[1:]), f"dsts[{k}]", src.dtype, dev)
        rows = shape[0]
        row = src.nbytes // rows if rows else src.element_size() * math.prod(shape[1:])
        _ROW_ARRAY.pack_into(d, k * _ROW_ARRAY.size, src.data_ptr(), dst.data_ptr(), rows,
                             dshape[0], row, 0)
    counts = list(map(min, keep, seq_lens))
    host = _i64([*src_starts, *seq_lens, *dst_starts, *counts])
    at = _i64_address(host)
    _check(load().ds4idx_evict_compact(_ptr(kept), kept.shape[1], B, at, at + 8 * B, at + 16 * B,
                                       at + 24 * B, n, ctypes.addressof(d),
                                       _stream_ptr(stream, dev)),
           "ds4idx_evict_compact")
    return dsts


def status_string(status: int) -> str:
    try:
        return load().ds4idx_status_string(int(status)).decode()
    except RuntimeError:
        return "library not loaded"


def _check(status: int, what: str):
    if status != OK:
        raise Ds4IdxError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current device's raw stream handle without building a Stream object (about 1 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device(t, name: str) -> int:
    """The device of a call: that of its first tensor. It has to be the current one, where the
    kernel is launched; ``_need`` holds the call's other tensors to it."""
    if t is None:
        raise ValueError(f"{name} is required")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _stream_ptr(stream, dev=None):
    """The stream of a call: the one given (it has to be of device ``dev``), else the current one."""
    if stream is not None:
        if dev is not None and getattr(stream, "device_index", dev) != dev:
            raise ValueError(f"stream is of cuda:{stream.device_index}, the tensors of cuda:{dev}")
        return stream.cuda_stream
    if _raw_stream is not None:
        if dev is not None:
            return _raw_stream(dev)
        if torch.cuda.is_initialized():
            return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _codes(t: torch.Tensor, dtype: int, name: str) -> torch.Tensor:
    if dtype == BF16:
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16 for a bf16 indexer")
        return t
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be float8_e4m3fn or uint8 E4M3 codes for an FP8 indexer")
    return t


def _new(shape, dtype, device, stream):
    """An output of a call on ``stream`` (None: the current one), from that stream's memory: what the
    current stream gave back may still be in use by its queued work. The current stream, on which
    the caller may go on with the output, is recorded as its user."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(t.device)
    if current != stream:
        t.record_stream(current)
    return t


def _need(t: torch.Tensor, shape, name: str, dtype=None, dev=None):
    """Raises unless t is a contiguous CUDA tensor of this shape (and dtype, and on device dev)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if ((t.is_cuda if dev is None else t.get_device() == dev) and t.shape == shape
            and t.is_contiguous() and (dtype is None or t.dtype == dtype)):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call's other tensors on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")


class Indexer:
    """One ds4idx handle (device workspace) for a dtype and maximum sizes."""

    def __init__(self, dtype: int = BF16, max_T: int = 65536, max_S: int = 65536,
                 max_batch: int = 1, n_heads: int = H_I, head_dim: int = D_I, topk: int = TOPK):
        self._lib = load()
        self.dtype = dtype
        self.topk = topk
        cfg = Config(n_heads, head_dim, topk, dtype, max_T, max_S, max_batch)
        h = ctypes.c_void_p()
        _check(self._lib.ds4idx_create(ctypes.byref(h), ctypes.byref(cfg)), "ds4idx_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.ds4idx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def score_topk(self, q, w, kcache, kscale=None, pos_offset: int = 0, out_idx=None,
                   out_score=None, stream=None, want_score: bool = True):
        """q [T,64,128], w [T,64] fp32, kcache [S,128], kscale [S] fp32 (FP8) -> (idx, score)."""
        T, S = q.shape[0], kcache.shape[0]
        q = _codes(q, self.dtype, "q")
        kcache = _codes(kcache, self.dtype, "kcache")
        _need(q, (T, H_I, D_I), "q")
        _need(w, (T, H_I), "w", torch.float32)
        _need(kcache, (S, D_I), "kcache")
        if kscale is not None:
            _need(kscale, (S,), "kscale", torch.float32)
        dev = q.device
        if out_idx is None:
            out_idx = _new((T, self.topk), torch.int32, dev, stream)
        if out_score is None and want_score:
            out_score = _new((T, self.topk), torch.float32, dev, stream)
        _need(out_idx, (T, self.topk), "out_idx", torch.int32)
        if out_score is not None:
            _need(out_score, (T, self.topk), "out_score", torch.float32)
        st = self._lib.ds4idx_score_topk(self._h, _ptr(q), _ptr(w), _ptr(kcache), _ptr(kscale),
                                         T, S, int(pos_offset), self.topk, _ptr(out_idx),
                                         _ptr(out_score), _stream_ptr(stream))
        _check(st, "ds4idx_score_topk")
        return out_idx, out_score

    def score_topk_batched(self, q, w, kcache, kscale, pos_offsets, out_idx=None, out_score=None,
                           stream=None):
        """q [B,T,64,128], w [B,T,64], kcache [B,S,128], kscale [B,S]; pos_offsets: B ints."""
        B, T, S = q.shape[0], q.shape[1], kcache.shape[1]
        q = _codes(q, self.dtype, "q")
        kcache = _codes(kcache, self.dtype, "kcache")
        _need(q, (B, T, H_I, D_I), "q")
        _need(w, (B, T, H_I), "w", torch.float32)
        _need(kcache, (B, S, D_I), "kcache")
        if kscale is not None:
            _need(kscale, (B, S), "kscale", torch.float32)
        dev = q.device
        if out_idx is None:
            out_idx = _new((B, T, self.topk), torch.int32, dev, stream)
        if out_score is None:
            out_score = _new((B, T, self.topk), torch.float32, dev, stream)
        _need(out_idx, (B, T, self.topk), "out_idx", torch.int32)
        _need(out_score, (B, T, self.topk), "out_score", torch.float32)
        pos = (ctypes.c_int64 * B)(*[int(x) for x in pos_offsets])
        st = self._lib.ds4idx_score_topk_batched(self._h, B, _ptr(q), _ptr(w), _ptr(kcache),
                                                 _ptr(kscale), T, S, ctypes.cast(pos, ctypes.c_void_p),
                                                 self.topk, _ptr(out_idx), _ptr(out_score),
                                                 _stream_ptr(stream))
        _check(st, "ds4idx_score_topk_batched")
        return out_idx, out_score

    def score_topk_varlen(self, q, w, cu_seqlens_q, kcache, kscale, seq_lens, pos_offsets,
                          kv_start=None, page_table=None, page_size: int = 0, out_idx=None,
                          out_score=None, stream=None):
        """Sequences of different lengths in one launch (see include/ds4idx.h).

        q [Q, 64, 128], w [Q, 64]: packed queries, sequence b owning rows
        cu_seqlens_q[b]..cu_seqlens_q[b+1]-1 (host ints, B + 1 of them). kcache [R, 128] (+ kscale
        [R]) is the key pool: sequence b's keys start at pool row kv_start[b], or are found through
        page_table [B, P] (int32, on the device) with page_size keys per page.
        seq_lens, pos_offsets: B host ints. Returns (out_idx, out_score), [Q, topk].
        """
        B = len(seq_lens)
        Q, R = q.shape[0], kcache.shape[0]
        q = _codes(q, self.dtype, "q")
        kcache = _codes(kcache, self.dtype, "kcache")
        _need(q, (Q, H_I, D_I), "q")
        _need(w, (Q, H_I), "w", torch.float32)
        _need(kcache, (R, D_I), "kcache")
        if kscale is not None:
            _need(kscale, (R,), "kscale", torch.float32)
        if len(cu_seqlens_q) != B + 1 or len(pos_offsets) != B:
            raise ValueError("cu_seqlens_q needs B + 1 entries and pos_offsets B")
        if page_table is not None:
            _need(page_table, tuple(page_table.shape), "page_table", torch.int32)
            if page_table.dim() != 2 or page_table.shape[0] != B:
                raise ValueError("page_table must be [B, pages_per_seq]")
        dev = q.device
        if out_idx is None:
            out_idx = _new((Q, self.topk), torch.int32, dev, stream)
        if out_score is None:
            out_score = _new((Q, self.topk), torch.float32, dev, stream)
        _need(out_idx, (Q, self.topk), "out_idx", torch.int32)
        _need(out_score, (Q, self.topk), "out_score", torch.float32)
        I64 = ctypes.c_int64
        cu = (I64 * (B + 1))(*[int(x) for x in cu_seqlens_q])
        sl = (I64 * B)(*[int(x) for x in seq_lens])
        po = (I64 * B)(*[int(x) for x in pos_offsets])
        ks = None if kv_start is None else (I64 * B)(*[int(x) for x in kv_start])
        vp = ctypes.c_void_p
        st = self._lib.ds4idx_score_topk_varlen(
            self._h, B, _ptr(q), _ptr(w), ctypes.cast(cu, vp), _ptr(kcache), _ptr(kscale), R,
            None if ks is None else ctypes.cast(ks, vp), _ptr(page_table), int(page_size),
            0 if page_table is None else int(page_table.shape[1]), ctypes.cast(sl, vp),
            ctypes.cast(po, vp), self.topk, _ptr(out_idx), _ptr(out_score), _stream_ptr(stream))
        _check(st, "ds4idx_score_topk_varlen")
        return out_idx, out_score

    def score_dense_debug(self, q, w, kcache, kscale=None, pos_offset: int = 0, out=None,
                          stream=None):
        """fp32 scores [T, S] as the selection kernels see them (-inf where not visible)."""
        T, S = q.shape[0], kcache.shape[0]
        q = _codes(q, self.dtype, "q")
        kcache = _codes(kcache, self.dtype, "kcache")
        _need(q, (T, H_I, D_I), "q")
        _need(w, (T, H_I), "w", torch.float32)
        _need(kcache, (S, D_I), "kcache")
        if kscale is not None:
            _need(kscale, (S,), "kscale", torch.float32)
        if out is None:
            out = _new((T, S), torch.float32, q.device, stream)
        _need(out, (T, S), "out", torch.float32)
        st = self._lib.ds4idx_score_dense_debug(self._h, _ptr(q), _ptr(w), _ptr(kcache),
                                                _ptr(kscale), T, S, int(pos_offset), _ptr(out),
                                                _stream_ptr(stream))
        _check(st, "ds4idx_score_dense_debug")
        return out

    def debug_wait_test(self, wait_limit_ns: int = 2_000_000_000, withhold: bool = False):
        """Test support: bounded-wait limit for later calls, and one withheld arrival."""
        _check(self._lib.ds4idx_debug_wait_test(self._h, int(wait_limit_ns), 1 if withhold else 0),
               "ds4idx_debug_wait_test")

    def sync_status(self, stream=None):
        _check(self._lib.ds4idx_sync_status(self._h, _stream_ptr(stream)), "ds4idx_sync_status")
