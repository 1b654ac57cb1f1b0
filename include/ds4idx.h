/*
 * ds4idx — Lightning Indexer for DeepSeek-V4-style sparse attention on GB300 (sm_103a).
 *
 * The operation. "DeepSeek V4 Flash 추론을 1.6초로 줄인 ds4 최적화" (aitrends), sections
 * 섹션별 상세 and 용어 해설, describes the Lightning Indexer as the kernel that picks, for every
 * query token, the key positions sparse attention will read, with a Top-512 selection after a
 * scorer. The pages print no formula; the score computed here is the DeepSeek indexer score
 *
 *     I[t,s] = kscale[s] * sum_{j < H_I} w[t,j] * max(0, sum_{i < d_I} q[t,j,i] * k[s,i])
 *
 * over H_I = 64 index heads of width d_I = 128, for every causally visible key
 * s <= p(t) = pos_offset + t (a token sees itself), with kscale[s] = 1 for bf16 caches. For each
 * query the library returns the top-k (k = 512) keys ordered by score descending, ties going to
 * the lower key index; when fewer than k keys are visible, all of them are returned and the
 * remaining slots are (-1, -inf). "DeepSeek V4 Flash는 단일 AMD MI300X에서 실행됩니다", section
 * 두 가지 핵심 정확성 수정 사항 (FP8 형식 불일치), gives the FP8 E4M3 indexer key cache; here
 * it is OCP E4M3FN (largest finite 448) with one fp32 scale per key.
 *
 * Arithmetic: products of bf16 (or E4M3) operands accumulate in fp32 on the tensor cores; the
 * ReLU, the weighted head sum and the key scale are fp32. Scores match an fp64 evaluation within
 * 1e-4 * (1 + |I|) for bf16 inputs.
 *
 * Conventions for every entry point:
 *  - All tensor arguments are DEVICE pointers on the current CUDA device, row-major, dense,
 *    16-byte aligned, owned by the caller. Nothing is copied or retained after the call.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream). Calls are asynchronous: they
 *    enqueue kernels on `stream` and return; outputs are valid once the stream has reached that
 *    point. No entry point synchronises the host except ds4idx_sync_status and ds4idx_destroy.
 *    Kernels are launched as programmatic dependents of the previous kernel on `stream`: their
 *    blocks may start (shared memory and tensor-memory setup) while that kernel finishes, but
 *    touch no global memory before it has completed, so stream order holds as usual.
 *  - A handle is not thread-safe: use one handle per stream / host thread. The handle owns a
 *    small device workspace (error word, per-split candidate lists) allocated at create; the
 *    compute entry points allocate nothing.
 *  - Return value: DS4IDX_OK (0) or a negative ds4idx_status. Argument errors are detected on
 *    the host before anything is enqueued. Inputs must be finite (not checked on the device).
 */
#ifndef DS4IDX_H_
#define DS4IDX_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DS4IDX_OK = 0,
  DS4IDX_ERR_INVALID_ARG = -1,    /* null pointer, misalignment, size out of range, mismatch */
  DS4IDX_ERR_UNSUPPORTED = -2,    /* shape/dtype not built (H_I != 64, d_I != 128, k != 512),
                                     or the current device is not sm_103 */
  DS4IDX_ERR_ALLOC = -3,          /* workspace allocation failed at create */
  DS4IDX_ERR_LAUNCH = -4,         /* a kernel launch or an enqueue failed */
  DS4IDX_ERR_DEVICE_TIMEOUT = -5, /* a kernel gave up on a bounded device-side wait */
  DS4IDX_ERR_CUDA = -6,           /* another CUDA runtime or driver call failed */
  DS4IDX_ERR_SCRATCH_LIMIT = -7   /* request needs more than the fixed scratch of the
                                     no-allocation entry point */
} ds4idx_status;

/* Element types. q and kcache of the indexer are BF16 or FP8_E4M3 codes; F32 is accepted as the
 * input of the FP8 cache writer only. */
typedef enum { DS4IDX_BF16 = 0, DS4IDX_FP8_E4M3 = 1, DS4IDX_F32 = 2 } ds4idx_dtype;

typedef struct {
  int32_t n_heads;   /* H_I; must be 64 */
  int32_t head_dim;  /* d_I; must be 128 */
  int32_t topk;      /* k; must be 512 */
  int32_t dtype;     /* ds4idx_dtype of q and kcache */
  int64_t max_T;     /* largest query count per sequence passed to any call (>= 1) */
  int64_t max_S;     /* largest key count per sequence (>= 1, < 2^31) */
  int64_t max_batch; /* largest B for ds4idx_score_topk_batched (1..64) */
} ds4idx_config;

typedef struct ds4idx_handle* ds4idx_t;

/* Creates a handle for the current CUDA device and allocates its workspace.
 * Errors: INVALID_ARG (null out/cfg, ranges), UNSUPPORTED (shape or device), ALLOC, CUDA.
 * On error *out is set to NULL. */
int ds4idx_create(ds4idx_t* out, const ds4idx_config* cfg);

/* Scores and selects for one sequence.
 *  q         [T, 64, 128]  bf16, or E4M3 codes (uint8) for FP8 handles. For FP8 the per-token q
 *                          scale is folded into w by the caller (w[t,j] * qscale[t]); this is exact
 *                          because ReLU is positively homogeneous.
 *  w         [T, 64]       fp32 head weights.
 *  kcache    [S, 128]      bf16, or E4M3 codes for FP8 handles.
 *  kscale    [S]           fp32 per-key scale (>= 0) for FP8; must be NULL for bf16.
 *  T         number of query tokens (0 <= T <= max_T; T = 0 is a no-op).
 *  S         number of keys in the cache (1 <= S <= max_S).
 *  pos_offset position of query 0 (>= 0); query t sits at p(t) = pos_offset + t and sees keys
 *            0..min(p(t), S - 1). A well-formed prefill or decode call has pos_offset + T <= S
 *            (every query's own key is in the cache); positions past the cache see all S keys.
 *  topk      must equal the handle's topk (512).
 *  out_idx   [T, topk] int32, written: key indices, best first; -1 in unused slots.
 *  out_score [T, topk] fp32, written: the scores of out_idx (-inf in unused slots); may be NULL.
 */
int ds4idx_score_topk(ds4idx_t h, const void* q, const float* w, const void* kcache,
                      const float* kscale, int64_t T, int64_t S, int64_t pos_offset, int32_t topk,
                      int32_t* out_idx, float* out_score, void* stream);

/* B independent sequences in one launch (batched decode or chunked prefill). Every array gains
 * a leading [B] dimension with a dense stride: q [B, T, 64, 128], w [B, T, 64],
 * kcache [B, S, 128], kscale [B, S] (FP8), out_idx / out_score [B, T, topk].
 * pos_offsets is a HOST array of B positions (>= 0), one per sequence.
 * 1 <= B <= max_batch. Other arguments as in ds4idx_score_topk. */
int ds4idx_score_topk_batched(ds4idx_t h, int32_t B, const void* q, const float* w,
                              const void* kcache, const float* kscale, int64_t T, int64_t S,
                              const int64_t* pos_offsets, int32_t topk, int32_t* out_idx,
                              float* out_score, void* stream);

/* Variable-length, optionally paged batch: B independent sequences, each with its own number
 * of queries, its own key count and its own position, in one launch (continuous-batching decode
 * and mixed chunked prefill). The pages have no interface for this; the concurrency sweep and
 * the hybrid KV-cache rows of "DeepSeek V4 Flash는 단일 AMD MI300X에서 실행됩니다" (동시성 스윕,
 * 프로덕션 수준 튜닝 세부 사항) are the serving setting it is for.
 *  q, w          packed queries of all sequences: q [Q, 64, 128], w [Q, 64] fp32, where
 *                Q = cu_seqlens_q[B]; sequence b owns rows cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1
 *                (cu_seqlens_q: HOST int64 [B + 1], starting at 0, non-decreasing; a sequence
 *                may have no query).
 *  kcache        the key pool [pool_rows, 128] (bf16 or E4M3 codes), pool_rows < 2^31;
 *  kscale        [pool_rows] fp32 for FP8 handles, NULL for bf16.
 *  Keys of sequence b (S_b = seq_lens[b] >= 1, HOST int64 [B]) are found either
 *   - contiguously: kv_start (HOST int64 [B]) gives the pool row of its key 0, or
 *   - through a page table: page_table (DEVICE int32 [B, pages_per_seq], 4-byte aligned) lists
 *     the pages of sequence b in key order; page_size keys per page (a multiple of 64); key s
 *     lives in pool row page_table[b][s / page_size] * page_size + s % page_size. Page ids are
 *     not checked on the host: an id outside the pool reads as zero keys (wrong results, no
 *     out-of-bounds access).
 *    Exactly one of kv_start and page_table is given.
 *  pos_offsets   HOST int64 [B]: the position of each sequence's first query (as in
 *                ds4idx_score_topk: query t sees keys 0 .. min(pos + t, S_b - 1)).
 *  out_idx / out_score  [Q, topk], rows packed like q. Key indices are positions within the
 *                sequence (0 .. S_b - 1), not pool rows.
 * Limits: B <= max_batch, every T_b <= max_T and S_b <= max_S of the handle. Key-range splits of
 * short sequences are fitted to the handle's workspace. Errors: INVALID_ARG, LAUNCH, CUDA. */
int ds4idx_score_topk_varlen(ds4idx_t h, int32_t B, const void* q, const float* w,
                             const int64_t* cu_seqlens_q, const void* kcache, const float* kscale,
                             int64_t pool_rows, const int64_t* kv_start,
                             const int32_t* page_table, int32_t page_size, int32_t pages_per_seq,
                             const int64_t* seq_lens, const int64_t* pos_offsets, int32_t topk,
                             int32_t* out_idx, float* out_score, void* stream);

/* Debug/test entry: the fp32 scores the selection kernels see, before selection.
 * out_scores [T, S] fp32, written: I[t,s] for visible s, -inf for s > p(t). Same inputs and
 * rules as ds4idx_score_topk; it runs the same scoring code path. */
int ds4idx_score_dense_debug(ds4idx_t h, const void* q, const float* w, const void* kcache,
                             const float* kscale, int64_t T, int64_t S, int64_t pos_offset,
                             float* out_scores, void* stream);

/* Synchronises `stream`, then reads and clears the handle's device error word.
 * Returns DEVICE_TIMEOUT if any kernel since the last check gave up on a bounded wait
 * (its outputs are then undefined), CUDA if the synchronisation reported an error, else OK. */
int ds4idx_sync_status(ds4idx_t h, void* stream);

/* Synchronises the device, frees the workspace and the handle. NULL is accepted (no-op). */
int ds4idx_destroy(ds4idx_t h);

/* Static English text for a status code. Never NULL. */
const char* ds4idx_status_string(int status);

/* Library ABI version: (major << 16) | minor. */
int ds4idx_version(void);

/* Number of kernels this library has enqueued in this process (all handles and entry points).
 * Instrumentation for benchmarks: a successful compute call adds the launches it made. */
uint64_t ds4idx_kernels_launched(void);

/* No-allocation variant of ds4idx_score_topk_batched. The pages have no counterpart: this is an
 * integration aid for callers that cannot allocate device memory when they call the indexer.
 * Examples are a serving engine that reserved all free HBM for its own KV-cache pool at start-up,
 * and a host framework whose allocator must account for every device byte. Neither can let a
 * library call cudaMalloc behind its back, and it may not be able to hold a ds4idx handle
 * either, since a handle allocates its workspace at create.
 *
 * This entry point takes no handle and allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library call). Its scratch, the per-split candidate lists of short sequences plus
 * an error word and the split counters, lives in one fixed array (16 MiB of lists, 1 MiB of
 * counters) compiled into the library as file-scope __device__ storage. Every GPU that loads the
 * library holds that array until the process exits.
 *  - dtype is a ds4idx_dtype. All other arguments, layouts and rules are those of
 *    ds4idx_score_topk_batched, with 1 <= B <= 64, 0 <= T, 1 <= S < 2^31 and topk = 512.
 *  - Limit: the array holds 2^21 list words (16 MiB) and the split counters (merge ticket and the
 *    splits' published bins) of 4096 query blocks. Short sequences (decode, small chunks) split
 *    their key range over several CTAs, and each split publishes a list of 512 words per query
 *    (1152 per one-query sequence). Here the split count steps down from the one
 *    ds4idx_score_topk_batched would use until the lists fit (B * T * splits * 512 <= 2^21); one
 *    split needs no list, so every valid call runs, only with fewer CTAs where the handle path
 *    would split further. Outputs are the same as the handle path's. DS4IDX_ERR_SCRATCH_LIMIT is
 *    returned only if a plan still did not fit.
 *  - Set-up: the first call on each device looks up the array's device address and sets kernel
 *    attributes, with that device current. Make that first call before any stream capture.
 *  - Argument errors return INVALID_ARG before anything is enqueued or the array is touched.
 *  - Sharing: all calls use the same array, and it keeps the previous call's contents. The error
 *    word and the split counters the call uses are cleared on `stream` at the start of every
 *    valid call; the candidate lists are always fully written before they are read. Calls that
 *    can overlap on the GPU (different streams or host threads without ordering between them)
 *    race on the array and corrupt each other's outputs, so order them, for example on one
 *    stream.
 *  - A kernel that gives up on a bounded device wait records it in the array's error word. This
 *    entry point cannot report it; callers that need that status use a handle and
 *    ds4idx_sync_status. */
int ds4idx_score_topk_batched_noalloc(int32_t dtype, int32_t B, const void* q, const float* w,
                                      const void* kcache, const float* kscale, int64_t T,
                                      int64_t S, const int64_t* pos_offsets, int32_t topk,
                                      int32_t* out_idx, float* out_score, void* stream);

/* ---- FP8 index-cache writer: the step before an FP8 indexer call.
 * "DeepSeek V4 Flash는 단일 AMD MI300X에서 실행됩니다", section 두 가지 핵심 정확성 수정 사항
 * (FP8 형식 불일치): the indexer key cache is written as FP8 E4M3, and the format's largest
 * finite value sets the scale. Here the format is OCP E4M3FN (largest finite 448) with one fp32
 * scale per token row:
 *     scale = absmax(row) / 448,  code[i] = E4M3(clamp(x[i] / scale, -448, 448)),
 * each fp32 operation correctly rounded, the conversion round-to-nearest-even; a row whose
 * scale is 0 gets codes 0. The results are bit-exact functions of the inputs. Inputs must be
 * finite. Both calls are asynchronous on `stream` and allocate nothing. */

/* Quantises n new key rows k [n, 128] (in_dtype DS4IDX_F32 or DS4IDX_BF16, 16-byte aligned)
 * into the index cache: row i goes to cache row slots[i] when `slots` (device int64 [n]) is
 * given, else to dst_offset + i. kcache [cache_rows, 128] uint8 E4M3 codes (16-byte aligned),
 * kscale [cache_rows] fp32. Slots outside [0, cache_rows) (e.g. -1 for padding tokens) are
 * skipped. Errors: INVALID_ARG (dtype, null or misaligned pointer, n < 0, a contiguous range
 * past cache_rows), LAUNCH. n = 0 is a no-op. */
int ds4idx_quantize_keys(const void* k, int32_t in_dtype, int64_t n, const int64_t* slots,
                         int64_t dst_offset, uint8_t* kcache, float* kscale, int64_t cache_rows,
                         void* stream);

/* Quantises the queries of an FP8 indexer call: q [T, 64, 128] (DS4IDX_F32 or DS4IDX_BF16)
 * with one scale per token over all 64 x 128 values into q_codes [T, 64, 128] uint8, and folds
 * the scale into the head weights, w_out[t, j] = w[t, j] * qscale[t] (fp32, correctly rounded;
 * exact in the score because ReLU is positively homogeneous). w [T, 64] fp32; qscale [T] fp32
 * receives the scales and may be NULL. w_out may equal w (in place). Errors: INVALID_ARG,
 * LAUNCH. T = 0 is a no-op. */
int ds4idx_quantize_queries(const void* q, int32_t in_dtype, int64_t T, const float* w,
                            uint8_t* q_codes, float* w_out, float* qscale, void* stream);

/* ---- Merge of key-sharded Top-k lists (the exchange step of a key-range-sharded indexer).
 * When the keys of a sequence are split into disjoint ranges (shards) and each shard's Top-k is
 * computed on its own (ds4idx_score_topk on that range), the union of the shards' lists holds
 * the global Top-k: a key among the k best of all keys is also among the k best of its shard.
 * This call merges them: for every row it takes the k largest (score, key) pairs of all lists,
 * ordered by score descending with ties to the lower key, padded with (-1, -inf).
 *  in_idx, in_score  DEVICE [n_lists, rows, topk] int32 / fp32: each list's indices are local to
 *                    its shard (-1 = empty slot); 1 <= n_lists <= 16.
 *  idx_offsets       HOST int64 [n_lists]: the first key of each shard, added to its indices
 *                    (merged keys must stay below 2^31).
 *  row0              HOST int64 [n_lists] or NULL: list l has no entries for rows < row0[l]
 *                    (queries that see none of its keys); NULL = all rows.
 *  out_idx, out_score DEVICE [rows, topk] (out_score may be NULL). topk must be 512.
 * Shards must be disjoint (a key in two lists would be kept twice). Asynchronous on `stream`,
 * allocates nothing. Errors: INVALID_ARG, LAUNCH, CUDA. */
int ds4idx_merge_topk(int32_t n_lists, int64_t rows, const int32_t* in_idx,
                      const float* in_score, const int64_t* idx_offsets, const int64_t* row0,
                      int32_t topk, int32_t* out_idx, float* out_score, void* stream);

/* ---- Sparse attention over the selected keys: the step that consumes the indexer's output.
 * "DeepSeek V4 Flash 추론을 1.6초로 줄인 ds4 최적화", 용어 해설 (희소 어텐션, Lightning Indexer):
 * sparse attention computes only some token pairs, and the indexer picks the positions. For
 * query token t and head h over its selected positions J(t) (one row of out_idx; -1 = empty):
 *     s_j = sm_scale * q[t,h,:] . kv[j,:],   out[t,h,:] = sum_j softmax(s)_j * kv[j, 0:d_v],
 *     lse[t,h] = log sum_j exp(s_j)          (natural log; -inf and out = 0 if J(t) is empty)
 * with one latent row per position shared by all heads (the value is the row's first d_v dims).
 *  q       DEVICE [T, n_heads, d_qk] bf16, 16-byte aligned.
 *  kv      DEVICE [kv_rows, d_qk] bf16 (1 <= kv_rows < 2^31), 16-byte aligned.
 *  idx     DEVICE [T, topk] int32: selected positions; position s of token t is kv row
 *          kv_row0[t] + s (kv_row0: DEVICE int64 [T], or NULL for 0). Positions whose row falls
 *          outside [0, kv_rows) are treated as empty. Selected positions must be distinct.
 *  out     DEVICE [T, n_heads, d_v] bf16; lse DEVICE [T, n_heads] fp32 or NULL.
 * Built shape: n_heads = 128, d_qk = 576, d_v = 512, topk = 512 (else UNSUPPORTED); sm_scale > 0.
 * Arithmetic: bf16 products with fp32 accumulation on the tensor cores, fp32 softmax, the
 * probabilities rounded to bf16 for the value product, the output rounded to bf16.
 * Asynchronous on `stream`, allocates nothing. Bounded device waits that run out are recorded
 * for ds4idx_sparse_attention_status. Errors: INVALID_ARG, UNSUPPORTED, LAUNCH, CUDA. */
int ds4idx_sparse_attention(const void* q, const void* kv, int64_t kv_rows, const int32_t* idx,
                            const int64_t* kv_row0, int64_t T, int32_t n_heads, int32_t d_qk,
                            int32_t d_v, int32_t topk, float sm_scale, void* out, float* lse,
                            void* stream);

/* Synchronises `stream`, then reads and clears the sparse-attention error word: DEVICE_TIMEOUT if
 * a kernel gave up on a bounded wait since the last check (outputs undefined), CUDA if the
 * synchronisation failed, else OK. */
int ds4idx_sparse_attention_status(void* stream);

/* ---- Rotary positions of queries and keys: the step before the cache writer, the indexer and the
 * attention. Every pair (a, b) of the rotated slice of a head of token t becomes
 *     scale * (a cos(x) - b sin(x), a sin(x) + b cos(x)),   x = positions[t] * inv_freq[pair],
 * where pair i is elements (2i, 2i + 1) (interleaved) or (i, i + rot_dim / 2) (halves). With
 * inverse != 0 the angle is negated (same scale): the transpose, which maps the gradient of the
 * output to the gradient of the input. The product with the frequencies that ds4idx_rotary_freqs
 * makes is exact modulo one turn at any position, so the angle is off by |position| times what the
 * frequency is; the rotation is fp32, rounded once to the tensor's type. */

typedef enum {
  DS4IDX_ROTARY_PLAIN = 0,  /* inv_freq[i] = base^(-2 i / rot_dim) */
  DS4IDX_ROTARY_LINEAR = 1, /* divided by factor */
  DS4IDX_ROTARY_YARN = 2    /* YaRN: pairs that turn more than beta_fast times within the original
                               context keep their frequency, those that turn less than beta_slow
                               times are divided by factor, a ramp joins them; scale is
                               0.1 ln(factor) + 1 */
} ds4idx_rotary_scaling;

/* One tensor of a rotary call. x and out point at the first rotated element of token 0, head 0
 * (DEVICE, aligned to an element); element (t, h, i) lies t * stride_t + h * stride_h + i elements
 * further (strides in elements; rotated elements adjacent). out may equal x with equal strides
 * (in place). Otherwise no out of a call may overlap itself (a stride of 0), another out or any x:
 * refused, as are an out and another tensor whose spans of memory interleave at different token
 * strides. Elements outside the slice are not touched.
 * 16-byte aligned pointers and strides move 16 bytes a thread; others 2 or 4. */
typedef struct {
  const void* x;
  void* out;
  int32_t dtype;       /* DS4IDX_BF16 or DS4IDX_F32 */
  int32_t interleaved; /* else halves */
  int32_t n_heads;     /* 1..65536 */
  int32_t reserved;
  int64_t x_stride_t, x_stride_h, out_stride_t, out_stride_h;
} ds4idx_rotary_tensor;

/* Host computation, no device access: fills freqs[rot_dim / 2] with the frequencies as 64-bit
 * fractions of a turn per position (inv_freq / 2 pi * 2^64) and *scale. rot_dim even, 2..256;
 * base > 1; factor >= 1; original_max_position >= 1 and 0 < beta_slow <= beta_fast for YaRN. A
 * frequency is off by at most (5 + ln base) * 2^-53 of it, (9 + ln base + min(factor, 256)) * 2^-53
 * with YaRN (double arithmetic), and 2^-65 turn. */
int ds4idx_rotary_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                        int64_t original_max_position, double beta_fast, double beta_slow,
                        uint64_t* freqs, float* scale);

/* Rotates 1..4 tensors of the same T tokens in one launch. tensors and freqs are HOST arrays (read
 * before the call returns); positions DEVICE int64 [T] (any sign). Asynchronous on `stream`,
 * allocates nothing. Errors: INVALID_ARG, LAUNCH, CUDA. T = 0 is a no-op. */
int ds4idx_rotary(int32_t n_tensors, const ds4idx_rotary_tensor* tensors, int64_t T,
                  int32_t rot_dim, const int64_t* positions, const uint64_t* freqs, float scale,
                  int32_t inverse, void* stream);

/* ---- The 4-bit latent cache: the latent rows of sparse attention (576 = 512 value dims + 64
 * rotary dims) in 416 bytes instead of 1152. One row:
 *   bytes   0..255  512 integers n in -7..7, stored as n + 8 in four bits: of each eight dims (one
 *                   little-endian 32-bit word) dim 2p stands in bits 4p..4p+3 and dim 2p + 1 in
 *                   bits 16+4p..16+4p+3;
 *   bytes 256..287  32 scale codes, one for each 16 dims: code c = 2^(c / 8 - 20) * (1 + (c % 8) / 8)
 *                   (integer division; 1e-6 .. 3840);
 *   bytes 288..415  the 64 rotary dims as bf16.
 * Dim i of the first 512 is n * scale, exact in bf16. A scale is the code nearest to absmax / 7 of
 * its 16 dims (ties to the even code, clamped to 0..255), n is x / scale rounded to nearest, ties
 * to even, clamped to -7..7: both are exact decisions, so the bytes are a function of the inputs.
 * Inputs must be finite. The cache pointer is 32-byte aligned. */

/* Writes n rows x [n, 576] (in_dtype DS4IDX_F32 or DS4IDX_BF16, 16-byte aligned) into cache rows
 * slots[i] (DEVICE int64 [n], distinct: of two rows for one slot each byte may come from either; rows
 * outside the cache, e.g. -1, are skipped) or dst_offset + i (slots NULL). Asynchronous, allocates nothing. Errors: INVALID_ARG, LAUNCH. n = 0 is a no-op. */
int ds4idx_quantize_latents(const void* x, int32_t in_dtype, int64_t n, const int64_t* slots,
                            int64_t dst_offset, uint8_t* cache, int64_t cache_rows, void* stream);

/* Reads n rows back as values: out [n, 576] (out_dtype DS4IDX_F32 or DS4IDX_BF16, both exact;
 * 16-byte aligned) from cache rows rows[i] (DEVICE int64 [n]; rows outside the cache read as zeros)
 * or start + i (rows NULL, start + n <= cache_rows). Errors as above. */
int ds4idx_read_latents(const uint8_t* cache, int64_t cache_rows, const int64_t* rows,
                        int64_t start, int64_t n, void* out, int32_t out_dtype, void* stream);

/* Where the tokens of a call find position s of their sequence in a pool of rows: pool row
 * kv_row0[t] + s (kv_row0 DEVICE int64 [T]; NULL = 0), or through a page table. */
typedef struct {
  const int64_t* kv_row0;    /* DEVICE int64 [T] or NULL; must be NULL with a page table */
  const int32_t* page_table; /* DEVICE int32 [n_seqs, pages_per_seq] or NULL */
  const int32_t* token_seq;  /* DEVICE int32 [T]: the table row of token t; NULL = row t */
  int32_t page_size;         /* positions per page (>= 1, any size) */
  int32_t pages_per_seq;
  int64_t n_seqs;
} ds4idx_placement;
/* A position past its table row, a table row outside 0..n_seqs-1, or a pool row outside the pool
 * makes the list entry empty: nothing out of range is read. */

/* Attention of q over the selected rows of a 4-bit latent cache. For token t, head h, over the
 * non-empty entries j of its list:
 *     s_j = sm_scale * q[t,h,:] . row_j,    out[t,h,:] = sum_j softmax(s)_j * row_j[0:512],
 *     lse[t,h] = log sum_j exp(s_j) (natural; -inf and out = 0 if the list is empty),
 *     weights[t,j] = sum_h softmax(s)_j (0 in empty entries).
 *  q        [T, n_heads, 576] bf16, 16-byte aligned; n_heads 1..128 (128 uses the tensor cores
 *           fully; fewer heads cost the same time).
 *  cache    [kv_rows, 416], 32-byte aligned, 1 <= kv_rows < 2^31.
 *  idx      [T, n_sel] int32 positions, 1 <= n_sel <= 512; negative = empty, anywhere in the list
 *           (the indexer's lists: n_sel = 512). Positions of a list must be distinct.
 *  where    HOST, may be NULL (row = position).
 *  out      [T, n_heads, 512] bf16, 32-byte aligned; lse [T, n_heads] fp32 or NULL; weights
 *           [T, n_sel] fp32 or NULL (summed in a fixed order).
 * Cache values are exact in bf16; products accumulate in fp32, softmax and sums are fp32, the
 * probabilities are rounded to bf16 for the value product. What a row of no entry holds (NaN
 * included) does not reach the results. Scores that are not finite follow the formulas: NaN among
 * them gives lse, out and the head's weights NaN; +infinity lse +infinity and out NaN; a list of
 * -infinity alone lse -infinity and out NaN, unlike an empty one. Few tokens (up to about half the
 * SMs) run a cluster of CTAs each. Asynchronous on `stream`, allocates nothing. Bounded device waits
 * that run out are recorded for ds4idx_sparse_attention_status.
 * Errors: INVALID_ARG, UNSUPPORTED (d_qk != 576, d_v != 512), LAUNCH, CUDA. T = 0 is a no-op. */
int ds4idx_sparse_attention_q4(const void* q, const uint8_t* cache, int64_t kv_rows,
                               const int32_t* idx, const ds4idx_placement* where, int64_t T,
                               int32_t n_heads, int32_t d_qk, int32_t d_v, int32_t n_sel,
                               float sm_scale, void* out, float* lse, float* weights,
                               void* stream);

/* ---- The 8-bit latent cache: a latent row in 640 bytes and an fp32 scale (kept apart, as the index
 * cache's scales are), between the 1152 of bf16 and the 416 of 4 bits. One row: bytes 0..511 the E4M3
 * (OCP E4M3FN) codes of the first 512 dims in order, bytes 512..639 the 64 rotary dims as bf16. The
 * scale is the least power of two 2^e, e in -24..7, with absmax <= 448 * 2^e (2^7 where none is: larger
 * values saturate); a code is the E4M3 number nearest to x / scale, ties to even. A dim is code * scale,
 * exact in bf16. The bytes are a function of the inputs, which must be finite. The cache pointer is
 * 32-byte aligned. */

/* Writes n rows x [n, 576] (in_dtype DS4IDX_F32 or DS4IDX_BF16, 16-byte aligned) into cache rows
 * slots[i] or dst_offset + i and their scales into scale [cache_rows]: as ds4idx_quantize_latents. */
int ds4idx_quantize_latents_fp8(const void* x, int32_t in_dtype, int64_t n, const int64_t* slots,
                                int64_t dst_offset, uint8_t* cache, float* scale, int64_t cache_rows,
                                void* stream);

/* Reads n rows back as values, as ds4idx_read_latents. */
int ds4idx_read_latents_fp8(const uint8_t* cache, const float* scale, int64_t cache_rows,
                            const int64_t* rows, int64_t start, int64_t n, void* out,
                            int32_t out_dtype, void* stream);

/* ---- A tree of drafted tokens: a decode step that verifies several drafted tokens at once. The latent
 * rows of the N drafted tokens (nodes) of a sequence stand in the cache behind its kv_lens[b] rows, node
 * j at position kv_lens[b] + j (whatever its depth; its rotary position is kv_lens[b] + depth). mask
 * [B, N] says which nodes a node sees: bit j of mask[b, i] is set where node j is i itself or lies above
 * it. A chain of tokens has the masks 1, 3, 7, ...; a mask of 0 is padding. */

typedef enum {
  DS4IDX_CACHE_BF16 = 0, /* rows of 576 bf16 */
  DS4IDX_CACHE_FP8 = 1,  /* rows of 640 bytes and their scales, as ds4idx_quantize_latents_fp8 writes */
  DS4IDX_CACHE_Q4 = 2    /* rows of 416 bytes, as ds4idx_quantize_latents writes */
} ds4idx_cache_format;

/* Attention of every node over all of its sequence's rows and the drafted rows that it sees:
 *     s_j = sm_scale * q[b,i,h,:] . row_j,    out[b,i,h,:] = sum_j softmax(s)_j * row_j[0:512],
 *     lse[b,i,h] = log sum_j exp(s_j) (natural),
 * over positions j < kv_lens[b], and j = kv_lens[b] + k where bit k of mask[b,i] is set.
 *  q        [B, n_nodes, n_heads, 576] bf16, 16-byte aligned; n_nodes 1..64, n_heads 1..128.
 *  cache    [kv_rows, ...] in `format`, 32-byte aligned, 1 <= kv_rows < 2^31; scale [kv_rows] fp32 for
 *           DS4IDX_CACHE_FP8 (powers of two, 2^-24 .. 2^7), else NULL. One that is negative or lies
 *           between powers of two makes NaN of the nodes that see its row.
 *  kv_lens  DEVICE int32 [B] (>= 0; less counts as 0), mask DEVICE int64 [B, n_nodes].
 *  where    HOST, may be NULL (row = position); its "tokens" are the B sequences. A position past a
 *           sequence's table row or outside the pool is not there; a sequence whose kv_row0 is negative
 *           has no rows.
 *  max_kv_len  the largest of kv_lens, or a bound of it: the work is laid out for it. A bound far above
 *           the lengths costs little (one sequence: 3 to 10%; 64 short ones: three quarters). With a longer
 *           sequence the results stay right and the call gets slower.
 *  out      [B, n_nodes, n_heads, 512] bf16, 32-byte aligned; lse [B, n_nodes, n_heads] fp32 or NULL.
 *           Of a node of mask 0, or that sees no row, out is 0 and lse -infinity.
 *  workspace  DEVICE, 16-byte aligned, the bytes that ds4idx_tree_attention_workspace gives for these
 *           sizes and this or a larger max_kv_len (may be 0, then NULL): partial sums of sequences whose
 *           keys are split. Calls that can overlap need one each.
 * Cache values are exact in bf16; products accumulate in fp32, softmax and sums are fp32, the
 * probabilities are rounded to bf16 for the value product and divided by the sum of the rounded ones.
 * Probabilities below 2^-126, beside 8-bit rows probabilities times the row's scale, lose bits or count as 0.
 * A term may be 2^48 (beside 8-bit and 4-bit rows 2^64) times the maximum that it is taken against, so
 * values of a bf16 cache stay finite in the sums below 2^80 / (rows of the sequence): below 2^49 always.
 * Beside an 8-bit cache the first 512 dims of a query are the sum of two 8-bit numbers: exact, or off by
 * at most 2^-21 of the query's largest value or of 2^-119, whichever is larger; rotary dims are finite
 * there and below 2^90, and a query that is not finite makes NaN of its output. What a row that is not seen
 * holds (NaN included) does not reach the results. Scores that are not finite follow the formulas, as in
 * ds4idx_sparse_attention_q4; the values of a drafted row that are not finite count as 0 (its scores still
 * make NaN of the nodes that see it). Asynchronous on `stream`, allocates nothing. Bounded device waits that
 * run out are recorded for ds4idx_sparse_attention_status.
 * Errors: INVALID_ARG, UNSUPPORTED (d_qk != 576, d_v != 512), LAUNCH, CUDA. B = 0 is a no-op. */
int ds4idx_tree_attention(const void* q, int32_t format, const void* cache, const float* scale,
                          int64_t kv_rows, const int32_t* kv_lens, const int64_t* mask,
                          const ds4idx_placement* where, int32_t B, int32_t n_nodes,
                          int32_t n_heads, int32_t d_qk, int32_t d_v, int64_t max_kv_len,
                          float sm_scale, void* out, float* lse, void* workspace,
                          int64_t workspace_size, void* stream);

/* *bytes: a workspace for calls of these sizes and every max_kv_len up to this one, on the current device
 * (with 152 SMs never more than 161 MB). Other batches, nodes or heads may need more, fewer of them too.
 * Errors: INVALID_ARG. */
int ds4idx_tree_attention_workspace(int32_t B, int32_t n_nodes, int32_t n_heads, int64_t max_kv_len,
                                    int64_t* bytes);

/* ---- Eviction by accumulated attention weight. Each pool row has a total, int64 in units of
 * 2^-32 (fixed point: integer adds commute, so the order of atomics does not change a result). */

/* total[row of (t, idx[t,j])] += round(weights[t,j] * 2^32) for every non-empty entry; weights
 * [T, n_sel] fp32 below 2^30 in size (others add nothing). n_sel >= 1, 1 <= pool_rows < 2^31.
 * Asynchronous, allocates nothing. Errors: INVALID_ARG, LAUNCH. T = 0 is a no-op. */
int ds4idx_evict_accumulate(int64_t* total, int64_t pool_rows, const float* weights,
                            const int32_t* idx, const ds4idx_placement* where, int64_t T,
                            int32_t n_sel, void* stream);

/* Chooses the rows that B sequences keep. Sequence b has seq_lens[b] >= 0 rows from pool row
 * starts[b] and keeps min(keep[b], seq_lens[b]) of them: all if keep[b] >= seq_lens[b], else its
 * first n_sink, its last n_recent and, of the others, those with the largest totals (ties to the
 * lower position). kept [B, width] int32 (DEVICE): the kept positions ascending, then -1; width >=
 * every count. starts, seq_lens, keep: HOST int64 [B]; 1 <= B <= 64; seq_lens <= 2^30;
 * 0 <= n_sink + n_recent <= keep[b]. Asynchronous, allocates nothing. Errors: INVALID_ARG, LAUNCH,
 * CUDA. */
int ds4idx_evict_select(const int64_t* total, int64_t pool_rows, int32_t B, const int64_t* starts,
                        const int64_t* seq_lens, const int64_t* keep, int64_t n_sink,
                        int64_t n_recent, int32_t* kept, int64_t width, void* stream);

/* One per-row array of a pool (latent rows, index keys, key scales, totals, ...). */
typedef struct {
  const void* src;
  void* dst;
  int64_t src_rows, dst_rows;
  int32_t row_bytes; /* 1..65536 */
  int32_t reserved;
} ds4idx_row_array;

/* Moves the kept rows of B sequences together: for every array, dst row dst_starts[b] + i = src row
 * src_starts[b] + kept[b][i], i < counts[b] (kept as written by ds4idx_evict_select, counts[b] =
 * min(keep[b], seq_lens[b])). 1 <= n_arrays <= 8. The rows written for a sequence in an array must not
 * overlap those of another sequence or array, nor a source range (src_starts[b] .. + src_lens[b]) of
 * any sequence in any array: refused, as their order is not defined. Source ranges may overlap. HOST:
 * arrays, src_starts, src_lens, dst_starts, counts; DEVICE: kept [B, width] (an entry outside 0..src_lens-1
 * leaves its row unwritten). Asynchronous, allocates nothing. Errors: INVALID_ARG, LAUNCH. */
int ds4idx_evict_compact(const int32_t* kept, int64_t width, int32_t B, const int64_t* src_starts,
                         const int64_t* src_lens, const int64_t* dst_starts, const int64_t* counts,
                         int32_t n_arrays, const ds4idx_row_array* arrays, void* stream);

/* Keeps the accepted path of each drafted tree: in every array, the row of position kv_lens[b] + j
 * becomes the row of position kv_lens[b] + path[b][j], j < n_accepted[b], and new_lens[b] = kv_lens[b] +
 * n_accepted[b], at most 2^31 - 1 (counts outside 0..n_nodes are clamped). In place: all rows of a path are
 * read before one is written, so that a path may name any nodes. An entry of path outside 0..n_nodes-1, or a
 * position that is not there, leaves its row as it is; of a negative length no position is there, and its sum
 * with n_accepted[b] is the new length all the same.
 *  kv_lens, n_accepted DEVICE int32 [B]; path DEVICE int32 [B, n_nodes], n_nodes 1..64; new_lens DEVICE
 *  int32 [B]; where as in ds4idx_tree_attention; rows: the pool's, of every array (1 <= rows < 2^31).
 *  arrays HOST, 0 <= n_arrays <= 8, src = dst and src_rows = dst_rows = rows in each.
 * No written array may overlap another or anything that the call reads: refused. The rows of two
 * sequences must differ. Asynchronous, allocates nothing. Errors: INVALID_ARG, LAUNCH. B = 0 is a
 * no-op. */
int ds4idx_tree_commit(const int32_t* kv_lens, const int32_t* path, const int32_t* n_accepted,
                       int32_t* new_lens, const ds4idx_placement* where, int32_t B, int32_t n_nodes,
                       int64_t rows, int32_t n_arrays, const ds4idx_row_array* arrays, void* stream);

/* Test support for the bounded device waits (the pages have no counterpart). Every mbarrier
 * wait in the kernels gives up after a limit (2 s by default), records DS4IDX_ERR_DEVICE_TIMEOUT
 * for ds4idx_sync_status, waits for its own copies and tensor-core work to finish, frees its
 * tensor memory and returns, so a lost arrival turns into an error status instead of a hang.
 * This call sets the limit used by the handle's later calls (1e6 <= wait_limit_ns <= 2e9) and,
 * with withhold != 0, makes the next calls of a four-query (T > 1) plan without key splits
 * withhold one arrival of their first CTA's first selector warp, so that CTA's epilogue wait for
 * the score ring runs out once the ring wraps (more than 30 key tiles in that CTA). Every copy
 * and MMA already issued completes on its own. Reset with (2000000000, 0).
 * Errors: INVALID_ARG (null handle, limit out of range). */
int ds4idx_debug_wait_test(ds4idx_t h, uint64_t wait_limit_ns, int32_t withhold);

/* The work decomposition a call would use, computed on the host alone (no device access), for
 * tests and capacity planning. num_sms: the device's SM count; B, T, S, pos_offsets[B] as in
 * ds4idx_score_topk_batched; fixed_scratch != 0 gives the plan of
 * ds4idx_score_topk_batched_noalloc. out[7] receives: queries per CTA, query blocks per
 * sequence, key splits, key tiles per split, CTAs in the grid, split-list words, split tickets.
 * Errors: INVALID_ARG. */
int ds4idx_plan_query(int32_t num_sms, int32_t B, int64_t T, int64_t S,
                      const int64_t* pos_offsets, int32_t fixed_scratch, int64_t* out);

#ifdef __cplusplus
}
#endif

#endif /* DS4IDX_H_ */
