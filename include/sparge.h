/*
 * sparge.h -- C ABI of the B200 (sm_100a) SpargeAttn sparse-attention forward.
 *
 * The method is the two-stage filtered sparse FlashAttention of "SpargeAttn:
 * Accurate and Training-free Sparse Attention Accelerating Any Model
 * Inference" (paper review page, section 三 技术架构, Algorithm 1):
 *   stage 1  block-mask prediction from mean-pooled Q/K blocks (Eq. 4-9);
 *   stage 2  block-sparse online-softmax attention with the per-warp lambda
 *            skip of P~V (Eq. 1-3);
 *   plus     the Hilbert-curve token permutation for visual tokens
 *            (same page, "HilbertCurve Permutation").
 *
 * Conventions shared by every entry point
 *   Layout     Q [B, Hq, N, d], K and V [B, Hkv, N, d], O [B, Hq, N, d],
 *              row-major with d contiguous; every base pointer 16-byte aligned.
 *              Query head h reads KV head h / (Hq / Hkv).
 *   Memory     Every pointer argument is DEVICE memory unless stated, allocated
 *              and owned by the caller.  The library allocates nothing, keeps no
 *              state between calls and is re-entrant for calls with distinct
 *              workspaces.
 *   Streams    Every call is asynchronous on the given stream; no call
 *              synchronises except sparge_device_status.
 *   Devices    A call runs on the device that owns its (first) device
 *              pointer and leaves the caller's current device as it was.
 *   Errors     Arguments are validated on the host before any launch:
 *              SPARGE_EINVAL (bad pointer, size or hyper-parameter),
 *              SPARGE_EUNSUPPORTED (valid but not implemented, e.g. d = 96,
 *              b_q != 128, b_k != 64, or more than 5952 key blocks: N > 380,928),
 *              SPARGE_EWORKSPACE (workspace too small), SPARGE_ECUDA (a CUDA
 *              runtime call or launch failed).  Nothing is launched when a call
 *              returns an error.  Kernels never trap: a device-side wait that
 *              runs out of time writes SPARGE_ETIMEOUT into the workspace
 *              status word and the kernel returns; sparge_device_status reads it.
 *   Blocks     bq = 128 query rows, bk = 64 key rows (the pages' b_q, b_k);
 *              c_w = bq / 32 = 4 warps of 32 query rows each for the lambda
 *              test; T_m = ceil(N / bq), T_n = ceil(N / bk).
 */
#ifndef SPARGE_H_
#define SPARGE_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPARGE_OK = 0,
  SPARGE_EINVAL = 1,
  SPARGE_EUNSUPPORTED = 2,
  SPARGE_ECUDA = 3,
  SPARGE_ETIMEOUT = 4,
  SPARGE_EWORKSPACE = 5,
  SPARGE_ERANGE = 6 /* a value did not fit its narrower form and was saturated: a bf16 V value
                       in fp16 (P~V runs in fp16), or the scale of a 4-bit cache group */
} sparge_status_t;

typedef enum { SPARGE_F16 = 0, SPARGE_BF16 = 1, SPARGE_F32 = 2 } sparge_dtype_t;

/* Hyper-parameters of one attention call (Algorithm 1 "Input" line). */
typedef struct {
  int32_t B, Hq, Hkv, N, d; /* d in {64, 128}; Hq % Hkv == 0; N >= 0            */
  int32_t bq, bk;           /* must be 128 and 64                               */
  float tau;                /* TopCdf mass, Eq. 8; (0, 1], >= 1 keeps all       */
  float theta;              /* self-similarity threshold, Eq. 7 and Eq. 9       */
  float lambda;             /* P~V skip threshold of Eq. 3, natural-log units;
                               <= 0, -INFINITY disables the skip                */
  float scale;              /* score scale, normally 1/sqrt(d) (Eq. 1)          */
  int32_t causal;           /* 1: key n is visible to query m iff n <= m        */
  int32_t qk_int8;          /* 1: per-block INT8 Q K^T with K mean smoothing
                               (Algorithm 1 steps 2 and 10; d = 128 only)       */
  sparge_dtype_t io_dtype;  /* dtype of Q, K, V: SPARGE_F16 or SPARGE_BF16      */
  sparge_dtype_t o_dtype;   /* dtype of O: io_dtype or SPARGE_F32               */
} sparge_params_t;

/* Per-call work counters, accumulated with atomics into caller-zeroed device
 * memory.  A "slice" is one warp's 32 query rows of one (tile, key block). */
typedef struct {
  unsigned long long tiles;          /* query tiles processed                    */
  unsigned long long qk_blocks;      /* Q_i K_j^T block products computed         */
  unsigned long long pv_blocks;      /* P~_ij V_j products issued (any slice on) */
  unsigned long long pv_slices;      /* slices whose P~V was kept                 */
  unsigned long long skipped_slices; /* slices skipped by the lambda test (Eq. 3) */
} sparge_stats_t;

/* Bytes of workspace that sparge_predict_mask and sparge_attn_fwd need for
 * these parameters.  The SAME workspace must be passed to both calls of one
 * forward: with qk_int8 the predictor writes the INT8 codes there and the
 * attention reads them.  Returns 0 for invalid parameters. */
size_t sparge_workspace_bytes(const sparge_params_t* p);

/* Hilbert permutation table (paper review page, "HilbertCurve Permutation";
 * rebuttal page, reply to Weakness 3).  Tokens are laid out as
 * [prefix_len text tokens | T x Hg x Wg grid, (t, y, x) row-major | rest].
 * Axes of extent 1 are dropped; the remaining axes, in order (t, y, x), index
 * a Hilbert curve on the smallest 2^b cube holding them (Skilling's transpose
 * form).  Writes perm[N] (device, int32) with y[p] = x[perm[p]]: prefix and
 * trailing tokens keep their place, grid tokens follow the curve.
 * ws: device workspace of sparge_hilbert_workspace_bytes(T, Hg, Wg) bytes. */
size_t sparge_hilbert_workspace_bytes(int32_t T, int32_t Hg, int32_t Wg);
sparge_status_t sparge_hilbert_index(int32_t N, int32_t prefix_len, int32_t T, int32_t Hg,
                                     int32_t Wg, int32_t* perm, void* ws, size_t ws_bytes,
                                     cudaStream_t stream);

/* y[b, h, p, :] = x[b, h, perm[p], :] for x, y [B, H, N, d] of dtype (16-bit
 * or f32).  perm is a device array of N int32 entries, normally a
 * permutation of 0..N-1 (e.g. from sparge_hilbert_index); a row whose entry
 * lies outside [0, N) is skipped (y's row is left as it was).  x and y must
 * not overlap (SPARGE_EINVAL).  A row of d elements must be a multiple of 16
 * bytes and B * H at most 65535 (SPARGE_EUNSUPPORTED otherwise); B, H or
 * N = 0 is a no-op.  HBM-bound: each row is read once and written once. */
sparge_status_t sparge_hilbert_permute(const void* x, void* y, int32_t B, int32_t H, int32_t N,
                                       int32_t d, sparge_dtype_t dtype, const int32_t* perm,
                                       cudaStream_t stream);

/* The inverse: x[b, h, perm[p], :] = y[b, h, p, :], under the same rules (a
 * row whose entry lies outside [0, N) is not written).  perm should be a
 * permutation: if two in-range entries are equal, both source rows are
 * written to the same destination row and which one remains is unspecified. */
sparge_status_t sparge_inverse_permute(const void* y, void* x, int32_t B, int32_t H, int32_t N,
                                       int32_t d, sparge_dtype_t dtype, const int32_t* perm,
                                       cudaStream_t stream);

/* Stage 1, Algorithm 1 steps 2-5 (Eq. 4-9): block means q_i, k_j, CosSim
 * self-similarities s_q, s_k (mean of the block's token cosine matrix), the
 * compressed map S_hat = scale * q k^T with -inf columns where s_k < theta
 * (and causal-future blocks), row softmax, TopCdf(tau), the fix-block rule.
 * Outputs (device):
 *   mask   [B, Hq, T_m, T_n] uint8 M_g (1 = compute block)
 *   kv_idx [B, Hq, T_m, T_n] int32: the kept j of each tile in ascending order,
 *          first kv_cnt entries valid (the rest are left unspecified)
 *   kv_cnt [B, Hq, T_m] int32
 *   s_q    [B, Hq, T_m] float, s_k [B, Hkv, T_n] float (both nullable)
 * With qk_int8 it also quantises Q and K - mean(K) per block into ws
 * (Algorithm 1 step 2): mean(K) is the per-head mean over all N tokens, summed
 * in float64 and rounded once to float32; per block delta = absmax / 127 and
 * code = round-half-even(x / delta) of the IEEE float32 quotient. */
sparge_status_t sparge_predict_mask(const sparge_params_t* p, const void* q, const void* k,
                                    uint8_t* mask, int32_t* kv_idx, int32_t* kv_cnt, float* s_q,
                                    float* s_k, void* ws, size_t ws_bytes, cudaStream_t stream);

/* The two halves of sparge_predict_mask, for callers that time or schedule
 * them apart.  sparge_predict_pool is Algorithm 1 steps 2-3 (Eq. 4-6): block
 * means, CosSim self-similarities and, with qk_int8, the INT8 codes of Q and
 * K - mean(K) with their scales, all written into ws (the HBM-bound pass over
 * Q and K).  sparge_predict_select is steps 4-5 (Eq. 7-9): S_hat, softmax,
 * TopCdf, the fix rule, mask / kv_idx / kv_cnt (and the optional s_q, s_k
 * copies) computed from what sparge_predict_pool left in the same ws, which
 * must therefore run first on the same stream (or be ordered before it).
 * Arguments, layouts and errors as for sparge_predict_mask; pool checks q and
 * k, select checks the outputs. */
sparge_status_t sparge_predict_pool(const sparge_params_t* p, const void* q, const void* k,
                                    void* ws, size_t ws_bytes, cudaStream_t stream);
sparge_status_t sparge_predict_select(const sparge_params_t* p, uint8_t* mask, int32_t* kv_idx,
                                      int32_t* kv_cnt, float* s_q, float* s_k, void* ws,
                                      size_t ws_bytes, cudaStream_t stream);

/* sparge_predict_mask without a workspace, for callers that cannot allocate
 * device memory at call time and have no workspace to pass in (a plugin whose
 * host framework owns every device buffer, a serving loop that must not call
 * the allocator after start-up).  The paper has no counterpart: this is a
 * deployment variant of the stage-1 predictor above, with the same outputs.
 * Its scratch (pooled block means and self-similarities) lives in one static
 * 32 MiB device array compiled into the library; every GPU that loads the
 * library holds that array until the process exits.  The predictor's regions
 * must fit: 256 + align256(B*Hq*T_m*d*4) + align256(B*Hkv*T_n*d*4)
 * + align256(B*Hq*T_m*4) + align256(B*Hkv*T_n*4) <= 32 MiB, else the call
 * returns SPARGE_EWORKSPACE (align256 rounds up to a multiple of 256).
 * qk_int8 = 1 returns SPARGE_EUNSUPPORTED (the INT8 codes must outlive the
 * call); otherwise a parameter set gets the same status as from
 * sparge_predict_mask (SPARGE_EINVAL or SPARGE_EUNSUPPORTED).  The first call
 * on each device looks up the array's device address there
 * (cudaGetSymbolAddress), so make that first call before any stream capture.
 * The call allocates nothing.  All calls share the array and it keeps the
 * last call's contents; each call rewrites every region it reads, so nothing
 * has to be cleared, but calls whose kernels overlap on the GPU (unordered
 * streams) race on it.  The predictor has no device-side waits, so these
 * calls leave no device status to read (there is no workspace to hold one). */
sparge_status_t sparge_predict_mask_noalloc(const sparge_params_t* p, const void* q,
                                            const void* k, uint8_t* mask, int32_t* kv_idx,
                                            int32_t* kv_cnt, float* s_q, float* s_k,
                                            cudaStream_t stream);

/* Compacts a caller-built mask [B, Hq, T_m, T_n] (uint8, nonzero = keep) into
 * the kv_idx / kv_cnt skip list sparge_attn_fwd consumes: Algorithm 1 step 9
 * visits, for query block i, the key blocks j with M_g[i, j] = 1 in ascending
 * order, and Eq. 2 skips the others; this is that visiting order.  Causal-
 * future blocks are kept if the mask keeps them (the attention masks them
 * anyway).  Outputs as for sparge_predict_mask; errors as for every entry
 * point (SPARGE_EINVAL for null or misaligned pointers). */
sparge_status_t sparge_mask_compact(const sparge_params_t* p, const uint8_t* mask,
                                    int32_t* kv_idx, int32_t* kv_cnt, cudaStream_t stream);

/* Stage 2, Algorithm 1 steps 6-17 (Eq. 1-3): for every query tile i, the key
 * blocks kv_idx[..., :kv_cnt] in the listed order: S = scale Q_i K_j^T (INT8
 * codes times the block scales with qk_int8), online softmax of Eq. 1, then
 * P~V for every 32-row warp slice whose max(m_local - m_new) >= lambda.
 * O_i = O / l; a row with l = 0 outputs 0.  P~V runs in fp16 with fp32
 * accumulation (V is converted from bf16 into ws when io_dtype is bf16).
 * stats: nullable device pointer to caller-zeroed counters.
 * ws: the workspace passed to sparge_predict_mask (required with qk_int8). */
sparge_status_t sparge_attn_fwd(const sparge_params_t* p, const void* q, const void* k,
                                const void* v, const int32_t* kv_idx, const int32_t* kv_cnt,
                                void* o, void* ws, size_t ws_bytes, sparge_stats_t* stats,
                                cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * Around the prompt pass: positions, pages and the tokens that follow.
 *
 * The paper has no counterpart of these calls.  They are what a serving
 * program runs next to the sparse prompt pass: rotary positions of Q and K
 * (fused with the Hilbert permutation), the block tables and slots of a paged
 * cache, the cache itself with K and V in 4 bits, and attention of new tokens
 * over it.  Conventions as above, except where strides are given.
 * ------------------------------------------------------------------------- */

/* Rotary positions with several axes (time, height, width, ...). */
typedef struct {
  int32_t B, H, N, d;     /* x, y: [B, H, N, d], channels contiguous, the rest strided     */
  int32_t rot;            /* channels that turn, the first rot of d; the others are copied */
  int32_t axes;           /* position axes, >= 1                                           */
  int32_t interleaved;    /* pair i is channels (i, i + rot/2), or with 1 (2i, 2i + 1)     */
  sparge_dtype_t dtype;   /* of x and y                                                    */
  int64_t x_stride[3];    /* elements between batches, heads and tokens of x, and of y;    */
  int64_t y_stride[3];    /*   each a multiple of 16 bytes                                 */
  int64_t pos_stride;     /* elements between the positions of two batches; 0 shares them  */
} sparge_rope_t;

/* y[b, h, p, :] = x[b, h, s, :] turned, s = perm[p] (perm == NULL: s = p): pair i, (u, v),
 * becomes (u cos a - v sin a, u sin a + v cos a) with a = pos[b, axis[i], s] * inv_freq[i].
 *   pos       device int32 [B or 1, axes, N]
 *   inv_freq  device float64 [rot/2], radians per position (any frequency scaling is in it)
 *   axis      device int32 [rot/2], which axis turns pair i, in [0, axes) (others: a = 0)
 *   perm      device int32 [N] or NULL; rows whose entry lies outside [0, N) are skipped.  An
 *             entry may come twice here, but not in the inverse
 * The angle is reduced in float64 turns, so far positions lose nothing: for |inv_freq| <= 1 its
 * error is below 2^-23 of a turn up to position 2^30.  The products are float32, rounded once
 * to dtype.
 * y may be x (same strides, no perm); any other overlap of the two extents is refused
 * (SPARGE_EINVAL), as is a written tensor whose rows may overlap: its strides, in ascending
 * order, must each step over what the smaller ones span (no stride of 0, so no broadcast).
 * SPARGE_EUNSUPPORTED: rows or strides that are no multiple of 16 bytes, or rot * element size
 * no multiple of 32 bytes. */
sparge_status_t sparge_rope_apply(const sparge_rope_t* p, const void* x, void* y,
                                  const int32_t* pos, const double* inv_freq,
                                  const int32_t* axis, const int32_t* perm, cudaStream_t stream);

/* The inverse, which is also the gradient of sparge_rope_apply (the rotation is
 * orthogonal): x[b, h, s, :] = y[b, h, p, :] turned by -a.  Same rules; with perm, rows of x
 * that no entry names are left as they were, and of rows that two entries name each 16 bytes are
 * one of the two's and which is unspecified (not their sum, as a gradient would have it). */
sparge_status_t sparge_rope_inverse(const sparge_rope_t* p, const void* y, void* x,
                                    const int32_t* pos, const double* inv_freq,
                                    const int32_t* axis, const int32_t* perm,
                                    cudaStream_t stream);

/* One step of a paged cache's bookkeeping, on the device: which requests get the pages
 * they need, their block tables, and the slot of every new token.
 *   new_len      int32 [R]: tokens that request r brings; 0: none; < 0: it has ended
 *   seq_len      int32 [R]: tokens it has in the cache so far
 *   block_table  int32 [R, max_pages], in and out: entry j is the page of tokens
 *                [j * page_size, (j + 1) * page_size)
 *   free_pages   int32 [num_pages], in and out: a stack of free page numbers
 *   free_count   int32 [1]: its height
 * In this order: the pages of ended requests are pushed (request by request, each in table
 * order); then requests with new tokens are admitted in order.  A request is admitted when
 * its tokens fit its table row and max_tokens slots and the pages it needs, together with
 * those of every earlier such request, are there; one that needs no new page is always
 * admitted then.  Pages are popped from the top, request by request.
 *   seq_len_out, free_count_out  the new values (may be seq_len and free_count themselves)
 *   cu_new       int32 [R + 1]: where each request's new tokens start (cu_q of the attention),
 *                those of requests that were not admitted counted too: their rows' attention
 *                means nothing
 *   slot_map     int32 [max_tokens]: page * page_size + offset of new token t; -1 for a
 *                token of a request that was not admitted and behind the last token
 *   admitted     int32 [R]: 0 for a request whose new tokens found no room, else 1
 * A request that is not admitted keeps its length and its pages.  Lengths outside
 * [0, max_pages * page_size] are taken as the nearer end, a height outside [0, num_pages]
 * likewise; what would be pushed past num_pages is dropped.  Page numbers are taken as they are; one whose
 * slots do not fit 32 bits gives slots below 0.
 * The outputs may not overlap one another or the inputs, apart from the two named above.
 * SPARGE_EUNSUPPORTED: R > 4096, num_pages or max_pages times page_size >= 2^31, or
 * max_tokens > 2^31 - 16. */
sparge_status_t sparge_kv_plan(int32_t R, int32_t page_size, int32_t max_pages,
                               int32_t num_pages, int32_t max_tokens, const int32_t* new_len,
                               const int32_t* seq_len, int32_t* block_table,
                               int32_t* free_pages, const int32_t* free_count,
                               int32_t* seq_len_out, int32_t* free_count_out, int32_t* cu_new,
                               int32_t* slot_map, int32_t* admitted, cudaStream_t stream);

/* A paged cache of K and V in 4 bits.  Every (token, KV head) row of d channels is cut into
 * d / group groups; each has one fp16 scale s = absmax / 7 (the quotient in float32, rounded
 * to fp16) and per channel the code c = round-half-even(x / s) of the IEEE float32 quotient,
 * clamped to [-7, 7] and held as c + 8.  The value is c * s.  A group whose s is 0 has codes
 * 0; a group with a NaN has s = NaN; s above 16376 is saturated (SPARGE_ERANGE), so that a
 * softmax weight times s stays in fp16.
 * Memory: uint8 [num_pages, Hkv, page_size / 16, tile], a tile holding 16 tokens:
 *   8d bytes      codes of K, token rows of d/2 bytes: byte b of 32-bit word (t, j), t < 4,
 *                 j < d/32, holds channels 32j + 8t + e, e = (0,2), (4,6), (1,3), (5,7) for
 *                 b = 0..3, the first in the low half
 *   8d bytes      codes of V, [d/64 w][8 g][16 p][4 i]: channels 64w + 16i + 2g (low half)
 *                 and 64w + 16i + 2g + 1 of the token k with p = 4((k%8)/2) + 2(k/8) + k%2
 *   64d/group     scales, fp16 [16 tokens][d/group of K, d/group of V]
 * which is the order in which the tensor-core fragments take them.  A token's bytes are its
 * own, so writes of different tokens never meet. */
typedef struct {
  int32_t Hkv, d;      /* d in {64, 128}                                      */
  int32_t group;       /* channels per scale: 32, 64 or 128, at most d        */
  int32_t page_size;   /* tokens per page: a multiple of 16                   */
  int32_t num_pages;   /* num_pages * page_size < 2^31                        */
} sparge_kv4_t;

/* Bytes of the cache; 0 for invalid or unsupported parameters.  Its base must be 16-byte
 * aligned.  No initial contents are needed: only written tokens are ever used. */
size_t sparge_kv4_bytes(const sparge_kv4_t* c);

/* Writes T tokens: row t of k and v goes to slot slot_map[t] = page * page_size + offset;
 * rows whose slot lies outside [0, num_pages * page_size) are skipped.  If two rows name one
 * slot, each byte of it is one of the two's and which is unspecified.
 * k, v: [T, Hkv, d] of dtype (16-bit), channels contiguous; *_stride: elements between tokens
 * and heads, multiples of 16 bytes.  status: nullable device int32 that receives
 * SPARGE_ERANGE (the first word of a workspace will do). */
sparge_status_t sparge_kv4_append(const sparge_kv4_t* c, int32_t T, const void* k,
                                  const int64_t k_stride[2], const void* v,
                                  const int64_t v_stride[2], sparge_dtype_t dtype,
                                  const int32_t* slot_map, void* cache, int32_t* status,
                                  cudaStream_t stream);

/* The values that T slots hold, c * s in float32 rounded once to dtype (16-bit or float32),
 * into rows of k and v (either nullable); rows whose slot lies outside the cache are left as
 * they were. */
sparge_status_t sparge_kv4_read(const sparge_kv4_t* c, int32_t T, const void* cache,
                                const int32_t* slot_map, void* k, const int64_t k_stride[2],
                                void* v, const int64_t v_stride[2], sparge_dtype_t dtype,
                                cudaStream_t stream);

/* Attention of new tokens over the cache. */
typedef struct {
  int32_t R;              /* requests                                                      */
  int32_t T;              /* rows of q and o                                               */
  int32_t Hq;             /* query heads; head h reads KV head h / (Hq / Hkv)              */
  int32_t max_q;          /* no request has more new tokens than this                      */
  int32_t max_pages;      /* width of the block table                                      */
  int32_t max_len;        /* no request is longer; 0: max_pages * page_size                */
  int32_t causal;         /* 1: a token sees the keys up to its own; 0: all of its request */
  float scale;            /* score scale in (0, 2^100], normally 1/sqrt(d)                 */
  sparge_dtype_t dtype;   /* of q and o: SPARGE_F16 or SPARGE_BF16                         */
  int64_t q_stride;       /* elements between tokens of q, heads are d apart               */
} sparge_kv4_attn_t;

/* Bytes of workspace for these parameters; 0 when they are invalid.  It must be zeroed once,
 * before its first use (and again after a device status of SPARGE_ETIMEOUT); calls of
 * different shapes may share one, if it is large enough for each and they do not overlap in
 * time. */
size_t sparge_kv4_workspace_bytes(const sparge_kv4_t* c, const sparge_kv4_attn_t* a);

/* o[t, h, :] = sum_n softmax_n(scale q[t, h] . k_n) v_n over the keys that token t sees.
 * Rows cu_q[r] .. cu_q[r + 1] - 1 of q and o are request r's newest tokens, the last of them
 * at position seq_len[r] - 1 (they are in the cache already).  A row that sees no key gives
 * 0 and lse -infinity; rows that belong to no request are left as they were.
 *   cache, block_table [R, max_pages], seq_len [R], cu_q [R + 1]: device, as sparge_kv_plan
 *     leaves them
 *   o    [T, Hq, d] of dtype; lse: nullable float32 [T, Hq], log of the sum of exponentials
 * Q is taken to fp16 with one power of two per row, products accumulate in float32, softmax
 * statistics are float32; a weight, and its product with V's scale, are rounded to fp16, held
 * times powers of two so that they keep all their bits down to a weight of 2^-24 of the row's
 * largest and, for a product, 2^-27 of what that weight and the KV head's largest scale would give
 * (where this scale is at least 2^-12; 2^-39 itself below), in the tiles of the next paragraph
 * down to a weight of 2^-20.
 * Requests with more than 64 rows for a KV head (new tokens times Hq / Hkv; of a call's only
 * request, max_q tokens) go through tiles of K and V in fp16: there the values c * s are taken
 * as they are for fp16 rows and rounded to fp16 (by up to 2^-11 of each) for bf16 rows (a token of
 * K or of V with a scale of 8192 or more: its other scales to multiples of 2^-23), and a
 * NaN scale of V makes every channel NaN in the rows that see its token, not its group's alone.
 * Keys at pages outside [0, num_pages) or behind max_len are left out; these, a length below
 * 0 and a cu_q that does not ascend within [0, T] by steps of at most max_q (such a request
 * is skipped) put SPARGE_EINVAL into the workspace's status word (sparge_device_status).
 * A call gives the same bits every time.  They depend on the whole call: the work is cut over all
 * of its requests, and of a call's only request max_q alone says which tiles it goes through.
 * SPARGE_EUNSUPPORTED: R or Hkv > 65535, or more than 2^31 - 1 rows of q times heads. */
sparge_status_t sparge_kv4_attn(const sparge_kv4_t* c, const sparge_kv4_attn_t* a,
                                const void* q, const void* cache, const int32_t* block_table,
                                const int32_t* seq_len, const int32_t* cu_q, void* o,
                                float* lse, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Synchronises the stream and returns the status word that kernels write to
 * the workspace (SPARGE_OK, SPARGE_ETIMEOUT, SPARGE_ERANGE or, from sparge_kv4_attn,
 * SPARGE_EINVAL), then clears it.
 * ws: the workspace of sparge_predict_mask / sparge_attn_fwd, or of sparge_kv4_attn. */
sparge_status_t sparge_device_status(void* ws, cudaStream_t stream);

/* Failure-detection self-test (no counterpart in the paper): launches one
 * CTA whose time-bounded mbarrier wait -- the same wait the attention kernel
 * uses -- is on a phase that nothing ever completes.  The wait gives up after
 * its 1 s limit and writes SPARGE_ETIMEOUT into the status word of ws, which
 * sparge_device_status then returns (and clears).  Nothing faults, traps or
 * hangs; the context stays usable.  ws: any workspace of at least 256 bytes. */
sparge_status_t sparge_selftest_wait_timeout(void* ws, cudaStream_t stream);

/* Static description of a status code (never NULL). */
const char* sparge_status_string(sparge_status_t s);

#ifdef __cplusplus
}
#endif

#endif /* SPARGE_H_ */
