/*
 * qdq.h -- GB300 (sm_103a) dequantize-and-multiply kernels for GGML Q8_0 / Q4_K
 * weight matrices against f32 activations (the token-decode hot path).
 *
 * Sources (rustdoc pages of the qualia_core_db crate):
 *   "Module cuda_lane", Functions:
 *     q8_0_gemv_oracle_into / try_q8_0_cuda_gemv   -> qdq_q8_0_gemv
 *     try_q4k_soa_gemv                              -> qdq_q4k_gemv
 *     try_q4k_soa_fused_swiglu                      -> qdq_q4k_swiglu
 *     try_q4k_soa_qkv                               -> qdq_q4k_qkv
 *     try_q4k_soa_ffn_block / _ffn_block_residual   -> qdq_q4k_ffn_residual
 *     preload_q4k_soa_weights (one-time upload)     -> qdq_q8_0_pack / qdq_q4k_pack
 *   "Module cuda_lane", Goal (batch prefill-shaped GEMMs on tensor cores) and
 *   "weight_cache.rs", try_cuda_batch_gemv          -> qdq_q8_0_gemm_batch / qdq_q4k_gemm_batch /
 *                                                      qdq_q4k_swiglu_batch
 *   "QTensorEngine", dispatch_output_top1_chunked   -> qdq_q8_0_logits_argmax
 *   "QTensorEngine", dispatch_output_topk_chunked   -> qdq_topk_rows / qdq_q8_0_logits_topk
 *   "QTensorEngine", embedding_pipeline (Q6_K dequant + matmul on the GPU),
 *     dispatch_quantized_token_embedding, dispatch_gemm_into (Q6_K)
 *                                                   -> qdq_q6k_pack / _gemv / _get_rows
 *
 * Conventions for every call
 *   - W is row-major n_out x n_in (rows = outputs, the GGML convention).
 *     Activations are packed batch x n_in f32, outputs batch x n_out f32
 *     ("weight_cache.rs", try_cuda_batch_gemv doc comment).
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates, frees or keeps a pointer after a call returns.
 *   - Every compute call is asynchronous and stream-ordered on `stream`
 *     (0 = the legacy default stream); nothing synchronises the host.
 *   - Calls return QDQ_OK or a negative status.  On a rejected argument (every
 *     status but QDQ_ERR_CUDA) nothing has been launched and every output
 *     buffer is untouched.  QDQ_ERR_CUDA from a call that launches several
 *     kernels (the FFN block, the batch GEMM, the argmax and top-k, QKV at batch > 1) can leave the
 *     kernels before the failing launch enqueued.  There is no fallback path:
 *     an unsupported shape is an error, never a silent slower route.
 *   - Kernels are launched with programmatic dependent launch: a kernel may
 *     start streaming its own weights while the previous kernel on the stream
 *     finishes, but it reads activations only after that kernel completed.
 *
 * Block formats (GGML, little-endian)
 *   Q8_0: 34-byte block per 32 weights: fp16 d, then int8 q[32]; w = d*q.
 *   Q4_K: 144-byte superblock per 256 weights: fp16 d, fp16 dmin, 12 bytes of
 *         eight 6-bit scales sc_j and eight 6-bit mins m_j, 128 bytes of 4-bit
 *         quants; sub-block j = weights 32j..32j+31; w = d*sc_j*q - dmin*m_j.
 *   Q6_K: 210-byte superblock per 256 weights: ql[128] (low 4 bits of each
 *         quant), qh[64] (high 2 bits), sixteen int8 scales, fp16 d (at byte
 *         208); weight e = d*scale[e/16]*(q_e - 32), q_e in 0..63, where weight
 *         128h + 32t + l (h < 2, t < 4, l < 32) takes its low 4 bits from the low
 *         (t < 2) or high (t >= 2) nibble of ql[64h + 32(t & 1) + l] and its high
 *         2 bits from bits 2t..2t+1 of qh[32h + l].
 *
 * Packed (device) formats -- produced once by qdq_*_pack, same byte count as
 * the GGML input, laid out as planes so that every kernel load is a 16-byte
 * aligned vector load:
 *   Q8_0 packed: [ q plane: n_out*n_in int8, row-major ]
 *                [ d plane: n_out*(n_in/32) fp16, row-major ]
 *   Q4_K packed: [ q plane: n_out*(n_in/2) bytes; weight e of a row is nibble
 *                  (e & 1) (0 = low) of byte e/2 ]
 *                [ header plane: n_out*(n_in/256) records of 16 bytes:
 *                  word0 = d | dmin << 16 (fp16 bits); words 1..3 form a
 *                  96-bit little-endian field with sc_j at bits 12j..12j+5
 *                  and m_j at bits 12j+6..12j+11 ]
 *   Q6_K packed: rows of qdq_q6k_packed_bytes(1, n_in) bytes (the 210/256
 *                bytes per weight padded to a multiple of 16; no padding when
 *                n_in % 2048 == 0): [ low-bit plane n_in/2 | high-bit plane
 *                n_in/4 | int8 scales n_in/16 | fp16 d n_in/128 | zeros ];
 *                32-weight block b: low bits at 16b (byte i of word c: weight
 *                8c+i in the low nibble, 8c+4+i in the high nibble), high bits
 *                at n_in/2 + 8b (byte i of word h: weights 16h+i, 16h+4+i,
 *                16h+8+i, 16h+12+i at bits 0-1, 2-3, 4-5, 6-7).
 */
#ifndef QDQ_H
#define QDQ_H

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes --------------------------------------------------------- */
#define QDQ_OK               0
#define QDQ_ERR_NULL        -1  /* a required pointer is NULL */
#define QDQ_ERR_DIMS        -2  /* a dimension is <= 0, not a whole number of blocks, or out of range */
#define QDQ_ERR_ALIGN       -3  /* a pointer does not meet the stated alignment */
#define QDQ_ERR_UNSUPPORTED -4  /* valid arguments this build does not handle (e.g. n_in too large) */
#define QDQ_ERR_CUDA        -5  /* a CUDA runtime call failed; see qdq_last_cuda_error() */
#define QDQ_ERR_ALIAS       -6  /* an output overlaps an input it may not overlap */
#define QDQ_ERR_SCRATCH     -7  /* the request does not fit the library's fixed scratch array, or the workspace's bytes */

/* Human-readable name of a status code (static string). */
const char *qdq_status_string(int status);
/* cudaError_t of the most recent QDQ_ERR_CUDA returned on the calling thread (0 if none). */
int qdq_last_cuda_error(void);
/* Library version string (static). */
const char *qdq_version(void);

/* ---- limits --------------------------------------------------------------- */
/* Largest supported batch for the GEMV-family calls. */
#define QDQ_MAX_GEMV_BATCH 8
/* Largest supported n_in for the GEMV-family calls (activations are staged in
 * shared memory: batch_group * n_in * 4 bytes per CTA). */
#define QDQ_MAX_GEMV_N_IN 32768

/* ---- one-time repack (the pages' preload step) ----------------------------
 * "Module cuda_lane", Functions: preload_q4k_soa_weights -- bulk upload once
 * at plan build.  Converts a row-major GGML matrix already resident on the
 * device into the packed planes above.  `ggml` and `packed` are device
 * pointers; `packed` must hold qdq_*_packed_bytes(n_out, n_in) bytes, be
 * 16-byte aligned and must not overlap `ggml`.  Q8_0 needs n_in % 32 == 0,
 * Q4_K needs n_in % 256 == 0.
 */
size_t qdq_q8_0_packed_bytes(int n_out, int n_in);   /* n_out*n_in/32*34, 0 on bad dims */
size_t qdq_q4k_packed_bytes(int n_out, int n_in);    /* n_out*n_in/256*144, 0 on bad dims */
int qdq_q8_0_pack(const void *ggml, void *packed, int n_out, int n_in, cudaStream_t stream);
int qdq_q4k_pack(const void *ggml, void *packed, int n_out, int n_in, cudaStream_t stream);

/* ---- dequantisation (verification aid) ------------------------------------
 * Writes the f32 weights of a packed matrix, row-major n_out x n_in, into
 * `out` (4-byte aligned).  Q8_0: d*q (exact in f32).  Q4_K: the single f32
 * rounding of d*sc_j*q - dmin*m_j.  Same block definitions as above.
 */
int qdq_q8_0_dequant(const void *W, float *out, int n_out, int n_in, cudaStream_t stream);
int qdq_q4k_dequant(const void *W, float *out, int n_out, int n_in, cudaStream_t stream);

/* ---- GEMV: y[b, r] = sum_k w[r, k] * x[b, k] -------------------------------
 * "Module cuda_lane", Functions: try_q8_0_cuda_gemv, q8_0_gemv_oracle_into,
 * try_q4k_soa_gemv.  W: packed (16-byte aligned).  x: batch x n_in f32,
 * 16-byte aligned.  y: batch x n_out f32, 4-byte aligned, must not overlap W
 * or x.  1 <= batch <= QDQ_MAX_GEMV_BATCH.  Error against the exact sum:
 * <= 1e-5 * sum_k |w[r,k]| |x[b,k]| for every finite input (f32 arithmetic; for
 * Q4_K also where d*sc_j*q and dmin*m_j cancel).  Batch 1 can opt into the
 * faster fixed-point arithmetic of QDQ_OPT_XS_FLOAT_X = 0, with the bound
 * stated there (the same holds for the SwiGLU, QKV and FFN calls below).
 */
int qdq_q8_0_gemv(const void *W, const float *x, float *y,
                  int n_out, int n_in, int batch, cudaStream_t stream);
int qdq_q4k_gemv(const void *W, const float *x, float *y,
                 int n_out, int n_in, int batch, cudaStream_t stream);

/* ---- fused SwiGLU expansion -------------------------------------------------
 * "Module cuda_lane", Functions: try_q4k_soa_fused_swiglu:
 *   mid[b, i] = silu(gate_i . x_b) * (up_i . x_b),  silu(z) = z / (1 + e^-z),
 * one kernel reading x once for both Q4_K matrices.  Wg, Wu: packed Q4_K
 * n_ff x n_embd.  x: batch x n_embd (16-byte aligned).  mid: batch x n_ff,
 * must not overlap any input.
 */
int qdq_q4k_swiglu(const void *Wg, const void *Wu, const float *x, float *mid,
                   int n_ff, int n_embd, int batch, cudaStream_t stream);

/* ---- Q6_K: repack, dequantisation, GEMV, embedding lookup -------------------
 * "QTensorEngine": embedding_pipeline (Q6_K embedding dequant + matmul on the
 * GPU, no CPU dequant), dispatch_quantized_token_embedding (raw quantised
 * embedding bytes uploaded, used without CPU dequant) and dispatch_gemm_into
 * (quantised GEMM into the caller's buffer, Q6_K).
 * qdq_q6k_packed_bytes: bytes of the packed matrix (0 on bad dims: n_in % 256).
 * qdq_q6k_pack: as qdq_q4k_pack, for GGML Q6_K input (n_out*n_in/256*210 bytes).
 * qdq_q6k_dequant: w = d*scale*(q - 32), exact in f32, into `out` (n_out x n_in).
 * qdq_q6k_gemv: as qdq_q8_0_gemv (same pointer, alignment, aliasing and batch
 *   rules); error <= 1e-5 * sum_k |w[r,k]| |x[b,k]| for every finite input.
 * qdq_q6k_get_rows: embedding lookup, out[i, :] = the dequantised row ids[i] of
 *   the packed n_rows x n_in matrix W, for i < n_ids (0 = nothing to do).  ids:
 *   int32 device array (4-byte aligned), read after the previous kernel on the
 *   stream; an id outside [0, n_rows) gives a row of NaN.  out: n_ids x n_in
 *   f32 (4-byte aligned), must not overlap W or ids.
 */
size_t qdq_q6k_packed_bytes(int n_out, int n_in);
int qdq_q6k_pack(const void *ggml, void *packed, int n_out, int n_in, cudaStream_t stream);
int qdq_q6k_dequant(const void *W, float *out, int n_out, int n_in, cudaStream_t stream);
int qdq_q6k_gemv(const void *W, const float *x, float *y, int n_out, int n_in, int batch, cudaStream_t stream);
int qdq_q6k_get_rows(const void *W, const int *ids, float *out, int n_ids, int n_rows, int n_in,
                     cudaStream_t stream);

/* ---- output projection with on-device argmax --------------------------------
 * "QTensorEngine", dispatch_output_top1_chunked (GPU block argmax, k = 1): the
 * output projection with an on-device argmax epilogue, so a decode step reads
 * back one token instead of the logits.
 *   logits[b, t] = W_t . x_b (a Q8_0 GEMV, as qdq_q8_0_gemv), then
 *   index[b] = the first t with the largest logits[b, t], value[b] = that logit
 *   (a NaN logit counts as the largest: the first NaN wins).
 * W: packed Q8_0 n_vocab x n_in (16-byte aligned).  x: batch x n_in (16-byte
 * aligned).  logits: batch x n_vocab f32 scratch the caller owns, overwritten
 * (4-byte aligned).  index (int32), value (f32): batch entries each, 4-byte
 * aligned.  No output may overlap an input or another output.  Two kernels on
 * `stream`; nothing is read back.
 */
int qdq_q8_0_logits_argmax(const void *W, const float *x, float *logits, int *index, float *value,
                           int n_vocab, int n_in, int batch, cudaStream_t stream);

/* ---- on-device top-k of the logits --------------------------------------------
 * "QTensorEngine", dispatch_output_topk_chunked (the logits stay on the GPU, a
 * top-k kernel reduces them per chunk, only K (id, logit) candidates are read
 * back).  For each of `batch` rows of n logits (row-major, 4-byte aligned):
 * index[b, j], value[b, j] (j < k, int32 / f32, 4-byte aligned) = the j-th entry
 * of the order NaN first (the first NaN first), then larger logits first, equal
 * logits (+0 == -0) by smaller index; value holds the logit's exact bits.
 * 1 <= k <= min(n, QDQ_MAX_TOPK).  workspace: qdq_topk_workspace_bytes(n, batch,
 * k) bytes of caller scratch (16-byte aligned, overwritten; the size depends on
 * the current device).  Outputs and workspace may overlap nothing.  Several
 * kernels on `stream`; k = 1 is the argmax kernel of qdq_q8_0_logits_argmax (the
 * same order), one launch, the workspace untouched.
 * qdq_q8_0_logits_topk: the Q8_0 output projection (as qdq_q8_0_logits_argmax)
 * followed by the top-k; logits: batch x n_vocab scratch the caller owns (it
 * receives the logits).  At batch 1 the projection's CTAs write the k best
 * (logit, index) keys of their own rows as they finish, and only merge kernels
 * follow; same results as the separate top-k.  k = 1 runs as
 * qdq_q8_0_logits_argmax.
 */
#define QDQ_MAX_TOPK 64
size_t qdq_topk_workspace_bytes(int n, int batch, int k);   /* 0 on bad arguments */
int qdq_topk_rows(const float *logits, int n, int batch, int k, void *workspace, int *index, float *value,
                  cudaStream_t stream);
int qdq_q8_0_logits_topk(const void *W, const float *x, float *logits, void *workspace, int *index, float *value,
                         int n_vocab, int n_in, int batch, int k, cudaStream_t stream);

/* ---- fused QKV projection ---------------------------------------------------
 * "Module cuda_lane", Functions: try_q4k_soa_qkv (one activation, one fused
 * kernel; GQA: K and V only for rows below n_kv):
 *   q[b, r] = Wq_r . x_b (r < n_q),  k[b, r] = Wk_r . x_b,  v[b, r] = Wv_r . x_b (r < n_kv).
 * Wq: packed Q4_K n_q x n_embd; Wk, Wv: packed Q4_K n_kv x n_embd, 1 <= n_kv <= n_q
 * (16-byte aligned).  x: batch x n_embd (16-byte aligned).  q: batch x n_q; k, v:
 * batch x n_kv (4-byte aligned); no output may overlap an input or another output.
 * Batch 1 is one kernel over the rows of Wq, Wk, Wv; batch 2..8 is three GEMV
 * launches.  Error bound as qdq_q4k_gemv.
 */
int qdq_q4k_qkv(const void *Wq, const void *Wk, const void *Wv, const float *x,
                float *q, float *k, float *v, int n_q, int n_kv, int n_embd, int batch,
                cudaStream_t stream);

/* ---- FFN block with on-device residual --------------------------------------
 * "Module cuda_lane", Functions: try_q4k_soa_ffn_block_residual:
 *   out = residual + W_down . swiglu(W_gate x, W_up x)
 * (pre-norm-free: x is used as given).  Two kernels on `stream`; `mid` stays
 * on the device.  Wg, Wu: packed Q4_K n_ff x n_embd; Wd: packed Q4_K
 * n_embd x n_ff.  x, residual, out: batch x n_embd.  mid_workspace: caller-
 * owned batch x n_ff f32 scratch, 16-byte aligned, overwritten.  out may be
 * exactly `residual` (in-place residual add) but may not overlap anything else.
 */
int qdq_q4k_ffn_residual(const void *Wg, const void *Wu, const void *Wd,
                         const float *x, const float *residual, float *out,
                         float *mid_workspace, int n_embd, int n_ff, int batch,
                         cudaStream_t stream);

/* ---- FFN block without caller scratch (allocates nothing) -------------------
 * No counterpart on the reference pages: an addition for callers that may not
 * allocate device memory -- e.g. a plug-in whose host application owns all GPU
 * memory through its own pool, or a decode loop that must not pay for
 * cudaMalloc/cudaFree.  Same operation, arguments and error behaviour as
 * qdq_q4k_ffn_residual, but `mid` lives in a fixed device array inside the
 * library (QDQ_NOALLOC_FFN_MAX_MID floats, 1 MiB, held by every GPU that loads
 * the library until the process exits); nothing is allocated.
 *   - batch * n_ff > QDQ_NOALLOC_FFN_MAX_MID returns QDQ_ERR_SCRATCH.
 *   - The first call on each device looks up the array's device address (with
 *     that device current); make that first call before any stream capture.
 *   - Every call shares the one array: calls that overlap on the GPU (other
 *     streams, other threads) race on it and must be serialised by the caller.
 */
#define QDQ_NOALLOC_FFN_MAX_MID 262144
int qdq_q4k_ffn_residual_noalloc(const void *Wg, const void *Wu, const void *Wd,
                                 const float *x, const float *residual, float *out,
                                 int n_embd, int n_ff, int batch, cudaStream_t stream);

/* ---- batch-prefill GEMMs on tensor cores -----------------------------------
 * "Module cuda_lane", Goal (tensor-core GEMM for batch prefill-shaped work)
 * and "weight_cache.rs", try_cuda_batch_gemv (hidden packed batch x n_in,
 * W row-major n_out x n_in, out batch x n_out; the reference pads to 16 and
 * trims, this call masks instead):
 *   Y[m, r] = sum_k bf16(X[m, k]) * bf16(w[r, k])   (f32 accumulation)
 * with w the exact f32 dequantised weight (Q8_0 d*q; Q4_K RN(d*sc*q - dmin*m)).
 * W: packed Q8_0 / Q4_K (16-byte aligned).  X: M x n_in f32 (16-byte aligned).
 * Y: M x n_out f32 (16-byte aligned), must not overlap W, X or workspace.
 * workspace: caller-owned scratch of qdq_gemm_batch_workspace_bytes(M, n_out,
 * n_in) bytes (0 when no device can be queried), 256-byte aligned, overwritten
 * with X rounded to bf16 when M > 32 (unused for M <= 32, where the kernel
 * rounds X itself; qdq_q4k_swiglu_batch: M > 16 and M <= 16).  K is split across the CTAs of a thread-block cluster when
 * the output tiles alone cannot fill the SMs; the splits' partial tiles are
 * added in shared memory, in a fixed order.
 * Requires n_in % 64 == 0 (Q4_K: % 256) and n_out % 128 == 0; M >= 1 (tail
 * masked).  Results do not depend on the order in which CTAs run (split-K
 * partials are added in a fixed order).
 * Error against the exact sum: <= 4e-3 * sum_k |w[r,k]| |X[m,k]|.
 * qdq_q4k_swiglu_batch: the SwiGLU expansion for M tokens ("Module cuda_lane",
 * try_q4k_soa_fused_swiglu, prefill-shaped): mid[m, i] = silu(g[m, i]) * u[m, i]
 * with g, u the two GEMMs above against Wg, Wu (packed Q4_K n_ff x n_embd), in
 * one kernel; workspace of qdq_q4k_swiglu_batch_workspace_bytes(M, n_ff, n_embd).
 */
size_t qdq_gemm_batch_workspace_bytes(int M, int n_out, int n_in);
int qdq_q8_0_gemm_batch(const void *W, const float *X, float *Y, void *workspace,
                        int n_out, int n_in, int M, cudaStream_t stream);
int qdq_q4k_gemm_batch(const void *W, const float *X, float *Y, void *workspace,
                       int n_out, int n_in, int M, cudaStream_t stream);
size_t qdq_q4k_swiglu_batch_workspace_bytes(int M, int n_ff, int n_embd);
int qdq_q4k_swiglu_batch(const void *Wg, const void *Wu, const float *X, float *mid, void *workspace,
                         int n_ff, int n_embd, int M, cudaStream_t stream);

/* ---- what stands between the projections of a decode step ---------------------
 * No counterpart on the reference pages (their attention, cache and norm live in another
 * engine): the operators that a model's layer needs between the projections above.
 * Activations are f32, f16 or bf16 (QDQ_TYPE_*); all sums, maxima and softmax
 * statistics are f32, and an output is rounded once to its type (attention rounds more for 16-bit types: below).
 * Strides count elements between consecutive rows (tokens).  Rows of one stride may lie beside one another, as slices of
 * one wide buffer do; of operands with different strides the whole spans may not overlap.  Where an int array on the
 * device (cu_new, cu, cu_q) says how many rows there are, the host compares the first row alone.
 * Norm weights and slopes count as weights: a kernel may read them while an earlier call of this library still runs.
 */
#define QDQ_TYPE_F32  0
#define QDQ_TYPE_F16  1
#define QDQ_TYPE_BF16 2

/* ---- RMS norm with the residual's addition ------------------------------------
 *   h = x + residual (x when residual is NULL),
 *   y = h / sqrt(mean(h^2) + eps) * weight (weight NULL: 1),
 * per row of n elements (1 <= n <= QDQ_MAX_NORM_N), rows >= 0 (0: nothing to do).
 * sum_out (may be NULL): h, rounded to the type (the norm uses h unrounded).
 * out (may be NULL): y in the type.  q8_out (may be NULL; n % 32 == 0, 16-byte aligned):
 * y as a packed Q8_0 matrix of rows x n (qdq_q8_0_packed_bytes(rows, n) bytes, layout
 * above): d = f16(max |y| / 127) over each 32, code = rint(y * (1 / d)) within
 * +-127, 0 where d is 0; a block with a NaN has d = NaN.  (The rounded d is divided by, so a code can differ by one
 * from a quantiser that divides by the unrounded one.)  The next call may take q8_out as its W.  out or q8_out is given.
 * x, residual, sum_out and out are aligned to their elements and weight to 4 bytes (16-byte
 * aligned rows are faster); strides are at least n.  sum_out may be exactly residual or x, and out exactly x
 * or residual (with its stride); outputs may overlap nothing else.
 */
#define QDQ_MAX_NORM_N 32768
int qdq_rms_norm(const void *x, const void *residual, const float *weight, void *sum_out, void *out, void *q8_out,
                 int type, int rows, int n, long long x_stride, long long residual_stride, long long sum_stride,
                 long long out_stride, float eps, cudaStream_t stream);

/* ---- paged 8-bit key/value cache ------------------------------------------------
 * A pool of n_pages pages of qdq_kv_page_bytes bytes; a page holds page_tokens tokens
 * (a multiple of QDQ_KV_BLOCK) of one sequence.  In a page each of the n_kv
 * heads has one record of page_bytes / n_kv bytes (a multiple of 128):
 *   key codes page_tokens x head_dim int8, value codes page_tokens x head_dim int8,
 *   key scales page_tokens / 16 f32, value scales page_tokens / 16 f32, zeros or anything.
 * A block is QDQ_KV_BLOCK consecutive tokens of a page (and so of a sequence); value = code * scale.
 * head_dim is 64, 96, 128, 192 or 256.  page_table: n_seqs rows of table_stride int32 page
 * ids; row s, entry i is the page of tokens i * page_tokens .. of sequence s.  Entries
 * past a sequence's tokens are not read.  kv_len (int32): tokens of each sequence,
 * the appended or querying ones included.  pages: 128-byte aligned; the int arrays 4-byte.
 *
 * qdq_kv_append quantises new tokens into the cache: the last cu_new[s + 1] - cu_new[s] of
 *   sequence s's kv_len[s] tokens are rows cu_new[s] .. of k and v (n_kv x
 *   head_dim elements per row, rows k_stride / v_stride elements apart; cu_new NULL:
 *   one token per sequence, row s).  max_new: an upper bound of the new tokens of a
 *   sequence (tokens past it are not appended).  Per block, head, and keys or values:
 *     s = max(s_old, max |x| / 127) over its new tokens (s_old: its scale, 0 if it held none),
 *     code = rint(x * (1 / s)) for new tokens, rint(code * (s_old / s)) for those it held,
 *   all f32; s below the smallest normal f32 counts as 0.  A new value that is
 *   not finite makes the block's scale NaN.  Tokens whose page id is outside [0, n_pages) or
 *   whose table entry does not exist are dropped; more new tokens than kv_len append nothing.
 * qdq_kv_read writes cu[s + 1] - cu[s] tokens of sequence s from token start[s] (start
 *   NULL: 0) to rows cu[s] .. of k and v; max_tokens bounds a sequence's tokens.  A
 *   token without a valid page reads as NaN.  The caller asks for tokens it has appended.
 * k and v are 16-byte aligned, their strides (>= n_kv * head_dim) whole 16 bytes.
 */
#define QDQ_KV_BLOCK 16
size_t qdq_kv_page_bytes(int page_tokens, int n_kv, int head_dim);   /* 0 on bad arguments */
int qdq_kv_append(void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                  int table_stride, const int *kv_len, const int *cu_new, int n_seqs, int max_new, const void *k,
                  const void *v, long long k_stride, long long v_stride, int type, cudaStream_t stream);
int qdq_kv_read(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                int table_stride, const int *start, const int *cu, int n_seqs, int max_tokens, void *k, void *v,
                long long k_stride, long long v_stride, int type, cudaStream_t stream);

/* ---- attention over the cache -----------------------------------------------------
 * For each query row i < n of sequence s (n = cu_q[s + 1] - cu_q[s], rows cu_q[s] .. of q;
 * cu_q NULL: one query per sequence, row s), at position pos = kv_len[s] - n + i, and
 * each of n_heads heads (n_heads a multiple of n_kv; head h reads cache head h / (n_heads / n_kv)):
 *   x[j] = scale * q . k[j];  softcap > 0: x[j] = softcap * tanh(x[j] / softcap);
 *   slopes (n_heads f32, may be NULL): x[j] -= slopes[h] * (pos - j);
 *   visible: j <= pos, and pos - j < window when window > 0;
 *   out = sum_j softmax(x)[j] v[j],  lse (n_heads f32 per query row, may be NULL) = log sum_j e^x[j].
 * Rounding: with f32 activations, and with 16-bit ones where max_q * (n_heads / n_kv) <= 8, the probabilities times
 * their value scales keep 2^-22 (two f16 parts, which end 2^-35 below the row's largest).  With 16-bit ones and more rows
 * they are rounded to f16 once (2^-11, as an f16 output), and query elements 2^-25 below their row's largest count
 * as 0; so a token's result moves within that when it is computed with others instead of alone.  With 16-bit
 * activations the cap's tanh is off by up to 2^-21, times softcap.
 * A row that sees no token gives zeros and lse -inf.  A value scale of 2^118 and more (values from 4e37) gives NaN.
 * A sequence with kv_len outside [0,
 * max_kv_len] or past its table row gives NaN, and so does a row that sees a token
 * with an invalid page or a NaN scale, and a query that is not finite.
 * max_kv_len, max_q: a call is cut into CTAs by them (and the workspace sized), so bounds near the lengths are faster.
 * max_q: an upper bound of a sequence's queries (rows past it are not written), at most 2^20; a cache head
 * serves at most 1024 heads.
 * q, out: head_dim elements per head, n_heads heads per row, rows q_stride /
 * out_stride elements apart, 16-byte aligned (strides whole 16 bytes).  out may overlap no other argument.
 * workspace: qdq_kv_attention_workspace_bytes(...) bytes (0 when no device can be queried), 256-byte aligned, ZEROED ONCE by
 * the caller before its first use; a call leaves it ready for the next one on the same stream, also one of
 * other sizes, types or windows, or of qdq_token_logprobs, that is given the same workspace and workspace_bytes.
 * Results do not depend on the order in which CTAs run; the last bits of a row do on the lengths of all sequences of
 * the call, which decide where its sums are cut.
 */
#define QDQ_MAX_KV_LEN 4194304   /* the largest max_kv_len */
size_t qdq_kv_attention_workspace_bytes(int n_seqs, int max_q, int max_kv_len, int n_heads, int n_kv, int head_dim);
int qdq_kv_attention(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                     int table_stride, const int *kv_len, const int *cu_q, int n_seqs, int max_q, int max_kv_len,
                     int n_heads, const void *q, long long q_stride, void *out, long long out_stride, float *lse,
                     const float *slopes, float scale, float softcap, int window, int type, void *workspace,
                     size_t workspace_bytes, cudaStream_t stream);

/* ---- log probabilities of given tokens ----------------------------------------------
 * For each of `rows` rows (row_stride elements apart) of n logits x (1 <= n <= 2^30):
 *   lse = log sum_i e^x[i];  logprob[r] = x[tokens[r]] - lse (NaN for a token outside [0, n));
 *   entropy[r] = -sum_i p[i] log p[i], p = softmax(x)  (a -inf logit counts 0; may be NULL);
 *   top_index / top_logprob [r, j] (j < k, 0 <= k <= min(n, QDQ_MAX_TOPK); ignored for k = 0):
 *   the j-th of the order of qdq_topk_rows, and its x - lse.
 * A row with a NaN or +inf, or without a logit above -inf, has NaN in all but top_index.
 * tokens and logprob: both given or both NULL.  workspace as for qdq_kv_attention
 * (qdq_token_logprobs_workspace_bytes, 256-byte aligned, zeroed once).  Outputs may overlap nothing.
 */
size_t qdq_token_logprobs_workspace_bytes(int rows, int n, int k);
int qdq_token_logprobs(const void *logits, long long row_stride, int type, const int *tokens, int rows, int n, int k,
                       float *logprob, float *entropy, int *top_index, float *top_logprob, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/* ---- drafted tokens ---------------------------------------------------------------------
 * Several tokens of a sequence run in one step: guesses of what follows, verified by the model's own
 * probabilities.  They are a tree: node i of n is row cu[s] + i, and the i-th of the sequence's last n
 * cached tokens; parent[row] is an earlier node's number (0 <= parent < i), or -1.  A node's depth is the number of its
 * ancestors, its position kv_len[s] - n + depth.  A step is
 *   qdq_kv_append_rope -> qdq_kv_tree_attention (every layer), qdq_verify_drafts, qdq_kv_keep (every layer's cache),
 * and then kv_len[s] -= n - 1 - accepted[s].  A tree has at most QDQ_MAX_TREE nodes; a node whose parent is
 * neither -1 nor earlier gives NaN (and its cache blocks do), or is not accepted.
 *
 * qdq_kv_append_rope norms and turns new tokens' queries and keys, and appends keys and values to the cache:
 *   q_weight, k_weight (head_dim f32 each, may be NULL: no norm): per head y = x / sqrt(mean(x^2) + eps) * weight;
 *   freqs (n_rot / 2 f32, radians per position; NULL: nothing is turned): pair i of a head's first n_rot elements,
 *     (a, b) -> (a cos t - b sin t, b cos t + a sin t) with t = position * freqs[i]; the pair is elements
 *     (2i, 2i + 1) where interleaved is 1, else (i, i + n_rot / 2).  n_rot: a multiple of 8, at most head_dim.
 *     For freqs up to 1 the angle is off by at most 2^-29 + position * 2^-52, and an f32's rounding, before cos and sin.
 *   q_out: the queries in the type (may be exactly q with its stride); keys go into the cache in f32, values as they are,
 *   by the definition of qdq_kv_append, whose other arguments, refusals and dropped tokens hold here.
 *   parent NULL: tokens one after the other (position = place in the cache).  q and q_out NULL with n_heads 0: keys and values alone.
 *   Where a sequence has more new tokens than kv_len, nothing is appended and its rows of q_out are NaN.
 *   Weights and freqs count as weights (above); they are 16-byte and 4-byte aligned.
 *
 * qdq_kv_tree_attention is qdq_kv_attention with cu_q and parent: node i sees the tokens before
 *   kv_len[s] - n, its ancestors and itself, of which the window hides those at positions too far before its own; bias by
 *   positions.  Same workspace (qdq_kv_attention_workspace_bytes), rounding and other rules.
 *   max_q: at most QDQ_MAX_TREE; a sequence with more rows gives NaN in its first max_q.
 *
 * qdq_verify_drafts accepts drafts of each sequence and draws its next token.  logits: n per row (type, row_stride
 *   elements apart), the target's after the row's token; cu NULL: one row per sequence (the next token alone).
 *   Row 0 is the sequence's last token, rows i > 0 are drafts tokens[row] under their parents (parent
 *   NULL: i - 1).  p = softmax(logits / temperature).  At the present node, first 0, with w = p: its children x in order
 *     accepted when uniform[row of x] * q(x) < w(x): the present node then, and w its p;
 *     else w = max(w - q, 0) / sum (as it was where the sum is 0).
 *   q = draft_probs (n f32 per row, draft_stride apart: what the children of the row's node were drawn from,
 *   independently); draft_probs NULL: 1 at x, so that w loses x.  Then, where no child is left:
 *     next_token[s] = the first i with w_0 + .. + w_i > uniform[row 0] * sum w,
 *     accepted[s] = the number of accepted drafts, path[s * max_rows ..] = 0, the accepted nodes, then -1.
 *   temperature 0: a child is accepted when it is the row's largest logit (the first of equals), which is next_token
 *   too; draft_probs and uniform are not read.  Else temperature is between 1e-6 and 1e6.
 *   A drafted token outside [0, n) is not accepted.  Numbers outside [0, 1) count as the nearest inside.  At a node
 *   whose row has a NaN or +inf, or nothing above -inf, no child is accepted and next_token is -1.  A sequence without
 *   rows gets accepted -1, next_token -1 and a path of -1.  max_rows: at most QDQ_MAX_TREE; rows past it do not count.
 *   A number may fall to either side of a border that lies as near as what decides is off: p by 2^-17 of itself (below 2^-126
 *   of the row's largest it counts as 0); after rejections, without draft_probs, w by 2^-16 of itself; with draft_probs
 *   w = max(p - b q, 0) / S, where b is the sum of the S before (first 0 and 1), max(p - b q, 0) by 2^-16 of p + b q for each
 *   rejection at the node, and S by what that is for all its tokens; the drawn token's sum by the same share of it.
 *   workspace: qdq_verify_drafts_workspace_bytes(...) bytes, 256-byte aligned; it may be shared as those above.
 *
 * qdq_kv_keep moves the cached tokens of the accepted paths: of sequence s's last n = cu[s + 1] - cu[s] tokens, node
 *   path[s * path_stride + i], i <= accepted[s], goes to place kv_len[s] - n + i (kv_len is not changed).  Per block
 *   that gets a token from elsewhere: its scale becomes the largest scale of its tokens' blocks, s, and
 *   every code rint(code * (s_of_its_block / s)); tokens that stay lose nothing where their scale is the largest.  A path's
 *   nodes are in growing order (as qdq_verify_drafts writes them); it ends before the first that is not, or is not below n.
 *   accepted below 0, or n above kv_len: nothing.  A token without a page counts as one of scale NaN.
 */
#define QDQ_MAX_TREE 64
int qdq_kv_append_rope(void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                       int table_stride, const int *kv_len, const int *cu_new, const int *parent, int n_seqs, int max_new,
                       int n_heads, const void *q, long long q_stride, void *q_out, long long q_out_stride, const void *k,
                       long long k_stride, const void *v, long long v_stride, const float *q_weight,
                       const float *k_weight, float eps, const float *freqs, int n_rot, int interleaved, int type,
                       cudaStream_t stream);
int qdq_kv_tree_attention(const void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table,
                          int table_stride, const int *kv_len, const int *cu_q, const int *parent, int n_seqs, int max_q,
                          int max_kv_len, int n_heads, const void *q, long long q_stride, void *out, long long out_stride,
                          float *lse, const float *slopes, float scale, float softcap, int window, int type,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream);
size_t qdq_verify_drafts_workspace_bytes(int n_seqs, int max_rows, int n);
int qdq_verify_drafts(const void *logits, long long row_stride, int type, const int *tokens, const int *cu, const int *parent,
                      int n_seqs, int max_rows, int n, const float *draft_probs, long long draft_stride,
                      const float *uniform, float temperature, int *accepted, int *path, int *next_token, void *workspace,
                      size_t workspace_bytes, cudaStream_t stream);
int qdq_kv_keep(void *pages, int n_pages, int page_tokens, int n_kv, int head_dim, const int *page_table, int table_stride,
                const int *kv_len, const int *cu, int n_seqs, const int *path, int path_stride, const int *accepted,
                cudaStream_t stream);

/* ---- pipeline health -------------------------------------------------------
 * Every wait inside the tensor-core pipeline is bounded (2 s wall clock); a
 * wait that runs out makes its CTA stop early instead of hanging, and counts
 * here.  Returns the count since the previous call and resets it (-1 on a
 * CUDA error).  Synchronous: it waits for the device.
 */
int qdq_pipeline_timeouts(void);

/* ---- debug build: device-side guards ----------------------------------------
 * A library built with -DQDQ_CHECKS (ggml_quantized_dequant_gb300._build.build(checks=True),
 * libqdq_checked.so) guards its shared-memory row buffers, blocks and lists, weight-row and
 * activation indices, output and workspace indices and bulk-copy alignment inside the kernels:
 * an index out of bounds skips that access and sets a bit of a device status word
 * (QDQ_CHECK_* in the library's internal header: 1 shared memory, 2 weight row,
 * 4 output, 8 copy alignment) instead of trapping.  qdq_check_status waits for the
 * device, returns the or of the bits since its previous call and clears them (-1
 * on a CUDA error); in the normal build it returns 0.  qdq_checks_enabled: 1 in
 * the debug build, else 0.
 */
int qdq_check_status(void);
int qdq_checks_enabled(void);

/* ---- launch round trip -------------------------------------------------------
 * "QTensorEngine", bench_empty_submit_roundtrip (the fixed submit-to-completion
 * latency, measured with no compute): launches one empty kernel (one thread) on
 * `stream`; a caller times n of these each followed by a synchronisation.
 */
int qdq_noop(cudaStream_t stream);

/* ---- launch options (same work, different launch shape; for measurement) -- */
#define QDQ_OPT_PDL          1  /* 1 (default): programmatic dependent launch on; 0: plain launches */
#define QDQ_OPT_L2_PREFETCH  2  /* L2 prefetch of weight rows.  0 (default): automatic -- the batch-1 direct-load kernel
                                   prefetches nothing, the ring kernel's Q8_0 GEMV prefetches the rows its first ring fill
                                   leaves out when they fit in half the L2; 1: every GEMV CTA prefetches all its rows first;
                                   2: every ring-kernel CTA prefetches the rows its first ring fill leaves out; 3: no prefetch */
#define QDQ_OPT_CTAS_PER_SM  3  /* GEMV-family CTAs per SM, 1..4; 0 (default): automatic (batch-1 direct-load kernel: as
                                   many as fit; ring kernel: 2 for the FFN kernels, else 1; batch 2..8: 1) */
#define QDQ_OPT_XS_GROUPS    4  /* batch-1 GEMV groups of slice warps per CTA, 0 = automatic (default: 1 in the
                                   direct-load kernel), 1..16 */
#define QDQ_OPT_XS_STAGES    5  /* batch-1 GEMV: ring slots per consumer group (ring kernel), or the register depth
                                   1 / 2 (direct-load kernel); 0 = automatic (default), 1..16 */
/* Arithmetic of the batch-1 kernels (qdq_q8_0_gemv and qdq_q4k_gemv at batch 1,
 * qdq_q4k_swiglu, qdq_q4k_qkv, the output projections and both FFN calls at batch 1):
 *   1 (default): weights converted exactly to f32 and multiplied with f32 FMAs
 *     (Q4_K: quants shifted by the sub-block's integer offset before they are
 *     summed): within 1e-5 sum |w||x| of the exact sum for every finite input.
 *   0 (opt-in, faster): each 32-activation block becomes 24-bit block fixed
 *     point X_j = rint(x_j 2^e), |X_j| <= 2^22, and block dot products are
 *     exact integer byte dot products, scaled in f32.  Error against the exact
 *     sum <= 2^-22 sum_blocks max_j |x_j| sum_j |w_j| + f32 rounding: a bound
 *     relative to each block's largest activation, so it exceeds
 *     1e-5 sum |w||x| where a row's weights sit on the small activations of
 *     blocks whose largest activation they skip.  A block with an inf or NaN
 *     activation gives NaN outputs. */
#define QDQ_OPT_XS_FLOAT_X   6
/* Batch-1 kernel of the f32 arithmetic: 0 (default) the direct-load kernel (weights straight into
 * registers, small CTAs of one group of slice warps, as many per SM as fit); 1 the shared-memory
 * ring kernel (a producer warp streams weights into a ring sized to half an SM, so that the next
 * kernel's CTA can start streaming beside it).  Same results within the stated bound; the
 * fixed-point arithmetic always runs in the ring kernel. */
#define QDQ_OPT_BATCH1_KERNEL 7
/* Kernel of qdq_kv_attention: 0 (default) automatic (by rows per cache head and work); 1 the decode kernel; 2 the
 * tensor-core kernel wherever it can run (head dims 64, 128, 192, or 256 with 16-bit types; more than 8 rows per
 * cache head for 16-bit types).  Results within the same bound.  Set it before the workspace is sized. */
#define QDQ_OPT_ATTN_KERNEL 8
/* Sets a process-wide option; returns the previous value, or QDQ_ERR_DIMS for a bad key/value. */
int qdq_set_option(int key, int value);

#ifdef __cplusplus
}
#endif

#endif /* QDQ_H */
