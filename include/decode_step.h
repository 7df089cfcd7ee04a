/*
 * decode_step.h — C ABI of the GB300 (sm_103a) single-token decode step.
 *
 * Every call takes plain pointers and sizes.  Unless stated otherwise:
 *  - Buffers are DEVICE pointers owned by the caller; the library allocates
 *    no device memory in any call (a decode step "runs with zero heap
 *    allocations", "Inside the engine", section 1, "CausalLM: the forward
 *    path").  Scratch space is a caller-supplied workspace whose size a
 *    *_workspace_bytes call reports; a workspace must be zero-filled before
 *    its first use and is left ready for the next call of the same operation
 *    and sizes by every call.  For another operation, or other sizes, it has to
 *    be zeroed again unless the calls say that they may share it.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream) and return before the GPU work finishes.
 *  - Every length argument is an element count.  Each buffer's real length
 *    is passed next to it and checked against the length the operation
 *    needs, as the "LLM inference kernels" page's contract checks do
 *    ("Status vocabulary and the shape checks (contract)", "Guarantees").
 *    On any refusal the call returns before launching anything and leaves
 *    every output untouched.
 *  - Only what the host can see is checked on the host.  Values that live in
 *    device memory (token ids, positions, sequence lengths) are checked by the
 *    kernels: an out-of-range value is clamped or skipped and a bit is set in
 *    the workspace's error word (see ds_workspace_error).
 *  - Identical inputs give bit-identical outputs run to run: no reduction
 *    depends on the order in which thread blocks finish.
 *  - fp32 activations and fp32 or bf16 weights, unless a call names others;
 *    KV cache fp32 or bf16; fp32 accumulation.
 */
#ifndef DECODE_STEP_H
#define DECODE_STEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(_WIN32)
#define DS_API
#else
#define DS_API __attribute__((visibility("default")))
#endif

/* A cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st *ds_stream_t;

/* ---------------------------------------------------------------------
 * Status vocabulary.  560-571 keep the numbers and meanings of the
 * "LLM inference kernels" page ("Status vocabulary and the shape checks
 * (contract)"); 572-577 are this library's additions in the unused part of
 * the same 560-579 range.
 * ------------------------------------------------------------------- */
enum {
    DS_OK = 560,                      /* ran; every output element is defined */
    DS_EMPTY_DIMENSION = 561,         /* a required dimension was < 1 */
    DS_A_LENGTH_MISMATCH = 562,       /* first operand's length != n */
    DS_B_LENGTH_MISMATCH = 563,       /* second operand's length != n */
    DS_DIMENSION_TOO_LARGE = 564,     /* a dimension exceeds DS_MAX_DIM */
    DS_CODE_OUT_OF_RANGE = 565,       /* ds_status_name's answer for an unknown code */
    DS_CACHE_LENGTH_MISMATCH = 566,   /* cache length / position out of range */
    DS_NEW_LENGTH_MISMATCH = 567,     /* appended values' length != n_new */
    DS_LOGITS_LENGTH_MISMATCH = 568,  /* logits length != n_rows * n */
    DS_GEMV_A_LENGTH_MISMATCH = 569,  /* matrix length != rows * cols */
    DS_GEMV_X_LENGTH_MISMATCH = 570,  /* vector length != the reduced dimension */
    DS_CACHE_CAPACITY_EXCEEDED = 571, /* an append would overrun the reserved cache */
    DS_BAD_DTYPE = 572,               /* dtype or layout code not supported here */
    DS_CUDA_ERROR = 573,              /* a CUDA runtime call failed */
    DS_WORKSPACE_TOO_SMALL = 574,     /* workspace NULL or smaller than required */
    DS_BAD_SAMPLING_PARAM = 575,      /* temperature/top_k/top_p outside their domain */
    DS_TOKEN_OUT_OF_RANGE = 576,      /* a host-visible token id outside [0, vocab) */
    DS_BAD_ARGUMENT = 577             /* NULL pointer, misaligned pointer or bad count */
};

/* Largest accepted dimension (per dimension), 1 << 24, as on the
 * "LLM inference kernels" page ("Status vocabulary and the shape checks"). */
#define DS_MAX_DIM (1LL << 24)

/* Storage dtypes.  DS_E4M3 (8-bit floating point: sign, 4 bits of exponent, 3
 * of mantissa, 0x7F and 0xFF NaN, no infinities) is taken where a call says so. */
enum { DS_F32 = 0, DS_BF16 = 1, DS_E4M3 = 2 };

/* RoPE layouts: pairs (p, p + head_dim/2) — the GPT-NeoX split-half
 * convention ("LLM inference kernels", "Two gaps, not three") — or pairs
 * (2p, 2p + 1) ("The forward pass end to end", "The code"). */
enum { DS_ROPE_HALF_SPLIT = 0, DS_ROPE_INTERLEAVED = 1 };

/* Bits of a workspace's error word (set by kernels, never by the host). */
enum {
    DS_ERR_TOKEN_RANGE = 1,   /* a device-side token id was outside [0, vocab); clamped */
    DS_ERR_POSITION = 2,      /* a device-side position or length exceeded the cache */
    DS_ERR_WAIT_TIMEOUT = 4,  /* a bounded wait inside a kernel gave up */
    DS_ERR_SAMPLING = 8,      /* a sampler row had no finite logits */
    DS_ERR_NO_BLOCKS = 16     /* a step's rows or new blocks did not fit (ds_paged_plan) */
};

/* Name of a status code ("ds_ok", "ds_a_length_mismatch", ...);
 * "ds_code_out_of_range" for anything else.  Static storage. */
DS_API const char *ds_status_name(int code);

/* The residual-add shape check of the "LLM inference kernels" contract:
 * 561 if n < 1, 564 if n > DS_MAX_DIM, 562 if a_len != n, 563 if b_len != n,
 * else 560.  Host only. */
DS_API int ds_residual_dims_check(int64_t n, int64_t a_len, int64_t b_len);

/* Copy a workspace's error word (int32 at byte 0 of every workspace) to
 * *host_word and clear it.  Synchronises `stream`. */
DS_API int ds_workspace_error(void *workspace, int32_t *host_word, ds_stream_t stream);

/* Number of streaming multiprocessors the library sizes its grids for on the
 * current device (0 when no device is usable). */
DS_API int ds_device_sm_count(void);

/* ---------------------------------------------------------------------
 * Projections
 * ------------------------------------------------------------------- */

/* Workspace bytes ds_gemv_transposed needs for a rows x cols matrix. */
DS_API size_t ds_gemv_workspace_bytes(int64_t rows, int64_t cols, int a_dtype);

/* y = A^T x: y[j] = sum_i A[i * cols + j] * x[i] for j < cols.
 * The transposed mat-vec of "LLM inference kernels" ("A parallel path for
 * one frozen kernel's known-slow shape"): A is row-major with `rows` input
 * rows and `cols` output columns, the layout of every decode-step projection.
 *   A: rows*cols elements of a_dtype (a_len must equal rows*cols, else 569)
 *   x: rows fp32 (x_len must equal rows, else 570); y: cols fp32 (y_len must
 *   equal cols, else 562); 561 / 564 for an empty / oversized dimension.
 *   workspace: ds_gemv_workspace_bytes(rows, cols, a_dtype) bytes, zeroed
 *   before first use.
 * Weight rows stream through shared memory with bulk asynchronous copies when
 * A is 16-byte aligned and cols * element size is a multiple of 16 bytes;
 * other shapes run a plain-load kernel with the same result definition. */
DS_API int ds_gemv_transposed(const void *A, int64_t a_len, int a_dtype, const float *x,
                              int64_t x_len, int64_t rows, int64_t cols, float *y,
                              int64_t y_len, void *workspace, size_t workspace_bytes,
                              ds_stream_t stream);

/* ds_gemv_transposed for callers that cannot allocate device memory (for
 * example a host whose device memory is all owned by its own allocator, or a
 * plug-in handed nothing but one operation's inputs and outputs).  The pages
 * have no counterpart of this call.  Same arguments, result and checks as
 * ds_gemv_transposed, minus the workspace: the split-reduction scratch comes
 * from a fixed area compiled into the library, which every GPU that loads the
 * library keeps (ds_gemv_transposed_noalloc_max_bytes() bytes, 1 MiB) until
 * the process exits.  A matrix on the streamed path (A 16-byte aligned and
 * cols * element size a multiple of 16 bytes) whose scratch
 * (ds_gemv_workspace_bytes) does not fit in the area is refused with
 * DS_DIMENSION_TOO_LARGE; any other matrix runs the plain-load kernel, which
 * uses no scratch.  The call allocates nothing: on the streamed path it clears
 * the band counters with one asynchronous memset, then launches the kernel on
 * `stream`.
 *  - The first call on a device (that device current) looks up the area's
 *    device address, which is kept for the life of the process; make that
 *    first call before any stream capture.  After cudaDeviceReset the kept
 *    address is stale: the call must not be used again in that process.
 *  - All calls share the one area and it keeps the last call's contents:
 *    calls whose GPU work overlaps (other streams, other threads) race on it
 *    and must be ordered by the caller.
 *  - A kernel's error bits (DS_ERR_*) collect in the area's error word across
 *    calls until ds_gemv_transposed_noalloc_error reads and clears it. */
DS_API int ds_gemv_transposed_noalloc(const void *A, int64_t a_len, int a_dtype, const float *x,
                                      int64_t x_len, int64_t rows, int64_t cols, float *y,
                                      int64_t y_len, ds_stream_t stream);
DS_API size_t ds_gemv_transposed_noalloc_max_bytes(void);
/* Copy the no-allocation area's error word (of the current device) to
 * *host_word and clear it, as ds_workspace_error does for a workspace.
 * Synchronises `stream`. */
DS_API int ds_gemv_transposed_noalloc_error(int32_t *host_word, ds_stream_t stream);

/* y = W x: y[r] = sum_c W[r * cols + c] * x[c] for r < rows — the
 * untransposed form the "LLM inference kernels" page uses for lm_head.
 *   W: rows*cols of w_dtype (569), x: cols fp32 (570), y: rows fp32 (562). */
DS_API int ds_gemv(const void *W, int64_t w_len, int w_dtype, const float *x, int64_t x_len,
                   int64_t rows, int64_t cols, float *y, int64_t y_len, ds_stream_t stream);

/* ---------------------------------------------------------------------
 * Batched projections (tensor cores)
 *
 * When one step decodes n sequences ("Inside the engine", section 4:
 * batched decode, one token per sequence per step) each projection applies
 * the same matrix to n activation vectors: a skinny GEMM, run on the tcgen05
 * tensor cores with bf16 operands and fp32 accumulation.  n is 1..256.
 * ------------------------------------------------------------------- */

/* Workspace bytes ds_gemm_transposed / ds_gemm need for n vectors and a
 * rows x cols matrix (either orientation); 0 for an unsupported shape. */
DS_API size_t ds_gemm_workspace_bytes(int64_t n, int64_t rows, int64_t cols);

/* Y[s][j] = sum_i A[i * cols + j] * X[s * rows + i] for s < n, j < cols:
 * ds_gemv_transposed's y = A^T x ("LLM inference kernels", "A parallel path
 * for one frozen kernel's known-slow shape") for the n rows of X at once.
 *   A: bf16 rows*cols (a_len, else 569); X: bf16 n*rows (x_len, else 570);
 *   Y: fp32 n*cols (y_len, else 562).  rows and cols multiples of 8, A and X
 *   16-byte aligned (577).  561 / 564 for an empty / oversized dimension
 *   (n > 256 included).  workspace: ds_gemm_workspace_bytes(n, rows, cols)
 *   bytes, zeroed before first use. */
DS_API int ds_gemm_transposed(const void *A, int64_t a_len, const void *X, int64_t x_len, int64_t n,
                              int64_t rows, int64_t cols, float *Y, int64_t y_len, void *workspace,
                              size_t workspace_bytes, ds_stream_t stream);

/* Y[s][r] = sum_c W[r * cols + c] * X[s * cols + c] for s < n, r < rows: the
 * untransposed form of the output head (ds_gemv) for n vectors.
 *   W: bf16 rows*cols (569); X: bf16 n*cols (570); Y: fp32 n*rows (562);
 *   cols a multiple of 8; other checks as ds_gemm_transposed. */
DS_API int ds_gemm(const void *W, int64_t w_len, const void *X, int64_t x_len, int64_t n, int64_t rows,
                   int64_t cols, float *Y, int64_t y_len, void *workspace, size_t workspace_bytes,
                   ds_stream_t stream);

/* ---------------------------------------------------------------------
 * 8-bit projections
 *
 * Weights and activations in e4m3 with an fp32 scale for each block: a
 * projection then streams half the bytes of bf16.  Weights are untransposed
 * ([out][in], ds_gemm's form) with a scale for each 128 x 128 block,
 * activations have one for each 128 values of a row.  A value stands for
 * code x scale.
 * ------------------------------------------------------------------- */

/* Rows (block_rows 1: activations) or a matrix (block_rows 128: weights) in
 * e4m3.  For each block of block_rows x 128 values (fewer at the ends):
 *   top = max |x|, at least 2^-96;  scale = top / 448;
 *   code = e4m3(x * (448 / top)), to nearest, ties to even;
 * top, quotients and product in fp32.  A block that holds a NaN or an infinity
 * has scale NaN and codes NaN.
 *   x: `rows` rows of `cols` fp32 or bf16 elements, x_stride elements apart;
 *   x_len counts the elements from x on ((rows - 1) * x_stride + cols at
 *   least, else 562).  q: codes, rows q_stride bytes apart (563 likewise; the
 *   bytes between rows stay as they were).  scales: fp32
 *   [ceil(rows / block_rows)][ceil(cols / 128)] (563).  q and scales overlap
 *   nothing (577).  561 / 564 for an empty / oversized dimension or stride,
 *   572 for another x_dtype, 577 for another block_rows.
 * Rows that start on 16 bytes (q on 8) are read 16 bytes at a time. */
DS_API int ds_fp8_quantize(const void *x, int64_t x_len, int x_dtype, int64_t x_stride, int64_t rows,
                           int64_t cols, int block_rows, void *q, int64_t q_len, int64_t q_stride,
                           float *scales, int64_t scales_len, ds_stream_t stream);

/* Workspace bytes ds_gemm_fp8 needs for these sizes; 0 for a dimension
 * < 1 or past DS_MAX_DIM. */
DS_API size_t ds_gemm_fp8_workspace_bytes(int64_t n, int64_t rows, int64_t cols);

/* Y[s][r] = sum_b x_scales[s][b] * w_scales[r / 128][b]
 *           * sum_{c in [128 b, 128 b + 128), c < cols} X[s][c] * W[r][c]
 * for s < n, r < rows: ds_gemm's untransposed product of e4m3 operands, the
 * products of a block summed by the tensor cores in fp32, the blocks in fp32,
 * the two scales multiplied first, in fp32 (past its range infinite or zero).
 * n is any count from a single token to a whole prompt.
 *   W: e4m3, rows w_stride bytes apart; w_scales: fp32 [ceil(rows / 128)]
 *   [ceil(cols / 128)] (569).  X: e4m3 [n], rows x_stride bytes apart;
 *   x_scales: fp32 [n][ceil(cols / 128)] (570).  Y: fp32 or bf16 (572), rows
 *   y_stride elements apart (562).  w_len, x_len, y_len count the elements
 *   from the pointer on, (count - 1) * stride + width at least.  W and X
 *   16-byte aligned, w_stride and x_stride multiples of 16 (577); cols need
 *   not be.  Y overlaps no input (577).  561 / 564 for an empty / oversized
 *   dimension or stride.  A NaN code or scale reaches the outputs whose sums
 *   it is part of and no other.
 *   workspace: ds_gemm_fp8_workspace_bytes(n, rows, cols) bytes, 256-byte
 *   aligned, zeroed before first use (and again after a DS_ERR_WAIT_TIMEOUT);
 *   calls whose GPU work may overlap need one each.  Calls of several sizes, of
 *   this operation and of ds_moe_layer, may share one that is as large as the
 *   largest of their answers (a larger n may need less). */
DS_API int ds_gemm_fp8(const void *W, int64_t w_len, int64_t w_stride, const float *w_scales,
                       int64_t w_scales_len, const void *X, int64_t x_len, int64_t x_stride,
                       const float *x_scales, int64_t x_scales_len, int64_t n, int64_t rows, int64_t cols,
                       void *Y, int64_t y_len, int y_dtype, int64_t y_stride, void *workspace,
                       size_t workspace_bytes, ds_stream_t stream);

/* ---------------------------------------------------------------------
 * Mixture of experts
 *
 * The feed-forward of a decoder whose tokens each go through a few of many
 * experts, for a decode step's tokens: of the weights only the chosen
 * experts' are read, once for each 32 tokens of an expert (16 with fp32 x and
 * e4m3 weights), one after the other.
 * ------------------------------------------------------------------- */

/* Workspace bytes ds_moe_layer needs; 0 for sizes that it refuses. */
DS_API size_t ds_moe_layer_workspace_bytes(int64_t n, int64_t d, int64_t ff, int n_experts, int top_k);

/* The whole layer for n tokens in one launch.  For token t
 *   l_e = sum_j x[t][j] * w_router[e][j], the top_k largest chosen (among
 *   equals the lower index; NaN above every number), chosen i being e_i;
 *   p_i = exp(l_{e_i}) / sum_e exp(l_e), over all experts, or with
 *   renormalize != 0 over the chosen ones;
 *   y[t] = (residual[t] +) sum_i p_i W_down[e_i] (silu(W_gate[e_i] x[t]) * (W_up[e_i] x[t])),
 *   silu(z) = z / (1 + e^-z) as in ds_silu_mul.
 *   x, residual (may be NULL) and y: [n][d] fp32 or bf16 (x_dtype; 570, 562).
 *   w_router: [n_experts][d] fp32 or bf16 (router_dtype).  w_gate_up:
 *   [n_experts][2][ff][d], an expert's gate rows and then its up rows; w_down:
 *   [n_experts][d][ff]; both bf16, or e4m3 with a scale for each 128 x 128
 *   block of every matrix (w_dtype): gate_up_scales [n_experts][2][ceil(ff /
 *   128)][ceil(d / 128)], down_scales [n_experts][ceil(d / 128)][ceil(ff /
 *   128)] (with bf16 NULL, else 577, and 0).  569 for a weight's or scale's length.
 *   expert_ids, expert_weights: e_i and p_i [n][top_k], either may be NULL.
 * Logits are held to some 2^-45 of the sum of their products' magnitudes
 * (products above 2^-102; of smaller ones fewer bits are left), and the choice of
 * experts is that of 64-bit arithmetic where logits are farther apart than that.
 * Sums are fp32, of factors of 24 bits (with e4m3 experts before a bf16 y the
 * intermediate has 16); y is rounded once.  Before e4m3 weights a value of x or
 * of the intermediate is held to 2^-37 (bf16 x: 2^-25, intermediate 2^-29) of
 * the largest of its 128, whatever its own size: a smaller one may be lost.
 * Weights are finite; a value of x that is not, or a product that overflows
 * fp32, makes outputs of its own token (and of no other) NaN or infinite.
 *   n <= 256, n_experts <= 512, top_k <= 16 (564), top_k <= n_experts (577);
 *   d and ff multiples of 8 with bf16 weights, of 16 with e4m3 (577); x, the
 *   router and the experts' matrices 16-byte aligned (577).  y may be x or
 *   residual itself; otherwise no output overlaps an input or another output
 *   (577).  workspace: ds_moe_layer_workspace_bytes(...) bytes, 256-byte
 *   aligned, zeroed before first use (and again after a DS_ERR_WAIT_TIMEOUT);
 *   calls whose GPU work may overlap need one each, others may share one, with
 *   ds_gemm_fp8 as well (see there).  A cooperative launch: its
 *   blocks wait for one another, so it runs when every SM has room for one. */
DS_API int ds_moe_layer(const void *x, int64_t x_len, int x_dtype, int64_t n, int64_t d,
                        const void *w_router, int64_t router_len, int router_dtype, int n_experts,
                        int top_k, int renormalize, const void *w_gate_up, int64_t gate_up_len,
                        const float *gate_up_scales, int64_t gate_up_scales_len, const void *w_down,
                        int64_t down_len, const float *down_scales, int64_t down_scales_len, int w_dtype,
                        int64_t ff, const void *residual, void *y, int64_t y_len, int32_t *expert_ids,
                        float *expert_weights, void *workspace, size_t workspace_bytes,
                        ds_stream_t stream);

/* ---------------------------------------------------------------------
 * Decode glue
 * ------------------------------------------------------------------- */

/* out[i] = a[i] + b[i] in fp32 for i < n ("LLM inference kernels",
 * "Residual add").  a_len/b_len must equal n (562/563); out has n elements and
 * may alias a or b. */
DS_API int ds_residual_add(const float *a, int64_t a_len, const float *b, int64_t b_len,
                           float *out, int64_t n, ds_stream_t stream);

/* residual += x (fp32, in place), then h = residual * (mean(residual^2) + eps)^(-1/2) * w,
 * the square sum accumulated in fp32 ("decode-ops", "Usage" and
 * "API — Method"; "The forward pass end to end", "The code", rmsnorm).
 * x may be NULL (plain RMSNorm; x_len ignored).  residual_len (562), x_len
 * (563), w_len and h_len (562) must equal n; w is fp32 or bf16. */
DS_API int ds_add_rmsnorm(float *residual, int64_t residual_len, const float *x, int64_t x_len,
                          const void *w, int64_t w_len, int w_dtype, float eps, float *h,
                          int64_t h_len, int64_t n, ds_stream_t stream);

/* Rotate q (n_qh heads) and k (n_kh heads, may be NULL with n_kh = 0) of
 * head_dim values each, in place, to position `pos`: pair p turns by
 * pos * base^(-2p/head_dim), the head_dim/2 angles formed once per call in fp64
 * on the host and rounded to fp32 ("decode-ops", "API — Method"), the rotation
 * applied in fp32 on the device.  layout: DS_ROPE_*.
 * q_len must be n_qh*head_dim (562), k_len n_kh*head_dim (563); head_dim
 * even and <= 1024 (577); pos >= 0 (566). */
DS_API int ds_rope(float *q, int64_t q_len, float *k, int64_t k_len, int64_t pos, int n_qh,
                   int n_kh, int head_dim, double base, int layout, ds_stream_t stream);

/* Reserved-capacity KV append: write the n_new fp32 values into
 * cache[cache_len, cache_len + n_new) in place, converted to cache_dtype
 * (bf16: round to nearest even) ("LLM inference kernels", "The hot loop
 * doesn't call kv_cache_append_flat").  `capacity` is the cache's reserved
 * element count.  561 for n_new < 1, 567 if new_len != n_new, 566 if
 * cache_len < 0, 571 if cache_len + n_new > capacity. */
DS_API int ds_kv_cache_append(void *cache, int cache_dtype, int64_t capacity, int64_t cache_len,
                              const float *new_vals, int64_t new_len, int64_t n_new,
                              ds_stream_t stream);

/* out[i] = silu(gate[i]) * up[i], silu(z) = z / (1 + e^-z), fp32
 * ("decode-ops", "Usage": silu_mul).  gate_len (562), up_len (563) equal n. */
DS_API int ds_silu_mul(const float *gate, int64_t gate_len, const float *up, int64_t up_len,
                       float *out, int64_t n, ds_stream_t stream);

/* ---------------------------------------------------------------------
 * Attention
 * ------------------------------------------------------------------- */

/* Workspace bytes for ds_gqa_decode_attn. */
DS_API size_t ds_attention_workspace_bytes(int n_seqs, int n_qh, int n_kvh, int head_dim,
                                           int64_t max_ctx);

/* Grouped-query attention of one new query token per sequence over its
 * cached positions ("The forward pass end to end", "The code":
 * forward_token's attention; split across the context and reduced, "Inside
 * the engine", section 1).  For sequence s and query head h, the KV head is
 * g = h / (n_qh / n_kvh); scores q_h . k_t * scale over t < seq_lens[s],
 * softmax, and out[s][h][:] = sum_t w_t v_t.
 *   q: [n_seqs][n_qh][head_dim] fp32.  out: same shape fp32.
 *   k_cache / v_cache: rows of n_kvh*head_dim elements of kv_dtype,
 *   `cache_rows` rows each; position t of sequence s is row
 *   blk * block_tokens + t % block_tokens with blk = block_table[s *
 *   max_blocks_per_seq + t / block_tokens], or, with block_table NULL,
 *   blk = s * max_blocks_per_seq + t / block_tokens (a contiguous slot per
 *   sequence, "Inside the engine", section 3).
 *   seq_lens: device int32 [n_seqs]; a length outside
 *   [1, max_blocks_per_seq*block_tokens] is clamped and flags DS_ERR_POSITION.
 *   n_qh must be a multiple of n_kvh; head_dim a multiple of 4 up to 128, or of 8 up to 256.
 *   workspace: ds_attention_workspace_bytes(...) with max_ctx >= every length. */
DS_API int ds_gqa_decode_attn(const float *q, const void *k_cache, const void *v_cache,
                              int kv_dtype, int64_t cache_rows, const int32_t *block_table,
                              int max_blocks_per_seq, int block_tokens, const int32_t *seq_lens,
                              int n_seqs, int n_qh, int n_kvh, int head_dim, float scale,
                              float *out, void *workspace, size_t workspace_bytes,
                              ds_stream_t stream);

/* ---------------------------------------------------------------------
 * A ragged step: chunks and single tokens of many requests in one launch
 *
 * "Inside the engine", section 2: a step runs prompt chunks and decode rows
 * side by side.  Sequence s of the step has n_s new positions (a chunk, one
 * token, or none) behind c_s cached ones; the new rows of all sequences lie
 * one after the other.  ds_paged_plan maps them to the pool, ds_rope_append
 * turns a layer's fused q|k|v rows and writes k and v, ds_gqa_chunk_attn
 * attends.  Calls whose GPU work may overlap (other streams, other graphs)
 * need a workspace each.
 * ------------------------------------------------------------------- */

DS_API size_t ds_paged_plan_workspace_bytes(void);

/* Block table entries, row starts, positions and cache slots of a step, from
 * lengths in device memory ("Inside the engine", section 3: the pool's blocks
 * and a request's block table).  Per sequence s, in order:
 *   blocks: ceil((c_s + n_s) / block_tokens) - ceil(c_s / block_tokens) are
 *     taken from the front of what is left of free_blocks and entered in
 *     block_table from entry ceil(c_s / block_tokens) on; other entries stay;
 *   row_starts[s] = sum of n_i over i < s; seq_lens[s] = c_s + n_s;
 *   row r of s: row_seq[r] = s, positions[r] = c_s + r - row_starts[s] and
 *     slots[r] = block * block_tokens + position % block_tokens, its cache row.
 *   cached_lens, new_lens: int32 [n_seqs]; free_blocks: int32 [n_free] (may be
 *   NULL when n_free is 0); block_table: int32 [n_seqs][max_blocks_per_seq],
 *   updated in place; row_starts: int32 [n_seqs + 1]; seq_lens: int32
 *   [n_seqs]; row_seq, positions, slots: int32 [max_rows], all -1 behind the
 *   last row, so a batch padded to max_rows can be captured in a graph;
 *   n_taken: int32 [1], how many of free_blocks are used up.  No output may
 *   overlap an input or another output (577): cached_lens for the next step
 *   is this one's seq_lens, in two buffers that take turns.
 * The lengths are not changed: the same call again gives the same answer.
 * A sequence with a negative length or one past its table row gets no rows
 * (DS_ERR_POSITION).  The first sequence whose rows pass max_rows or whose
 * blocks pass n_free ends the step: it and all behind it get no rows and no
 * blocks (DS_ERR_NO_BLOCKS).  A sequence without rows has seq_lens[s] = c_s (a
 * negative c_s gives 0, one past the table row the row's reach).
 * A block number outside the cache's cache_rows / block_tokens whole blocks
 * gives slot -1 (a new one also table entry -1) and DS_ERR_POSITION.
 * 561 for a count < 1 (n_free may be 0), 564 past DS_MAX_DIM or 4096
 * sequences.  One launch, no host copy, capturable. */
DS_API int ds_paged_plan(const int32_t *cached_lens, const int32_t *new_lens, int n_seqs,
                         const int32_t *free_blocks, int64_t n_free, int block_tokens, int64_t cache_rows,
                         int32_t *block_table, int max_blocks_per_seq, int32_t *row_starts,
                         int32_t *seq_lens, int32_t *row_seq, int32_t *positions, int32_t *slots,
                         int64_t max_rows, int32_t *n_taken, void *workspace, size_t workspace_bytes,
                         ds_stream_t stream);

DS_API size_t ds_rope_append_workspace_bytes(void);

/* Rotary positions and K/V write of a step's rows ("Inside the engine",
 * section 1: qkPrep).  Row r of qkv holds n_qh query heads, n_kvh key heads
 * and n_kvh value heads of head_dim elements, the fused projection's output,
 * rows row_stride elements apart.  The first rot_dim dims of every q and k
 * head are rotated: pair p turns by
 *   positions[axis(p)][r] * base^(-2p / rot_dim),  axis(p) = pair_axis[p],
 * pairs laid out over the rot_dim dims as in ds_rope (DS_ROPE_*); dims behind
 * them stay.  With one axis this is the rotation of ds_rope; with several
 * (time, height, width of an image's or a video's patches) each pair turns by
 * the axis it is given, in runs or interleaved, as pair_axis says.  The angle
 * is exact to 2^-33 of a turn at any position for bases from 1e-8 up (below,
 * frequencies of billions of turns a position lose digits); the rotation is
 * fp32, rounded once to the output's type.
 *   q_out: [n_rows][n_qh][head_dim]; the rotated k and v as it is go to row
 *   slots[r] of k_cache / v_cache (rows of n_kvh * head_dim elements).
 *   qkv, q_out and the caches are fp32 or bf16 each (572).
 *   positions: device int32 [n_axes][n_rows]; pair_axis: HOST bytes
 *   [rot_dim / 2], each < n_axes (NULL for one axis), read before the call
 *   returns; slots: device int32 [n_rows].
 * A row with a negative slot is padding: it may hold anything and nothing is
 * written for it (its q_out stays).  A slot past the cache or a negative position skips the
 * row and flags DS_ERR_POSITION.  Two rows with one slot: each element of the
 * cache row is one's or the other's.
 * qkv_len (562) must reach the last row's end and row_stride its width; q_len
 * must be n_rows * n_qh * head_dim (563).  head_dim <= 256, rot_dim even and
 * <= head_dim, n_axes <= 8, base finite and > 0 (577).  No output may overlap
 * qkv or another output (577).  Rows with 16-byte aligned buffers, row_stride and
 * head_dim multiples of 8 and rot_dim of 16 move 16 bytes at a time (whole
 * rows by bulk copies from 2,048 rows on, rows of padding included); others one
 * element. */
DS_API int ds_rope_append(const void *qkv, int64_t qkv_len, int qkv_dtype, int64_t row_stride,
                          int64_t n_rows, const int32_t *positions, int n_axes, const uint8_t *pair_axis,
                          int n_qh, int n_kvh, int head_dim, int rot_dim, double base, int layout,
                          void *q_out, int64_t q_len, int q_dtype, void *k_cache, void *v_cache,
                          int kv_dtype, int64_t cache_rows, const int32_t *slots, void *workspace,
                          size_t workspace_bytes, ds_stream_t stream);

/* Workspace bytes of ds_gqa_chunk_attn for up to n_rows rows; 0 for an
 * unsupported shape. */
DS_API size_t ds_chunk_attention_workspace_bytes(int n_seqs, int64_t n_rows, int n_qh, int n_kvh,
                                                 int head_dim);

/* Grouped-query attention of every sequence's new rows over its cached
 * positions, its new ones included ("Inside the engine", section 1: causal
 * flash attention over a chunk).  Sequence s holds rows row_starts[s] ..
 * row_starts[s + 1] - 1; with n of them and L = seq_lens[s], row j attends
 * positions 0 .. L - n + j: out = softmax over t of (q . k_t * scale), times
 * v_t, KV head g = h / (n_qh / n_kvh) as in ds_gqa_decode_attn.  One row per
 * sequence is a decode step, any mix of lengths runs in one launch.
 *   q, out: [n_rows][n_qh][head_dim], both fp32 or both bf16 (q_dtype), not
 *   overlapping; k_cache, v_cache, cache_rows, block_table (NULL: contiguous
 *   slots), max_blocks_per_seq, block_tokens as in ds_gqa_decode_attn, fp32
 *   or bf16 (kv_dtype).  row_starts: device int32 [n_seqs + 1], seq_lens:
 *   device int32 [n_seqs].
 * A row that attends nothing (L < n) is zero.  Rows of no sequence (in front
 * of row_starts[0], behind row_starts[n_seqs]) stay as they were.  What the
 * cache holds at positions a row does not attend, NaN and infinities
 * included, does not reach it; what it does attend counts as in the formula
 * (but an infinite value may show although its weight is zero).
 * Row starts that fall or pass n_rows and lengths outside the table row are
 * clamped (an element of a row that two sequences then claim is one's or the
 * other's), a block number outside the cache reads block 0; all flag
 * DS_ERR_POSITION.
 * A bf16 cache with head_dim 64 or 128 and block_tokens a multiple of 8 runs
 * on the tensor cores.  There bf16 q has each weight of the softmax rounded to
 * bf16 before it meets v (2^-8 of the weight at most; sums stay fp32 and take
 * it unrounded): on normal inputs outputs are 2.0e-3 to 2.3e-3 from 64 bits in
 * the mean, of which their own rounding makes 1.5e-3 to 1.7e-3.  fp32 q keeps the digits of fp32
 * products.  fp32 caches, other heads and other pages run on the plain cores,
 * in fp32 throughout and slower the longer the chunks (2,048 bf16 rows of 32
 * heads: 62 us, with heads of 80 or pages of 7 positions 1,012); their tile
 * follows n_rows / n_seqs, rows of padding included.
 * q_len = out_len = n_rows * n_qh * head_dim (562, 563); n_qh a multiple of
 * n_kvh, head_dim a multiple of 4 up to 256, scale finite and > 0, q, out and
 * the caches 16-byte aligned (577); contiguous slots and one block at least
 * must fit the cache (571).  No allocation, no host copy, capturable. */
DS_API int ds_gqa_chunk_attn(const void *q, int64_t q_len, int q_dtype, int64_t n_rows,
                             const int32_t *row_starts, const int32_t *seq_lens, int n_seqs,
                             const void *k_cache, const void *v_cache, int kv_dtype, int64_t cache_rows,
                             const int32_t *block_table, int max_blocks_per_seq, int block_tokens,
                             int n_qh, int n_kvh, int head_dim, float scale, void *out, int64_t out_len,
                             void *workspace, size_t workspace_bytes, ds_stream_t stream);

/* ---------------------------------------------------------------------
 * Picking the next token
 * ------------------------------------------------------------------- */

DS_API size_t ds_argmax_workspace_bytes(int n_rows, int64_t n);

/* ids[r] = first index of the maximum of row r of logits [n_rows][n]
 * ("LLM inference kernels", "KV-cache growth and greedy argmax": ties go to
 * the first id; "decode-ops", "Correctness": exact against torch.argmax, NaN
 * ranking above every number).  max_logit (optional) gets the row maxima.
 * logits_len must be n_rows*n (568). */
DS_API int ds_greedy_argmax(const float *logits, int64_t logits_len, int n_rows, int64_t n,
                            int32_t *ids, float *max_logit, void *workspace,
                            size_t workspace_bytes, ds_stream_t stream);

DS_API size_t ds_sample_workspace_bytes(int n_rows, int64_t n);

/* Per row r of logits [n_rows][n], with the explicit uniform draw u[r] in
 * [0,1): temperature -> top-k -> softmax over the survivors -> top-p ->
 * renormalise -> inverse CDF at u ("decode-ops", "API — Method", the
 * HuggingFace warper order).  In this order: l' = l / T (fp32); survivors =
 * the top_k largest l', ties to the lower index, in descending order;
 * e_i = exp(l'_i - l'_max) (fp32); p_i = e_i / (sum of e over the
 * survivors); keep the prefix whose exclusive running sum of p is < top_p (at
 * least one; top_p >= 1 keeps all); token = first kept survivor whose
 * inclusive running sum exceeds u * (sum of kept p), else the last kept.
 * The running sums are exact sums of the e_i, each rounded to a multiple of
 * 2^-F of the largest (F = min(46, 63 - ceil(log2 n)): 2^-46 at a 128,256
 * vocabulary), so the token does not depend on summation order.
 *   temperature <= 0: greedy (first index of the maximum).
 *   top_k: any value; <= 0 or >= n means no top-k cut.
 *   top_p in (0, 1].  575 for a parameter outside its domain.
 *   u: device fp32 [n_rows]; ids: device int32 [n_rows].
 * A row whose largest scaled logit is NaN or infinite gets the first index of
 * that value and sets DS_ERR_SAMPLING in the workspace's error word.
 * Each row runs as one cluster of up to 8 thread blocks; no allocation, no
 * workspace beyond the error word. */
DS_API int ds_sample(const float *logits, int64_t logits_len, int n_rows, int64_t n,
                     float temperature, int top_k, float top_p, const float *u, int32_t *ids,
                     void *workspace, size_t workspace_bytes, ds_stream_t stream);

/* ---------------------------------------------------------------------
 * The decode step
 * ------------------------------------------------------------------- */

/* Model shape ("The forward pass end to end", "The code": Config, with the
 * head dimension explicit). */
typedef struct {
    int32_t vocab, d, n_layer, n_qh, n_kvh, head_dim, ff;
    int32_t rope_layout; /* DS_ROPE_* */
    double rope_base;
    float eps;           /* RMSNorm epsilon */
    int32_t tied;        /* 1: the output head is the embedding table */
    int32_t w_dtype;     /* DS_F32 or DS_BF16, for emb, out and projections */
    int32_t kv_dtype;    /* DS_F32 or DS_BF16 */
    int32_t max_seqs;    /* largest n_seqs a step will be given, 1..256.  Above 1 every step
                          * runs the batched path: the projections as GEMMs over the batch on
                          * the tcgen05 tensor cores ("Inside the engine", section 4: batched
                          * decode), which needs bf16 weights (else 572) and a head_dim that
                          * divides 128 (else 577). */
    int32_t max_ctx;     /* largest position + 1 a step will see */
    /* Long-context RoPE scaling as Llama 3.1 checkpoints define it (not on the
     * pages): pair p's frequency f = rope_base^(-2p/head_dim), wavelength
     * w = 2 pi / f, becomes f where w < rope_orig_max_pos / rope_high_freq_factor,
     * f / rope_factor where w > rope_orig_max_pos / rope_low_freq_factor, and
     * (1 - s) f / rope_factor + s f in between, with
     * s = (rope_orig_max_pos / w - rope_low_freq_factor) /
     *     (rope_high_freq_factor - rope_low_freq_factor).
     * rope_factor 0 (a zeroed struct): no scaling.  Otherwise rope_factor >= 1,
     * 0 < rope_low_freq_factor < rope_high_freq_factor and rope_orig_max_pos > 0
     * (else 577).  Applies to every position of the model's RoPE table. */
    double rope_factor;
    double rope_low_freq_factor, rope_high_freq_factor;
    double rope_orig_max_pos;
} ds_model_config;

/* Device pointers to the weights, in this storage layout:
 *   emb [vocab][d]; out [vocab][d] (ignored when tied); final_norm [d] fp32;
 *   per layer (host arrays of n_layer device pointers):
 *   n1, n2 [d] fp32;  wqkv [d][(n_qh + 2 n_kvh) head_dim] with the q columns,
 *   then k, then v;  wo [n_qh head_dim][d];  wgu [d][2 ff] with the gate
 *   columns, then up;  wd [ff][d].  Projections are [in][out] row-major and
 *   applied as y = W^T x.  The library keeps the pointers, not copies: the
 *   weights must outlive the model. */
typedef struct {
    const void *emb;
    const void *out;
    const float *final_norm;
    const float *const *n1;
    const void *const *wqkv;
    const void *const *wo;
    const float *const *n2;
    const void *const *wgu;
    const void *const *wd;
    /* Optional QK-norm, as Qwen3 checkpoints define it (not on the pages):
     * host arrays of n_layer device pointers to fp32 [head_dim] weights, or
     * both NULL (no QK-norm; a zeroed struct has none).  Every q head is
     * scaled by 1 / sqrt(mean of its head_dim squares + eps) and by q_norm,
     * every k head likewise with k_norm, after the projection and before
     * RoPE; v is untouched.  One set without the other: 577. */
    const float *const *q_norm;
    const float *const *k_norm;
} ds_model_weights;

/* The KV cache: per layer one K and one V buffer of rows of n_kvh*head_dim
 * elements (kv_dtype), addressed as in ds_gqa_decode_attn ("Inside the
 * engine", section 3: KvPool holds one K and one V buffer per layer). */
typedef struct {
    void *const *k;             /* host array of n_layer device pointers */
    void *const *v;             /* host array of n_layer device pointers */
    int64_t rows;               /* rows each per-layer buffer holds */
    int32_t block_tokens;       /* positions per block */
    int32_t max_blocks;         /* blocks per sequence */
    const int32_t *block_table; /* device int32 [max_seqs][max_blocks], or NULL */
} ds_kv_cache;

/* Sampling parameters for a whole step (see ds_sample); NULL means greedy. */
typedef struct {
    float temperature;
    int32_t top_k;
    float top_p;
} ds_sampling;

typedef struct ds_model ds_model;

/* Bytes of the model workspace (activations, split reductions, RoPE table,
 * error word) for a configuration. */
DS_API size_t ds_model_workspace_bytes(const ds_model_config *cfg);

/* Validate the configuration and weights, carve the caller's workspace
 * (zeroed here) and build the RoPE table (angles in fp64 on the device).
 * Synchronises the device.  The model object lives in host memory. */
DS_API int ds_model_create(const ds_model_config *cfg, const ds_model_weights *weights,
                           void *workspace, size_t workspace_bytes, ds_model **out);
DS_API void ds_model_destroy(ds_model *model);

/* Workspace pointer of a model (its error word is at byte 0). */
DS_API void *ds_model_workspace(ds_model *model);

/* Flags of ds_decode_step. */
#define DS_STEP_ADVANCE 1u     /* after picking: tokens[s] = next_ids[s], pos[s] += 1 (on device) */
#define DS_STEP_PHASE_TIMES 2u /* record a device timestamp at every phase boundary of the step */
#define DS_STEP_TRACE 4u       /* also record per-CTA timestamps inside every phase (see ds_model_trace) */

/* One decode step for n_seqs sequences: for each sequence s, token
 * tokens[s] at position pos[s] ("The forward pass end to end", "What a
 * forward step does"; "LLM inference kernels", "How this composes into a
 * decode step").  A model with max_seqs 1 runs the step as one persistent
 * kernel; a model with max_seqs > 1 runs the batched path (one launch per
 * operation, projections on the tensor cores, each fp32 activation handed to
 * them as a bf16 pair hi + lo, 16 significant bits), every sequence at its own
 * position in its own blocks of the K/V cache.  The step: embed; per layer
 * RMSNorm -> fused q|k|v projection -> RoPE on
 * q and k with the K/V write at pos ("Inside the engine", section 1: qkPrep)
 * -> attention over positions 0..pos -> output projection + residual ->
 * RMSNorm -> fused gate|up projection with SiLU-gate -> down projection +
 * residual; final RMSNorm -> output head -> greedy argmax (sampling NULL) or
 * the sampler with draws u[s].
 *   tokens, pos: device int32 [n_seqs]; next_ids: device int32 [n_seqs];
 *   u: device fp32 [n_seqs] (sampling only); logits_out: optional device fp32
 *   [n_seqs][vocab].  n_seqs in [1, max_seqs].
 * Bad device-side tokens/positions are clamped/skipped and flag the model's
 * error word. */
DS_API int ds_decode_step(ds_model *model, const ds_kv_cache *kv, int32_t *tokens, int32_t *pos,
                          int n_seqs, const ds_sampling *sampling, const float *u,
                          int32_t *next_ids, float *logits_out, unsigned flags,
                          ds_stream_t stream);

/* n_steps greedy decode steps of one sequence in ONE kernel launch: step i
 * decodes tokens[0] at pos[0] + i and feeds its pick to step i + 1 on the
 * device, so the weight stream runs on from one step's output head into the
 * next step's first layer without a launch in between ("Inside the engine",
 * section 4: the decode loop's steps issued back to back on the device).
 * Each step is a whole ds_decode_step (same result, same K/V writes).
 *   ids_out: optional device int32 [n_steps], the pick of every step;
 *   next_ids: device int32 [1], the last pick.  With DS_STEP_ADVANCE,
 *   tokens[0] and pos[0] end at the last pick and pos[0] + n_steps.
 * Batch-1 models (max_seqs 1) on the persistent step kernel only (577
 * otherwise); n_steps >= 1 (561); logits are not written. */
DS_API int ds_decode_steps(ds_model *model, const ds_kv_cache *kv, int32_t *tokens, int32_t *pos, int n_steps,
                           int32_t *ids_out, int32_t *next_ids, unsigned flags, ds_stream_t stream);

/* stepSeq(sequence, tokens, offset, count): `count` prompt tokens of one
 * sequence at positions offset .. offset + count - 1, run as chunks of at
 * most max_seqs rows, each chunk one batch of rows through the batched path
 * ("Inside the engine", section 1: prefill runs a chunk of prompt tokens as a
 * batch of rows through the batched projections; decode is the one-token
 * chunk of the same step).  Row j of a chunk is the token at position
 * offset + c0 + j: its K and V are written to sequence `seq`'s blocks and it
 * attends positions 0 .. offset + c0 + j of that sequence (earlier chunks'
 * rows and its own chunk's earlier rows included), so the cache ends as
 * `count` decode steps would leave it.  Only the last token goes through the
 * final norm, the head and the greedy argmax.
 *   tokens: device int32 [count] (tokens_len must equal count, else 562);
 *   seq in [0, max_seqs) (577; with a block table, its row seq, else the
 *   contiguous slot seq); next_id: device int32 [1], the greedy pick after
 *   the last token; logits_out: optional device fp32 [vocab], that token's
 *   logits (the model's own buffer is used when NULL).
 * Models with max_seqs > 1 only (577 otherwise); count >= 1 (561);
 * offset >= 0 and offset + count within the cache and max_ctx (571).
 * Uses the model's workspace: calls on one model are serialised on a stream. */
DS_API int ds_step_seq(ds_model *model, const ds_kv_cache *kv, const int32_t *tokens, int64_t tokens_len,
                       int32_t seq, int32_t offset, int32_t count, int32_t *next_id, float *logits_out,
                       ds_stream_t stream);

/* Device timestamps (ns, globaltimer) of the last step run with
 * DS_STEP_PHASE_TIMES: [0] start, then the start of every phase in order
 * (per layer: q|k|v, attention, o, gate|up, down), then the head, then the
 * end — 5*n_layer + 3 values for a batch-1 step.  Copies at most cap values
 * to ns_out (host), the count to *n_out; synchronises `stream`. */
DS_API int ds_model_phase_times(ds_model *model, uint64_t *ns_out, int cap, int *n_out,
                                ds_stream_t stream);

/* Per-CTA timestamps (ns) of the last step run with DS_STEP_TRACE, laid out
 * [phase][cta][5]: phase start, prologue done, last weight stage consumed,
 * epilogue done, and the producer warp's last weight request of the phase
 * (zero where a point does not apply).  Phases as in ds_model_phase_times.
 * Copies at most cap_words values; *n_ctas gets the CTA count. */
DS_API int ds_model_trace(ds_model *model, uint64_t *out, size_t cap_words, size_t *n_words,
                          int *n_ctas, ds_stream_t stream);

/* A decode step captured once as a CUDA graph and replayed ("Inside the
 * engine", section 4: the launch sequence of a step replayed as a captured
 * graph).  Arguments as ds_decode_step; the pointed-to device buffers are
 * read at every launch, so with DS_STEP_ADVANCE each launch decodes the next
 * token.  Capture uses `stream`, which must not be capturing already. */
typedef struct ds_step_graph ds_step_graph;
DS_API int ds_step_graph_create(ds_model *model, const ds_kv_cache *kv, int32_t *tokens,
                                int32_t *pos, int n_seqs, const ds_sampling *sampling,
                                const float *u, int32_t *next_ids, float *logits_out,
                                unsigned flags, ds_stream_t stream, ds_step_graph **out);
DS_API int ds_step_graph_launch(ds_step_graph *graph, ds_stream_t stream);
DS_API void ds_step_graph_destroy(ds_step_graph *graph);

/* Per-kernel timing of one decode step: the step's kernels are launched one
 * at a time on `stream` with CUDA events around each, `reps` times, and the
 * mean duration of each launch slot is written to ms_out[i] with its kernel
 * kind in kinds_out[i] (DS_KIND_*).  *n_out gets the number of slots (at most
 * cap).  Runs the step `reps` times: with DS_STEP_ADVANCE the state advances. */
enum {
    DS_KIND_EMBED = 0,
    DS_KIND_QKV = 1,
    DS_KIND_ATTENTION = 2,
    DS_KIND_O_PROJ = 3,
    DS_KIND_GATE_UP = 4,
    DS_KIND_DOWN = 5,
    DS_KIND_HEAD = 6,
    DS_KIND_SAMPLE = 7,
    DS_KIND_COUNT = 8
};
/* Mean duration, in microseconds, of one launch of the step's kernels of one
 * kind (DS_KIND_*, not DS_KIND_SAMPLE), measured with CUDA events around
 * `reps` passes over all of that kind's launches of a step (every layer's),
 * launched back to back on `stream` as in a step.  The kernels read and write
 * the model's buffers and the cache row at pos[0] as a step would (the
 * residual stream is left changed), but tokens and pos are not advanced.
 * Synchronises `stream`. */
DS_API int ds_decode_kernel_time(ds_model *model, const ds_kv_cache *kv, int32_t *tokens,
                                 int32_t *pos, int kind, int reps, float *us_per_launch,
                                 ds_stream_t stream);

DS_API int ds_decode_step_profile(ds_model *model, const ds_kv_cache *kv, int32_t *tokens,
                                  int32_t *pos, int n_seqs, const ds_sampling *sampling,
                                  const float *u, int32_t *next_ids, float *logits_out,
                                  unsigned flags, int reps, float *ms_out, int32_t *kinds_out,
                                  int cap, int *n_out, ds_stream_t stream);

/* ---------------------------------------------------------------------
 * Continuous-batching scheduler slice over the paged K/V pool (host only)
 * ("Inside the engine", section 2: admission, chunks, preemption, resume).
 * It decides, step by step, which requests run, as prompt chunks or decode
 * rows, and which pool blocks each one's block-table row maps; the caller
 * runs the rows (ds_step_seq for a chunk, ds_decode_step for decode rows)
 * and reports back.  Policy (the page's, read for a pool whose blocks hold
 * every layer's K/V of block_tokens positions):
 *   - a request's tokens are its prompt plus what it has generated; its
 *     cached prefix is the positions whose K/V sit in its blocks;
 *   - admission, strictly first come first served over the waiting list
 *     (preempted requests first, by preemption order, then new ones by
 *     submission): the head is admitted when a block-table row is free and
 *     the free blocks cover all its tokens plus headroom_blocks; those
 *     blocks are taken (lowest block numbers first); otherwise admission
 *     stops for this step;
 *   - chunks: a request with uncached tokens runs them in chunks of at most
 *     `chunk`; the chunk that reaches the last token also yields the next
 *     token; a request whose tokens are all cached but the last runs one
 *     decode row (the last token), which yields the next token;
 *   - preemption: a decode row whose position needs a new block takes the
 *     lowest free one; with none free, the youngest running request (last
 *     submitted) is preempted — its blocks and row freed, its cache
 *     forgotten — until one is free or the request itself was the youngest;
 *     older requests claim blocks first;
 *   - resume: a preempted request waits ahead of new ones, first preempted
 *     first, and recomputes its whole prefix (prompt and generated tokens)
 *     through the chunked path;
 *   - completion: a request that has generated max_new tokens, or that the
 *     caller reports finished, frees its blocks and row at ds_sched_commit;
 *     the next plan admits into them.
 * ------------------------------------------------------------------- */
typedef struct {
    int32_t n_blocks;        /* blocks in the pool */
    int32_t block_tokens;    /* positions per block */
    int32_t max_blocks;      /* block-table width: blocks per request at most */
    int32_t max_running;     /* block-table rows: requests running at once (a model's max_seqs) */
    int32_t chunk;           /* prompt tokens a request runs per step at most */
    int32_t headroom_blocks; /* free blocks demanded beyond a request's tokens at admission */
} ds_sched_config;

/* One row of a planned step. */
typedef struct {
    int64_t request; /* the caller's id */
    int32_t slot;    /* block-table row (the sequence index the kernels address) */
    int32_t offset;  /* position of the row's first token */
    int32_t count;   /* tokens: a chunk of the prompt (or of a resumed prefix), or 1 */
    int32_t decode;  /* 1: the decode row of a request whose tokens are all cached but the last */
    int32_t yields;  /* 1: the row ends at the request's last token and yields its next one */
} ds_sched_row;

typedef struct ds_sched ds_sched;

/* 561 for a count < 1 (headroom_blocks may be 0), 564 beyond DS_MAX_DIM,
 * 577 for NULL.  The scheduler lives in host memory. */
DS_API int ds_sched_create(const ds_sched_config *cfg, ds_sched **out);
DS_API void ds_sched_destroy(ds_sched *sched);

/* Queue a request (ids unique among live requests, else 577): prompt_len >= 1
 * and max_new >= 1 (561); prompt_len + max_new - 1 positions must fit one
 * block-table row (571). */
DS_API int ds_sched_submit(ds_sched *sched, int64_t request, int32_t prompt_len, int32_t max_new);

/* Plan the next step: admit, grow, preempt, and list one row per running
 * request, oldest first, in rows[0 .. *n_rows) (cap >= max_running, else
 * 574).  block_table (host int32 [max_running][max_blocks]) receives every
 * row's blocks, -1 past a request's blocks and in free rows.  preempted
 * (optional, capacity max_running) receives the ids preempted by this plan,
 * *n_preempted their count.  A plan must be committed before the next one
 * (577 otherwise). */
DS_API int ds_sched_plan(ds_sched *sched, ds_sched_row *rows, int32_t cap, int32_t *n_rows,
                         int32_t *block_table, int64_t *preempted, int32_t *n_preempted);

/* The planned step ran: every row's tokens are cached, the rows that yield
 * add a generated token, and requests that reached max_new or appear in
 * finished[0 .. n_finished) free their blocks and rows.  577 without a plan
 * to commit. */
DS_API int ds_sched_commit(ds_sched *sched, const int64_t *finished, int32_t n_finished);

/* Counts: [0] free blocks, [1] running, [2] waiting, [3] finished,
 * [4] preemptions so far. */
DS_API int ds_sched_stats(const ds_sched *sched, int64_t *out5);

/* Generated tokens of a live or finished request (-1: unknown id). */
DS_API int64_t ds_sched_generated(const ds_sched *sched, int64_t request);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_STEP_H */
