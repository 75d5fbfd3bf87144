/*
 * qmm.h -- C ABI of libqmm: block-quantized weights times dense activations,
 * with the dequantization fused into the kernels, on one NVIDIA GB300 (sm_103a).
 *
 * The problem statement follows ferrox-cuda 0.21.0 src/mul_mm.rs (the `BODY_SRC`
 * GEMM body and `validate_shape`): a weight matrix of `M` rows, each row a run of
 * `K / block_elems` contiguous blocks in their on-disk (GGUF) byte layout; `N`
 * activation rows of `K` values; an fp32 output written token-major,
 * Y[n * M + m] = sum_k W[m, k] * X[n * K + k].
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers (cudaMalloc / PyTorch CUDA tensors)
 *     on the current CUDA device. The library never takes ownership; the caller
 *     keeps every buffer alive until the work queued on `stream` has finished.
 *     qdequant, qgemv, qgemm_grouped and qgemm_noalloc never allocate device
 *     memory. qgemm (and qgemm_ex) with N > 8 on the tensor-core path may grow
 *     a per-device workspace that the library owns (see qgemm); qmm_shutdown
 *     frees it.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream). Every call
 *     is asynchronous with respect to the host: it validates, queues kernels on
 *     `stream` and returns.
 *   - Errors in arguments (shape, kind, dtype, null or misaligned pointers, too
 *     small buffers) are reported synchronously as a qmm_status BEFORE anything
 *     is launched; nothing is written. A zero-sized shape is QMM_ERR_EMPTY_SHAPE
 *     and launches nothing (ferrox-cuda mul_mm.rs, `MulMmUnsupported::EmptyShape`).
 *   - A failed launch returns QMM_ERR_CUDA. Device-side conditions (a bounded
 *     wait that ran out) are latched in a device flag and reported by
 *     qmm_check_device_error().
 *   - There is no fallback to a different computation and no CPU path: a format
 *     this library does not implement is QMM_ERR_BAD_KIND (ferrox-cuda
 *     mul_mm.rs, `kind_by_name`: an unknown format is reported to the caller,
 *     who chooses another implementation).
 *   - Every output element is written exactly once per call (no accumulation
 *     into the output), so sentinel-prefilled outputs are fully overwritten.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define QMM_API __attribute__((visibility("default")))
#else
#define QMM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Block formats. Geometry (bytes per block / elements per block):
 *   Q8_0 34/32, Q4_0 18/32, Q5_0 22/32, Q4_K 144/256, Q5_K 176/256,
 *   Q6_K 210/256, Q2_K 84/256, Q3_K 110/256, IQ4_NL 18/32, IQ4_XS 136/256,
 *   MXFP4 17/32 (ferrox-cuda mul_mm.rs `KINDS` and its geometry test;
 *   ferrox-cuda 0.20.0 src/mul_mm_kinds/codebook.rs for the codebook rows;
 *   Vulkore examples/llm/quant_test.cpp `kFormats`);
 *   Q4_1 20/32, Q5_1 24/32, Q8_1 36/32: the kinds that ferrox-cuda 0.21.0
 *   mul_mm.rs lists as having no mul_mm kernel, in the public GGUF layouts --
 *   Q4_1 and Q5_1 are Q4_0 and Q5_0 with unsigned codes and an f16 min after
 *   the f16 scale (w = d*q + m); Q8_1 is Q8_0 with an f16 field after d (d
 *   times the sum of the codes) that no element reads (w = d*q). */
typedef enum {
    QMM_Q8_0 = 0,
    QMM_Q4_0 = 1,
    QMM_Q5_0 = 2,
    QMM_Q4_K = 3,
    QMM_Q5_K = 4,
    QMM_Q6_K = 5,
    QMM_Q2_K = 6,
    QMM_Q3_K = 7,
    QMM_IQ4_NL = 8,
    QMM_IQ4_XS = 9,
    QMM_MXFP4 = 10,
    QMM_Q4_1 = 11,
    QMM_Q5_1 = 12,
    QMM_Q8_1 = 13,
    QMM_NKINDS = 14
} qmm_kind;

/* Activation element type. f32 activations must be 4-byte aligned, f16
 * (IEEE binary16) and bfloat16 activations 2-byte aligned. The products take
 * QMM_F32 and QMM_F16; the rotary, cache and attention operators take all
 * three. */
typedef enum { QMM_F32 = 0, QMM_F16 = 1, QMM_BF16 = 2 } qmm_dtype;

/* Status codes. The shape refusals mirror ferrox-cuda mul_mm.rs
 * `MulMmUnsupported`. */
typedef enum {
    QMM_OK = 0,
    QMM_ERR_EMPTY_SHAPE = 1,             /* M, K, N or n_assign is 0 */
    QMM_ERR_BAD_KIND = 2,                /* kind outside qmm_kind */
    QMM_ERR_BAD_DTYPE = 3,               /* x_dtype outside qmm_dtype */
    QMM_ERR_COLS_NOT_BLOCK_ALIGNED = 4,  /* K not a multiple of block_elems */
    QMM_ERR_WEIGHTS_TOO_SMALL = 5,       /* w_bytes < M * row_bytes (or experts) */
    QMM_ERR_ACTIVATIONS_TOO_SMALL = 6,   /* x_elems < rows needed * K */
    QMM_ERR_NULL_POINTER = 7,
    QMM_ERR_MISALIGNED = 8,              /* activation/output pointer alignment */
    QMM_ERR_BAD_EXPERT_ID = 9,           /* bad n_experts / expert stride */
    QMM_ERR_CUDA = 10,                   /* a CUDA runtime call failed */
    QMM_ERR_DEVICE_TIMEOUT = 11,         /* a device-side bounded wait ran out */
    QMM_ERR_UNIMPLEMENTED = 12,
    QMM_ERR_BAD_ARGUMENT = 13,           /* negative size or other bad scalar */
    QMM_ERR_OUTPUT_TOO_SMALL = 14,       /* y_elems < outputs to write */
    QMM_ERR_WORKSPACE_IN_CAPTURE = 15,   /* workspace would grow during stream capture */
    QMM_ERR_NOALLOC_LIMIT = 16,          /* qgemm_noalloc: scratch needed exceeds its fixed array */
    QMM_ERR_WORKSPACE_TOO_SMALL = 17,    /* caller-provided workspace smaller than required */
    QMM_ERR_CACHE_TOO_SMALL = 18,        /* key-value cache smaller than its pages */
    QMM_ERR_BAD_SLOT = 19                /* cache slot, page id or sequence length out of range */
} qmm_status;

/* Geometry of `kind`: bytes and elements of one block. Returns QMM_OK or
 * QMM_ERR_BAD_KIND / QMM_ERR_NULL_POINTER. Host only, no CUDA call. */
QMM_API int qmm_kind_info(int kind, size_t* block_bytes, size_t* block_elems);

/* Bytes of one weight row of K elements: (K / block_elems) * block_bytes.
 * 0 when kind is bad or K is not a positive multiple of block_elems. */
QMM_API size_t qmm_row_bytes(int kind, int64_t K);

/* Static, NUL-terminated description of a status code (never NULL). */
QMM_API const char* qmm_status_str(int status);

/* GGUF name of a kind ("Q4_0", ...), or NULL for a bad kind. */
QMM_API const char* qmm_kind_name(int kind);

/*
 * qdequant -- expand `rows` x `cols` quantized weights to fp32.
 *
 *   out[r * cols + k] = value of element k of weight row r
 *
 * Element values follow each format's definition (Vulkore quant_test.cpp, the
 * `ref::` CPU references; ferrox-cuda codebook.rs for IQ4_NL / IQ4_XS / MXFP4).
 * Bit-exact: every product in every format is exact in fp32; the affine-min
 * formats (Q4_K, Q5_K, Q2_K) round once, at the final subtraction. No flush of
 * subnormals (MXFP4 with small E8M0 scales yields fp32 subnormals).
 *
 *   blocks       device, rows * qmm_row_bytes(kind, cols) bytes, any alignment
 *   blocks_bytes size of `blocks` in bytes (checked)
 *   out          device fp32, rows * cols elements, 4-byte aligned
 *   out_elems    size of `out` in elements (checked)
 */
QMM_API int qdequant(int kind, const void* blocks, size_t blocks_bytes, int64_t rows, int64_t cols,
             float* out, size_t out_elems, void* stream);

/*
 * qgemv -- decode GEMV, y[m] = sum_k W[m, k] * x[k] (one activation row).
 * Exactly qgemm with N = 1 (inferencelayer 0.2.8 src/cublas_prefill.rs,
 * `Q4_GEMV_KERNEL`: the decode-time GEMV, bound by reading the weights).
 *
 *   W        device, M * row_bytes bytes, any alignment (16-byte aligned W with
 *            16-byte-multiple rows takes the streaming fast path)
 *   w_bytes  size of W in bytes (checked)
 *   x        device, K activations of x_dtype
 *   x_elems  size of x in elements (checked)
 *   y        device fp32, M elements, 4-byte aligned; y_elems its size
 */
QMM_API int qgemv(int kind, const void* W, size_t w_bytes, const void* x, int x_dtype, size_t x_elems,
          float* y, size_t y_elems, int64_t M, int64_t K, void* stream);

/*
 * qgemm -- Y[n * M + m] = sum_k W[m, k] * X[n * K + k] for n < N, m < M
 * (ferrox-cuda mul_mm.rs `BODY_SRC`: src0 = W, src1 = X, dst token-major).
 * Small N runs the weight-streaming GEMV kernels; large N the tcgen05
 * tensor-core GEMM. fp32 activations reach the tensor cores as two f16 rows
 * per token: a pre-pass scales each token row by the power of two that puts
 * its largest magnitude in [2^9, 2^10) and splits it into hi = f16(x) and
 * lo = f16(x - hi) (together exact to about 2^-22 relative); the epilogue adds
 * the two products and removes the scale. This doubles the tensor-core work of
 * the call against f16 activations. With f16 activations, Q4_K, Q5_K, Q2_K,
 * Q4_1 and Q5_1 carry the sums of each 32 (Q2_K: 16) consecutive activations
 * in f16: their magnitudes must stay below 65504.
 *
 *   W, w_bytes   as qgemv
 *   X            device, N * K activations of x_dtype, row-major; x_elems its size
 *   Y            device fp32, N * M elements; y_elems its size
 *
 * Accuracy: |Y - Y_exact| <= 1e-3 * sum_k |W[m,k] * X[n,k]| + 1e-6 per element.
 * One condition on the tensor-core path: MXFP4 folds each block's exponent
 * into its f16 operands relative to the largest exponent of its 256-element
 * group. This is exact while the eight exponents of a group span at most 23.
 * At 24 the codes +-0.5 and +-1.5 of the smallest block round to even; a block
 * 25 or more below the largest contributes nothing. The bound then holds while
 * the group's largest-exponent block carries a nonzero code against
 * activations of comparable magnitude (quantizers derive a block's exponent
 * from its largest value). The GEMV (N <= 8) and qdequant have no such limit.
 *
 * Workspace: the tensor-core path keeps its scratch in a per-device workspace
 * the library owns and grows on demand (cudaMalloc): the f16 (hi, lo) rows of
 * fp32 activations and their scales (4 * N * K + 4 * N bytes), for Q4_K,
 * Q5_K, Q2_K, Q4_1 and Q5_1 the per-group activation sums (N * K/16 f16
 * values at most, twice that for fp32 activations), and, when the
 * 128 x 128 output tiles do not fill the GPU evenly, the partial tiles of
 * the tiles whose K range several CTAs share (2 * 64 KiB per SM). Those
 * partial sums are added in a fixed order by a second kernel, so results are
 * deterministic. Growth is refused during stream capture
 * (QMM_ERR_WORKSPACE_IN_CAPTURE): make one call of the largest shape before
 * capturing. Concurrent calls on different streams of one device share that
 * workspace and must not overlap.
 */
QMM_API int qgemm(int kind, const void* W, size_t w_bytes, const void* X, int x_dtype, size_t x_elems,
          float* Y, size_t y_elems, int64_t M, int64_t K, int64_t N, void* stream);

/* Per-call flags of qgemm_ex. */
enum {
    /* W is not written by any work still in flight on `stream` (the normal
     * case for model weights). The weight-streaming GEMV (N <= 8) may then
     * start reading W while the preceding kernel on the stream is still
     * running (programmatic dependent launch); activations are read, and
     * outputs written, only after that kernel has completed, with or without
     * the flag. Other paths ignore it. */
    QMM_FLAG_WEIGHTS_CONST = 1,
    /* Y holds IEEE binary16 (QMM_FLAG_Y_F16) or bfloat16 (QMM_FLAG_Y_BF16)
     * values instead of fp32: each output is the fp32 result rounded to
     * nearest even once, at the store. Y must then be 2-byte aligned and
     * y_elems counts 16-bit elements. At most one of the two. */
    QMM_FLAG_Y_F16 = 2,
    QMM_FLAG_Y_BF16 = 4
};

/*
 * qgemm_ex -- qgemm with per-call flags (a bitwise OR of QMM_FLAG_* values;
 * unknown bits are QMM_ERR_BAD_ARGUMENT). qgemm and qgemv are qgemm_ex with
 * flags 0.
 */
QMM_API int qgemm_ex(int kind, const void* W, size_t w_bytes, const void* X, int x_dtype, size_t x_elems,
                     float* Y, size_t y_elems, int64_t M, int64_t K, int64_t N, uint32_t flags,
                     void* stream);

/*
 * qgemm_noalloc -- qgemm on the tensor-core path that never allocates device
 * memory. The pages have no counterpart to it. It is for callers that cannot
 * let a library call cudaMalloc: serving runtimes that reserve all of the
 * GPU's memory at start-up and hand out only their own pools (a cudaMalloc
 * from a library then fails or steals from the pool), and callers on a hot
 * path where an allocation's implicit device synchronisation is not allowed.
 *
 * It computes what qgemm computes, with the same arguments, layouts and
 * accuracy (one CTA per output tile, never shared K ranges, so the rounding
 * of the sums can differ from qgemm's), but only on the tensor-core path:
 * f16 activations, K a multiple of 256, 16-byte aligned W and X, rows a
 * multiple of 16 bytes (QMM_ERR_UNIMPLEMENTED otherwise). The per-group
 * activation sums that Q4_K, Q5_K, Q2_K, Q4_1 and Q5_1 need go to a fixed
 * 4 MiB device array compiled into the library (held on every GPU that loads
 * it, until the process exits) instead of a grown workspace; a problem whose
 * sums need more, N * (K / 256) * 32 bytes for Q4_K / Q5_K / Q4_1 / Q5_1 or
 * N * (K / 256) * 64 bytes for Q2_K above 4 MiB, returns QMM_ERR_NOALLOC_LIMIT
 * before anything is launched. Each call rewrites all the scratch it reads,
 * so nothing is left to clear between calls. The array is shared by every call: calls that can
 * overlap on the GPU (different streams, same device) race on it and must
 * be ordered by the caller. The first call on a device looks the array's
 * address up with cudaGetSymbolAddress (no allocation), once per device.
 */
QMM_API int qgemm_noalloc(int kind, const void* W, size_t w_bytes, const void* X, int x_dtype,
                          size_t x_elems, float* Y, size_t y_elems, int64_t M, int64_t K, int64_t N,
                          void* stream);

/*
 * qgemm_grouped -- expert-indexed product (a mixture-of-experts layer's
 * routed matmul). For each assignment r < n_assign:
 *
 *   Y[r * M + m] = sum_k W_e[m, k] * X[x_row[r] * K + k],  e = expert_id[r]
 *
 * where W_e = W + e * expert_stride bytes holds expert e's M x K weights. Each
 * assignment writes its own output row (no top-k combine).
 *
 * On the weight-streaming kernel, the assignments are bucketed by expert on
 * the device. Every touched expert's rows are then read from memory once per
 * block of up to four of its assignments. That kernel needs 16-byte aligned W,
 * expert_stride and row bytes multiples of 16, n_experts <= 1024 and
 * n_assign <= 4096. Other shapes run on the generic kernel, one pass per
 * assignment. Accuracy is as for qgemm.
 *
 *   W               device, n_experts experts of M rows each; w_bytes its size
 *   expert_stride   bytes between experts (>= M * row_bytes)
 *   X               device activations, n_x_rows rows of K; x_elems its size
 *   x_row, expert_id device int32 arrays of n_assign entries. Values are read
 *                   on the device: an out-of-range expert id or x row makes
 *                   that assignment's output row NaN and latches
 *                   QMM_ERR_BAD_EXPERT_ID for qmm_check_device_error().
 *   Y               device fp32, n_assign * M elements; y_elems its size
 */
QMM_API int qgemm_grouped(int kind, const void* W, size_t w_bytes, size_t expert_stride, int n_experts,
                  const void* X, int x_dtype, size_t x_elems, int64_t n_x_rows,
                  const int32_t* x_row, const int32_t* expert_id, int64_t n_assign,
                  float* Y, size_t y_elems, int64_t M, int64_t K, void* stream);

/*
 * qrepack -- load-time repack of Q8_0 / Q4_0 weights into the layout
 * qgemm_repacked reads (the Vulkore examples/llm/quant_test.cpp page's
 * repacked fast path: scales split from codes, everything aligned, checked to
 * reconstruct every element bit-exactly). Rows stay contiguous and keep their
 * byte count; each 256-element unit of a row holds the code fields of its
 * eight blocks back to back (16 bytes per Q4_0 block, 32 per Q8_0 block, in
 * the block's own element order), then the eight f16 scales (16 bytes).
 *
 *   W, w_bytes     device, rows x cols native blocks
 *   out, out_bytes device, qrepack_bytes(kind, rows, cols) bytes (the same
 *                  size as the native tensor); any alignment for W and out,
 *                  16 bytes for qgemm_repacked
 * cols must be a multiple of 256; other kinds are QMM_ERR_UNIMPLEMENTED.
 */
QMM_API int qrepack(int kind, const void* W, size_t w_bytes, int64_t rows, int64_t cols, void* out,
                    size_t out_bytes, void* stream);

/* Bytes of the repacked tensor (0 for an unsupported kind or shape). */
QMM_API size_t qrepack_bytes(int kind, int64_t rows, int64_t cols);

/*
 * qgemm_repacked -- qgemm (N <= 8 activation rows) on a tensor repacked by
 * qrepack, with the reduction over K optionally split: split ways of K / split
 * elements each (split a divisor of K / 256; 0 = chosen so that every SM gets
 * about two items of rows; 1 = not split). Each K-slice of every row is
 * streamed by its own CTA work item and the partial products are added by a
 * second kernel in slice order (deterministic), the split-k matvec plus
 * reduce of the same page. flags as qgemm_ex.
 *
 * Scratch for split > 1 (the partial products, split * N * M fp32) lives in a
 * per-device workspace the library grows on demand; growth during stream
 * capture is refused (QMM_ERR_WORKSPACE_IN_CAPTURE), qmm_shutdown frees it.
 */
QMM_API int qgemm_repacked(int kind, const void* R, size_t r_bytes, const void* X, int x_dtype, size_t x_elems,
                           float* Y, size_t y_elems, int64_t M, int64_t K, int64_t N, int split, uint32_t flags,
                           void* stream);

/*
 * qmoe_ffn -- one mixture-of-experts feed-forward layer over block-quantized
 * experts (the decoder layer whose per-token weight traffic the inferencelayer
 * 0.2.8 src/cublas_prefill.rs page quotes for Qwen3-30B-A3B). For token t and
 * routing slot j < top_k, with e = topk_ids[t * top_k + j] and weight
 * topk_w[t * top_k + j]:
 *
 *   g, u = rows [0, d_ff) and [d_ff, 2 d_ff) of W_gu_e times x_t
 *   h    = silu(g) * u,   silu(v) = v / (1 + e^-v)          (SwiGLU)
 *   o    = W_down_e h
 *   Y[t] = sum_j topk_w[t * top_k + j] * o                 (in slot order)
 *
 * The projections run on the expert-grouped streaming GEMV (each touched
 * expert's rows stream once per block of up to four of its assignments); the
 * down projection computes silu(g) * u while it stages its activations. The
 * routing weights are applied as given (normalise them first if the model
 * does). Accuracy: within what qgemm's per-product bar implies through SwiGLU
 * and the down projection.
 *
 *   W_gu, w_gu_bytes     device, n_experts experts every gu_stride bytes, each
 *                        2 d_ff rows of d_model elements (gate rows first)
 *   W_down, w_down_bytes device, experts every down_stride bytes, each d_model
 *                        rows of d_ff elements
 *   X                    device fp32 [T][d_model], 16-byte aligned
 *   topk_ids, topk_w     device int32 / fp32 [T][top_k]; an expert id out of
 *                        range gives NaN in its token's row of Y and latches
 *                        QMM_ERR_BAD_EXPERT_ID for qmm_check_device_error()
 *   Y                    device fp32 [T][d_model]
 *   workspace            device scratch owned by the caller, 256-byte aligned,
 *                        at least qmoe_ffn_workspace_bytes(T, top_k, d_model,
 *                        d_ff) bytes; the library allocates nothing. Calls that
 *                        overlap on the GPU must not share a workspace.
 *
 * Both projections must take the streaming kernel: 16-byte aligned weights,
 * strides and rows that are multiples of 16 bytes, n_experts <= 1024 and
 * T * top_k <= 4096 (QMM_ERR_UNIMPLEMENTED otherwise).
 */
QMM_API int qmoe_ffn(int kind, const void* W_gu, size_t w_gu_bytes, size_t gu_stride, const void* W_down,
                     size_t w_down_bytes, size_t down_stride, int n_experts, const float* X, size_t x_elems,
                     int64_t T, int64_t d_model, int64_t d_ff, const int32_t* topk_ids, const float* topk_w,
                     int top_k, float* Y, size_t y_elems, void* workspace, size_t workspace_bytes, void* stream);

/* Scratch bytes qmoe_ffn needs for these sizes (0 for a non-positive size). */
QMM_API size_t qmoe_ffn_workspace_bytes(int64_t T, int top_k, int64_t d_model, int64_t d_ff);

/*
 * The operators around the attention of a decoder layer, for serving: rotary
 * positions, a paged key-value cache, and the attention of one new token a
 * sequence over it. They take f32, f16 or bf16 activations with strides (in
 * elements; the last dimension is contiguous), so that q, k and v may be views
 * of one fused projection. They never allocate device memory, copy nothing to
 * the host and can be captured in a graph.
 *
 * Key-value cache. Keys and values live in two buffers of `n_pages` pages of
 * `page_size` tokens (a power of two, 8 to 4096), pages `page_stride` bytes
 * apart (a multiple of 16, at least qkv_page_bytes; larger strides let
 * layers share one allocation). In a page, head h has a unit of page_size
 * rows of head_dim values (head_dim a multiple of 32):
 *   QMM_KV_F16 / QMM_KV_BF16  the values, [page_size][head_dim]
 *   QMM_KV_Q8_0               int8 codes [page_size][head_dim], then f16 scales
 *                             [page_size][head_dim / 32]; value = scale * code
 *                             (a scale of either sign; qkv_store writes none
 *                             below zero).
 *                             The bytes per token are those of Q8_0 blocks.
 *   QMM_KV_Q4_0               4-bit codes plus 8, [page_size][head_dim / 2] bytes
 *                             (elements 2 j in the low and 2 j + 1 in the high half
 *                             of byte j), then f16 scales [page_size][head_dim / 32];
 *                             value = scale * code, code in [-8, 7], a scale
 *                             of either sign. The bytes per token are those of
 *                             Q4_0 blocks.
 * Slot s of the cache is row s % page_size of page s / page_size.
 */
typedef enum { QMM_KV_F16 = 0, QMM_KV_BF16 = 1, QMM_KV_Q8_0 = 2, QMM_KV_Q4_0 = 4 } qmm_kv_format;   /* (3 is none) */

/* Bytes of one page of keys (or of values); 0 for a format, page size, head
 * count or head dim the cache does not take. Host only, no CUDA call. */
QMM_API size_t qkv_page_bytes(int fmt, int page_size, int n_kv_heads, int head_dim);

/* Which elements of a head make a pair. */
typedef enum { QMM_ROPE_HALF = 0, QMM_ROPE_INTERLEAVED = 1 } qmm_rope_layout;

/* Frequency scalings for contexts longer than a model was trained on. */
typedef enum {
    QMM_ROPE_PLAIN = 0,   /* f_i = base^(-2 i / rot_dim) */
    QMM_ROPE_LINEAR = 1,  /* f_i / factor (positions interpolated) */
    QMM_ROPE_BASE = 2,    /* base replaced by base * factor^(rot_dim / (rot_dim - 2)) */
    QMM_ROPE_RAMP = 3,    /* pairs that make more than `fast` turns in orig_len positions are kept, fewer than `slow`
                             divided by factor, a linear ramp over the pair index between; mscale = 0.1 ln(factor) + 1 */
    QMM_ROPE_BANDS = 4    /* the same with the blend linear in the number of turns, and mscale = 1 */
} qmm_rope_scaling;

/*
 * qrope_turns -- the frequency table of qrope, computed on the host in double.
 * Entry i is the turns per position of pair i, f_i / (2 pi), as a 64-bit
 * fraction (2^64 = one turn): position * entry modulo 2^64 is then the exact
 * phase, at any position. Callers with frequencies of their own fill the table
 * the same way. Copy it to the device once.
 *
 *   turns    host, rot_dim / 2 entries;  mscale  host, the factor on the
 *            rotated values that the scaling asks for
 *   factor   >= 1, not read by QMM_ROPE_PLAIN; orig_len, fast > slow > 0 are
 *            read by QMM_ROPE_RAMP and QMM_ROPE_BANDS (customary: 32 and 1,
 *            4 and 1)
 */
QMM_API int qrope_turns(double base, int rot_dim, int scaling, double factor, double orig_len, double fast,
                        double slow, uint64_t* turns, float* mscale);

/*
 * qrope -- rotary positions on T tokens of H heads of D values (D <= 2048). For pair
 * i < rot_dim / 2, with a = 2 pi positions[t] * turns[i] / 2^64:
 *
 *   y1 = mscale (x1 cos a - x2 sin a),   y2 = mscale (x2 cos a + x1 sin a)
 *
 * (x1, x2) are elements i and i + rot_dim / 2 of the head (QMM_ROPE_HALF) or 2i
 * and 2i + 1 (QMM_ROPE_INTERLEAVED); elements from rot_dim (even, <= D) on are
 * copied. fp32 arithmetic, one rounding at the store. The gradient of the
 * input is the same call on the output's gradient with negated positions.
 *
 *   X, Y        device, dtype, element (t, h, d) at t * ts + h * hs + d; x_elems,
 *               y_elems their sizes. Y may be X with the same strides (in place).
 *               Otherwise they share no element, nor do two rows of Y
 *               (QMM_ERR_BAD_ARGUMENT); Y between rows of X has X's token stride
 *   positions   device int32 [T], any sign;  turns  device [rot_dim / 2]
 */
QMM_API int qrope(const void* X, int dtype, size_t x_elems, int64_t x_ts, int64_t x_hs, const int32_t* positions,
                  const uint64_t* turns, int rot_dim, int layout, float mscale, void* Y, size_t y_elems, int64_t y_ts,
                  int64_t y_hs, int64_t T, int64_t H, int64_t D, void* stream);

/*
 * qkv_store -- writes the keys and values of T tokens into the cache, rotating
 * the keys first when positions and turns are given (both NULL: stored as they
 * are), in one kernel. f16 and bf16 caches round once (to nearest even; an
 * fp32 value beyond the f16 range becomes Inf). QMM_KV_Q8_0 quantises each 32
 * consecutive values: d = f16(max |x| / 127), code = x / d rounded to nearest,
 * in [-127, 127]; d = 0 gives codes 0; a block holding an Inf or NaN, or whose
 * d overflows f16, gets d = NaN, so that it reads back as NaN. QMM_KV_Q4_0 the
 * same with d = f16(m / -8) for the value m of largest magnitude (the first of
 * them) and codes in [-8, 7]. Its keys are rotated as a plain fp32 computation
 * rotates them (the angle rounded to fp32, cos and sin within 3e-7).
 *
 *   K, V     device, dtype, element (t, h, d) at t * ts + h * hs + d; sizes in
 *            elements
 *   slots    device int64 [T]: the token's slot, or -1 to skip it. Slots other
 *            than -1 must be distinct. One outside the cache writes nothing and
 *            latches QMM_ERR_BAD_SLOT for qmm_check_device_error().
 *   k_cache, v_cache  device, cache_bytes bytes each, 16-byte aligned
 */
QMM_API int qkv_store(int fmt, const void* K, size_t k_elems, int64_t k_ts, int64_t k_hs, const void* V,
                      size_t v_elems, int64_t v_ts, int64_t v_hs, int dtype, const int64_t* slots,
                      const int32_t* positions, const uint64_t* turns, int rot_dim, int layout, float mscale,
                      void* k_cache, void* v_cache, size_t cache_bytes, int64_t n_pages, int64_t page_stride,
                      int page_size, int64_t T, int n_kv_heads, int head_dim, void* stream);

/*
 * qkv_load -- reads T slots of the cache back as dense rows [T][n_kv_heads]
 * [head_dim] of dtype (rounded once). Slot -1 gives zeros; one outside the cache
 * gives NaN and latches QMM_ERR_BAD_SLOT. K and V are 16-byte aligned, kv_elems
 * the size of each.
 */
QMM_API int qkv_load(int fmt, const int64_t* slots, const void* k_cache, const void* v_cache, size_t cache_bytes,
                     int64_t n_pages, int64_t page_stride, int page_size, void* K, void* V, int dtype, size_t kv_elems,
                     int64_t T, int n_kv_heads, int head_dim, void* stream);

/*
 * qattn_decode -- attention of one new token a sequence over the paged cache.
 * For sequence b and query head h, with kv head h / (n_q_heads / n_kv_heads),
 * keys k_j and values v_j of positions j in [max(0, len_b - window), len_b):
 *
 *   s_j = scale q . k_j        (softcap c > 0: c tanh(s_j / c))
 *   out[b][h] = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse[b][h] = ln sum_j e^{s_j}
 *
 * The new token's own key is in the cache already (qkv_store first). Position
 * j is row j % page_size of page block_table[b][j / page_size]. A sequence of
 * length 0 gives zeros and lse = -inf. Whatever the cache holds outside the
 * range, NaN included, has no effect; an Inf or NaN inside it makes the heads
 * that see it Inf or NaN. Long sequences are split over the GPU and joined in a
 * fixed order: results are deterministic.
 *
 * Accuracy. Scores, the softmax's maximum and sum, and outputs are held in fp32;
 * q and the weights enter the products as sums of 16-bit terms. With fp32 q (or q
 * of another 16-bit type than the cache's; f16 for Q8_0) those carry 22 bits or
 * more and the result is as near as a plain fp32 computation's. With q of the
 * cache's type the weights carry 22 bits (16 over bf16), and sums over up to 16384
 * keys are cut off, not rounded, to 24: 2^-16 and less of the result, before the
 * output's one rounding to 16 bits (over Q4_0 f16 and bf16 q count as the cache's type).
 * Small weights count where the keys of the large ones have values near zero. f16 terms
 * (every format but bf16) then hold a key's part to 2^-36 of the largest weight times the
 * largest |v| (Q4_0: of its 32 dims); with fp32 q, or of another 16-bit type than the cache's,
 * weights of less than 2^-32 (Q4_0: 2^-21) of the largest are scaled up first, so that a
 * part of values near that |v| keeps 5 bits (f16: 7, Q4_0: 15) and more; below 2^-104 of the
 * largest weight nothing is left.
 * Scores in log2 units (times 1.4427) have to
 * be finite floats, and |scale| times the largest |q| of a row below 2^136.
 *
 *   q            device, dtype, element (b, h, d) at b * q_bs + h * q_hs + d
 *   block_table  device int32, row b at b * table_stride, table_width page ids;
 *                entries past a sequence's length are not used
 *   seq_lens     device int32 [B], 0 .. max_len. A length outside that range,
 *                or a page id outside the cache, gives NaN in that sequence's
 *                heads and latches QMM_ERR_BAD_SLOT.
 *   max_len      host bound on seq_lens, at most table_width * page_size. The
 *                split goes by it, not by the lengths: under a bound far above
 *                them most of the GPU idles (one sequence of 6900 tokens, 8 heads
 *                of 128, f16: 11 us under a bound of 6900, 60 us under 131072)
 *   window       0: the whole sequence
 *   out          device, dtype, [B][n_q_heads][head_dim]: q itself where that
 *                is contiguous, or apart from it (QMM_ERR_BAD_ARGUMENT); lse  fp32
 *                [B][n_q_heads] or NULL
 *   workspace    device scratch of the caller, 16-byte aligned, at least
 *                qattn_decode_workspace_bytes(...) bytes (may be NULL where
 *                that is 0 or qattn_decode_splits is 1); calls that overlap
 *                must not share it
 * head_dim is 64, 96, 128, 192 or 256 (QMM_ERR_UNIMPLEMENTED otherwise).
 */
QMM_API int qattn_decode(int fmt, const void* q, int dtype, size_t q_elems, int64_t q_bs, int64_t q_hs,
                         const void* k_cache, const void* v_cache, size_t cache_bytes, int64_t n_pages,
                         int64_t page_stride, int page_size, const int32_t* block_table, size_t table_elems,
                         int64_t table_stride, int table_width, const int32_t* seq_lens, int max_len, int64_t B,
                         int n_q_heads, int n_kv_heads, int head_dim, float scale, int window, float softcap,
                         void* out, size_t out_elems, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Scratch bytes qattn_decode asks for on the current device (0: none, or an
 * argument it refuses). They do not shrink as B, max_len or window (0 counting
 * as the longest) grow: one workspace of the largest serves every smaller call. */
QMM_API size_t qattn_decode_workspace_bytes(int fmt, int dtype, int64_t B, int n_q_heads, int n_kv_heads, int head_dim,
                                            int max_len, int window);

/* Parts that qattn_decode splits sequences of max_len into on the current
 * device; with 1 it uses no workspace. 0: an argument it refuses. */
QMM_API int qattn_decode_splits(int fmt, int dtype, int64_t B, int n_q_heads, int n_kv_heads, int head_dim, int max_len,
                                int window);

/*
 * qrmsnorm -- RMS norm of T x H rows of D values, with the residual's addition
 * before it. For each row, in fp32:
 *
 *   h = x + residual             (h = x without a residual)
 *   residual_out = h             (rounded to the residual's type, if asked for)
 *   y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)
 *
 * The norm takes h before it is rounded for residual_out. H = 1 norms tokens; more
 * norm each head of a projection's rows. A row whose sum of squares passes
 * the fp32 range (values of about 2^60 and more) gives zeros, one that holds a
 * NaN gives NaN, and one that holds an Inf what the formula does: NaN in its place (in
 * QMM_NORM_Q8_0 rows its block) and zeros elsewhere; with eps = 0 one of zeros, or of values so small that
 * all squares vanish in fp32 (below 2^-75), is divided by zero.
 *
 *   X             device, x_dtype, element (t, h, d) at t * x_ts + h * x_hs + d
 *   residual      device, r_dtype, the same at r_ts, r_hs, or NULL
 *   residual_out  device, r_dtype, at ro_ts, ro_hs, or NULL; may be residual, or X
 *                 where that has its type, with the same strides
 *   weight        device fp32 [D], or NULL for ones (weight_offset is then not read)
 *   Y             device, element (t, h, d) at t * y_ts + h * y_hs + d of y_fmt:
 *                 QMM_F32, QMM_F16 or QMM_BF16 (rounded once); or
 *                 QMM_NORM_Q8_0: rows of D / 32 Q8_0 blocks (D a multiple of 32), as
 *                 qdequant and the products' weights have them, rounded as
 *                 QMM_KV_Q8_0 is by qkv_store; y_ts, y_hs and y_elems then count
 *                 bytes (strides even). Y may be X (QMM_F32 and so on of X's type) with
 *                 the same strides.
 * Otherwise no output shares memory with another or with an input, nor do two
 * rows of an output (QMM_ERR_BAD_ARGUMENT). D is at most 2^20, T * H below 2^31.
 */
enum { QMM_NORM_Q8_0 = 16 };
QMM_API int qrmsnorm(const void* X, int x_dtype, size_t x_elems, int64_t x_ts, int64_t x_hs, const void* residual,
                     int r_dtype, size_t r_elems, int64_t r_ts, int64_t r_hs, void* residual_out, size_t ro_elems,
                     int64_t ro_ts, int64_t ro_hs, const float* weight, size_t weight_elems, float weight_offset,
                     float eps, void* Y, int y_fmt, size_t y_elems, int64_t y_ts, int64_t y_hs, int64_t T, int64_t H,
                     int64_t D, void* stream);

/* Scores of qmoe_route. */
typedef enum { QMM_SCORE_SOFTMAX = 0, QMM_SCORE_SIGMOID = 1 } qmm_score;

/*
 * qmoe_route -- the experts of each token and their weights, as qmoe_ffn and
 * qgemm_grouped take them. For a token with logits x:
 *
 *   s_e = e^{x_e} / sum e^x  (softmax)  or  1 / (1 + e^{-x_e})  (sigmoid)
 *   c_e = s_e + bias_e                  (c = s without a bias)
 *   n_groups > 1: a group's value is the sum of its group_top (1 or 2) largest c;
 *     the experts of the top_groups best groups stay
 *   ids: the top_k largest c of those that stay, the largest first
 *   w_j = s_{ids_j}, divided by their sum if renorm, times scale
 *
 * Equal values go to the lower index. They are compared as 64 bits have them, not as
 * fp32 does: where fp32's rounding could decide (in a few rows of a thousand),
 * the row is computed in 64 bits. Without a bias, groups of group_top 2 aside,
 * the logits themselves are compared; with one, also of zeros, scores that 64 bits do
 * not tell apart are equal (sigmoids of logits past 37; what is below 2^-53 of the
 * bias), and values within 2^-49 of the largest's magnitude are in the order that this
 * computation rounds them to. A NaN logit or bias counts as the largest
 * value; weights are NaN where the formula is (softmax: all of the token's). Logits
 * of -Inf have s = 0, a row of only those all s = 0; a bias of -Inf puts an
 * expert behind all others. Where the chosen logits are all -Inf renormalised
 * weights are zero. Ids are always distinct and in range.
 *
 *   logits    device, dtype, token t's n_experts values at t * stride
 *   bias      device fp32 [n_experts], or NULL
 *   ids, weights  device int32 / fp32 [T][top_k]; out_elems the size of each
 * n_experts is at most 1024, top_k and n_groups at most 32 (QMM_ERR_UNIMPLEMENTED);
 * n_groups divides n_experts, group_top is at most a group's experts and top_k at
 * most the experts that stay (QMM_ERR_BAD_ARGUMENT).
 */
QMM_API int qmoe_route(const void* logits, int dtype, size_t elems, int64_t stride, const float* bias, int score,
                       int n_groups, int top_groups, int group_top, int top_k, int renorm, float scale, int32_t* ids,
                       float* weights, size_t out_elems, int64_t T, int n_experts, void* stream);

/*
 * qmm_check_device_error -- synchronize `stream`, then read and clear the
 * device-side error latch of the current device. Returns QMM_OK,
 * QMM_ERR_DEVICE_TIMEOUT (a bounded wait in a kernel ran out; that kernel's
 * output is unspecified), QMM_ERR_BAD_EXPERT_ID, QMM_ERR_BAD_SLOT, or
 * QMM_ERR_CUDA.
 */
QMM_API int qmm_check_device_error(void* stream);

/*
 * qmm_selftest_wait_timeout -- test of the failure path (the pages have no
 * counterpart). Queues on `stream` one small kernel that waits on a shared-
 * memory barrier nothing ever completes, gives up after `cycles` SM clock
 * cycles (1 .. 2^32), and latches the same timeout status a real kernel's
 * bounded wait would. The next qmm_check_device_error() then returns
 * QMM_ERR_DEVICE_TIMEOUT and clears it; the CUDA context stays usable. No
 * trap, fault or unbounded wait is involved. Returns QMM_OK, or
 * QMM_ERR_BAD_ARGUMENT / QMM_ERR_CUDA without launching.
 */
QMM_API int qmm_selftest_wait_timeout(int64_t cycles, void* stream);

/* Kernel-path override, for tests and experiments: 0 = automatic (default),
 * 1 = force the generic CUDA-core kernels, 2 = force the streaming GEMV for
 * qgemm (N <= 8), 3 = force the tensor-core GEMM for qgemm. Applies to the
 * later calls of the calling host thread only (thread-local). Returns that
 * thread's previous value, or -1 for an unknown value (setting unchanged). */
QMM_API int qmm_set_path(int path);

/* Which kernel family the most recent successful call on this host thread
 * launched: 1 generic, 2 streaming GEMV, 3 tensor-core GEMM, 4 dequant,
 * 5 grouped GEMV, 6 MoE layer, 7 repacked (split-K) GEMV, 8 rotary, 9 cache
 * store, 10 cache load, 11 decode attention, 12 RMS norm, 13 routing; 0 before
 * any call. */
QMM_API int qmm_last_path(void);

/* Number of kernels this library has launched since load (all threads). */
QMM_API uint64_t qmm_launch_count(void);

/*
 * qmm_shutdown -- frees the per-device workspaces qgemm grows (activation
 * sums, partial tiles; see qgemm) on every device that has one, and forgets
 * the device addresses of the library's own device arrays (its error latch
 * and qgemm_noalloc's scratch), which the next call looks up again. cudaFree
 * waits for the work in flight on that device first. Later calls grow the
 * workspaces again as needed. Call it before anything that tears down a
 * device's context (cudaDeviceReset): addresses cached across that would be
 * stale. Not to be called while another thread is inside the library.
 * Returns QMM_OK, or QMM_ERR_CUDA if a free failed (the remaining ones are
 * still attempted). The current device is left as it was.
 */
QMM_API int qmm_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
