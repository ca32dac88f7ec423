/*
 * qk.h -- C ABI of libqk: matrix products over GGUF block-quantized weights
 * on one GB300 (sm_103a), with the blocks unpacked inside the dot product.
 *
 * Block formats (one block = a fixed number of weights along a row):
 *   Q4_K  256 weights in 144 bytes: fp16 d, fp16 dmin, 12 bytes holding eight
 *         6-bit sub-block scales and eight 6-bit mins, 128 bytes of 4-bit
 *         codes; weight = (d*sc)*q - dmin*m.  ("Hitchhiker's Guide -- Lab 01:
 *         Air-Gapped LLM Serving", section 11.2, Q4_K super-block figure;
 *         "12 -- llama.cpp / GGUF / Local Inference Mastery", "Q4_K_M -- bit
 *         layout in exquisite detail", figure and dequantization pseudo-code.)
 *   Q6_K  256 weights in 210 bytes: 128 bytes of low code nibbles, 64 bytes
 *         of high code bit pairs, sixteen int8 scales (one per 16 weights),
 *         fp16 d; weight = d*sc*(q - 32).  ("12 -- llama.cpp / GGUF", "Other
 *         k-quants at a glance": 256-weight super-block, 6.6 bits/weight.)
 *   Q8_0  32 weights in 34 bytes: fp16 d, 32 int8 codes; weight = d*q.
 *         ("Hitchhiker's Guide", section 11.1: the Q4_0 structure with 8-bit
 *         codes.)
 *   Q5_0  32 weights in 22 bytes: fp16 d, a 32-bit word of fifth bits, 16
 *         bytes of nibbles; weight = d*(q - 16).  ("Local LLM inference",
 *         "The mmap backend": one of the block types of a Q4_K_M file.)
 *   Q4_0  32 weights in 18 bytes: fp16 d, 16 bytes of nibbles (low nibbles
 *         elements 0-15, high nibbles 16-31); weight = d*(q - 8).
 *         ("Hitchhiker's Guide", section 11.1, Q4_0 block figure; "How LLM
 *         Inference Engines Work", "Loading GGUF Models", the Q4_0
 *         dequantizer.)
 *   Q5_K  256 weights in 176 bytes: fp16 d, fp16 dmin, the 12 scale bytes
 *         of Q4_K, 32 bytes of fifth code bits (bit 2c + h of byte l for
 *         weight 64c + 32h + l), 128 bytes of low nibbles placed as Q4_K's
 *         codes; weight = (d*sc)*q - dmin*m, q in 0..31.  The pages give only
 *         its size ("12 -- llama.cpp / GGUF", "Other k-quants at a glance":
 *         256-weight super-block, 5.5-5.7 bits/weight); the layout is the
 *         GGUF k-quant one.
 *   Q2_K  256 weights in 84 bytes, sixteen 16-weight groups: 16 bytes of
 *         (4-bit scale, 4-bit min) per group, 64 bytes of 2-bit codes (code
 *         l of group 8t + 2j + k is bits 2j.. of byte 32t + 16k + l), fp16 d,
 *         fp16 dmin; weight = (d*sc)*q - dmin*m.  (Pages: 2.5-2.6 bits/weight
 *         on 256-weight super-blocks, same table; layout: GGUF.)
 *   Q3_K  256 weights in 110 bytes: 32 bytes of high-bit mask, 64 bytes of
 *         2-bit codes placed as Q2_K's, 12 bytes of sixteen 6-bit scales
 *         (stored + 32), fp16 d; a code is its 2 bits minus 4 unless its
 *         mask bit (bit 4t + j of byte 16k + l) is set; weight = (d*sc)*q.
 *         (Pages: 3.4-4.0 bits/weight, same table; layout: GGUF.)
 * The bit placement inside the Q4_K scale bytes, the Q6_K code bytes and the
 * Q5_0 block is the k-quant / GGUF packing: low nibbles of a group of bytes
 * are the first weights, high nibbles the next ("How LLM Inference Engines
 * Work", "Loading GGUF Models").
 *
 * Matrix layout: a weight matrix W has `rows` output rows and `cols` inputs.
 * Each row is cols / block_elems blocks laid back to back along cols; row r
 * starts at byte r * qk_row_bytes(type, cols).  Rows follow each other with
 * no padding (so Q6_K rows of 11008 weights start at 9030-byte steps, not on
 * 16-byte boundaries).
 *
 * Ownership and memory: every pointer argument is DEVICE memory owned by the
 * caller, except where a function says otherwise.  The library allocates no
 * device memory; scratch space comes from the caller as a workspace.
 *
 * Streams: `stream` is a cudaStream_t (NULL = the legacy default stream).
 * Every compute call is asynchronous on it and returns once the work is
 * queued.  Argument errors are detected on the host before anything is
 * queued; nothing is launched when a call returns an error.
 *
 * Errors: every call returns a qk_status; qk_last_error() gives a text for
 * the last failure on the calling thread.  Waits inside the kernels are
 * bounded; a wait that runs out sets a device status word instead of
 * hanging, and qk_device_status() reports it as QK_ERR_TIMEOUT.
 */
#ifndef QK_H_
#define QK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Quant types.  The numbers are this library's own. */
typedef enum {
    QK_Q4_K = 1, QK_Q6_K = 2, QK_Q8_0 = 3, QK_Q5_0 = 4, QK_Q4_0 = 5, QK_Q5_K = 6, QK_Q2_K = 7, QK_Q3_K = 8
} qk_type;

typedef enum {
    QK_OK = 0,
    QK_ERR_TYPE = 1,      /* unknown quant type                                 */
    QK_ERR_SHAPE = 2,     /* negative size, cols not a multiple of block_elems  */
    QK_ERR_ALIGN = 3,     /* a pointer breaks its stated alignment              */
    QK_ERR_NULL = 4,      /* a required pointer is NULL                         */
    QK_ERR_WORKSPACE = 5, /* workspace smaller than the matching *_workspace()  */
    QK_ERR_CUDA = 6,      /* the CUDA runtime reported an error                 */
    QK_ERR_TIMEOUT = 7,   /* a bounded wait inside a kernel ran out             */
    QK_ERR_ARG = 8,       /* any other invalid argument                         */
    QK_ERR_FORMAT = 9,    /* a GGUF image is malformed or truncated             */
    QK_ERR_IO = 10        /* a file could not be opened or mapped               */
} qk_status;

/* Output element types of qk_dequant. */
enum { QK_OUT_F32 = 0, QK_OUT_BF16 = 1 };

/* Version of this ABI. */
int qk_version(void);

/* Bytes per block (144, 210, 34, 22) and weights per block (256, 256, 32,
 * 32); 0 for an unknown type.  ("Hitchhiker's Guide", 11.2: 144 bytes =
 * 4.5 bits per weight.) */
size_t qk_block_bytes(int type);
int qk_block_elems(int type);

/* Bytes of one row of `cols` weights; 0 for an unknown type or when cols is
 * not a multiple of the block size. */
size_t qk_row_bytes(int type, int64_t cols);

/* Dequantize W [rows, cols] into out [rows, cols] row-major, as fp32
 * (out_dtype QK_OUT_F32) or bf16 (QK_OUT_BF16, round to nearest even).
 * Each weight is computed in fp32 by the type's formula above, in the order
 * written ((d*sc)*q - dmin*m for Q4_K); fp32 results are exact except for
 * the final subtraction of Q4_K.
 * W: 16-byte aligned.  out: 16-byte aligned.  rows == 0 queues nothing. */
qk_status qk_dequant(int type, const void* W, int64_t rows, int64_t cols,
                     void* out, int out_dtype, void* stream);

/* Quantize fp32 weights into packed blocks: the write side of the format.
 * The pages name the k-quant quantizer ("12 -- llama.cpp / GGUF / Local
 * Inference Mastery", reading list: quantize_row_q4_K) without giving it,
 * and describe plain quantization as minimising the weight-space error
 * ("Hitchhiker's Guide -- Lab 01", 11.3); this is the plain min/max scheme,
 * each quotient an IEEE fp32 division and each code clamp(round half away
 * from zero(quotient)):
 *   Q4_K per 32-weight sub-block: lo = min(0, min w), hi = max w,
 *        sc_f = (hi - lo)/15, m_f = -lo; d = fp16(max sc_f / 63),
 *        dmin = fp16(max m_f / 63); sc = cr(sc_f/d, 0..63),
 *        m = cr(m_f/dmin, 0..63); q = cr((w + dmin*m) / (d*sc), 0..15).
 *   Q5_K the same with 31 in place of 15.
 *   Q2_K per 16 weights: the Q4_K scheme with 3 in place of 15 and 4-bit
 *        sc, m (d = fp16(max sc_f / 15), dmin = fp16(max m_f / 15)).
 *   Q3_K per 16 weights: s = max|w| / 4, d = fp16(max s / 31),
 *        sc = cr(s/d, -32..31), q = cr(w / (d*sc), -4..3).
 *   Q6_K per 16 weights: s = max|w| / 32, d = fp16(max s / 127),
 *        sc = cr(s/d, -128..127), q = cr(w / (d*sc), -32..31) + 32.
 *   Q8_0 / Q5_0 / Q4_0 per 32: d = fp16(max|w| / 127 | 15 | 7),
 *        q = cr(w/d) + 0 | 16 | 8, clamped to the code range.
 * A zero divisor gives the offset code; NaN inputs are not rejected (they are
 * skipped by the maxima and a NaN quotient takes the lowest code).
 *   w   fp32 [rows, cols] row-major, 16-byte aligned.
 *   out rows * qk_row_bytes(type, cols) bytes, 4-byte aligned; fully
 *       overwritten.
 * Deterministic; the bytes do not depend on the launch.  rows == 0 or
 * cols == 0 queues nothing.  Errors: QK_ERR_TYPE, QK_ERR_SHAPE (cols not a
 * multiple of the block size, negative sizes), QK_ERR_NULL, QK_ERR_ALIGN. */
qk_status qk_quantize(int type, const float* w, int64_t rows, int64_t cols, void* out, void* stream);

/* Decode attention over a block-quantized KV cache ("Hitchhiker's Guide --
 * Lab 01", 13.2: K and V cached as q8_0, or q4_0 at a quality cost, and read
 * inside attention; grouped-query attention shares each kv head among
 * n_heads / n_kv query heads).  One query token:
 *   s_t = scale * sum_i q[h, i] K[t, g, i],  g = h / (n_heads / n_kv),
 *   p = softmax(s) over t = 0 .. T-1,  out[h, i] = sum_t p_t V[t, g, i].
 *   type   QK_Q8_0, QK_Q5_0 or QK_Q4_0 (the cache's block type).
 *   q      fp32 [n_heads, d], device, 4-byte aligned.
 *   K, V   [T, n_kv, d]: each (t, g) row is d / 32 blocks (so a cache row
 *          of all kv heads is qk_row_bytes(type, n_kv * d) bytes, written by
 *          qk_quantize from fp32 [T, n_kv * d]); device, 16-byte aligned.
 *   d      32, 64, 128 or 256; n_heads a multiple of n_kv, at most 8 query
 *          heads per kv head; 1 <= T <= 65535 * 256.
 *   out    fp32 [n_heads, d]; ws at least qk_attn_decode_workspace bytes.
 * Positions are split over CTAs (one CTA per kv head and range of
 * positions, about T / (2 SMs / n_kv) of them; shapes whose per-thread state
 * does not fit take chunks of 192 or 256), the cache streamed once; each
 * range keeps its max score, sum of exponentials and weighted value sum, and
 * a second launch combines the ranges (log-sum-exp) in a fixed order:
 * deterministic.  Scores on the fp16 tensor-core MMA (exact codes, each
 * query element as two fp16 terms after a power-of-two scale per 32-block),
 * fp32 softmax; the p V sums in fp32, or for Q8_0 / Q4_0 with d = 128 and
 * up to four query heads per kv head on the MMA with p d as two fp16 terms
 * after a power-of-two scale per 128 positions.  Accuracy: |out - out_exact|
 * <= 2e-4 * sum_t p_t |V[t, g, i]| + 1e-6.
 * Errors: QK_ERR_TYPE, QK_ERR_SHAPE, QK_ERR_NULL, QK_ERR_ALIGN,
 * QK_ERR_WORKSPACE. */
size_t qk_attn_decode_workspace(int type, int64_t T, int n_heads, int n_kv, int d);
qk_status qk_attn_decode(int type, const float* q, const void* K, const void* V, int64_t T, int n_heads, int n_kv, int d,
                         float scale, float* out, void* ws, size_t ws_bytes, void* stream);

/* Importance-weighted quantization ("Hitchhiker's Guide -- Lab 01", 11.3,
 * the importance matrix: minimise sum_i E[x_i^2] (w_i - w^_i)^2 rather than
 * the plain weight-space error).  imp[c] is the mean squared activation met
 * by weight column c (fp32 [cols], finite and >= 0; the same for every row).
 * The page gives the objective, not the search; per group (the 32-weight
 * block of Q8_0 / Q5_0 / Q4_0, the 32-weight sub-block of Q4_K / Q5_K, the
 * 16-weight group of Q6_K / Q3_K / Q2_K):
 *   s0 (and m0) = the plain quantizer's group scale (and min); for k = 0..20
 *   the candidate scale s0 * (90 + k) / 100 rounds the codes, a weighted
 *   least-squares refit gives the scale (scale and min jointly where the type
 *   has a min; kept only with a positive determinant, a positive scale and a
 *   non-negative min), and the candidate of least weighted error wins (the
 *   first on ties).  The block is then assembled as by qk_quantize with
 *   those group values, and kept only if its weighted error (summed per
 *   group, then over groups) is no more than the plain block's; otherwise
 *   the plain block is written.  fp32 throughout, sums in index order, so
 *   the bytes are deterministic.  All-zero importances give qk_quantize's
 *   bytes.
 *   w    device fp32 [rows, cols], 16-byte aligned.
 *   imp  device fp32 [cols], 4-byte aligned.
 *   out  rows * qk_row_bytes(type, cols) bytes, 4-byte aligned.
 * One lane per 32 weights (it searches its own groups; the codes of a
 * candidate take one reciprocal of its scale, with the division's rounding
 * reproduced exactly), a warp per 32 groups.
 * Errors as qk_quantize. */
qk_status qk_quantize_imatrix(int type, const float* w, int64_t rows, int64_t cols, const float* imp, void* out,
                              void* stream);

/* Fused decode FFN gate: h[n] = SiLU(g[n]) * u[n] with g = Wg x, u = Wu x
 * (batch 1) and SiLU(z) = z / (1 + e^-z) ("How LLM Inference Engines
 * Work", "SwiGLU Feed-Forward Network": the gate projection passes through
 * SiLU and multiplies the up projection element-wise; SiLU is not written
 * out on the page, the standard z * sigmoid(z) is used).  One launch: the
 * same CTAs walk their rows of Wg and then of Wu (x prepared once), and
 * write h only; g and u never reach memory.
 *   Wg, Wu [rows, cols] packed blocks of the same type, 16-byte aligned.
 *   x      fp32 [cols], 16-byte aligned.
 *   h      fp32 [rows], 4-byte aligned; fully overwritten.
 * Accuracy: g and u each as qk_gemv (1e-4 * sum|w x| + 1e-6), then the fp32
 * epilogue (expf, one division, one product).  No limit on cols beyond the
 * format's.
 * rows == 0 queues nothing; cols == 0 zero-fills h. */
qk_status qk_gemv_swiglu(int type, const void* Wg, const void* Wu, int64_t rows, int64_t cols,
                         const float* x, float* h, void* stream);

/* Most tokens, experts per token and experts of a qk_moe_ffn call. */
#define QK_MOE_MAX_TOK 64
#define QK_MOE_MAX_K 16
#define QK_MOE_MAX_EXP 512

/* A mixture-of-experts layer for a few tokens (a decode batch, a drafted
 * tree), over packed expert weights:
 *   l = R x [n_exp],  the k largest of l (of equals the lowest index),
 *   gate_j = scale * exp(l_j) / sum exp(l)   over the k chosen (norm) or over
 *            all experts (norm == 0),
 *   out = sum_j gate_j * Wd_j (SiLU(Wg_j x) * (Wu_j x))   over the chosen.
 *   type, Wg, Wu  packed blocks [n_exp, rows, cols], one type for both;
 *   type_down, Wd packed blocks [n_exp, cols, rows] of any type; 16-byte
 *          aligned (the layouts of a GGUF file's expert tensors).
 *   router fp32 [n_exp, cols], 16-byte aligned; ids and gate are then written.
 *          NULL: ids and gate are given (any other router); a pair whose id is
 *          outside 0 .. n_exp - 1 adds nothing, an id that a token has twice
 *          counts twice.  norm and scale are then ignored.
 *   x      fp32 [n_tok, cols], 16-byte aligned; n_tok 0 .. QK_MOE_MAX_TOK.
 *   ids    int32 [n_tok, k], gate fp32 [n_tok, k], by falling logit; k 1 ..
 *          QK_MOE_MAX_K and at most n_exp.
 *   out    fp32 [n_tok, cols], apart from x; fully overwritten.
 *   ws     at least qk_moe_workspace(..) bytes, 16-byte aligned.
 * Every expert that some token chose is read once per four or eight of its
 * tokens.  Three launches, four with a router.  Accuracy: each product is
 * within 2^-17 * sum_k (|scale code| + |min|) |x_k| + 1e-6 of its exact value
 * (for the types without a min that is sum |w x|, but Q6_K's codes count as 0 ..
 * 63 with a min of 32 scales); in practice the layer is 2 to 5e-7 of its norm
 * off.  The SiLU and the sum over experts are fp32; the router's logits are fp32
 * sums.
 * A logit that is NaN ranks first and gives NaN gates for its token.
 * Deterministic.
 * n_tok == 0 queues nothing.  Errors: QK_ERR_TYPE, QK_ERR_SHAPE (also rows or
 * cols below 1 or above 2^16), QK_ERR_NULL, QK_ERR_ALIGN, QK_ERR_ARG (scale
 * not finite), QK_ERR_WORKSPACE. */
size_t qk_moe_workspace(int type, int type_down, int n_exp, int64_t rows, int64_t cols, int k, int64_t n_tok);
qk_status qk_moe_ffn(int type, const void* Wg, const void* Wu, int type_down, const void* Wd, int n_exp, int64_t rows,
                     int64_t cols, const float* router, int k, int norm, float scale, const float* x, int64_t n_tok,
                     int32_t* ids, float* gate, float* out, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes qk_gemv needs for this problem: 0 for every shape (the
 * kernel prepares its activations in shared memory).  Kept so that callers
 * written against a workspace-taking GEMV need no change. */
size_t qk_gemv_workspace(int type, int64_t rows, int64_t cols, int64_t M);

/* Fused dequant-GEMV: y[m, n] = sum_k w[n, k] * x[m, k] for m < M,
 * n < rows, with every weight unpacked in registers inside the dot product
 * and never written out ("Local LLM inference", "The mmap backend": blocks
 * dequantized inside the dot product; each weight decoded once per input
 * batch and reused across its rows).  fp32 activations, fp32 accumulation.
 *   W  [rows, cols] packed blocks, 16-byte aligned.
 *   x  fp32 [M, cols] row-major, 16-byte aligned.
 *   y  fp32 [M, rows] row-major, 4-byte aligned; fully overwritten.
 *   ws, ws_bytes  ignored (no shape needs a workspace; NULL, 0 is fine).
 * Kernel: the fp16 warp MMA with exact integer codes (the code minus an
 * integer offset) and x as two fp16 terms per element after a power-of-two
 * scale per 32-element block; one launch for M == 1, one per pair of
 * activation rows otherwise (each launch streams W once).
 * Accuracy: |y - y_exact| <= 1e-4 * sum_k |w x| + 1e-6 per output.  The
 * per-element error model behind it: |x - (hi + lo) 2^e| <= 2^-22 |x| +
 * 2^(e-25), with 2^e <= 2^-14 times the block's largest magnitude when e > 0
 * (so elements down to 2^-17 of that magnitude keep 22 significant bits);
 * codes are exact, and a weight that is exactly zero contributes exactly
 * zero.  So blocks holding massive activations (tested at 1e3, 1e4
 * and 1e5 times the others, beside zero and tiny weights) stay within the
 * bound; the remaining terms are fp32 roundings of the block sums and scales.
 * Results are deterministic run to run (fixed reduction order).
 * rows == 0 or M == 0 queues nothing; cols == 0 zero-fills y. */
qk_status qk_gemv(int type, const void* W, int64_t rows, int64_t cols,
                  const float* x, int64_t M, float* y,
                  void* ws, size_t ws_bytes, void* stream);

/* Most matrices one qk_gemv_batch call takes. */
#define QK_GEMV_BATCH_MAX 8

/* Decode GEMV over several matrices that read the same activation vector, in
 * one launch: y_i[n] = sum_k W_i[n, k] * x[k] for i < n_mat, n < rows[i].
 * In a decoder layer the query, key and value projections are applied to the
 * same hidden state ("How LLM Inference Engines Work", Grouped-Query
 * Attention (GQA) and KV Cache), and so are the gate and up projections of
 * the feed-forward block (same page, SwiGLU Feed-Forward Network).  One call
 * per such group prepares x once and spreads the rows of all its matrices
 * over the GPU, instead of paying a launch and a ramp per matrix.
 *   type, cols  common to all matrices.
 *   W     host array of n_mat device pointers, W[i] = packed blocks
 *         [rows[i], cols], 16-byte aligned.
 *   rows  host array of n_mat row counts (0 allowed: that matrix is skipped).
 *   x     fp32 [cols] (one activation row), 16-byte aligned, device.
 *   y     host array of n_mat device pointers, y[i] = fp32 [rows[i]], 4-byte
 *         aligned; fully overwritten.
 * The host arrays are read during the call only.  No workspace, no limit on
 * cols beyond the format's.  n_mat outside 1..QK_GEMV_BATCH_MAX is
 * QK_ERR_ARG.  Kernel, accuracy and determinism as qk_gemv with M == 1. */
qk_status qk_gemv_batch(int type, int n_mat, const void* const* W, const int64_t* rows, int64_t cols,
                        const float* x, float* const* y, void* stream);

/* qk_gemv for callers that cannot allocate device memory.  The pages have no
 * counterpart; this is a convenience of this library.  Some callers of a
 * decode GEMV are not allowed to allocate: plug-in code running inside a
 * host runtime that owns every device allocation, code under a fixed memory
 * budget that must not grow its footprint while serving, and paths that
 * cannot afford the device-wide synchronization that cudaMalloc / cudaFree
 * can cause.  They call this instead of qk_gemv and pass no workspace.
 *   Arguments, results, accuracy and errors are those of qk_gemv; argument
 *   errors are reported exactly as qk_gemv reports them.
 *   Scratch: none.  The GEMV kernel prepares its activations in shared
 *   memory, so no shape needs a workspace; this call allocates nothing and
 *   holds no device memory of its own.
 *   Set-up: the first qk_* call on a device looks up the library's device
 *   status word; make it before starting any stream capture.  A
 *   cudaDeviceReset() unloads the module and leaves that address stale, so
 *   make no qk_* call on a device after resetting it. */
qk_status qk_gemv_noalloc(int type, const void* W, int64_t rows, int64_t cols,
                          const float* x, int64_t M, float* y, void* stream);

/* Workspace bytes qk_gemm needs (0 when none). */
size_t qk_gemm_workspace(int type, int64_t rows, int64_t cols, int64_t M);

/* Tensor-core dequant-GEMM for prefill: Y[m, n] = sum_k w[n, k] * X[m, k]
 * with X in bf16 and fp32 accumulation; weight tiles are unpacked to bf16 in
 * shared memory and fed to the tensor cores.  ("12 -- llama.cpp / GGUF":
 * prompt processing is big GEMMs of high arithmetic intensity.)
 *   W  [rows, cols] packed blocks, 16-byte aligned.
 *   X  bf16 [M, cols] row-major, 16-byte aligned; cols * 2 bytes must be a
 *      multiple of 16 (always true: cols is a multiple of 32).
 *   Y  fp32 [M, rows] row-major, 16-byte aligned; fully overwritten.
 *   ws as for qk_gemv.
 * Accuracy: |Y - Y_exact(bf16 X)| <= 5e-3 * sum_k |w x|; the weights are
 * rounded to bf16 before the product (Q8_0, Q5_0 and Q6_K codes and most
 * Q4_K weights are exact in bf16 up to the block scale).
 * M == 0 or rows == 0 queues nothing; cols == 0 zero-fills Y.  rows above
 * 65535 * 128 = 8,388,480 is QK_ERR_SHAPE. */
qk_status qk_gemm(int type, const void* W, int64_t rows, int64_t cols,
                  const void* X_bf16, int64_t M, float* Y,
                  void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * A paged, block-quantized KV cache of many requests, and one verification
 * step of speculative decoding over it.
 *
 * The cache is two pools (K and V) of n_pages pages.  A page holds `page`
 * consecutive positions of one request for every kv head, head by head:
 *   pool [n_pages][n_kv][page][d], each (page, head, position) row d / 32
 *   blocks of a 32-weight type (Q8_0, Q5_0 or Q4_0),
 * so one head's part of a page is contiguous and a multiple of 16 bytes (it
 * is what attention fetches with one copy).  page is 16, 32, 64, 128 or 256;
 * d is 32, 64, 128 or 256.  Position p of request r lives in page
 * table[r * table_stride + p / page] at p % page; its slot is
 * (page id) * page + p % page.  A pool needs n_pages * qk_kv_page_bytes
 * bytes, 16-byte aligned.  Requests, lengths and tables are int32 arrays in
 * device memory, so a step's launches need nothing from the host and can be
 * captured into a graph.
 *
 * A page id or slot outside the pool is never followed: the row concerned is
 * skipped (attention: not visible) and qk_device_status() then reports
 * QK_ERR_ARG.  A slot of -1 is a token without a place and is skipped
 * silently. */

/* Most drafted tokens of one request (the width of a tree mask). */
#define QK_TREE_MAX 64
/* Most positions of one request that attention walks (indexes inside a tile
 * past the last one still fit 32 bits). */
#define QK_TREE_MAX_POS 2147483392
/* Most requests one qk_kv_plan call takes. */
#define QK_PLAN_MAX_REQ 8192

/* Bytes of one page of one pool; 0 when the type, n_kv, d or page is not one
 * of the above. */
size_t qk_kv_page_bytes(int type, int n_kv, int d, int page);

/* Page bookkeeping of a step: requests whose lengths change give pages back
 * and take pages, and every token to be written gets its slot.  One launch.
 *   have   int32 [n_req]: positions the request holds pages for (before).
 *   want   int32 [n_req]: positions it shall hold pages for (after); 0 frees
 *          all of them.
 *   start  int32 [n_req]: the first position to be written; the tokens of
 *          request r are positions start[r] .. want[r] - 1 (none when
 *          start[r] >= want[r]).
 *   table  int32 [n_req, table_stride], updated in place: with P_old =
 *          ceil(have / page) and P_new = ceil(want / page), entries P_old ..
 *          P_new - 1 are written; no other entry changes (entries past a
 *          request's pages are stale, not cleared).
 *   free_pages int32 [free_cap]: a stack of free page ids, *n_free of them
 *          (device int32).  The pages given back (in request order, each
 *          request's by rising index) are pushed first; then each growing
 *          request, in order, takes its pages from the top.  Only entries at
 *          *n_free and above are written, and the count after the call goes
 *          to *n_free_out, which must not be n_free itself: the call gives
 *          the same results when repeated on the same buffers.
 *   granted int32 [n_req]: 1, or 0 when the running sum of pages taken up to
 *          and including this request exceeds what is free, or when its
 *          numbers are not valid (negative, or more pages than table_stride).
 *          A request that is refused keeps the pages it had.
 *   cu     int32 [n_req + 1]: running sum of the requests' token counts (a
 *          refused request's tokens count, an invalid request has none).
 *   slots  int64 [cap], pos int32 [cap], req int32 [cap]: of token i (in
 *          request order, positions rising) its slot (-1 when refused), its
 *          position and its request; entries past the last token are -1.
 *          Tokens past cap are not written.  pos and req may be NULL.
 * All integers; the result does not depend on the launch.  n_req == 0 sets
 * cu[0] = 0, *n_free_out = *n_free and the token arrays to -1.
 * Errors: QK_ERR_SHAPE (negative sizes, n_req above QK_PLAN_MAX_REQ, a page
 * size that is not listed), QK_ERR_NULL, QK_ERR_ALIGN, QK_ERR_ARG (n_free_out
 * == n_free). */
qk_status qk_kv_plan(const int32_t* have, const int32_t* start, const int32_t* want, int64_t n_req, int page,
                     int32_t* table, int64_t table_stride, int32_t* free_pages, int64_t free_cap, const int32_t* n_free,
                     int32_t* n_free_out, int32_t* granted, int32_t* cu, int64_t* slots, int32_t* pos, int32_t* req,
                     int64_t cap, void* stream);

/* Quantize n_tok tokens' K and V rows into the cache (one launch for both).
 *   k, v   [n_tok, n_kv, d], dtype QK_OUT_F32 or QK_OUT_BF16, aligned to the
 *          element; k_stride and v_stride elements from token to token (at
 *          least n_kv * d), so slices of a fused projection's output serve
 *          as they are.  Rows that start on 16-byte boundaries are read
 *          faster.
 *   slots  int64 [n_tok]; -1 is skipped; the others are distinct.
 * The blocks are byte for byte those qk_quantize writes for the same values.
 * n_tok == 0 queues nothing.
 * Errors: QK_ERR_TYPE, QK_ERR_SHAPE, QK_ERR_NULL, QK_ERR_ALIGN, QK_ERR_ARG
 * (dtype). */
qk_status qk_kv_append(int type, const void* k, const void* v, int dtype, int64_t n_tok, int64_t k_stride, int64_t v_stride,
                       int n_kv, int d, const int64_t* slots, void* K, void* V, int64_t n_pages, int page, void* stream);

/* Norms of query and key heads with the position rotation in the same pass:
 * rows in, rows out.  For a head x [d] of token i,
 *   y = (x * inv) * w,  inv = 1 / sqrt(sum_e x_e^2 / d + eps)   (w given; else y = x)
 *   a = pos[i] * freq[j],  j < rot / 2:
 *   (y_p, y_q) -> (y_p cos a - y_q sin a, y_q cos a + y_p sin a)
 * with (p, q) = (j, j + rot / 2), or (2j, 2j + 1) when pairs is non-zero; the
 * elements from rot on are not turned.
 *   q [n_tok, n_heads, d], k [n_tok, n_kv, d], dtype QK_OUT_F32 or
 *          QK_OUT_BF16, aligned to the element; q_stride and k_stride elements
 *          from token to token, so that slices of a fused projection's output
 *          serve as they are.  n_heads or n_kv may be 0 (that pointer is then
 *          ignored).
 *   d      32, 64, 128 or 256; rot a multiple of 16, 0 .. d (0: no rotation;
 *          pos and freq are then ignored).
 *   pos    int32 [n_tok], any value; freq fp32 [rot / 2], angle per position
 *          (frequency scaling of any kind goes in here).  A frequency that is
 *          not finite, or 2^64 and more, gives NaN.
 *   q_norm, k_norm fp32 [d] or NULL (no norm); eps >= 0 and finite.
 *   q_out, k_out like q and k with their own strides, of out_dtype, aligned to
 *          the element.  In place (the same pointer, stride and type) is fine,
 *          any other overlap is not.
 * Rows on 16-byte boundaries are read and written faster.
 * Every square, sum, quotient, root and product above is rounded to fp32 by
 * itself, the squares are added by neighbours (x0^2 + x1^2, .., then those
 * sums by neighbours), and cos and sin are the fp32 nearest to their exact
 * values, up to one value in some ten thousand that is the next one: the angle of
 * a position is kept to 2^-96 of a turn, so far positions lose nothing.  (A cos
 * or sin that is nearly zero, as at frequencies below 2^-46, is within half a step
 * of fp32 and 2^-84 + |pos| 2^-93.)  Results are then rounded once to out_dtype.
 * n_tok == 0, or no heads, queues nothing.  Errors: QK_ERR_SHAPE, QK_ERR_NULL,
 * QK_ERR_ALIGN, QK_ERR_ARG (dtype, eps). */
qk_status qk_norm_rope(const void* q, const void* k, int dtype, int64_t n_tok, int64_t q_stride, int64_t k_stride, int n_heads,
                       int n_kv, int d, const int32_t* pos, const float* q_norm, const float* k_norm, float eps,
                       const float* freq, int rot, int pairs, void* q_out, void* k_out, int out_dtype, int64_t qo_stride,
                       int64_t ko_stride, void* stream);

/* qk_norm_rope on the way into the paged cache, and qk_kv_append, in one
 * launch: keys normed, rotated and quantized into their slots, values
 * quantized, queries normed, rotated and written as bf16 for qk_attn_tree.
 * Arguments as those two calls'; the cached bytes are those that qk_kv_append
 * writes for qk_norm_rope's fp32 keys.  pos is the position that a token is
 * rotated by (in a drafted tree its depth after the text), apart from the
 * place that slots gives its row.  n_heads == 0: no queries.
 *   q_out  bf16 [n_tok, n_heads, d], q_out_stride elements from token to token.
 * Errors: those of the two calls. */
qk_status qk_kv_append_rope(int type, const void* q, const void* k, const void* v, int dtype, int64_t n_tok, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, int n_heads, int n_kv, int d, const int32_t* pos,
                            const float* q_norm, const float* k_norm, float eps, const float* freq, int rot, int pairs,
                            const int64_t* slots, void* K, void* V, int64_t n_pages, int page, void* q_out,
                            int64_t q_out_stride, void* stream);

/* Keep the accepted path of each request's drafted tree: the rows at
 * positions base[r] + path[r * path_stride + j] move to base[r] + j, for j <
 * n_path[r], in both pools, as if all were read before any is written.
 *   base, n_path int32 [n_req]; path int32 [n_req, path_stride], entries 0 ..
 *   QK_TREE_MAX - 1.  n_path above path_stride or QK_TREE_MAX is cut to it;
 *   a row whose source or target has no page is left as it is.
 * Errors as qk_kv_append. */
qk_status qk_kv_compact(int type, void* K, void* V, int64_t n_pages, int page, int n_kv, int d, const int32_t* table,
                        int64_t table_stride, const int32_t* base, const int32_t* path, int64_t path_stride,
                        const int32_t* n_path, int64_t n_req, void* stream);

/* Attention of a tree of drafted tokens over the paged cache: the tokens of
 * all requests in one call.  Request r has tokens cu[r] .. cu[r + 1] - 1 (rows
 * of q; n of them) and ctx[r] committed positions; the K and V rows of its
 * token j are in the cache at position ctx[r] + j (qk_kv_append before).
 * For token i of the request, query head h and kv head g = h / (n_heads /
 * n_kv):
 *   s_t = scale * sum_e q[i, h, e] K[t, g, e],   t < ctx[r]: every one,
 *         t = ctx[r] + j: those with bit j of the token's mask set,
 *   out[i, h] = sum_t softmax(s)_t V[t, g].
 * With scale 0 that is the plain mean of the visible V.  A query head with a
 * NaN or an infinity, and a scale that is one, give NaN.  A token that sees no
 * position gives zeros, whatever its query.  What a token does not see
 * never reaches its result, whatever it holds (NaN and infinities included);
 * stale bytes past a request's last position are not used.
 *   q      bf16 [n_tok, n_heads, d], q_stride elements from token to token (a
 *          multiple of 8), 16-byte aligned.
 *   ctx    int32 [n_req], cu int32 [n_req + 1] (non-decreasing, within 0 ..
 *          n_tok).  Requests may have no tokens.  Positions past
 *          QK_TREE_MAX_POS or past the table are not visible and reported as
 *          a page outside the pool is.
 *   mask   uint64 [n_tok], bit j = the request's token j is visible (its own
 *          bit included where it sees itself); NULL = a plain chain: token i
 *          sees tokens 0 .. i.  n_req requests with one token each and mask
 *          NULL is ordinary batched decoding.
 *   max_q  at least the most tokens of one request, at most QK_TREE_MAX;
 *          tokens past it are not computed.
 *   out    bf16 [n_tok, n_heads, d], out_stride elements from token to token,
 *          2-byte aligned, apart from the inputs; rows of no request are not
 *          written.
 *   ws     at least qk_attn_tree_workspace(..) bytes, 16-byte aligned;
 *          max_pos = table_stride * page.
 * Cached values (code * d) and probabilities are rounded to fp16 as operands
 * of the tensor cores; scores, softmax statistics and sums are fp32.
 * Accuracy, with A the largest |scale| sum_e |q_e K_te| of a visible
 * position: |out - out_exact| <= 2^-8 |out_exact| + (2^-10 (1 + A) + 2^-13)
 * sum_t p_t |V[t]| + 2^-32 sum_t |V[t]|, and 2 to 4 % above the rounding of
 * the output in practice.  qk_attn_decode, which keeps the codes exact and
 * hands out fp32, has a bound that does not grow with A and takes less time
 * for one token over one request's cache (32,000 positions, Q8_0, 32 / 8 heads
 * of 128: 25 us against 36).  Cached K values beyond fp16's range (|w| that
 * rounds past 65504) give NaN for the tokens that see them.
 * At most 64 query heads to a kv head, n_req up to 65,535.  n_tok == 0 or
 * n_req == 0 queues nothing.  Errors: QK_ERR_TYPE, QK_ERR_SHAPE (also when the
 * tables could hold about 2^31 tiles or more), QK_ERR_NULL, QK_ERR_ALIGN,
 * QK_ERR_WORKSPACE. */
size_t qk_attn_tree_workspace(int type, int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d);
qk_status qk_attn_tree(int type, const void* q, int64_t n_tok, int64_t q_stride, const void* K, const void* V,
                       int64_t n_pages, int page, const int32_t* table, int64_t table_stride, const int32_t* ctx,
                       const int32_t* cu, const uint64_t* mask, int64_t n_req, int max_q, int n_heads, int n_kv, int d,
                       float scale, void* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream);

/* Penalties for repeated tokens, biases and grammar masks on logits, as a
 * sampler wants them before it picks.  Rows cu[r] .. cu[r + 1] - 1 belong to
 * request r.  With c the number of times token v stands in the request's
 * history and among the row's drafted ancestors,
 *   y = x > 0 ? x / rep[r] : x * rep[r],  then  y - freq[r] * c - pres[r]   (c > 0; else y = x)
 *   y + bias of token v (if listed; after the penalties, so that a bias shifts
 *   the result by its own value whatever rep is: samplers that add biases to
 *   the logits first differ for tokens that have both),
 *   -inf where the row's grammar bit of v is 0.
 *   logits [n_rows, vocab], dtype QK_OUT_F32 or QK_OUT_BF16, aligned to the
 *          element, row_stride elements from row to row; out likewise (its
 *          own out_stride; out == logits with equal strides is fine, any
 *          other overlap is not).  fp32 arithmetic, rounded once.
 *   hist   int32 [n_req, hist_stride], the first hist_len[r] of them;
 *          hist_stride below 2^20 - 64.  rep, pres, freq fp32 [n_req].
 *   draft  int32 [n_rows], the drafted token of each row, and mask uint64
 *          [n_rows] as in qk_attn_tree: bit j = the request's row j is an
 *          ancestor (the row itself too, when its own bit is set).  mask NULL:
 *          rows cu[r] .. the row itself; a request whose history and rows come
 *          to 2^20 or more then has its drafted tokens left out, which
 *          qk_device_status() reports as QK_ERR_ARG.  draft NULL: no drafted
 *          tokens.
 *   bias_tok int32, bias_val fp32 [n_req, bias_stride], the first
 *          bias_len[r]; of entries with the same token the last counts;
 *          bias_stride at most 4095; bias_tok NULL: no biases.
 *   grammar uint32 [n_rows, grammar_stride], bit v % 32 of word v / 32; NULL:
 *          no masks.
 * Token ids outside 0 .. vocab - 1 are ignored.  Rows of no request get the
 * grammar mask only.  Deterministic.  n_rows == 0 or vocab == 0 queues
 * nothing.  Errors: QK_ERR_SHAPE, QK_ERR_NULL, QK_ERR_ALIGN, QK_ERR_ARG. */
qk_status qk_logits_process(const void* logits, int dtype, int64_t n_rows, int64_t vocab, int64_t row_stride,
                            const int32_t* cu, int64_t n_req, const int32_t* hist, int64_t hist_stride,
                            const int32_t* hist_len, const float* rep, const float* pres, const float* freq,
                            const int32_t* draft, const uint64_t* mask, const int32_t* bias_tok, const float* bias_val,
                            int64_t bias_stride, const int32_t* bias_len, const uint32_t* grammar, int64_t grammar_stride,
                            void* out, int64_t out_stride, void* stream);

/* Drafted trees judged against the target's probabilities, from given random
 * numbers: the accepted path of every request (as qk_kv_compact wants it), its
 * tokens, and one token more.  Rows cu[r] .. cu[r + 1] - 1 of the logits are
 * the nodes of request r's tree, as in qk_attn_tree and qk_logits_process; row
 * i of them predicts what follows node i.  Node 0 is the root (a token that
 * stands already), the parent of another node is its nearest ancestor: the
 * highest bit of its mask below its own (mask NULL: a chain).  Nodes without an
 * ancestor, and nodes past QK_TREE_MAX of a request, are never reached.
 * With e_v = exp((x_v - max x) / temp[r]) for the logits x of the node that the
 * path has reached (fp32; in sums each weight counts as a whole number of 2^-46
 * of the largest, for more than 65,536 tokens of 2^-45 and so on, so that they
 * depend on the row alone; comparisons are in 64 bits), its children are tried by
 * rising index; child c with token y = draft[c] is taken when
 *   u_accept[c] * q_y * sum_v W_v < W_y,
 * probs NULL (drafts picked without probabilities): q = 1, and W = e without
 *   the tokens of the children refused before;
 * probs given: q = the node's row of probs, the probabilities that its
 *   children were drawn from (each on its own), and W_v = max(e_v - tau q_v, 0)
 *   with tau (as fp32) the sum of the sums of W at the refusals before.
 * Where none is taken, the token after the path is the first v with
 * sum_{v' <= v} W_v' > u_sample[r] * sum W (of e, where W has nothing left).  So
 * with u uniform in [0, 1) the tokens are distributed as the target's, whatever
 * was drafted.  A temperature below 2^-20 (or NaN) is greedy: the child that
 * carries the largest logit's token (the lowest of equals), and that token at
 * the end.
 *   logits [n_rows, vocab], dtype QK_OUT_F32 or QK_OUT_BF16, aligned to the
 *          element, row_stride elements from row to row.  NaN counts as -inf; a
 *          row with +inf has its mass there; a row of -inf only gives the
 *          token -1 and no child.
 *   draft  int32 [n_rows]; tokens outside 0 .. vocab - 1 are refused.
 *   probs  fp32 [n_rows, vocab], probs_stride elements from row to row, or NULL.
 *   temp, u_sample fp32 [n_req]; u_accept fp32 [n_rows].
 *   path   int32 [n_req, path_stride]: the path's nodes from the root on;
 *          tokens int32, the same shape: the tokens of path[1], path[2], .. and
 *          the token after the path; n_path int32 [n_req] of each (0 for a
 *          request without rows); entries behind them are -1.  A path ends at
 *          path_stride nodes (the last one's children are then not tried).
 *   ws     at least qk_verify_workspace(..) bytes (0 for some sizes: ws may
 *          then be NULL), 16-byte aligned.
 * Deterministic.  n_req == 0 queues nothing.  n_req is at most 2^27.
 * Errors: QK_ERR_SHAPE (also vocab or path_stride below 1), QK_ERR_NULL,
 * QK_ERR_ALIGN, QK_ERR_ARG, QK_ERR_WORKSPACE. */
size_t qk_verify_workspace(int64_t n_rows, int64_t n_req, int64_t vocab);
qk_status qk_verify_tree(const void* logits, int dtype, int64_t n_rows, int64_t vocab, int64_t row_stride, const int32_t* cu,
                         int64_t n_req, const int32_t* draft, const uint64_t* mask, const float* temp, const float* u_accept,
                         const float* u_sample, const float* probs, int64_t probs_stride, int32_t* path, int64_t path_stride,
                         int32_t* n_path, int32_t* tokens, void* ws, size_t ws_bytes, void* stream);

/* Test hook: unpack nblocks consecutive blocks into their integer fields.
 *   codes int16 [nblocks * block_elems]: Q4_K 0..15, Q5_K 0..31, Q6_K 0..63,
 *         Q8_0 -128..127, Q5_0 0..31, Q4_0 0..15, Q2_K 0..3, Q3_K -4..3.
 *   sc    int16 [nblocks * 16]: Q4_K / Q5_K 6-bit scales in slots 0..7, Q6_K
 *         the sixteen int8 scales, Q2_K the 4-bit scales, Q3_K the scales
 *         (-32..31); other slots and types 0.
 *   mins  uint8 [nblocks * 16]: Q4_K / Q5_K 6-bit mins (8 used), Q2_K 4-bit
 *         mins; 0 elsewhere.
 *   d, dmin fp32 [nblocks]: the decoded binary16 fields (dmin 0 unless the
 *         type has one: Q4_K, Q5_K, Q2_K).
 * All outputs device memory, any may be NULL.  W 16-byte aligned. */
qk_status qk_unpack(int type, const void* W, int64_t nblocks, int16_t* codes,
                    int16_t* sc, uint8_t* mins, float* d, float* dmin, void* stream);

/* Test hook: the most (token, expert) pairs, 4 or 8, that qk_moe_ffn multiplies
 * an expert's weights with at a time, in its gate and up products (down == 0) or
 * its down product, for these sizes on a GPU of `sms` SMs (0: the current
 * device's).  0 for sizes that the call refuses, and for no tokens. */
int qk_test_moe_group(int type, int type_down, int n_exp, int64_t rows, int64_t cols, int k, int64_t n_tok, int down, int sms);

/* Diagnostic of the failure-detection path; the pages have no counterpart.
 * Every mbarrier wait inside the library's kernels is bounded (2 s): when it
 * runs out the kernel records a timeout in the device status word, drains
 * its copies in flight, releases its tensor memory and returns, so the
 * context stays usable.  This call queues one thread that waits, through
 * the same bounded wait, on a barrier nothing arrives on, with the limit
 * shortened to limit_us microseconds (1 .. 10,000,000; else QK_ERR_ARG).
 * Afterwards qk_device_status() reports QK_ERR_TIMEOUT (and clears it). */
qk_status qk_test_stalled_wait(uint32_t limit_us, void* stream);

/* The same inside attention: qk_attn_tree in which each CTA's copies of V stop
 * before its tile number `tile` (from 0, counted over its units) and the wait
 * for them is limited to limit_us (1 .. 2,000,000; else QK_ERR_ARG).  A CTA that
 * comes so far gives up, and the call's results are then invalid; nothing
 * outside out and ws is written. */
qk_status qk_test_attn_tree_stalled(uint32_t limit_us, uint32_t tile, int type, const void* q, int64_t n_tok,
                                    int64_t q_stride, const void* K, const void* V, int64_t n_pages, int page,
                                    const int32_t* table, int64_t table_stride, const int32_t* ctx, const int32_t* cu,
                                    const uint64_t* mask, int64_t n_req, int max_q, int n_heads, int n_kv, int d, float scale,
                                    void* out, int64_t out_stride, void* ws, size_t ws_bytes, void* stream);

/* Synchronize `stream`, then read and clear this device's kernel status
 * word: QK_OK, QK_ERR_TIMEOUT when a bounded wait ran out since the last
 * call (the affected outputs are then invalid), or QK_ERR_ARG when a paged
 * call met a page id or slot outside its pool or qk_logits_process a request
 * with more tokens than it counts. */
qk_status qk_device_status(void* stream);

/* ------------------------------------------------------------------------
 * GGUF container reader (host code; no GPU involved).  The file the blocks
 * come in ("12 -- llama.cpp / GGUF / Local Inference Mastery", "Part 1 --
 * The GGUF format (bit-level)"): header (magic "GGUF", version uint32,
 * tensor_count uint64, metadata_kv_count uint64), metadata entries
 * (length-prefixed key, value type, value), tensor infos (name, n_dims,
 * shape, ggml type, offset), padding to the alignment, tensor data.
 * Versions 2 and 3, little-endian.  The value-type codes (0 u8, 1 i8, 2 u16,
 * 3 i16, 4 u32, 5 i32, 6 f32, 7 bool, 8 string, 9 array, 10 u64, 11 i64,
 * 12 f64), the ggml tensor types (0 F32, 1 F16, 2 Q4_0, 6 Q5_0, 8 Q8_0,
 * 10 Q2_K, 11 Q3_K, 12 Q4_K, 13 Q5_K, 14 Q6_K, 30 BF16 are sized here;
 * others are listed with nbytes 0)
 * and the "general.alignment" key (uint32 power of two, default 32) follow
 * the GGUF specification the page cites.
 * Every length, count and offset is checked against the image before use;
 * a malformed or truncated image gives QK_ERR_FORMAT and no handle.  Tensor
 * data is never copied: qk_gguf_tensor gives a pointer into the image.  A
 * handle is read-only and may be used from several threads. */
typedef struct qk_gguf qk_gguf;

typedef struct {
    const char* name;      /* NUL-terminated, valid while the handle is open      */
    uint32_t n_dims;       /* 1..4                                                */
    int64_t dims[4];       /* dims[0] innermost (a weight matrix: cols, rows); 1 past n_dims */
    uint32_t ggml_type;
    int qk_type;           /* this library's type id (QK_Q4_K ...), -1 for others */
    uint64_t offset;       /* absolute byte offset in the image                   */
    uint64_t nbytes;       /* data bytes; 0 when the type's size is not known here */
    const void* data;      /* image + offset                                      */
} qk_gguf_tensor_info;

/* Open `path` read-only (memory-mapped) and parse it.  *out is NULL on error
 * (QK_ERR_IO, QK_ERR_FORMAT, QK_ERR_NULL). */
qk_status qk_gguf_open(const char* path, qk_gguf** out);
/* Parse an image the caller owns; it must outlive the handle. */
qk_status qk_gguf_parse(const void* data, uint64_t size, qk_gguf** out);
/* Release the handle (and its mapping).  NULL is ignored. */
void qk_gguf_close(qk_gguf* g);

uint32_t qk_gguf_version(const qk_gguf* g);
int64_t qk_gguf_n_kv(const qk_gguf* g);
int64_t qk_gguf_n_tensors(const qk_gguf* g);
uint64_t qk_gguf_alignment(const qk_gguf* g);
uint64_t qk_gguf_data_offset(const qk_gguf* g);   /* start of the tensor data section */
const void* qk_gguf_image(const qk_gguf* g);

/* Metadata entry i (0 .. n_kv-1); the index of `key`, or -1. */
int64_t qk_gguf_find_kv(const qk_gguf* g, const char* key);
const char* qk_gguf_kv_key(const qk_gguf* g, int64_t i);   /* NULL when out of range */
int qk_gguf_kv_type(const qk_gguf* g, int64_t i);          /* -1 when out of range */
/* Scalar values: integers of any width and bools as int64 (a uint64 above
 * INT64_MAX gives QK_ERR_TYPE), floats as double; QK_ERR_TYPE for another
 * type, QK_ERR_ARG for a bad index. */
qk_status qk_gguf_kv_int(const qk_gguf* g, int64_t i, int64_t* v);
qk_status qk_gguf_kv_float(const qk_gguf* g, int64_t i, double* v);
/* A string value (not NUL-terminated: *len bytes), NULL when not a string. */
const char* qk_gguf_kv_str(const qk_gguf* g, int64_t i, uint64_t* len);
/* Arrays: element type and count; element j as int64 / double / string. */
qk_status qk_gguf_kv_array(const qk_gguf* g, int64_t i, int* elem_type, uint64_t* n);
qk_status qk_gguf_kv_array_int(const qk_gguf* g, int64_t i, uint64_t j, int64_t* v);
qk_status qk_gguf_kv_array_float(const qk_gguf* g, int64_t i, uint64_t j, double* v);
const char* qk_gguf_kv_array_str(const qk_gguf* g, int64_t i, uint64_t j, uint64_t* len);

/* Tensor i (0 .. n_tensors-1); the index of `name`, or -1. */
int64_t qk_gguf_find_tensor(const qk_gguf* g, const char* name);
qk_status qk_gguf_tensor(const qk_gguf* g, int64_t i, qk_gguf_tensor_info* info);

/* Text of the last error on the calling thread ("" if none). */
const char* qk_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* QK_H_ */
