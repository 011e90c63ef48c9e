/*
 * qll.h -- C ABI of libqll.so, the quantized linear layer y = x.W^T for one
 * AMD Instinct MI355X (gfx950).
 *
 * Sources (web pages, cited by title and section):
 *  [CPU]   llama.cpp visual guide, lesson 31 "CPU backend", section "How the
 *          quantized dot product works" (block_q4_0, the Q4_0 x Q8_0 dot).
 *  [FAST]  Fucina course "Chapter 06 -- Going fast on CPUs": 6.1 "Where the
 *          time goes" (GEMM naming, decode is bandwidth-bound, prefill is
 *          compute-bound), 6.3 "The kernel contract: small, unchecked,
 *          allocation-free", 6.4 "The scalar backend is the specification".
 *  [BACK]  Fucina reference "Backends": 9.2 (the kernel contract: validate
 *          once above, kernels below are unchecked), 9.7 "Quantized matmul
 *          dispatch" (per-call Q8_0 activation quantization; pre-quantized
 *          LHS entries), 9.9 "GPU offload" (an entry reports that it did not
 *          run instead of failing silently).
 *  [LOOM]  Loom "Plan 9 SIMD Forward", section "BitNet ternary MAD kernel".
 *
 * Conventions shared by every entry point
 *  - Data pointers are DEVICE pointers owned by the caller.  The library never
 *    allocates, frees or retains them.  Base addresses must be 16-byte aligned
 *    (every PyTorch/hipMalloc allocation is).  Tensors are dense, row-major.
 *  - `stream` is a hipStream_t passed as `void *` (NULL = the default stream),
 *    so that this header needs no HIP include.  Every call checks
 *    its arguments on the host in O(1), enqueues its kernel(s) on `stream` and
 *    returns without synchronising.  On error nothing is enqueued.  Faults
 *    during execution surface at the caller's next synchronisation.
 *  - Return value: QLL_OK (0) or a negative QLL_ERR_* code; qll_status_string
 *    names it.  Argument checks run before any HIP call, so an invalid call
 *    never touches the device.
 *  - Calls are reentrant; the library keeps no mutable global state besides
 *    a once-per-device architecture check.  Output buffers must not overlap
 *    inputs.
 *  - Not checked (undefined): NaN/Inf inputs, Q4_0 codes > 15 or ternary
 *    codes > 2 handed to the pack entries (the low bits are used), ternary
 *    code 3 inside packed words, act_sum inconsistent with xq.
 *
 * Byte formats (little-endian, packed)
 *  - block_q4_0 (18 B): u16 d (IEEE binary16 bits), u8 qs[16].  Element t < 16
 *    is the low nibble of qs[t], element t >= 16 the high nibble of qs[t-16];
 *    weight = d * (code - 8)  [CPU].
 *  - block_q8_0 (34 B): u16 d (binary16), int8 qs[32]; value ~ d * qs.
 *  - Q4_0 weights W: [n][k/32] blocks, row j = output feature j.
 *    Q8_0 activations X: [m][k/32] blocks.
 *  - Ternary weights: uint32 [n][k/16]; code s of a word (s = 0..15, weight
 *    index 16*word + s) sits at bits 2s..2s+1; code = weight + 1 in {0,1,2}
 *    [LOOM].
 */
#ifndef QLL_H
#define QLL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    QLL_OK = 0,
    QLL_ERR_NULL = -1,      /* a required pointer is NULL */
    QLL_ERR_SHAPE = -2,     /* a size is < 1, not a multiple of the block, or too large */
    QLL_ERR_ALIGN = -3,     /* a base address is not 16-byte aligned */
    QLL_ERR_WORKSPACE = -4, /* ws is NULL or smaller than qll_workspace_bytes() */
    QLL_ERR_LAUNCH = -5,    /* the HIP launch itself failed */
    QLL_ERR_DEVICE = -6,    /* no usable device, or the current device is not gfx950 */
    QLL_ERR_SCRATCH = -7,   /* qll_q4_0_q8_0_gemm_noalloc: the shape needs more than its static scratch */
    QLL_ERR_VALUE = -8      /* an argument that is not a size has a value outside its documented set */
};

/* Operations that may need a caller-owned device workspace. */
enum {
    QLL_OP_SGEMM = 1,
    QLL_OP_Q4_0_Q8_0_GEMM = 2,
    QLL_OP_TERNARY_GEMM = 3,
    QLL_OP_Q4_0_REPACKED_GEMM = 4,
    QLL_OP_Q8_0_REPACKED_GEMM = 5,
    QLL_OP_GEMM_NT_BF16 = 6, /* qll_gemm_nt with QLL_DTYPE_BF16 weights */
    QLL_OP_GEMM_NT_F16 = 7,  /* qll_gemm_nt with QLL_DTYPE_F16 weights on the bf16 matrix core */
    QLL_OP_GEMM_NT_F32 = 8,  /* qll_gemm_nt with QLL_DTYPE_F32 weights on the bf16 matrix core */
    QLL_OP_SGEMM_BF16 = 9,   /* qll_sgemm at m > 1 on the bf16 matrix core */
    QLL_OP_Q4_0_GEMV_F32 = 10, /* qll_q4_0_q8_0_gemv_f32's optional workspace */
    QLL_OP_Q4_0_LINEAR = 11,         /* qll_q4_0_q8_0_linear (the repacked form: QLL_OP_Q4_0_REPACKED_GEMM) */
    QLL_OP_Q4_0_GATED = 12,          /* qll_q4_0_q8_0_gated */
    QLL_OP_Q4_0_REPACKED_GATED = 13, /* qll_q4_0_repacked_q8_0_gated */
    QLL_OP_TOKEN_LOGPROBS = 14       /* qll_token_logprobs: n is its v, k its top */
};

/* Bytes of device workspace `op` needs at this shape (0 if none); SIZE_MAX if
 * the shape is invalid. */
size_t qll_workspace_bytes(int op, int64_t m, int64_t n, int64_t k);

/* Element types of the weights of qll_gemm_nt. */
enum { QLL_DTYPE_F32 = 0, QLL_DTYPE_BF16 = 1, QLL_DTYPE_F16 = 2 };

/* Activations of the linear and gated entries: none, max(x, 0),
 * x Phi(x) (the erf form), 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))),
 * x / (1 + exp(-x)). */
enum { QLL_ACT_NONE = 0, QLL_ACT_RELU = 1, QLL_ACT_GELU = 2, QLL_ACT_GELU_TANH = 3, QLL_ACT_SILU = 4 };

/* Static string naming a status code. */
const char *qll_status_string(int status);

/* ---------------------------------------------------------------- packing */

/* Encode Q4_0 weights on the device: codes uint8[n][k] (0..15, weight index
 * t of row j at codes[j*k + t]) and scales uint16[n][k/32] (binary16 bits)
 * -> w block_q4_0[n][k/32] in the layout above [CPU].  k % 32 == 0. */
int qll_pack_q4_0(const uint8_t *codes, const uint16_t *d_bits, void *w, int64_t n, int64_t k, void *stream);

/* Encode ternary codes uint8[n][k] (0..2) into uint32[n][k/16], LSB first
 * [LOOM].  k % 16 == 0. */
int qll_pack_ternary(const uint8_t *codes, uint32_t *w, int64_t n, int64_t k, void *stream);

/* ------------------------------------------------- Q4_0 x Q8_0 (decode, prefill) */

/* Quantize f32 activations x[m][k] to Q8_0 blocks xq[m][k/32] ([BACK] 9.7:
 * the activation rows are quantized per call).  Per 32-block: amax = max|x|,
 * d = amax/127 (IEEE f32 division), q = round-half-away(x/d) (IEEE f32
 * division) clamped to +-127, d stored as binary16 rounded to nearest even;
 * a block whose f32 d is 0 stores q = 0.  Bit-exact with the oracle.
 * k % 32 == 0. */
int qll_quantize_q8_0(const float *x, void *xq, int64_t m, int64_t k, void *stream);

/* Decode GEMV (m = 1): y[j] = sum_b f32(dw[j,b]) * f32(dx[b]) * sumi[j,b],
 * sumi[j,b] = sum_t (qw[j,b,t] - 8) * qx[b,t] exact in int32 [CPU]; the float
 * sum over b is accumulated in f32 in an order of the kernel's choosing
 * (tolerance 1e-4 * sum_b |term_b| against an f64 sum).  w: block_q4_0[n][k/32],
 * xq: block_q8_0[k/32], y: float[n].  k % 32 == 0 and k <= 49152 (else
 * QLL_ERR_SHAPE: the activation row is staged in LDS).  Bandwidth-bound: every
 * weight byte is read once ([FAST] 6.1). */
int qll_q4_0_q8_0_gemv(const void *w, const void *xq, float *y, int64_t n, int64_t k, void *stream);

/* Prefill GEMM: Y[m][n] = X.W^T with the same per-block arithmetic as the
 * GEMV for every (i, j).  xq: block_q8_0[m][k/32], w: block_q4_0[n][k/32],
 * y: float[m][n].  k % 32 == 0, and k < 2^24 when m > 8 (else QLL_ERR_SHAPE:
 * the kernels address 32 activation rows, or a 128-row panel, with 32-bit
 * offsets).  ws/ws_bytes: device workspace of at least
 * qll_workspace_bytes(QLL_OP_Q4_0_Q8_0_GEMM, m, n, k) bytes (nonzero for
 * the 128-row GEMM, m > 64): the call first
 * writes the activations there in the matrix-core operand form (exact f16
 * codes, scale bits, bias terms), then split-k partial sums when it splits
 * k; contents on return are unspecified.  m == 1 runs the GEMV kernel;
 * 2 <= m <= 32 (the small-m band that [BACK] 9.9 gates apart from the
 * general GEMM, one row-dot per weight row in 9.9.2) runs kernels that load
 * every weight once for all m rows -- a GEMV-shaped one, or one that forms
 * 16 x 16 tiles of block sums on the int8 matrix core -- and 33 <= m <= 64
 * runs them on groups of at most 32 activation rows;
 * none of these needs a workspace.  At m == 1 the GEMV's limit k <= 49152
 * applies. */
int qll_q4_0_q8_0_gemm(const void *w, const void *xq, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                       size_t ws_bytes, void *stream);

/* Bytes of the static device scratch of qll_q4_0_q8_0_gemm_noalloc (per device). */
#define QLL_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* qll_q4_0_q8_0_gemm for callers that cannot allocate device memory or pass
 * a workspace (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc): the same kernels, the same results bit for bit,
 * with the workspace taken from a static device array of
 * QLL_NOALLOC_SCRATCH_BYTES (64 MiB) that each device holds from the first
 * call until the process ends.  The call itself allocates nothing.  Shapes
 * whose qll_workspace_bytes(QLL_OP_Q4_0_Q8_0_GEMM, m, n, k) exceeds that
 * size return QLL_ERR_SCRATCH with nothing enqueued (every 8B-class layer at
 * m = 512 fits); the small-m kernels (m <= 64, see above) need no scratch.  All calls on one device share its
 * array and leave their contents there: two calls whose executions overlap
 * on one device (different streams, or graphs replayed concurrently) race
 * and give undefined results, so serialise them.  Other arguments and
 * errors as qll_q4_0_q8_0_gemm. */
int qll_q4_0_q8_0_gemm_noalloc(const void *w, const void *xq, float *y, int64_t m, int64_t n, int64_t k,
                               void *stream);

/* Quantize-fused decode: Y[m][n] = Q8_0(X).W^T for 1 <= m <= 8, from the f32
 * activation rows x: float[m][k] ([BACK] 9.7 quantizes the activation per
 * call), quantized to Q8_0 with exactly the arithmetic of qll_quantize_q8_0
 * and dotted with the per-block arithmetic of qll_q4_0_q8_0_gemm.
 * w: block_q4_0[n][k/32], y: float[m][n], k % 32 == 0; QLL_ERR_SHAPE for m
 * outside [1, 8].
 * ws is optional.  Where qll_workspace_bytes(QLL_OP_Q4_0_GEMV_F32, m, n, k)
 * is nonzero and ws (16-byte aligned, caller-owned, contents not preserved)
 * holds at least that many bytes, the rows are quantized once into ws and
 * the kernel qll_q4_0_q8_0_gemm runs for this shape runs on them: two
 * launches from this one call, as fast as the pair, and the result is that
 * of qll_quantize_q8_0 followed by qll_q4_0_q8_0_gemm bit for bit.
 * Otherwise (ws NULL or smaller, or no workspace needed: m == 1 with a short
 * row and a matrix that one pass of the resident workgroups covers) a single
 * GEMV-shaped launch quantizes the rows inside every workgroup, which is
 * faster only at that size: the same Q8_0 codes and block sums, the float
 * sum over the blocks in that kernel's order (bit for bit the pair's result
 * where qll_q4_0_q8_0_gemm also runs a GEMV-shaped kernel: m == 1, k < 256,
 * m == 2 with n >= 8192, m <= 4 with n >= 32768). */
int qll_q4_0_q8_0_gemv_f32(const void *w, const float *x, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                           size_t ws_bytes, void *stream);

/* ------------------------------------- Q4_0 repacked for the matrix core (prefill) */

/* Bytes of the repacked form of Q4_0 weights W[n][k/32] (SIZE_MAX if the
 * shape is invalid): ceil(n/128) * (k/32) * 3328. */
size_t qll_q4_0_repacked_bytes(int64_t n, int64_t k);

/* Load-time repack of Q4_0 weights into the matrix-core operand form (the
 * packed right-hand side of [BACK] 9.7: rewritten once, reused by every
 * call).  w: block_q4_0[n][k/32]; wp: qll_q4_0_repacked_bytes(n, k) bytes,
 * written in full.  Layout, for 128-row tiles t (rows past n are zero) and
 * blocks b, chunk c = t*(k/32) + b: first the codes, 3072 B per chunk at
 * 3072*c -- the six dwords of row r (r < 128) hold the 6-bit e3m2 codes of
 * w = code - 8 for the block's elements 0..31 (element e at bits 6e), dwords
 * 0..3 at 16*r and dwords 4..5 at 2048 + 8*r; then the scales, the binary16
 * d of row r at byte 2*(128*c + r) of that second region.  Lossless: every
 * w in [-8, 7] is exact in e3m2.  k % 32 == 0. */
int qll_q4_0_repack(const void *w, void *wp, int64_t n, int64_t k, void *stream);

/* Prefill GEMM on repacked weights: Y[m][n] = X.W^T with exactly the
 * per-block arithmetic of qll_q4_0_q8_0_gemm (exact int32 block sums [CPU],
 * f32 scaling; tolerance 1e-4 * sum_b |term_b| against an f64 sum), computed
 * on the matrix core's 6-bit block-scaled path.  wp: the output of
 * qll_q4_0_repack for (n, k); xq: block_q8_0[m][k/32]; y: float[m][n];
 * k % 32 == 0 and k < 2^24 (else QLL_ERR_SHAPE: the kernel addresses the
 * blocks of a row with 32-bit offsets), m >= 1.  ws/ws_bytes: at least
 * qll_workspace_bytes(QLL_OP_Q4_0_REPACKED_GEMM, m, n, k) bytes: the call
 * writes the activations there in operand form (6-bit codes of h and l with
 * q = 16h + l, and d), then split-k partial sums when it splits k; contents on
 * return are unspecified. */
int qll_q4_0_repacked_q8_0_gemm(const void *wp, const void *xq, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                                size_t ws_bytes, void *stream);

/* ------------------------------------------- Q4_0 packed for the decode GEMV */

/* Bytes of the decode-packed form of Q4_0 weights W[n][k/32] (SIZE_MAX if the
 * shape is invalid): n * (16 * (k/32) + 16 * ceil(k/256)) -- 18 bytes per
 * block, as the block_q4_0 array, when k % 256 == 0. */
size_t qll_q4_0_decode_packed_bytes(int64_t n, int64_t k);

/* Load-time repack of Q4_0 weights for the decode GEMV (the packed
 * right-hand side of [BACK] 9.7, with aligned 128-bit loads in place of the
 * 18-byte block stride).  w: block_q4_0[n][k/32]; wp:
 * qll_q4_0_decode_packed_bytes(n, k) bytes, written in full.  Layout, row j
 * at j * (16 * nb + 16 * ceil(nb/8)) with nb = k/32: the nb blocks' 16 nibble
 * bytes (their Q4_0 order) at 16 * b, then their binary16 d at 16 * nb + 2 * b,
 * the scale plane padded with zeros to a multiple of 16 bytes.  k % 32 == 0. */
int qll_q4_0_decode_pack(const void *w, void *wp, int64_t n, int64_t k, void *stream);

/* Decode GEMV on decode-packed weights: y[n] = x.W^T, the arithmetic of
 * qll_q4_0_q8_0_gemv per block (exact int32 block sum, f32 d_w*d_x scaling,
 * tolerance 1e-4 * sum_b |term_b| against an f64 sum; the order of the f32
 * sum differs, so the two are not equal bit for bit).  wp: the output of
 * qll_q4_0_decode_pack for (n, k); xq: block_q8_0[k/32]; y: float[n];
 * k % 32 == 0 and k <= 49152 (the activation row is staged whole in LDS). */
int qll_q4_0_decode_packed_q8_0_gemv(const void *wp, const void *xq, float *y, int64_t n, int64_t k, void *stream);

/* ------------------------------------------------ Q8_0 weights x Q8_0 activations */

/* Weights quantized to Q8_0 blocks too ([BACK] 9.7: a Q8_0-quantized
 * right-hand side against the per-call Q8_0 activation).  Per output and
 * block: sumi = sum_t qw[t] * qx[t] exact in int32, term = f32(dw) * f32(dx)
 * * sumi, summed in f32 (tolerance 1e-4 * sum_b |term_b| against an f64
 * sum).  Weight codes may take the whole int8 range. */

/* Decode GEMV (m = 1): w: block_q8_0[n][k/32], xq: block_q8_0[k/32],
 * y: float[n].  k % 32 == 0 and k <= 49152 (the activation row is staged in
 * LDS).  Bandwidth-bound: every weight byte is read once. */
int qll_q8_0_q8_0_gemv(const void *w, const void *xq, float *y, int64_t n, int64_t k, void *stream);

/* Bytes of the repacked form of Q8_0 weights W[n][k/32] (SIZE_MAX if the
 * shape is invalid): ceil(n/128) * (k/32) * 6400. */
size_t qll_q8_0_repacked_bytes(int64_t n, int64_t k);

/* Load-time repack of Q8_0 weights into the matrix-core operand form
 * ([BACK] 9.7's packed RHS): every code is split exactly as q = 16h + l with
 * l in [-8, 7] and h in [-8, 8] (both e3m2 values).  Layout, for 128-row
 * tiles t (rows past n are zero) and blocks b, chunk c = t*(k/32) + b: the
 * codes first, 6144 B per chunk at 6144*c -- the six dwords of e3m2 codes of
 * h for row r at 16*r (dwords 0..3) and 2048 + 8*r (dwords 4..5), the same
 * for l at 3072 + 16*r and 5120 + 8*r, element e at bits 6e -- then the
 * binary16 d of row r at byte 2*(128*c + r) of the scale region.  Lossless.
 * w: block_q8_0[n][k/32]; wp: qll_q8_0_repacked_bytes(n, k) bytes, written
 * in full.  k % 32 == 0. */
int qll_q8_0_repack(const void *w, void *wp, int64_t n, int64_t k, void *stream);

/* Prefill GEMM on repacked Q8_0 weights: Y[m][n] = X.W^T with the per-block
 * arithmetic above, the exact block sum taken by two 6-bit block-scaled MFMAs
 * (16 h_w and l_w against 16 h_x + l_x).  wp: the output of qll_q8_0_repack;
 * xq: block_q8_0[m][k/32]; y: float[m][n]; k % 32 == 0 and k < 2^24 (else
 * QLL_ERR_SHAPE), m >= 1.  ws/ws_bytes: at least
 * qll_workspace_bytes(QLL_OP_Q8_0_REPACKED_GEMM, m, n, k) bytes
 * (prepared activations, then split-k partials); contents on return are
 * unspecified. */
int qll_q8_0_repacked_q8_0_gemm(const void *wp, const void *xq, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                                size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- f32 */

/* C[m][n] = A[m][k] . B[k][n], all f32 row-major (the plain orientation of
 * [FAST] 6.4), accumulated in f32 (tolerance 1e-5 * sum_p |a*b| against an
 * f64 sum).  m == 1 runs a split-k GEMV whose partial sums go to ws in a
 * fixed order (results are bit-identical from run to run) and takes n < 2^30; ws: at
 * least qll_workspace_bytes(QLL_OP_SGEMM, 1, n, k) bytes.  m > 1 runs on the bf16
 * matrix core when ws holds at least qll_workspace_bytes(QLL_OP_SGEMM_BF16, m,
 * n, k) bytes and k % 16 == 0 (the workspace size selects the algorithm, as
 * in BLAS libraries): A and B (transposed on the way) are each split exactly
 * into three bf16 parts and the part products a_i b_j with i + j <= 4 are
 * accumulated (each one left out is at most 2^-27 of a * b); otherwise (ws
 * NULL or smaller) on the f32 matrix core.  Contents of ws on return
 * unspecified. */
int qll_sgemm(const float *a, const float *b, float *c, int64_t m, int64_t n, int64_t k, void *ws, size_t ws_bytes,
              void *stream);

/* Transposed-B GEMM, the linear layer's own orientation ([FAST] 6.6: W stored
 * [n][k], each output a two-stream dot): Y[m][n] = X[m][k] . W^T, x f32
 * row-major, w of element type w_dtype (QLL_DTYPE_F32, _BF16 or _F16)
 * row-major [n][k], y f32 [m][n].  bf16 and f16 weights are used exactly as
 * stored ([FAST] on reduced precision: bf16 is the top half of an f32; f16 is
 * converted once per load) and never written back as f32; the activations are
 * never rounded; accumulation in f32 (tolerance 1e-5 * sum_p |x * w| against
 * an f64 sum).  m == 1 runs a row-dot GEMV (bandwidth-bound: W is read once).
 * m > 1 runs a matrix-core GEMM: on the f32 matrix core with the weights
 * widened in registers, or, when k % 16 == 0, on the bf16 matrix core with
 * every activation split exactly into three bf16 parts: bf16 weights as
 * stored (each bf16 x bf16 product is exact in f32, so the same products are
 * accumulated), and, when a workspace is passed, f16 weights split exactly
 * into two bf16 parts and f32 weights into three, accumulating the part
 * products x_i w_j with i + j <= 4 (five of six, resp. six of nine; each one
 * left out is at most 2^-27 of x * w).  Any k >= 1.  ws/ws_bytes: bf16
 * weights need at least qll_workspace_bytes(QLL_OP_GEMM_NT_BF16, m, n, k)
 * bytes (the split activations and, when K is split, partial sums; 0 when
 * that path does not run); f16 and f32 weights take the bf16 matrix core when
 * ws holds at least qll_workspace_bytes(QLL_OP_GEMM_NT_F16, resp.
 * QLL_OP_GEMM_NT_F32, m, n, k) bytes (also the weight planes, 2 bytes per
 * weight and plane), and the f32 matrix core otherwise (ws NULL or smaller).
 * Contents on return unspecified.  QLL_ERR_SHAPE for an unknown w_dtype. */
int qll_gemm_nt(const float *x, const void *w, int w_dtype, float *y, int64_t m, int64_t n, int64_t k, void *ws,
                size_t ws_bytes, void *stream);

/* ---------------------------------------------------------------- ternary */

/* Per-row int8 activations [LOOM]: act_scale[i] = 127 / max|x[i,:]| (IEEE
 * f32), xq = round-half-away(x * act_scale) (f32 product) clamped to +-127,
 * act_sum[i] = sum_t xq[i,t].  A row whose amax is 0 or whose scale is not
 * finite gets xq = 0, act_scale = 0, act_sum = 0.  Bit-exact with the oracle.
 * x: float[m][k], xq: int8[m][k], act_scale: float[m], act_sum: int32[m].
 * Any k >= 1. */
int qll_quantize_i8_rows(const float *x, int8_t *xq, float *act_scale, int32_t *act_sum, int64_t m, int64_t k,
                         void *stream);

/* Ternary linear [LOOM]: dot[i,j] = sum_t code[j,t] * xq[i,t] - act_sum[i]
 * (exact int32; equal to sum_t (code - 1) * xq by the ternary identity), then
 * y[i,j] = dot * w_scale / act_scale[i] (0 where act_scale[i] == 0).
 * w: uint32[n][k/16], xq: int8[m][k], y: float[m][n].  k % 16 == 0.
 * The GEMV is the m = 1 case (qll_ternary_gemm with m == 1 runs it): there
 * k <= 65536 (else QLL_ERR_SHAPE: the activation row is staged in LDS). */
int qll_ternary_gemv(const uint32_t *w, float w_scale, const int8_t *xq, const float *act_scale,
                     const int32_t *act_sum, float *y, int64_t n, int64_t k, void *stream);
int qll_ternary_gemm(const uint32_t *w, float w_scale, const int8_t *xq, const float *act_scale,
                     const int32_t *act_sum, float *y, int64_t m, int64_t n, int64_t k, void *stream);

/* ------------------------------------- Q4_0 linear layer with its epilogue */

/* Y[m][n] = act(X.W^T + bias) + residual, the products those of
 * qll_q4_0_q8_0_gemm (the same kernels, limits on k and workspace, which
 * QLL_OP_Q4_0_LINEAR names) and the epilogue applied to each f32 sum before
 * it is stored: bias float[n] or NULL, act a QLL_ACT_* value, residual
 * float[m][n] or NULL.  residual may be y itself (an accumulation in place);
 * otherwise y must not overlap an input.  Without bias, activation and
 * residual the result is that of qll_q4_0_q8_0_gemm bit for bit up to m = 16;
 * above, the order of the f32 sum can differ, and from m = 17 on small and
 * middle-sized matrices this entry is the faster one (m = 128, 1024 -> 1024: 4.3
 * against 19.5 us), since the plain one keeps its bits.
 * QLL_ERR_VALUE for an unknown act. */
int qll_q4_0_q8_0_linear(const void *w, const void *xq, const float *bias, int act, const float *residual, float *y,
                         int64_t m, int64_t n, int64_t k, void *ws, size_t ws_bytes, void *stream);

/* The same on weights repacked by qll_q4_0_repack: the products of
 * qll_q4_0_repacked_q8_0_gemm, its limits and its workspace. */
int qll_q4_0_repacked_q8_0_linear(const void *wp, const void *xq, const float *bias, int act, const float *residual,
                                  float *y, int64_t m, int64_t n, int64_t k, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------ Q4_0 gated projection (GLU) */

/* Y[m][n] = act(X.Wg^T) * (X.Wu^T), the two projections of a gated
 * feed-forward block and their product in one kernel: neither projection is
 * written to memory.  wg, wu: block_q4_0[n][k/32]; xq: block_q8_0[m][k/32];
 * y: float[m][n]; each product with the arithmetic of qll_q4_0_q8_0_gemm
 * (exact int32 block sums, f32 scaling).  k % 32 == 0 and k < 2^24.
 * ws/ws_bytes: at least qll_workspace_bytes(QLL_OP_Q4_0_GATED, m, n, k) bytes
 * (0 for m <= 64 with k >= 256, for m == 1 and for other small products);
 * contents on return are unspecified. */
int qll_q4_0_q8_0_gated(const void *wg, const void *wu, const void *xq, int act, float *y, int64_t m, int64_t n,
                        int64_t k, void *ws, size_t ws_bytes, void *stream);

/* Bytes of the repacked form of a gate and up pair W[n][k/32] (SIZE_MAX if the
 * shape is invalid): ceil(n/64) * (k/32) * 3328. */
size_t qll_q4_0_repacked_gated_bytes(int64_t n, int64_t k);

/* Load-time repack of a gate and up pair for qll_q4_0_repacked_q8_0_gated: the
 * layout of qll_q4_0_repack with rows 0..63 of 128-row tile t holding rows
 * 64 t .. 64 t + 63 of wg and rows 64..127 the same rows of wu (rows past n
 * zero).  wp: qll_q4_0_repacked_gated_bytes(n, k) bytes, written in full. */
int qll_q4_0_repack_gated(const void *wg, const void *wu, void *wp, int64_t n, int64_t k, void *stream);

/* qll_q4_0_q8_0_gated on a repacked pair, on the 6-bit matrix-core path of
 * qll_q4_0_repacked_q8_0_gemm.  m >= 1; ws/ws_bytes: at least
 * qll_workspace_bytes(QLL_OP_Q4_0_REPACKED_GATED, m, n, k) bytes. */
int qll_q4_0_repacked_q8_0_gated(const void *wp, const void *xq, int act, float *y, int64_t m, int64_t n, int64_t k,
                                 void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------- norms into activations */

/* Residual sum, root-mean-square norm and quantization of the stream in one
 * pass, the step before a linear layer.  For every row
 *     h = T(f32(x) + f32(residual))   (h = x where residual is NULL)
 *     v_t = h_t * weight_t / rms,  rms = sqrt(sum_t h_t^2 / k + eps)
 * with T the stream's type `dtype` (QLL_DTYPE_F32, _BF16 or _F16; the sum is
 * rounded to it once, to nearest even, and the norm is taken of the rounded
 * sum).  h, where not NULL, receives the sum; it may be x or residual itself
 * (the update in place) and must not overlap an input otherwise.  x,
 * residual, h: [m][k] of type T; weight: float[k], finite; eps >= 0 and finite (else
 * QLL_ERR_VALUE, like an unknown dtype).  k < 2^24 (else QLL_ERR_SHAPE, as in
 * the GEMMs that take the result).
 *
 * The codes are those of exact products and a correctly rounded f64 quotient:
 * with p_t = h_t * weight_t and A = max |p_t| over the block (or row),
 *     q_t = round-half-away(127 * p_t / A)      (0 where A is 0)
 * -- rms cancels from them -- so they do not depend on how a kernel splits
 * the row.  Against qll_quantize_q8_0 on an f32 v they can differ by one at
 * values within f32 rounding of a border. */

/* Q8_0 blocks: d = binary16(f32(A / (127 rms))) per 32-block.  xq:
 * block_q8_0[m][k/32].  k % 32 == 0.  In a row whose h has NaN or an infinity in
 * it, d is NaN in every block, and the codes are unspecified. */
int qll_rmsnorm_q8_0(const void *x, int dtype, const void *residual, const float *weight, float eps, void *h,
                     void *xq, int64_t m, int64_t k, void *stream);

/* int8 rows: act_scale = f32(127 rms / A) and act_sum = sum_t q_t per row; a
 * row with A = 0, or whose act_scale is not finite (one with NaN or an infinity
 * in its h among them), gets q = 0, act_scale = 0 and act_sum = 0.  xq: int8[m][k], act_scale: float[m], act_sum: int32[m].
 * Any k >= 1. */
int qll_rmsnorm_i8_rows(const void *x, int dtype, const void *residual, const float *weight, float eps, void *h,
                        int8_t *xq, float *act_scale, int32_t *act_sum, int64_t m, int64_t k, void *stream);

/* ------------------------------------------------- token log probabilities */

/* What is read off the logits of a vocabulary projection.  For every row
 * x[0..v) of logits: [m][v] of type dtype (QLL_DTYPE_F32, _BF16 or _F16), with
 * M = max x, S = sum_j exp(x_j - M) and log p_j = x_j - M - log S:
 *   logprob[m][t]      log p of the row's t given tokens (int32 ids); NaN for
 *                      an id outside [0, v) (padding), which is not read
 *   entropy[m]         -sum_j p_j log p_j, in nats
 *   top_ids[m][top],   the `top` largest logits, largest first, the lower
 *   top_logprob        index first among equal ones, and their log p
 * t == 0 leaves tokens and logprob unused (may be NULL), top == 0 top_ids and
 * top_logprob; entropy may be NULL.  A logit of -inf is a masked token: p = 0,
 * log p = -inf.  In a row with nothing but -inf, or with NaN or +inf in it,
 * every float output is NaN (its top_ids are the lowest indices, resp.
 * unspecified ids below v).
 * Sums are f32 over eight or sixteen logits and f64 beyond; every float output is
 * within 2^-18 (1 + |value|) of the exact one (the largest error measured, over
 * random, flat, rising and masked rows, is 2^-20 (1 + |value|)).  1 <= v <= 2^20, t >= 0,
 * 0 <= top <= min(64, v) (else QLL_ERR_SHAPE); QLL_ERR_VALUE for an unknown
 * dtype.  ws/ws_bytes: at least qll_workspace_bytes(QLL_OP_TOKEN_LOGPROBS, m,
 * v, top) bytes; contents on return are unspecified. */
int qll_token_logprobs(const void *logits, int dtype, const int32_t *tokens, int64_t t, float *logprob,
                       float *entropy, int64_t top, int32_t *top_ids, float *top_logprob, int64_t m, int64_t v,
                       void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLL_H */
