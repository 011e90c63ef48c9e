// Internal header of libqll.so: device helpers shared by the kernels and the
// launcher declarations called by the C-ABI layer (abi.hip).  Kernels below
// the ABI are unchecked: the ABI validates shapes, pointers and alignment
// once, then launches (the kernel contract of Fucina course "Chapter 06 --
// Going fast on CPUs", 6.3).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qll {

// 16-byte vector of dwords that only promises 4-byte alignment: global
// dwordx4 loads need no more on gfx950, and the 18- and 34-byte block formats
// only give dword alignment for pairs of blocks.
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float half_bits_to_float(uint32_t bits)
{
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(bits & 0xffffu));
}

// f32 -> binary16 bits, round to nearest even (v_cvt_f16_f32 in the default
// rounding mode).
__device__ __forceinline__ uint16_t float_to_half_bits(float f)
{
    return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// Low 32 bits of ({hi, lo} >> s).
__device__ __forceinline__ uint32_t funnel(uint32_t hi, uint32_t lo, uint32_t s)
{
    return __builtin_amdgcn_alignbit(hi, lo, s);
}

// Signed 4x8-bit dot product accumulated into c (v_dot4_i32_i8).
__device__ __forceinline__ int32_t sdot4(uint32_t a, uint32_t b, int32_t c)
{
    return __builtin_amdgcn_sdot4((int32_t)a, (int32_t)b, c, false);
}

__device__ __forceinline__ u32x4 load4_a4(const uint8_t *p)
{
    return *reinterpret_cast<const u32x4_a4 *>(p);
}

// One wave-wide global -> LDS load: lane l reads 16 bytes at base + off (base
// uniform, in scalar registers; the address need only be 2-byte aligned) and the
// wave writes them to LDS at lds + 16 l.  Inline assembly keeps these loads out of
// the compiler's wait bookkeeping, and so out of its hazard bookkeeping too: a load
// that takes its LDS address from M0 has to come one wait state or more after the
// scalar write of M0, which the s_nop is for.
__device__ __forceinline__ void lds_dma16(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16(const void *base, uint32_t off,
                                          const __attribute__((address_space(3))) void *lds)
{
    lds_dma16(base, off, (uint32_t)(uintptr_t)lds);
}
// The same with two bytes a lane, zero-extended to lds + 4 l.
__device__ __forceinline__ void lds_dma2(const void *base, uint32_t off,
                                         const __attribute__((address_space(3))) void *lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ushort %0, %1" ::"v"(off), "s"(base),
                 "s"((uint32_t)(uintptr_t)lds)
                 : "memory", "m0");
}

// Q8_0 code of x for the block scale d (IEEE f32 division, ties away from
// zero, clamped to +-127; d = 0 gives 0).
__device__ __forceinline__ int quant_code(float x, float d)
{
    if (d == 0.0f)
        return 0;
    float r = roundf(x / d);
    r = fminf(fmaxf(r, -127.0f), 127.0f);
    return (int)r;
}

// Q8_0 block at byte offset o of `base` (o % 4 is 0 or 2) -> binary16 d bits
// and the 32 int8 codes as 8 dwords.  Reads only bytes of this block and, when
// o % 4 == 2, the two bytes before it (inside the same buffer, since o >= 34).
__device__ __forceinline__ void load_q8_0_block(const uint8_t *base, int64_t o, uint32_t &d, uint32_t q[8])
{
    if ((o & 3) == 0) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(base + o);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            w[i] = p[i];
        uint32_t tail = *reinterpret_cast<const uint16_t *>(base + o + 32);
        d = w[0] & 0xffffu;
#pragma unroll
        for (int i = 0; i < 7; i++)
            q[i] = funnel(w[i + 1], w[i], 16);
        q[7] = funnel(tail, w[7], 16);
    } else {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(base + o - 2);
        uint32_t w0 = p[0];
        d = w0 >> 16;
#pragma unroll
        for (int i = 0; i < 8; i++)
            q[i] = p[i + 1];
    }
}

// ------------------------------------------------------------ epilogues

// Activations of the fused linear and gated entries (the ABI's QLL_ACT_*).
enum { QLL_A_NONE = 0, QLL_A_RELU = 1, QLL_A_GELU = 2, QLL_A_GELU_TANH = 3, QLL_A_SILU = 4 };

// x / (1 + exp(-t)) with the hardware's exp2 and reciprocal (each within about
// one unit in the last place; exp2's argument rounding adds |t| 2^-24 relative
// where exp(-t) counts): exp(-t) = inf gives x * 0.
__device__ __forceinline__ float times_sigmoid(float x, float t)
{
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * t));
}

__device__ __forceinline__ float act_relu(float x) { return x < 0.0f ? 0.0f : x; } // NaN stays
// x Phi(x) = x - h for x >= 0 and h for x < 0, h = x erfc(|x| / sqrt(2)) / 2, with
// erfc(|x| / sqrt(2)) = t 2^(G(t) - x^2 log2(e) / 2), t = 1 / (1 + 0.4 |x|).  G is a
// polynomial fitted to that definition in f64 on |x| <= 14 (beyond, h is below
// 1e-36); with its coefficients in f32 it gives erfc within 2.7e-7 relative, most at
// |x| = 0.05, and within 1e-7 from 1 on.  In f32 the value is within 10 half steps
// (2^-24 relative) from -2 on.  Below, the exponent's rounding counts, up to 0.85 x^2
// of them: 21 down to -5, 83 (5e-6) down to -10.  About 20 instructions; with the
// library's erfcf a kernel of 128 x 128 tiles took 4 us longer (14.2 against 10.2 us
// for one tile of five blocks).
__device__ __forceinline__ float act_gelu(float x)
{
    const float xc = fminf(fmaxf(x, -14.0f), 14.0f), t = __builtin_amdgcn_rcpf(fmaf(0.4f, fabsf(xc), 1.0f));
    float g = 0.27634788f;
    g = fmaf(g, t, -1.4145187f);
    g = fmaf(g, t, 2.825165f);
    g = fmaf(g, t, -2.542245f);
    g = fmaf(g, t, 0.7925071f);
    g = fmaf(g, t, -0.26599124f);
    g = fmaf(g, t, 0.5378745f);
    g = fmaf(g, t, 1.4383701f);
    g = fmaf(g, t, -1.6475099f);
    const float h = 0.5f * xc * (t * __builtin_amdgcn_exp2f(fmaf(-0.72134752f * xc, xc, g)));
    return x < 0.0f ? h : x - h; // NaN: x - h
}
// 0.5 (1 + tanh(u)) = sigmoid(2 u)
__device__ __forceinline__ float act_gelu_tanh(float x)
{
    return times_sigmoid(x, 1.59576912f * (x + 0.044715f * x * x * x));
}
__device__ __forceinline__ float act_silu(float x) { return times_sigmoid(x, x); }

__device__ __forceinline__ float activate(float x, int act)
{
    switch (act) { // uniform
    case QLL_A_RELU: return act_relu(x);
    case QLL_A_GELU: return act_gelu(x);
    case QLL_A_GELU_TANH: return act_gelu_tanh(x);
    case QLL_A_SILU: return act_silu(x);
    default: return x;
    }
}

// The 16 values of a matrix-core tile register group, the choice made once.
template <typename V16>
__device__ __forceinline__ void activate16(V16 &v, int act)
{
    switch (act) { // uniform
    case QLL_A_RELU:
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = act_relu(v[i]);
        break;
    case QLL_A_GELU:
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = act_gelu(v[i]);
        break;
    case QLL_A_GELU_TANH:
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = act_gelu_tanh(v[i]);
        break;
    case QLL_A_SILU:
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = act_silu(v[i]);
        break;
    default: break;
    }
}

// What a product kernel does with output (i, j) of [m][n], as a template
// argument, so that the plain entries keep their kernels.
struct PlainEpilogue { // y = v
    static constexpr bool kLinear = false, kGated = false;
    __host__ __device__ PlainEpilogue rows(int64_t, int64_t) const { return *this; }
};
struct LinearEpilogue { // y = act(v + bias[j]) + res[i][j]; bias and res may be null, res may be y
    static constexpr bool kLinear = true, kGated = false;
    const float *bias, *res;
    int act;
    // the same for rows i0, i0 + 1, ... as rows 0, 1, ...
    __host__ __device__ LinearEpilogue rows(int64_t i0, int64_t n) const { return {bias, res ? res + i0 * n : nullptr, act}; }
};
struct GatedEpilogue { // y = act(v of w) * (v of wu); raw: both products as planes (a k-split's partials)
    static constexpr bool kLinear = false, kGated = true;
    const uint8_t *wu; // null where the weights are interleaved at load time
    int act;
    bool raw;
    __host__ __device__ GatedEpilogue rows(int64_t, int64_t) const { return *this; }
};

template <class EP>
__device__ __forceinline__ float epilogue(const EP &ep, float v, int64_t i, int64_t j, int64_t n)
{
    if constexpr (EP::kLinear) {
        v = activate(ep.bias ? v + ep.bias[j] : v, ep.act);
        return ep.res ? v + ep.res[i * n + j] : v;
    }
    return v;
}

// ------------------------------------------------------------ grids

// A grid has fewer than 2^32 threads in each dimension.  More wrap around without
// an error, and the launch leaves the rest undone.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks * threads < (int64_t)1 << 32; }

// `count` units (rows, blocks) in launches of at most `part`: launch(first, number).
template <class F>
inline hipError_t launch_parts(int64_t count, int64_t part, const F &launch)
{
    for (int64_t first = 0; first < count; first += part) {
        launch(first, count - first < part ? count - first : part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}
constexpr int64_t kPartThreads = (int64_t)1 << 31; // threads of such a launch

// ------------------------------------------------------------ launchers
// Each returns a hipError_t of the launch; arguments are already validated.

hipError_t launch_pack_q4_0(const uint8_t *codes, const uint16_t *d_bits, uint8_t *w, int64_t n, int64_t k,
                            hipStream_t s);
hipError_t launch_pack_ternary(const uint8_t *codes, uint32_t *w, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_quantize_q8_0(const float *x, uint8_t *xq, int64_t nblocks, hipStream_t s);
hipError_t launch_quantize_i8_rows(const float *x, int8_t *xq, float *act_scale, int32_t *act_sum, int64_t m,
                                   int64_t k, hipStream_t s);
hipError_t launch_q4_0_q8_0_gemv(const uint8_t *w, const uint8_t *xq, float *y, int64_t n, int64_t k,
                                 hipStream_t s);
// y[i] = sum of parts[s * count + i] over the splits s, in split order (the
// split-k GEMMs' second launch).
hipError_t launch_sum_splits(const float *parts, float *y, int64_t count, int splits, hipStream_t s);
hipError_t launch_q4_0_q8_0_gemm(const uint8_t *w, const uint8_t *xq, float *y, int64_t m, int64_t n, int64_t k,
                                 void *ws, hipStream_t s);
// Small-m decode: Q8_0 activations at 1 <= m <= 64 (groups of at most 32
// rows above 32; m <= kMaxMSmall when k >= kMaxKMfma), or, in the
// quantize-fused entry, f32 activations quantized to Q8_0 inside the launch
// (1 <= m <= kMaxMSmall).
constexpr int64_t kMaxMSmall = 8;
hipError_t launch_q4_0_q8_0_gemv_m(const uint8_t *w, const uint8_t *xq, float *y, int64_t m, int64_t n, int64_t k,
                                   hipStream_t s);
// Small m on the int8 matrix core (1 <= m <= kMaxMMfma, kMinKMfma <= k <
// kMaxKMfma: a stage is eight blocks, and 32 activation rows are addressed
// with 32-bit offsets): Q8_0 activations, no workspace.
constexpr int64_t kMaxMMfma = 32;
constexpr int64_t kMinKMfma = 256, kMaxKMfma = (int64_t)1 << 24;

// Whether the Q4_0 x Q8_0 GEMM entry runs the small-m kernels (no
// workspace) rather than the 128-row GEMM: m <= 8 at any k; otherwise
// k < kMaxKMfma and m <= 64, above 32 as groups of at most 32 activation
// rows (each group re-reads the weights, which beats the GEMM's padding of m
// to 128 rows up to there: at m = 64, 4096 -> 14336 33 against 44 us,
// 4096 -> 128256 206 against 234 us; at m = 96 the GEMM wins).
inline bool q4_small_m_path(int64_t m, int64_t n, int64_t k)
{
    (void)n;
    return m <= kMaxMSmall || (k < kMaxKMfma && m <= 64);
}
hipError_t launch_q4_0_q8_0_small_m_mfma(const uint8_t *w, const uint8_t *xq, float *y, int64_t m, int64_t n,
                                         int64_t k, hipStream_t s);
// With ws (at least q4_0_gemv_f32_workspace bytes, nonzero), the rows are
// quantized into ws by the quantize kernel and the Q8_0 decode kernel runs
// on them; with ws == nullptr, one launch quantizes inside each workgroup.
hipError_t launch_q4_0_q8_0_gemv_f32(const uint8_t *w, const float *x, float *y, int64_t m, int64_t n, int64_t k,
                                     uint8_t *ws, hipStream_t s);
size_t q4_0_gemv_f32_workspace(int64_t m, int64_t n, int64_t k);
size_t q4_0_q8_0_gemm_workspace(int64_t m, int64_t n, int64_t k);
// The same products with an epilogue, on the same kernels and workspaces.
//
// From 17 rows: groups of 16 rows in one launch.  Up to 64 rows, instead of one
// group of 32 rows after another: more and smaller workgroups count for more than
// reading the weights again (m = 37 in us, 1440 -> 4099 9.4 -> 8.0, 4096 -> 4096 13.2 ->
// 10.5, 8192 -> 8192 38.3 -> 32.3; m = 64, 4096 -> 6144 29.0 -> 18.1), but on tall and large
// matrices, which fill the CUs with 32 rows (14336 x 4096: m = 32 19.0 -> 19.9, m = 37
// 28.8 -> 31.8).  Above 64 rows, instead of the GEMM and its activation prepass and
// split sum, while the work is small (m = 128, 1024 -> 1024 19.5 -> 4.3, 2048 -> 2048 22.2
// -> 7.9, 4096 -> 4096 29.7 -> 20.7; 3.2e9 products are even: m = 192, 4096 -> 4096 34.3
// and 34.2; m = 256 35.9 -> 40.5), and so are the outputs, many of which favour the
// GEMM where k is short (512 -> 4096: m = 512 27.4 -> 19.3, m = 1024 30.1 -> 33.1).
inline bool q4_small_work(int64_t m, int64_t n, int64_t k)
{
    return m <= 4096 && n < 32768 && m * n <= ((int64_t)1 << 21) && m * n <= (((int64_t)3 << 30) - 1) / k;
}
inline bool q4_row_groups(int64_t m, int64_t n, int64_t k)
{
    if (m <= 16 || k < kMinKMfma || k >= kMaxKMfma)
        return false;
    return m <= 64 ? n < 12288 || (n < 32768 && n * k < ((int64_t)1 << 25)) : q4_small_work(m, n, k);
}
// The linear entry without a workspace: those groups, the kernels of the plain
// product up to 64 rows, and groups of eight rows where rows have fewer than eight
// blocks and, above 16 rows, the outputs are few (m = 128, 64 -> 1024 19.3 -> 11.3 us, m = 256 19.6 ->
// 20.4).
inline bool q4_linear_small(int64_t m, int64_t n, int64_t k)
{
    if (m <= kMaxMSmall)
        return true;
    if (k < kMinKMfma)
        return m <= 16 || m * n <= ((int64_t)1 << 18);
    return (m <= 64 && k < kMaxKMfma) || q4_row_groups(m, n, k);
}
hipError_t launch_sum_splits_linear(const float *parts, float *y, int64_t m, int64_t n, int splits,
                                    const LinearEpilogue &ep, hipStream_t s);
hipError_t launch_q4_0_q8_0_gemv_linear(const uint8_t *w, const uint8_t *xq, float *y, int64_t n, int64_t k,
                                        const LinearEpilogue &ep, hipStream_t s);
hipError_t launch_q4_0_q8_0_gemv_m_linear(const uint8_t *w, const uint8_t *xq, float *y, int64_t m, int64_t n,
                                          int64_t k, const LinearEpilogue &ep, hipStream_t s);
hipError_t launch_q4_0_q8_0_small_m_mfma_linear(const uint8_t *w, const uint8_t *xq, float *y, int64_t m, int64_t n,
                                                int64_t k, const LinearEpilogue &ep, hipStream_t s);
hipError_t launch_q4_0_q8_0_gemm_linear(const uint8_t *w, const uint8_t *xq, float *y, int64_t m, int64_t n,
                                        int64_t k, const LinearEpilogue &ep, void *ws, hipStream_t s);
hipError_t launch_q4_0_packed_gemm_linear(const uint8_t *wp, const uint8_t *xq, float *y, int64_t m, int64_t n,
                                          int64_t k, const LinearEpilogue &ep, void *ws, hipStream_t s);
// Gated products y = act(X.Wg^T) * (X.Wu^T): the GEMV at m = 1 up to
// kMaxKQ4Gemv, the small-m matrix-core kernel where q4_gated_small holds
// (groups of at most 32 rows; above 64 rows m = 128, 1024 -> 2 x 1024 19.2 -> 4.9 us, 4096 ->
// 2 x 4096 34.7 -> 29.2; m = 192 44.8 -> 47.4), the 128-row GEMM otherwise.
inline bool q4_gated_small(int64_t m, int64_t n, int64_t k)
{
    return m == 1 || (k >= kMinKMfma && (m <= 64 || q4_small_work(m, n, k)));
}
hipError_t launch_q4_0_gated_gemv(const uint8_t *wg, const uint8_t *wu, const uint8_t *xq, int act, float *y,
                                  int64_t n, int64_t k, hipStream_t s);
hipError_t launch_q4_0_gated_small_m(const uint8_t *wg, const uint8_t *wu, const uint8_t *xq, int act, float *y,
                                     int64_t m, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_sum_splits_gated(const float *parts, float *y, int64_t m, int64_t n, int splits, int act,
                                   hipStream_t s);
size_t q4_0_gated_gemm_workspace(int64_t m, int64_t n, int64_t k);
hipError_t launch_q4_0_gated_gemm(const uint8_t *wg, const uint8_t *wu, const uint8_t *xq, int act, float *y,
                                  int64_t m, int64_t n, int64_t k, void *ws, hipStream_t s);
size_t q4_0_repacked_gated_bytes(int64_t n, int64_t k);
hipError_t launch_q4_0_repack_gated(const uint8_t *wg, const uint8_t *wu, uint8_t *wp, int64_t n, int64_t k,
                                    hipStream_t s);
size_t q4_0_packed_gated_workspace(int64_t m, int64_t n, int64_t k);
hipError_t launch_q4_0_packed_gated(const uint8_t *wp, const uint8_t *xq, int act, float *y, int64_t m, int64_t n,
                                    int64_t k, void *ws, hipStream_t s);
// Decode GEMV with Q8_0 weights.
hipError_t launch_q8_0_q8_0_gemv(const uint8_t *w, const uint8_t *xq, float *y, int64_t n, int64_t k, hipStream_t s);
// Transposed-B (W stored [n][k]) f32 GEMV and GEMM with f32, bf16 or f16
// weights (the values of the ABI's QLL_DTYPE_*).
enum { QLL_W_F32 = 0, QLL_W_BF16 = 1, QLL_W_F16 = 2 };
hipError_t launch_gemv_nt(const float *x, const void *w, int wfmt, float *y, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_sgemm_nt(const float *a, const void *w, int wfmt, float *c, int64_t m, int64_t n, int64_t k,
                           hipStream_t s);
bool gemm_nt_bf16_core_shape(int64_t m, int64_t k);
size_t gemm_nt_workspace(int wfmt, int64_t m, int64_t n, int64_t k);
hipError_t launch_gemm_nt_bf16_mfma(const float *x, const void *w, int wfmt, float *y, int64_t m, int64_t n,
                                    int64_t k, void *ws, hipStream_t s, bool b_kn = false);
// Load-time repack of Q4_0 weights and the GEMM on them (6-bit matrix-core path).
size_t q4_0_repacked_bytes(int64_t n, int64_t k);
// Decode-packed Q4_0 weights (groups of eight blocks: nibbles, then scales).
size_t q4_0_packed_bytes(int64_t n, int64_t k);
hipError_t launch_q4_0_pack_decode(const uint8_t *w, uint8_t *wp, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_q4_0_packed_gemv(const uint8_t *w, const uint8_t *xq, float *y, int64_t n, int64_t k,
                                   hipStream_t s);
hipError_t launch_q4_0_repack(const uint8_t *w, uint8_t *wp, int64_t n, int64_t k, hipStream_t s);
size_t q4_0_packed_gemm_workspace(int64_t m, int64_t n, int64_t k);
hipError_t launch_q4_0_packed_gemm(const uint8_t *wp, const uint8_t *xq, float *y, int64_t m, int64_t n, int64_t k,
                                   void *ws, hipStream_t s);
size_t q8_0_repacked_bytes(int64_t n, int64_t k);
hipError_t launch_q8_0_repack(const uint8_t *w, uint8_t *wp, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_q8_0_packed_gemm(const uint8_t *wp, const uint8_t *xq, float *y, int64_t m, int64_t n, int64_t k,
                                   void *ws, hipStream_t s);
hipError_t launch_sgemv(const float *x, const float *b, float *c, int64_t n, int64_t k, float *ws, hipStream_t s);
size_t sgemv_workspace(int64_t n, int64_t k);
hipError_t launch_sgemm(const float *a, const float *b, float *c, int64_t m, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_ternary_gemv(const uint32_t *w, float w_scale, const int8_t *xq, const float *act_scale,
                               const int32_t *act_sum, float *y, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_ternary_gemm(const uint32_t *w, float w_scale, const int8_t *xq, const float *act_scale,
                               const int32_t *act_sum, float *y, int64_t m, int64_t n, int64_t k, hipStream_t s);

// Residual sum, root-mean-square norm and quantization of the stream (dtype: a
// QLL_W_* value) to Q8_0 blocks or int8 rows; res and h may be null.
hipError_t launch_rmsnorm_q8_0(const void *x, int dtype, const void *res, const float *w, float eps, void *h,
                               uint8_t *xq, int64_t m, int64_t k, hipStream_t s);
hipError_t launch_rmsnorm_i8_rows(const void *x, int dtype, const void *res, const float *w, float eps, void *h,
                                  int8_t *xq, float *act_scale, int32_t *act_sum, int64_t m, int64_t k,
                                  hipStream_t s);
// Token log probabilities, entropy and the `top` best of each row of logits.
constexpr int64_t kMaxLpVocab = (int64_t)1 << 20, kMaxLpTop = 64;
size_t token_logprobs_workspace(int64_t m, int64_t v, int64_t top);
hipError_t launch_token_logprobs(const void *logits, int dtype, const int32_t *tokens, int64_t nt, float *logprob,
                                 float *entropy, int64_t top, int32_t *top_ids, float *top_logprob, int64_t m,
                                 int64_t v, void *ws, hipStream_t s);

// 4-bit weights with group scales (q4g.h has the packed form; fmt: the ABI's
// QLL_Q4G_* bits; dtypes: QLL_W_* values): packing, the linear layer, and the
// experts of a mixture-of-experts layer with the router that chooses them.
size_t q4g_packed_bytes(int64_t n, int64_t k, int64_t group, int fmt);
hipError_t launch_q4g_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int64_t group, int fmt,
                           uint8_t *wp, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_q4g_from_q4_0(const uint8_t *w, uint8_t *wp, int64_t n, int64_t k, hipStream_t s);
hipError_t launch_q4g_linear(const uint8_t *wp, int64_t group, int fmt, const void *x, int dtype, const float *bias,
                             int act, const void *res, void *y, int y_dtype, int64_t m, int64_t n, int64_t k, void *ws,
                             hipStream_t s);
size_t q4g_linear_workspace(int64_t m, int64_t n, int64_t k);
// f32 values (a multiple of eight of them) as three bf16 parts, one after another.
hipError_t launch_q4g_split(const void *x, void *parts, int64_t count, hipStream_t s);
constexpr int64_t kMaxExperts = 1024, kMaxTop = 32;
constexpr int64_t kMaxMoeN = (int64_t)1 << 20; // the experts' inner size: 32-bit offsets into the gated products
size_t moe_route_workspace(int64_t m, int64_t e);
hipError_t launch_moe_route(const void *x, int dtype, const void *w, int w_dtype, const float *bias, int sigmoid,
                            int renorm, float scale, int32_t *ids, float *weights, int64_t top, int64_t m, int64_t e,
                            int64_t k, void *ws, hipStream_t s);
size_t q4g_moe_workspace(int64_t m, int64_t n, int64_t top);
hipError_t launch_q4g_moe(const void *x, int dtype, const int32_t *ids, const float *weights, int64_t top,
                          const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, int64_t group, int fmt, int act,
                          const void *res, void *y, int64_t m, int64_t n, int64_t k, int64_t e, void *ws,
                          hipStream_t s);

// Largest k the LDS-staged decode kernels accept (the activation of one row
// is kept whole in LDS).
constexpr int64_t kMaxKQ4Gemv = 49152;
constexpr int64_t kMaxKTernaryGemv = 65536;

} // namespace qll
