// 4-bit codes with one scale (f16 or bf16) and, where present, one 4-bit zero
// point per group of 32, 64 or 128 weights of a row:
//     w[j][t] = s[j][t / g] * (c[j][t] - z[j][t / g]),   z = 8 where there is none.
// The packed form and the product of one wave on it, shared by the linear
// layer (q4g.hip) and the experts (moe.hip).
//
// Packed form of W[n][k], three regions one after another, each a multiple of
// 256 bytes, for tiles of 16 rows (index rt, rows past n zero) and 128 weights
// (index kt, weights past k zero):
//   codes   tile (rt, kt) at 1024 * (rt * KT + kt), KT = ceil(k / 128): 16 bytes a
//           lane of a wave, lane l holding row l % 16; dword j (matrix-core step j) has the
//           weights 32 j + 8 (l / 16) + 0..7 of the tile, number 2 p at bits 4 p, number
//           2 p + 1 at bits 16 + 4 p, so that a shift and a mask give two neighbours in
//           the halves of a register
//   scales  for chunks of 512 weights (index ks, KS = ceil(k / 512)), 16 rows a chunk and 512 / g
//           scales a row: 1024 / g bytes at (rt * KS + ks) * 16 + row
//   zeros   the same with 4 bits each, lowest first: 256 / g bytes a row
// One wave-wide load of 16 bytes a lane fetches a tile without a gap, and it is four
// operands of the 16 x 16 x 32 matrix instruction as they stand.
#pragma once

#include "common.h"

namespace qll {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kQ4gBf16 = 1, kQ4gZeros = 2; // the ABI's QLL_Q4G_*

struct Q4gShape {
    int64_t rt, kt, ks;                     // tiles of 16 rows, of 128 weights, chunks of 512
    int64_t scales, zeros, bytes;           // byte offsets of the regions, and the end
    __host__ __device__ Q4gShape(int64_t n, int64_t k, int64_t group, int fmt)
        : rt((n + 15) / 16), kt((k + 127) / 128), ks((k + 511) / 512)
    {
        scales = rt * kt * 1024;
        zeros = scales + rt * ks * 16 * (1024 / group);
        bytes = (zeros + ((fmt & kQ4gZeros) ? rt * ks * 16 * (256 / group) : 0) + 255) / 256 * 256;
    }
};

// Element types of the activation rows (the ABI's QLL_DTYPE_* values).
enum { Q4G_X_F32 = 0, Q4G_X_BF16 = 1, Q4G_X_F16 = 2 };

// What a lane reads of one row tile: its 16 bytes of codes, its row's scales and zeros.
struct Q4gRows {
    const uint8_t *codes, *scales, *zeros; // zeros null: every zero point is 8
    bool bf16;
    __device__ Q4gRows() {}
    __device__ Q4gRows(const uint8_t *wp, const Q4gShape &sh, int64_t rt, int group, int fmt, int lane)
        : codes(wp + rt * sh.kt * 1024 + lane * 16),
          scales(wp + sh.scales + (rt * sh.ks * 16 + lane % 16) * (1024 / group)),
          zeros((fmt & kQ4gZeros) ? wp + sh.zeros + (rt * sh.ks * 16 + lane % 16) * (256 / group) : nullptr),
          bf16(fmt & kQ4gBf16)
    {
    }
};

template <int TX>
struct Q4gFrag { // eight consecutive activations
    u32x4 v;
};
template <>
struct Q4gFrag<Q4G_X_F32> {
    u32x4 v, w;
};

// Two f32 -> their upper halves as a pair of bf16 (truncated).
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi)
{
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}
__device__ __forceinline__ float below_bf16(float x) // what truncation to bf16 leaves, exact
{
    return x - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xffff0000u);
}

// One 128-weight tile as a wave holds it in flight.
template <int TX, int GRP, int RTN, int C>
struct Q4gStage {
    u32x4 codes[RTN];
    uint32_t scale[RTN][GRP == 32 ? 2 : 1], zero[RTN];
    Q4gFrag<TX> x[4][C];
};

// The product of RTN row tiles with 16 C activation rows over tiles [t0, t1) of k,
// one wave.  The activation rows are the matrix instruction's A operand (16 rows) and
// the weights its B operand (16 columns), so that the accumulator's column is the lane's own weight
// row, whose scale the lane holds: A row a = 4 h + i of a column group is activation h + 4 i (so that
// up to four activations use one accumulator register a lane, I = 1), and y[r][c][i]
// of lane l is activation l / 16 + 4 i of group c with row l % 16 of tile r.
//
// f32 and bf16 activations: the weight operand is 16 + c as bf16 (exact; three
// instructions two weights), the group's sum of activations comes from the same
// instruction with ones, and s * (D - (16 + z) * S) is the group's part.  The
// difference loses up to 31 / |c - z| of f32's precision, a few bits of 24.  f32 activations
// are split exactly into three bf16 parts.  f16 activations: the weights become
// c - z in f16, exact, by the bits of 1024 + c and one packed subtraction.
//
// D stages of tiles are in flight: D - 1 tiles are asked for ahead of the one in use.
template <int TX, int GRP, int RTN, int C, int I, int D>
struct Q4gWave {
    using Stage = Q4gStage<TX, GRP, RTN, C>;
    static constexpr int kGroups = 128 / GRP, kSteps = GRP / 32; // groups a tile, matrix steps a group
    f32x4 y[RTN][C];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < RTN; r++)
#pragma unroll
            for (int c = 0; c < C; c++)
                y[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // x[c]: this lane's activation row of group c (A row lane % 16), advanced by 8 (lane / 16) elements
    __device__ __forceinline__ static void load(Stage &st, const Q4gRows (&rows)[RTN], const uint8_t *const (&x)[C],
                                                int64_t t, int64_t k)
    {
        const int64_t chunk = t >> 2;
        const int at = (int)(t & 3);
#pragma unroll
        for (int r = 0; r < RTN; r++) {
            st.codes[r] = *reinterpret_cast<const u32x4 *>(rows[r].codes + t * 1024);
            const uint8_t *s = rows[r].scales + chunk * (16 * (1024 / GRP)) + at * (256 / GRP);
            if constexpr (GRP == 32) {
                const uint2 v = *reinterpret_cast<const uint2 *>(s);
                st.scale[r][0] = v.x, st.scale[r][1] = v.y;
            } else if constexpr (GRP == 64)
                st.scale[r][0] = *reinterpret_cast<const uint32_t *>(s);
            else
                st.scale[r][0] = *reinterpret_cast<const uint16_t *>(s);
            if (rows[r].zeros) {
                const uint8_t *z = rows[r].zeros + chunk * (16 * (256 / GRP));
                if constexpr (GRP == 32)
                    st.zero[r] = *reinterpret_cast<const uint16_t *>(z + at * 2);
                else if constexpr (GRP == 64)
                    st.zero[r] = z[at];
                else
                    st.zero[r] = z[at >> 1] >> (4 * (at & 1));
            } else
                st.zero[r] = 0x8888u;
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            // past k (a tile's last steps) the weights have scale 0: any activations of the row do
            const int64_t at_k = t * 128 + 32 * j < k ? t * 128 + 32 * j : k - 32;
#pragma unroll
            for (int c = 0; c < C; c++) {
                if constexpr (TX == Q4G_X_F32) {
                    const u32x4 *p = reinterpret_cast<const u32x4 *>(x[c] + at_k * 4);
                    st.x[j][c].v = p[0], st.x[j][c].w = p[1];
                } else
                    st.x[j][c].v = *reinterpret_cast<const u32x4 *>(x[c] + at_k * 2);
            }
        }
    }

    __device__ __forceinline__ static bf16x8 widen(uint32_t w) // 16 + c of the eight codes
    {
        constexpr uint32_t m = 0x00780078u, b = 0x41804180u;
        const u32x4 v = {((w << 3) & m) | b, ((w >> 1) & m) | b, ((w >> 5) & m) | b, ((w >> 9) & m) | b};
        return __builtin_bit_cast(bf16x8, v);
    }
    // c - z: 1024 + c as f16 bits at a nibble's place, 1024 + 16 c one place up
    __device__ __forceinline__ static f16x8 widen16(uint32_t w, f16x2 less1024, f16x2 less64)
    {
        constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, b = 0x64006400u;
        const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
        const uint32_t u = w >> 8;
        const f16x2 p0 = __builtin_bit_cast(f16x2, (w & lo) | b) + less1024;
        const f16x2 p1 = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (w & hi) | b), sixteenth, less64);
        const f16x2 p2 = __builtin_bit_cast(f16x2, (u & lo) | b) + less1024;
        const f16x2 p3 = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (u & hi) | b), sixteenth, less64);
        return f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }

    __device__ __forceinline__ static f32x4 mul(bf16x8 a, bf16x8 b, f32x4 acc)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
    }

    __device__ __forceinline__ void use(const Stage &st, bool bf16)
    {
        const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < kGroups; g++) {
            float s[RTN];
            uint32_t z[RTN];
#pragma unroll
            for (int r = 0; r < RTN; r++) {
                const uint32_t pair = st.scale[r][g / 2], bits = g & 1 ? pair >> 16 : pair & 0xffffu;
                s[r] = bf16 ? __builtin_bit_cast(float, bits << 16) : half_bits_to_float(bits);
                z[r] = (st.zero[r] >> (4 * g)) & 15u;
            }
            f32x4 d[RTN][C], sum[C];
#pragma unroll
            for (int c = 0; c < C; c++) {
                sum[c] = none;
#pragma unroll
                for (int r = 0; r < RTN; r++)
                    d[r][c] = none;
            }
#pragma unroll
            for (int e = 0; e < kSteps; e++) {
                const int j = g * kSteps + e;
                if constexpr (TX == Q4G_X_F16) {
                    f16x8 w[RTN];
#pragma unroll
                    for (int r = 0; r < RTN; r++)
                        w[r] = widen16(st.codes[r][j], __builtin_bit_cast(f16x2, 0xe400e400u + z[r] * 0x00010001u),
                                       __builtin_bit_cast(f16x2, 0xd400d400u + z[r] * 0x00100010u));
#pragma unroll
                    for (int c = 0; c < C; c++)
#pragma unroll
                        for (int r = 0; r < RTN; r++)
                            d[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                __builtin_bit_cast(f16x8, st.x[j][c].v), w[r], d[r][c], 0, 0, 0);
                } else {
                    constexpr int P = TX == Q4G_X_F32 ? 3 : 1;
                    const u32x4 one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
                    bf16x8 w[RTN];
#pragma unroll
                    for (int r = 0; r < RTN; r++)
                        w[r] = widen(st.codes[r][j]);
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        bf16x8 a[P];
                        if constexpr (TX == Q4G_X_F32)
                            split(st.x[j][c], a);
                        else
                            a[0] = __builtin_bit_cast(bf16x8, st.x[j][c].v);
#pragma unroll
                        for (int p = P - 1; p >= 0; p--) { // small parts first
                            sum[c] = mul(a[p], __builtin_bit_cast(bf16x8, one), sum[c]);
#pragma unroll
                            for (int r = 0; r < RTN; r++)
                                d[r][c] = mul(a[p], w[r], d[r][c]);
                        }
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < RTN; r++)
#pragma unroll
                for (int c = 0; c < C; c++)
#pragma unroll
                    for (int i = 0; i < I; i++) {
                        if constexpr (TX == Q4G_X_F16)
                            y[r][c][i] = fmaf(s[r], d[r][c][i], y[r][c][i]);
                        else
                            y[r][c][i] = fmaf(s[r], fmaf(-(16.0f + (float)z[r]), sum[c][i], d[r][c][i]), y[r][c][i]);
                    }
        }
    }

    // f32 -> three bf16 parts by truncation: 8 + 8 + 8 bits, exact
    __device__ __forceinline__ static void split(const Q4gFrag<Q4G_X_F32> &f, bf16x8 (&a)[3])
    {
        u32x4 p[3];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t b0 = i < 2 ? f.v[2 * i] : f.w[2 * i - 4], b1 = i < 2 ? f.v[2 * i + 1] : f.w[2 * i - 3];
            const float x0 = __builtin_bit_cast(float, b0), x1 = __builtin_bit_cast(float, b1);
            const float r0 = below_bf16(x0), r1 = below_bf16(x1);
            p[0][i] = upper_halves(x0, x1);
            p[1][i] = upper_halves(r0, r1);
            p[2][i] = upper_halves(below_bf16(r0), below_bf16(r1));
        }
#pragma unroll
        for (int i = 0; i < 3; i++)
            a[i] = __builtin_bit_cast(bf16x8, p[i]);
    }

    __device__ __forceinline__ void run(const Q4gRows (&rows)[RTN], const uint8_t *const (&x)[C], int64_t t0,
                                        int64_t t1, int64_t k)
    {
        if (t0 >= t1)
            return;
        Stage st[D];
#pragma unroll
        for (int i = 0; i < D; i++)
            load(st[i], rows, x, t0 + i < t1 ? t0 + i : t1 - 1, k);
        int64_t t = t0;
        for (; t + D < t1; t += D) {
#pragma unroll
            for (int i = 0; i < D; i++) {
                use(st[i], rows[0].bf16);
                load(st[i], rows, x, t + D + i < t1 ? t + D + i : t1 - 1, k);
            }
        }
#pragma unroll
        for (int i = 0; i < D; i++)
            if (t + i < t1)
                use(st[i], rows[0].bf16);
    }
};

// f32 -> an element of type `dtype` at p[i], rounded to nearest even.
__device__ __forceinline__ void store_as(void *p, int64_t i, float v, int dtype)
{
    if (dtype == QLL_W_F32)
        static_cast<float *>(p)[i] = v;
    else if (dtype == QLL_W_BF16)
        static_cast<__bf16 *>(p)[i] = (__bf16)v;
    else
        static_cast<_Float16 *>(p)[i] = (_Float16)v;
}
__device__ __forceinline__ float load_as(const void *p, int64_t i, int dtype)
{
    if (dtype == QLL_W_F32)
        return static_cast<const float *>(p)[i];
    if (dtype == QLL_W_BF16)
        return (float)static_cast<const __bf16 *>(p)[i];
    return (float)static_cast<const _Float16 *>(p)[i];
}

} // namespace qll
