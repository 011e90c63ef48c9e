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

// How a lane finds activations: rows of one of the ABI's element types, or rows
// of two or three bf16 parts, part by part, which the gated products are kept in.
enum { Q4G_X_F32 = 0, Q4G_X_BF16 = 1, Q4G_X_F16 = 2, Q4G_X_PARTS2 = 3, Q4G_X_PARTS3 = 4 };
constexpr int q4g_x_size(int tx) { return tx == Q4G_X_F32 ? 4 : 2; }
constexpr int q4g_x_parts(int tx) { return tx == Q4G_X_F32 || tx == Q4G_X_PARTS3 ? 3 : tx == Q4G_X_PARTS2 ? 2 : 1; }

// One row tile (uniform over a wave; the lanes' offsets are added to each load).
struct Q4gRows {
    const uint8_t *codes, *scales, *zeros; // zeros null: every zero point is 8
    __device__ Q4gRows() {}
    __device__ Q4gRows(const uint8_t *wp, const Q4gShape &sh, int64_t rt, int group, int fmt)
        : codes(wp + rt * sh.kt * 1024), scales(wp + sh.scales + rt * sh.ks * 16 * (1024 / group)),
          zeros((fmt & kQ4gZeros) ? wp + sh.zeros + rt * sh.ks * 16 * (256 / group) : nullptr)
    {
    }
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

// The product of RTN row tiles with up to C * 16 / PK activation rows over tiles
// [t0, t1) of k, one wave.  The activations are the matrix instruction's A operand (16
// rows) and the weights its B operand (16 columns), so that the accumulator's column is the lane's
// own weight row, whose scale the lane holds.
//
// PK = 4, 2 or 1: with few activation rows, A's 16 rows hold PK steps of 32 weights of each,
// row a the step a % PK of activation a / PK, so that one register quad serves PK steps.  Every
// product with the weights of step p is right in the rows with a % PK = p and unused in the
// others.  Against one step an operand this loads a quarter (PK = 4) of the operands, most of
// whose rows were empty, and for f32 splits a quarter.  y[r][c][i] of lane l is activation
// (l / 16) * 4 / PK + i of group c with row l % 16 of tile r.
//
// f32 and bf16 activations: the weight operand is 16 + c as bf16 (exact; two
// instructions two weights), the group's sum S of activations comes from the same
// instruction with ones, and s * (D - (16 + z) * S) is the group's part.  The
// difference loses up to 31 / |c - z| of f32's precision, a few bits of 24.  f32 activations
// are split exactly into three bf16 parts.  f16 activations: the weights become
// c - z in f16, exact, by the bits of 1024 + c and one packed subtraction.
//
// D tiles are in flight: a tile's registers are asked for again as soon as it is used.
template <int TX, int GRP, int RTN, int C, int PK, int D>
struct Q4gWave {
    static constexpr int kGroups = 128 / GRP, kSteps = GRP / 32; // groups a tile, steps a group
    static constexpr int kQuads = 4 / PK, kLoads = TX == Q4G_X_F32 ? 2 : q4g_x_parts(TX), P = q4g_x_parts(TX);
    static constexpr int N = 4 / PK; // activations of a group a lane ends up with
    float y[RTN][C][N];

    struct Stage { // one 128-weight tile in flight
        u32x4 codes[RTN], x[kQuads][C][kLoads];
        uint32_t scale[RTN][GRP == 32 ? 2 : 1], zero[RTN];
    };
    // Bases are uniform over the wave and offsets 32 bits, so that a load takes one register
    // of address (64-bit addresses of a lane cost up to 30 a stage).
    struct Rows {
        Q4gRows w[RTN];
        const uint8_t *x;
        uint32_t at[C]; // byte offset of activation row_of(lane) of group c
        int64_t part;   // bytes from one part of it to the next (Q4G_X_PARTS*)
        int last;       // k - 32
        bool bf16;      // scales are bf16
        int lane;
    };

    // which activation of a group this lane's A row is
    __device__ __forceinline__ static int row_of(int lane) { return lane % 16 / PK; }
    // which one y[..][i] is
    __device__ __forceinline__ static int out_of(int lane, int i) { return lane / 16 * N + i; }

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int r = 0; r < RTN; r++)
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int i = 0; i < N; i++)
                    y[r][c][i] = 0.0f;
    }

    template <class T>
    __device__ __forceinline__ static T fetch(const uint8_t *base, uint32_t at)
    {
        return *reinterpret_cast<const T *>(base + at);
    }

    __device__ __forceinline__ static void load(Stage &st, const Rows &rows, int t)
    {
        const int64_t chunk = t >> 2;
        const int at = t & 3;
        const uint32_t lane = rows.lane, row = lane % 16;
#pragma unroll
        for (int r = 0; r < RTN; r++) {
            st.codes[r] = fetch<u32x4>(rows.w[r].codes + (int64_t)t * 1024, lane * 16);
            const uint8_t *s = rows.w[r].scales + chunk * (16 * (1024 / GRP)) + at * (256 / GRP);
            if constexpr (GRP == 32) {
                const uint2 v = fetch<uint2>(s, row * (1024 / GRP));
                st.scale[r][0] = v.x, st.scale[r][1] = v.y;
            } else if constexpr (GRP == 64)
                st.scale[r][0] = fetch<uint32_t>(s, row * (1024 / GRP));
            else
                st.scale[r][0] = fetch<uint16_t>(s, row * (1024 / GRP));
            if (rows.w[r].zeros) {
                const uint8_t *z = rows.w[r].zeros + chunk * (16 * (256 / GRP)) + (GRP == 32 ? at * 2 : GRP == 64 ? at : at >> 1);
                if constexpr (GRP == 32)
                    st.zero[r] = fetch<uint16_t>(z, row * (256 / GRP));
                else
                    st.zero[r] = fetch<uint8_t>(z, row * (256 / GRP));
            } else
                st.zero[r] = 0x8888u;
        }
#pragma unroll
        for (int q = 0; q < kQuads; q++) {
            // past k (a tile's last steps) the weights have scale 0: any activations of the row do
            const int step = t * 128 + 32 * (q * PK + (int)(lane % PK));
            const uint32_t at_k = ((uint32_t)(step < rows.last ? step : rows.last) + 8 * (lane / 16)) * q4g_x_size(TX);
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int i = 0; i < kLoads; i++)
                    st.x[q][c][i] = TX == Q4G_X_F32 ? fetch<u32x4>(rows.x + 16 * i, rows.at[c] + at_k)
                                                    : fetch<u32x4>(rows.x + i * rows.part, rows.at[c] + at_k);
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

    __device__ __forceinline__ static f32x4 mul(u32x4 a, bf16x8 b, f32x4 acc)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b, acc, 0, 0, 0);
    }
    __device__ __forceinline__ static f32x4 mul16(u32x4 a, f16x8 b, f32x4 acc)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), b, acc, 0, 0, 0);
    }

    // f32 -> three bf16 parts by truncation: 8 + 8 + 8 bits, exact
    __device__ __forceinline__ static void split(const u32x4 (&f)[2], u32x4 (&a)[3])
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float x0 = __builtin_bit_cast(float, (uint32_t)f[i / 2][2 * (i % 2)]);
            const float x1 = __builtin_bit_cast(float, (uint32_t)f[i / 2][2 * (i % 2) + 1]);
            const float r0 = below_bf16(x0), r1 = below_bf16(x1);
            a[0][i] = upper_halves(x0, x1);
            a[1][i] = upper_halves(r0, r1);
            a[2][i] = upper_halves(below_bf16(r0), below_bf16(r1));
        }
    }

    __device__ __forceinline__ void use(const Stage &st, bool bf16, int t)
    {
        const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
        const u32x4 one = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        u32x4 x[kQuads][C][P];
#pragma unroll
        for (int q = 0; q < kQuads; q++)
#pragma unroll
            for (int c = 0; c < C; c++) {
                if constexpr (TX == Q4G_X_F32)
                    split(st.x[q][c], x[q][c]);
                else
#pragma unroll
                    for (int p = 0; p < P; p++)
                        x[q][c][p] = st.x[q][c][p];
            }
        f32x4 sum[C];
#pragma unroll
        for (int g = 0; g < kGroups; g++) {
            float s[RTN];
            uint32_t z[RTN];
#pragma unroll
            for (int r = 0; r < RTN; r++) {
                const uint32_t pair = st.scale[r][g / 2], bits = g & 1 ? pair >> 16 : pair & 0xffffu;
                s[r] = bf16 ? __builtin_bit_cast(float, bits << 16) : half_bits_to_float(bits);
                z[r] = (st.zero[r] >> (GRP == 128 ? 4 * (t & 1) : 4 * g)) & 15u;
            }
            f32x4 d[RTN][C][PK];
#pragma unroll
            for (int e = 0; e < kSteps; e++) {
                const int j = g * kSteps + e, q = j / PK, b = j % PK;
                if constexpr (TX == Q4G_X_F16) {
#pragma unroll
                    for (int r = 0; r < RTN; r++) {
                        const f16x8 w = widen16(st.codes[r][j], __builtin_bit_cast(f16x2, 0xe400e400u + z[r] * 0x00010001u),
                                                __builtin_bit_cast(f16x2, 0xd400d400u + z[r] * 0x00100010u));
#pragma unroll
                        for (int c = 0; c < C; c++)
                            d[r][c][b] = mul16(x[q][c][0], w, e < PK ? none : d[r][c][b]);
                    }
                } else {
                    if (j % PK == 0) // a new quad: the sums of its steps, on top of the group's so far
#pragma unroll
                        for (int c = 0; c < C; c++)
#pragma unroll
                            for (int p = P - 1; p >= 0; p--) // small parts first
                                sum[c] = mul(x[q][c][p], __builtin_bit_cast(bf16x8, one),
                                             e == 0 && p == P - 1 ? none : sum[c]);
#pragma unroll
                    for (int r = 0; r < RTN; r++) {
                        const bf16x8 w = widen(st.codes[r][j]);
#pragma unroll
                        for (int c = 0; c < C; c++)
#pragma unroll
                            for (int p = P - 1; p >= 0; p--)
                                d[r][c][b] = mul(x[q][c][p], w, e < PK && p == P - 1 ? none : d[r][c][b]);
                    }
                }
            }
            // the group's steps within a quad: rows b0 .. b0 + count - 1 of every activation's PK
            constexpr int count = kSteps < PK ? kSteps : PK;
            const int b0 = g * kSteps % PK;
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int i = 0; i < N; i++) {
                    float whole = 0.0f;
                    if constexpr (TX != Q4G_X_F16) {
                        whole = sum[c][i * PK + b0];
#pragma unroll
                        for (int b = 1; b < count; b++)
                            whole += sum[c][i * PK + b0 + b];
                    }
#pragma unroll
                    for (int r = 0; r < RTN; r++) {
                        float v = d[r][c][b0][i * PK + b0];
#pragma unroll
                        for (int b = 1; b < count; b++)
                            v += d[r][c][b0 + b][i * PK + b0 + b];
                        if constexpr (TX != Q4G_X_F16)
                            v = fmaf(-(16.0f + (float)z[r]), whole, v);
                        y[r][c][i] = fmaf(s[r], v, y[r][c][i]);
                    }
                }
        }
    }

    // The scheduling fences keep a stage's work together: without them the compiler widens
    // the codes of several stages at once and runs out of registers.
    __device__ __forceinline__ void run(const Rows &rows, int t0, int t1)
    {
        if (t0 >= t1)
            return;
        Stage st[D];
#pragma unroll
        for (int i = 0; i < D; i++)
            load(st[i], rows, t0 + i < t1 ? t0 + i : t1 - 1);
        int t = t0;
        for (; t + D < t1; t += D) {
#pragma unroll
            for (int i = 0; i < D; i++) {
                use(st[i], rows.bf16, t + i);
                __builtin_amdgcn_sched_barrier(0);
                load(st[i], rows, t + D + i < t1 ? t + D + i : t1 - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int i = 0; i < D; i++) {
            if (t + i < t1)
                use(st[i], rows.bf16, t + i);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

__device__ __forceinline__ int wave_number() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// The lane as a value the compiler knows nothing about: what depends on it is computed
// where it is used, not ahead of a loop over tiles or of all branches at once, where it would hold
// registers.
__device__ __forceinline__ int opaque_lane()
{
    int lane = threadIdx.x % 64;
    asm volatile("" : "+v"(lane));
    return lane;
}

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
