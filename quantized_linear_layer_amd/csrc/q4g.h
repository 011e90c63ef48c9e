// 4-bit codes with one scale (f16 or bf16) and, where present, one 4-bit zero
// point per group of 32, 64 or 128 weights of a row:
//     w[j][t] = s[j][t / g] * (c[j][t] - z[j][t / g]),   z = 8 where there is none.
// The packed form and the product of one wave on it, shared by the linear
// layer (q4g.hip) and the experts (moe.hip).
//
// Packed form of W[n][k], three regions one after another and zero bytes up to a multiple of
// 256, for tiles of 16 rows (index rt, rows past n zero) and 128 weights
// (index kt, weights past k zero):
//   codes   tile (rt, kt) at 1024 * (rt * KT + kt), KT = ceil(k / 128): 16 bytes a
//           lane of a wave, lane l holding row l % 16; dword j (matrix-core step j) has the
//           weights 32 j + 8 (l / 16) + 0..7 of the tile, number 2 p at bits 4 p, number
//           2 p + 1 at bits 16 + 4 p, so that a shift and a mask give two neighbours in
//           the halves of a register
//   scales  for pieces of 512 weights (index ks, KS = ceil(k / 512)), 16 rows a piece and 512 / g
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
    int64_t rt, kt, ks;                     // tiles of 16 rows, of 128 weights, pieces of 512
    int64_t scales, zeros, end, bytes;      // byte offsets of the regions, their end, and that of all bytes
    __host__ __device__ Q4gShape(int64_t n, int64_t k, int64_t group, int fmt)
        : rt((n + 15) / 16), kt((k + 127) / 128), ks((k + 511) / 512)
    {
        scales = rt * kt * 1024;
        zeros = scales + rt * ks * 16 * (1024 / group);
        end = zeros + ((fmt & kQ4gZeros) ? rt * ks * 16 * (256 / group) : 0);
        bytes = (end + 255) / 256 * 256;
    }
};

__device__ __forceinline__ int wave_number() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// How activations lie in memory: rows of one of the ABI's element types, or rows of two or
// three bf16 parts, part by part.
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
// Eight f32 -> three bf16 parts by truncation: 8 + 8 + 8 bits, exact.
__device__ __forceinline__ void split3(u32x4 lo, u32x4 hi, u32x4 &a, u32x4 &b, u32x4 &c)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t b0 = i < 2 ? lo[2 * i] : hi[2 * i - 4], b1 = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
        const float x0 = __builtin_bit_cast(float, b0), x1 = __builtin_bit_cast(float, b1);
        const float r0 = below_bf16(x0), r1 = below_bf16(x1);
        a[i] = upper_halves(x0, x1);
        b[i] = upper_halves(r0, r1);
        c[i] = upper_halves(below_bf16(r0), below_bf16(r1));
    }
}

// The product of RTN row tiles with up to C * 16 / PK activation rows, one wave.  The
// activations are the matrix instruction's A operand (16 rows) and the weights its B operand (16
// columns), so that the accumulator's column is the lane's own weight row, whose scale the lane holds.
//
// PK = 4, 2 or 1: with few activation rows, A's 16 rows hold PK steps of 32 weights of each,
// row a the step a % PK of activation a / PK, so that one register quad serves PK steps.  Every
// product with the weights of step p is right in the rows with a % PK = p and unused in the
// others.  Against one step an operand this moves a quarter (PK = 4) of the operands, most of
// whose rows were empty.  y[r][c][i] of lane l is activation (l / 16) * 4 / PK + i of group c
// with row l % 16 of tile r.
//
// The weight operand is c - z, exact in bf16 and f16: a weight of 0 adds nothing, however large its
// activation.  For bf16 that takes 17 instructions for eight weights.  16 + c takes nine, with the group's sum S of
// activations from the same matrix instruction and D - (16 + z) S as the group's part (4096 -> 14336, one
// bf16 row: 8.6 us in place of 10.1; from eight rows on the two are alike), but D and S then carry the rounding
// of an outlier whose own weight is 0 (an outlier 10^4 times the others: 160 times an f32 product's error).
// f32 activations are split exactly into three bf16 parts.
//
// Codes are loaded by tiles of 128 weights, scales and zero points by pieces of 512: loads of
// a few bytes cost nearly as much as those of 16 (4096 -> 14336, one row: 10.8 us with a load of
// scales and one of zero points a tile, 8.0 without).
template <int TX, int GRP, int RTN, int C, int PK>
struct Q4gTile {
    static constexpr int kGroups = 128 / GRP, kSteps = GRP / 32; // groups a tile, steps a group
    static constexpr int kQuads = 4 / PK, P = q4g_x_parts(TX), N = 4 / PK;
    static constexpr int kScaleWords = 256 / GRP, kZeroWords = GRP == 32 ? 2 : 1;
    static constexpr int kPieceLoads = RTN * (GRP == 32 ? 2 : 1); // without zero points
    static_assert(C == 1 || PK == 1, "several steps an operand only with one column group");
    float y[RTN][C][N];

    struct Piece { // scales and zero points of 512 weights
        uint32_t scale[RTN][kScaleWords], zero[RTN][kZeroWords];
    };

    // which activation of a group this lane's A row is, and which one y[..][i] is
    __device__ __forceinline__ static int row_of(int lane) { return lane % 16 / PK; }
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

    // Bases are uniform over the wave and offsets 32 bits, so that a load takes one register of
    // address; the offset is opaque, or the compiler adds it to the base ahead of the loop and holds
    // 64-bit addresses of every stream and stage.
    template <class V>
    __device__ __forceinline__ static V fetch(const uint8_t *base, uint32_t at)
    {
        asm volatile("" : "+v"(at));
        return *reinterpret_cast<const V *>(base + at);
    }
    __device__ __forceinline__ static void load_tile(u32x4 (&codes)[RTN], const Q4gRows (&w)[RTN], int t, uint32_t lane)
    {
#pragma unroll
        for (int r = 0; r < RTN; r++)
            codes[r] = fetch<u32x4>(w[r].codes + (int64_t)t * 1024, lane * 16);
    }
    __device__ __forceinline__ static void load_piece(Piece &p, const Q4gRows (&w)[RTN], int piece, uint32_t lane)
    {
        const uint32_t row = lane % 16;
#pragma unroll
        for (int r = 0; r < RTN; r++) {
            const uint8_t *s = w[r].scales + (int64_t)piece * (16 * (1024 / GRP));
            if constexpr (GRP == 128) {
                const uint2 v = fetch<uint2>(s, row * 8);
                p.scale[r][0] = v.x, p.scale[r][1] = v.y;
            } else
#pragma unroll
                for (int i = 0; i < kScaleWords / 4; i++) {
                    const u32x4 v = fetch<u32x4>(s + 16 * i, row * (1024 / GRP));
#pragma unroll
                    for (int b = 0; b < 4; b++)
                        p.scale[r][4 * i + b] = v[b];
                }
            if (w[r].zeros) {
                const uint8_t *z = w[r].zeros + (int64_t)piece * (16 * (256 / GRP));
                if constexpr (GRP == 128)
                    p.zero[r][0] = fetch<uint16_t>(z, row * 2);
                else if constexpr (GRP == 64)
                    p.zero[r][0] = fetch<uint32_t>(z, row * 4);
                else {
                    const uint2 v = fetch<uint2>(z, row * 8);
                    p.zero[r][0] = v.x, p.zero[r][1] = v.y;
                }
            } else
#pragma unroll
                for (int i = 0; i < kZeroWords; i++)
                    p.zero[r][i] = 0x88888888u;
        }
    }

    // (w & m) | b in one instruction: it takes no literals, so the constants stay in registers, where the
    // compiler would rather have two instructions with a literal each.
    __device__ __forceinline__ static uint32_t and_or(uint32_t w, uint32_t m, uint32_t b)
    {
        asm("" : "+s"(m));
        asm("" : "+v"(b));
        return (w & m) | b;
    }
    // c - z as bf16: 1024 + c as f16 bits (1024 + 16 c where the code is one place up), less 1024 + z (a sixteenth
    // of it less 64 + z) in f32 by one mixed fma a weight, whose upper half is the bf16.
    __device__ __forceinline__ static bf16x8 widen(uint32_t w, float less1024, float less64)
    {
        constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, b = 0x64006400u;
        float one = 1.0f, sixteenth = 0.0625f; // opaque: a product with 1 would become a conversion and a sum
        asm("" : "+s"(one), "+s"(sixteenth));
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const f16x2 p = __builtin_bit_cast(f16x2, and_or(i < 2 ? w : w >> 8, i & 1 ? hi : lo, b));
            const float by = i & 1 ? sixteenth : one, less = i & 1 ? less64 : less1024;
            v[i] = upper_halves(fmaf((float)p[0], by, less), fmaf((float)p[1], by, less));
        }
        return __builtin_bit_cast(bf16x8, v);
    }
    // c - z as f16: the same bits, one packed subtraction or fma for two weights
    __device__ __forceinline__ static f16x8 widen16(uint32_t w, uint32_t z)
    {
        constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u, b = 0x64006400u;
        const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
        const f16x2 less1024 = __builtin_bit_cast(f16x2, 0xe400e400u + z * 0x00010001u); // -1024 - z
        const f16x2 less64 = __builtin_bit_cast(f16x2, 0xd400d400u + z * 0x00100010u);   // -64 - z
        const uint32_t u = w >> 8;
        const f16x2 p0 = __builtin_bit_cast(f16x2, and_or(w, lo, b)) + less1024;
        const f16x2 p1 = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, and_or(w, hi, b)), sixteenth, less64);
        const f16x2 p2 = __builtin_bit_cast(f16x2, and_or(u, lo, b)) + less1024;
        const f16x2 p3 = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, and_or(u, hi, b)), sixteenth, less64);
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

    // Tile j of a piece; operand(q, c, p): part p of quad q of column group c.
    template <class X>
    __device__ __forceinline__ void use(const u32x4 (&codes)[RTN], const Piece &piece, int j, const X &operand, bool bf16)
    {
        const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t which = bf16 ? ~0u : 0u;
        asm("" : "+v"(which));
        // a quad's operands are asked for while the one before it is multiplied
        u32x4 xs[2][C][P];
        const auto ask = [&](int q) {
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int p = 0; p < P; p++)
                    xs[q & 1][c][p] = operand(q, c, p);
        };
        ask(0);
#pragma unroll
        for (int g = 0; g < kGroups; g++) {
            const int number = j * kGroups + g; // of the piece's groups
            float s[RTN];
            uint32_t z[RTN];
#pragma unroll
            for (int r = 0; r < RTN; r++) {
                const uint32_t pair = piece.scale[r][number / 2];
                const uint32_t as_bf16 = number & 1 ? pair & 0xffff0000u : pair << 16;
                const uint32_t as_f16 = __builtin_bit_cast(uint32_t, half_bits_to_float(number & 1 ? pair >> 16 : pair));
                s[r] = __builtin_bit_cast(float, (as_bf16 & which) | (as_f16 & ~which)); // one instruction, no branch
                z[r] = (piece.zero[r][number / 8] >> (4 * (number & 7))) & 15u;
            }
            f32x4 d[RTN][C][PK];
#pragma unroll
            for (int e = 0; e < kSteps; e++) {
                const int step = g * kSteps + e, q = step / PK, b = step % PK;
                u32x4 (&x)[C][P] = xs[q & 1];
                if (step % PK == 0 && q + 1 < kQuads)
                    ask(q + 1);
                if constexpr (TX == Q4G_X_F16) {
#pragma unroll
                    for (int r = 0; r < RTN; r++) {
                        const f16x8 w = widen16(codes[r][step], z[r]);
#pragma unroll
                        for (int c = 0; c < C; c++)
                            d[r][c][b] = mul16(x[c][0], w, e < PK ? none : d[r][c][b]);
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < RTN; r++) {
                        const float less1024 = __builtin_bit_cast(float, 0xc4800000u | z[r] << 13); // by their bits
                        const float less64 = __builtin_bit_cast(float, 0xc2800000u | z[r] << 17);
                        const bf16x8 w = widen(codes[r][step], less1024, less64);
#pragma unroll
                        for (int c = 0; c < C; c++)
#pragma unroll
                            for (int p = P - 1; p >= 0; p--)
                                d[r][c][b] = mul(x[c][p], w, e < PK && p == P - 1 ? none : d[r][c][b]);
                    }
                }
            }
            // the group's steps within a quad: rows b0 .. b0 + count - 1 of every activation's PK
            constexpr int count = kSteps < PK ? kSteps : PK;
            const int b0 = g * kSteps % PK;
#pragma unroll
            for (int c = 0; c < C; c++)
#pragma unroll
                for (int i = 0; i < N; i++)
#pragma unroll
                    for (int r = 0; r < RTN; r++) {
                        float v = d[r][c][b0][i * PK + b0];
#pragma unroll
                        for (int b = b0 + 1; b < b0 + count; b++)
                            v += d[r][c][b][i * PK + b];
                        y[r][c][i] = fmaf(s[r], v, y[r][c][i]);
                    }
            if constexpr (RTN * C >= 8) // one group at a time, or they run out of registers
                __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Up to 16 / PK activation rows, each wave with its operands in registers beside the codes: for
// few rows, whose operands are few and the same for all waves of a CU, and for small
// products.  D of a piece's four tiles are in flight, and the next ones from each one's use on.  The
// scheduling fences keep a tile's work together: without them the compiler widens the codes of several
// tiles at once and runs out of registers.
template <int TX, int GRP, int RTN, int PK, int D>
struct Q4gWave : Q4gTile<TX, GRP, RTN, 1, PK> {
    using Tile = Q4gTile<TX, GRP, RTN, 1, PK>;
    using Piece = typename Tile::Piece;
    static constexpr int kLoads = TX == Q4G_X_F32 ? 2 : Tile::P, kQuads = Tile::kQuads;

    struct From { // row tiles and the activations
        Q4gRows w[RTN];
        const uint8_t *x;
        uint32_t at;  // byte offset of activation row_of(lane)
        int64_t part; // bytes from one part of it to the next (Q4G_X_PARTS*)
        int last, kt; // k - 32, tiles
    };
    struct Slot {
        u32x4 codes[RTN], x[kQuads][kLoads];
    };
    Slot slot[D];
    Piece next;

    __device__ __forceinline__ static void load(Slot &s, const From &f, int t, uint32_t lane)
    {
        Tile::load_tile(s.codes, f.w, t < f.kt ? t : f.kt - 1, lane);
#pragma unroll
        for (int q = 0; q < kQuads; q++) {
            // past k (a tile's last steps) the weights have scale 0: any activations of the row do
            const int step = t * 128 + 32 * (q * PK + (int)(lane % PK));
            const uint32_t at = f.at + ((uint32_t)(step < f.last ? step : f.last) + 8 * (lane / 16)) * q4g_x_size(TX);
#pragma unroll
            for (int i = 0; i < kLoads; i++)
                s.x[q][i] = Tile::template fetch<u32x4>(f.x + (TX == Q4G_X_F32 ? 16 * i : i * f.part), at);
        }
    }
    // the first loads
    __device__ __forceinline__ void start(const From &f, int piece, uint32_t lane)
    {
        Tile::load_piece(next, f.w, piece, lane);
#pragma unroll
        for (int j = 0; j < D; j++)
            load(slot[j], f, 4 * piece + j, lane);
    }
    // Piece `piece` of `now_f`; MORE: with the loads of the one after it, piece `after` of f.  WHOLE: it has
    // all four tiles (a branch around a tile costs copies of the sums).
    template <bool MORE, bool WHOLE>
    __device__ __forceinline__ void use_piece(const From &now_f, int piece, const From &f, int after, bool bf16, uint32_t lane)
    {
        const Piece now = next;
        const int tiles = now_f.kt - 4 * piece;
        if constexpr (MORE)
            Tile::load_piece(next, f.w, after, lane);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            Slot &s = slot[j % D];
            if (WHOLE || j < tiles) {
                u32x4 x[kQuads][Tile::P];
#pragma unroll
                for (int q = 0; q < kQuads; q++) {
                    if constexpr (TX == Q4G_X_F32)
                        split3(s.x[q][0], s.x[q][1], x[q][0], x[q][1], x[q][2]);
                    else
#pragma unroll
                        for (int p = 0; p < Tile::P; p++)
                            x[q][p] = s.x[q][p];
                }
                Tile::use(s.codes, now, j, [&](int q, int, int p) { return x[q][p]; }, bf16);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (j + D < 4)
                load(s, now_f, 4 * piece + j + D, lane);
            else if constexpr (MORE)
                load(s, f, 4 * after + j + D - 4, lane);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // pieces [p0, p1)
    __device__ __forceinline__ void run(const From &f, int p0, int p1, bool bf16, uint32_t lane)
    {
        if (p0 >= p1)
            return;
        start(f, p0, lane);
        for (int p = p0; p + 1 < p1; p++)
            use_piece<true, true>(f, p, f, p + 1, bf16, lane);
        use_piece<false, false>(f, p1 - 1, f, 0, bf16, lane);
    }
};

// lds_dma16 with a base that the compiler may hold in vector registers or bring back from them:
// five wait states between that and the load's use of it.
__device__ __forceinline__ void lds_operand16(const uint8_t *base, uint32_t off, uint32_t lds)
{
    const uint64_t b = (uint64_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)b), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"((uint64_t)hi << 32 | lo),
                 "s"(__builtin_amdgcn_readfirstlane((int)lds))
                 : "memory", "m0");
}

// More rows: a workgroup of up to eight waves with the activations in LDS, in the order of
// the matrix instruction's operands.  A wave that fetches them itself moves, for every KB of
// codes, 2 KB (8 rows) to 4 KB (16) of them through a path that gives 12 to 15 bytes a
// clock and CU whatever cache they come from (14336 -> 4096, 16 rows: 19 us, with the operands
// left out 10).  Waves take row tiles, or parts of every chunk of activations: kChunk
// elements of T rows, which loads straight into LDS bring in while the chunk before it is in use.
template <int TX, int GRP, int RTN, int C, int PK>
struct Q4gBlock : Q4gTile<TX, GRP, RTN, C, PK> {
    using Tile = Q4gTile<TX, GRP, RTN, C, PK>;
    using Piece = typename Tile::Piece;
    static_assert(TX != Q4G_X_F32, "f32 rows come as parts");
    static constexpr int T = 16 * C / PK, P = Tile::P, kQuads = Tile::kQuads;
    static constexpr int kBase = 16384 / (T * P) / 512 * 512; // 32 KB
    static constexpr int kChunk = kBase < 512 ? 512 : kBase;
    static constexpr int kPieces = kChunk / 512;
    static constexpr int kTileBytes = kQuads * C * P * 1024, kBuffer = kChunk / 128 * kTileBytes;

    struct X { // what a lane fetches: rows row_of(lane) of each column group
        const uint8_t *base;
        uint32_t at[C]; // byte offset, ~0 for no row
        int64_t part;
        int k;
    };

    // LDS of the chunks in flight (of one, if there is only one)
    __host__ __device__ static constexpr int lds_bytes(int64_t k)
    {
        return k > kChunk ? 2 * kBuffer : (int)((k + 127) / 128) * kTileBytes;
    }

    // operand (q, c, p) of tile t of a chunk at (((t * kQuads + q) * C + c) * P + p) * 1024 + lane * 16
    __device__ __forceinline__ static void fetch_x(const X &src, int chunk, uint32_t lds, int lane)
    {
        const int wave = wave_number(), waves = blockDim.x / 64, kt = (src.k + 127) / 128 - chunk * (kChunk / 128);
        const int count = (kt < kChunk / 128 ? kt : kChunk / 128) * kQuads;
        for (int i = wave; i < count; i += waves) { // tile i / kQuads, quad i % kQuads
            const int step = chunk * kChunk + i / kQuads * 128 + 32 * (i % kQuads * PK + lane % PK);
            const uint32_t at_k = ((uint32_t)(step < src.k - 32 ? step : src.k - 32) + 8 * (lane / 16)) * 2;
#pragma unroll
            for (int c = 0; c < C; c++)
                if (src.at[c] != ~0u)
#pragma unroll
                    for (int p = 0; p < P; p++)
                        lds_operand16(src.base + p * src.part, src.at[c] + at_k, lds + ((i * C + c) * P + p) * 1024);
        }
    }

    // Every wave's loads into LDS but for those after them, then all waves' are seen by all.  `after`: the
    // wave has asked for a whole piece's codes and scales since.
    __device__ __forceinline__ static void arrive(bool after)
    {
        if (after)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(4 * RTN + Tile::kPieceLoads < 63 ? 4 * RTN + Tile::kPieceLoads : 63) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }

    // A piece, whose four tiles are in flight; MORE: with the loads of the piece `after` it (then it has all four tiles; a branch around
    // a tile costs copies of the sums).
    template <bool MORE>
    __device__ __forceinline__ void use_piece(u32x4 (&codes)[4][RTN], Piece &next, const Q4gRows (&w)[RTN], int piece,
                                              int after, int kt, const uint8_t *at, bool bf16, uint32_t lane)
    {
        const Piece now = next;
        if constexpr (MORE)
            Tile::load_piece(next, w, after, lane);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (MORE || 4 * piece + j < kt)
                Tile::use(codes[j], now, j, [&](int q, int c, int p) {
                    return *reinterpret_cast<const u32x4 *>(at + j * kTileBytes + ((q * C + c) * P + p) * 1024);
                }, bf16);
            __builtin_amdgcn_sched_barrier(0);
            if (MORE)
                Tile::load_tile(codes[j], w, 4 * after + j < kt ? 4 * after + j : kt - 1, lane);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Chunks [x0, x1) of the activations.  The wave is part kw of KW (which divides kPieces) of the
    // ones on its row tiles.  Every wave of the workgroup calls it alike; `busy` is false
    // for one that has no rows.  staged: the one chunk is in LDS already; else all waves are done with LDS.
    // Next to nothing is asked for that is not used: the load path is what bounds short rows.
    __device__ __forceinline__ void run(const Q4gRows (&w)[RTN], bool busy, const X &src, int x0, int x1, int kw, int KW,
                                        bool bf16, bool staged, const uint8_t *lds, uint32_t lane)
    {
        const int kt = (src.k + 127) / 128, per = kPieces / KW, last = x1 - 1;
        const int whole = (src.k + 511) / 512, ks = x1 * kPieces < whole ? x1 * kPieces : whole; // pieces end here
        const uint32_t base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)lds;
        u32x4 codes[4][RTN];
        Piece next;
        if (!staged)
            fetch_x(src, x0, base, lane);
        int piece = x0 * kPieces + kw * per;
        const bool some = busy && piece < ks;
        if (some) {
            Tile::load_piece(next, w, piece, lane);
#pragma unroll
            for (int i = 0; i < 4; i++)
                Tile::load_tile(codes[i], w, 4 * piece + i < kt ? 4 * piece + i : kt - 1, lane);
        }
        if (!staged)
            arrive(some);
        const uint8_t *at = lds + kw * per * 4 * kTileBytes + lane * 16;
        for (int xc = x0; xc < last; xc++) { // whole chunks
            fetch_x(src, xc + 1, base + ((xc - x0 + 1) & 1) * kBuffer, lane);
            if (busy)
                for (int r = 0; r < per; r++) {
                    piece = xc * kPieces + kw * per + r;
                    int after = r + 1 < per ? piece + 1 : (xc + 1) * kPieces + kw * per;
                    after = after < ks ? after : ks - 1; // a wave without a piece in the last chunk: not used
                    use_piece<true>(codes, next, w, piece, after, kt, at + ((xc - x0) & 1) * kBuffer + r * 4 * kTileBytes, bf16,
                                    lane);
                }
            arrive(busy);
        }
        piece = last * kPieces + kw * per;
        if (!busy || piece >= ks)
            return;
        const int end = piece + per < ks ? piece + per : ks;
        at += ((last - x0) & 1) * kBuffer;
        if constexpr (kPieces > 1)
            for (; piece + 1 < end; piece++, at += 4 * kTileBytes)
                use_piece<true>(codes, next, w, piece, piece + 1, kt, at, bf16, lane);
        use_piece<false>(codes, next, w, piece, 0, kt, at, bf16, lane);
    }
};

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
