// 4-bit weights with group scales: packing, and the linear layer
//     Y = act(X.W^T + bias) + residual
// on f32, bf16 or f16 activations as they are.  q4g.h has the packed form and
// the product of one wave.
#include "q4g.h"

namespace qll {
namespace {

// ------------------------------------------------------------ packing

// Where the codes come from: one byte each, or the nibbles of block_q4_0.
struct CodeBytes {
    const uint8_t *codes;
    __device__ uint32_t eight(int64_t row, int64_t t, int64_t k) const
    {
        const uint2 v = *reinterpret_cast<const uint2 *>(codes + row * k + t);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t c = ((e < 4 ? v.x : v.y) >> (8 * (e & 3))) & 15u;
            w |= c << (4 * (e >> 1) + 16 * (e & 1));
        }
        return w;
    }
};
struct CodeBlocks {
    const uint8_t *w;
    __device__ uint32_t eight(int64_t row, int64_t t, int64_t k) const
    {
        const uint8_t *qs = w + (row * (k / 32) + t / 32) * 18 + 2 + t % 16; // t % 8 == 0
        const int shift = t % 32 >= 16 ? 4 : 0;
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 8; e++)
            v |= ((uint32_t)(qs[e] >> shift) & 15u) << (4 * (e >> 1) + 16 * (e & 1));
        return v;
    }
};

// Where the scales come from, and the zero points.
struct ScaleArray {
    const uint16_t *scales;
    const uint8_t *zeros;
    __device__ uint32_t scale(int64_t row, int64_t g, int64_t groups) const { return scales[row * groups + g]; }
    __device__ uint32_t zero(int64_t row, int64_t g, int64_t groups) const { return zeros[row * groups + g] & 15u; }
};
struct ScaleBlocks {
    const uint8_t *w;
    __device__ uint32_t scale(int64_t row, int64_t g, int64_t groups) const
    {
        return *reinterpret_cast<const uint16_t *>(w + (row * groups + g) * 18);
    }
    __device__ uint32_t zero(int64_t, int64_t, int64_t) const { return 0; }
};

// A tile of codes.
template <class Codes>
__device__ __forceinline__ void pack_codes(const Codes &codes, uint8_t *wp, const Q4gShape &sh, int64_t tile, int64_t n,
                                           int64_t k)
{
    const int lane = threadIdx.x % 64;
    const int64_t row = tile / sh.kt * 16 + lane % 16, t = tile % sh.kt * 128 + lane / 16 * 8;
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (row < n && t + 32 * j < k)
            v[j] = codes.eight(row, t + 32 * j, k);
    *reinterpret_cast<u32x4 *>(wp + tile * 1024 + lane * 16) = v;
}

// Scales (and zero points) of one row and 512 weights.
template <class Scales>
__device__ __forceinline__ void pack_scales(const Scales &from, uint8_t *scales, uint8_t *zeros, int64_t ks, int64_t item,
                                            int64_t n, int64_t groups, int group)
{
    const int64_t row = item / 16 / ks * 16 + item % 16, piece = item / 16 % ks;
    const int per = 512 / group;
    uint16_t *s = reinterpret_cast<uint16_t *>(scales) + item * per;
    uint64_t z = 0;
    for (int g = 0; g < per; g++) {
        const int64_t at = piece * per + g;
        const bool in = row < n && at < groups;
        s[g] = in ? (uint16_t)from.scale(row, at, groups) : (uint16_t)0;
        if (zeros && in)
            z |= (uint64_t)from.zero(row, at, groups) << (4 * g);
    }
    if (zeros)
        for (int b = 0; b < per / 2; b++)
            zeros[item * (per / 2) + b] = (uint8_t)(z >> (8 * b));
}

// The first workgroups pack the codes, a tile a wave, the others the scales, an item a thread: one
// launch, as many a small matrix is packed (an expert's, one at a time: 8.8 us, the host's).  14336 x 4096 with zero
// points: 28 us (90 MB, 3.1 TB/s).
template <class Codes, class Scales>
__global__ void __launch_bounds__(256) q4g_pack_kernel(Codes codes, Scales from, uint8_t *wp, int64_t first, int64_t n,
                                                       int64_t k, int group, int fmt)
{
    const Q4gShape sh(n, k, group, fmt);
    const int64_t tiles = sh.rt * sh.kt, block = first + blockIdx.x, code_blocks = (tiles + 3) / 4;
    if (block < code_blocks) {
        const int64_t tile = block * 4 + threadIdx.x / 64;
        if (tile < tiles)
            pack_codes(codes, wp, sh, tile, n, k);
    } else {
        const int64_t item = (block - code_blocks) * 256 + threadIdx.x;
        if (sh.end + item < sh.bytes) // the first of them, the bytes behind the regions too
            wp[sh.end + item] = 0;
        if (item < sh.rt * sh.ks * 16)
            pack_scales(from, wp + sh.scales, (fmt & kQ4gZeros) ? wp + sh.zeros : nullptr, sh.ks, item, n, k / group, group);
    }
}

template <class Codes, class Scales>
hipError_t pack(const Codes &codes, const Scales &from, int64_t group, int fmt, uint8_t *wp, int64_t n, int64_t k,
                hipStream_t s)
{
    const Q4gShape sh(n, k, group, fmt);
    const int64_t blocks = (sh.rt * sh.kt + 3) / 4 + (sh.rt * sh.ks * 16 + 255) / 256;
    return launch_parts(blocks, kPartThreads / 256, [&](int64_t first, int64_t count) {
        q4g_pack_kernel<<<(unsigned)count, 256, 0, s>>>(codes, from, wp, first, n, k, (int)group, fmt);
    });
}

// ------------------------------------------------------------ linear layer

struct Q4gLinear {
    const uint8_t *wp;
    const void *x;
    const float *bias;
    const void *res;
    void *y;
    float *part; // sums of parts of k, [part][m][n]
    int64_t m, n, k, row0, tok0; // row0, tok0: this launch's first workgroup of row tiles, first activation row
    int fmt, act, y_dtype;
    int kw, parts, tok_groups; // waves along k of a workgroup, workgroups along k, groups of activation rows
    int rw;                    // sets of kw waves of a workgroup
};

// The sums of a workgroup's waves: RTN row tiles and C column groups each, sets of kw waves adding up
// in LDS; then the epilogue, or a part of k as it is.
template <int RTN, int C, int N>
__device__ __forceinline__ void q4g_outputs(const Q4gLinear &a, const float (&y)[RTN][C][N], int64_t rt0, int64_t tok0,
                                            float *sums, int lane)
{
    constexpr int kOuts = RTN * C * N, kTokens = 4 * N; // kTokens: of a column group
    const int wave = wave_number(), kw = wave % a.kw, set = wave - kw;
    if (a.kw > 1) {
        __syncthreads(); // LDS is read
#pragma unroll
        for (int o = 0; o < kOuts; o++)
            sums[(wave * kOuts + o) * 64 + lane] = y[o / (C * N)][o / N % C][o % N];
        __syncthreads();
    }
#pragma unroll
    for (int o = 0; o < kOuts; o++) {
        if (a.kw > 1 && o % a.kw != kw) // the set's waves take turns
            continue;
        const int r = o / (C * N), c = o / N % C, i = o % N;
        float v = y[r][c][i];
        if (a.kw > 1) {
            v = sums[(set * kOuts + o) * 64 + lane];
            for (int p = 1; p < a.kw; p++)
                v += sums[((set + p) * kOuts + o) * 64 + lane];
        }
        const int64_t j = (rt0 + r) * 16 + lane % 16, t = tok0 + kTokens * c + lane / 16 * N + i;
        if (j >= a.n || t >= a.m)
            continue;
        if (a.parts > 1) {
            a.part[(blockIdx.y * a.m + t) * a.n + j] = v;
            continue;
        }
        v = activate(a.bias ? v + a.bias[j] : v, a.act);
        if (a.res)
            v += load_as(a.res, t * a.n + j, a.y_dtype);
        store_as(a.y, t * a.n + j, v, a.y_dtype);
    }
}

// Few activation rows, or a small product: the waves of a set share its row tiles' pieces of k;
// groups of 16 / PK activation rows along y.  Four steps an operand while there are four rows, each wave
// fetching them: 4096 -> 14336, one bf16 row, 8.8 to 9.8 us (31 MB, 3.5 TB/s; loading alone would take 6.1): 613 vector
// instructions a wave, which are half of that time, and waves that wait a third of theirs to issue; one f32 row 13.4
// (947, three times the matrix instructions).  512 -> 512 takes 4.2 us, of which 1.8 is an empty
// launch's and the rest one trip to memory for a wave, the sums and the store.  1440 -> 4099 on 37 rows of f32 13 us:
// three groups read the codes, and a wave's 96 matrix instructions and 1968 others wait for
// one tile at a time (more in flight takes more registers than two workgroups a CU leave).
template <int TX, int GRP, int RTN, int PK, int D>
__global__ void __launch_bounds__(512, 4) q4g_few_kernel(Q4gLinear a)
{
    using Wave = Q4gWave<TX, GRP, RTN, PK, D>;
    extern __shared__ float few_sums[]; // [8][RTN * N][64]
    const Q4gShape sh(a.n, a.k, GRP, a.fmt);
    const int lane = threadIdx.x % 64, wave = wave_number(), kw = wave % a.kw;
    const int64_t rt = ((a.row0 + blockIdx.x) * a.rw + wave / a.kw) * RTN, tok0 = a.tok0 + (int64_t)blockIdx.y * (16 / PK);
    Wave w;
    w.clear();
    if (rt < sh.rt) {
        typename Wave::From f;
        const int64_t rows = a.m - tok0; // past the last row: its values again
        const uint32_t row = Wave::row_of(lane) < rows ? Wave::row_of(lane) : (uint32_t)rows - 1;
#pragma unroll
        for (int r = 0; r < RTN; r++) // past the last tile: the last one again, not stored
            f.w[r] = Q4gRows(a.wp, sh, rt + r < sh.rt ? rt + r : sh.rt - 1, GRP, a.fmt);
        f.x = static_cast<const uint8_t *>(a.x) + tok0 * a.k * q4g_x_size(TX), f.at = row * (uint32_t)a.k * q4g_x_size(TX);
        f.part = 0, f.last = (int)a.k - 32, f.kt = (int)sh.kt;
        const int ks = (int)sh.ks, per = (ks + a.kw - 1) / a.kw, p0 = kw * per;
        w.run(f, p0, p0 + per < ks ? p0 + per : ks, a.fmt & kQ4gBf16, lane);
    }
    q4g_outputs(a, w.y, rt, tok0, few_sums, lane);
}

// More rows.  Workgroups eight apart land on the same XCD: those of one set of rows follow
// each other there, so that its weights stay in that L2.
//
// 16 rows, 14336 -> 4096: 13 to 14 us (33 MB, 2.4 TB/s), 2 to 4 to add up the parts; four waves a SIMD that wait for
// memory and for instructions to issue, each weight widened for one operand of 16 rows.  512 rows, 4096 ->
// 14336 in f16: 97 to 99 us (610 TFLOP/s; 91 back to back; bf16 112 and 105): some 5700 vector instructions a wave (bf16
// 7650) against 1024 of the matrix core, which widen the codes (nine for eight weights, 17 as bf16, again in each of
// the eight workgroups that share them) and scale each group's sum, and a wait for all eight waves every 512 weights.  64 x 32 outputs a wave: 64 x 64
// takes 106 us and twice as long at 128 rows, 16 x 64 152; sixteen waves at 128 registers spill.
template <int TX, int GRP, int RTN, int C, int PK, int WPS>
__global__ void __launch_bounds__(512, WPS) q4g_linear_kernel(Q4gLinear a)
{
    using Block = Q4gBlock<TX, GRP, RTN, C, PK>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const Q4gShape sh(a.n, a.k, GRP, a.fmt);
    const int lane = threadIdx.x % 64, wave = wave_number(), kw = wave % a.kw;
    const int64_t b = blockIdx.x, tg = b / 8 % a.tok_groups, rg = b / 8 / a.tok_groups * 8 + b % 8;
    const int64_t rt0 = ((a.row0 + rg) * a.rw + wave / a.kw) * RTN;
    const int64_t tok0 = a.tok0 + tg * Block::T;
    typename Block::X src;
    src.base = static_cast<const uint8_t *>(a.x) + tok0 * a.k * 2;
    src.part = a.m * a.k * 2, src.k = (int)a.k;
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int row = 16 / PK * c + Block::row_of(lane);
        src.at[c] = tok0 + row < a.m ? (uint32_t)row * (uint32_t)a.k * 2 : ~0u; // 64 rows: below 2^32 bytes
    }
    Q4gRows rows[RTN];
#pragma unroll
    for (int r = 0; r < RTN; r++) // past the last tile: the last one again, not stored
        rows[r] = Q4gRows(a.wp, sh, rt0 + r < sh.rt ? rt0 + r : sh.rt - 1, GRP, a.fmt);
    const int chunks = (int)((a.k + Block::kChunk - 1) / Block::kChunk), per = (chunks + a.parts - 1) / a.parts;
    const int x0 = blockIdx.y * per, x1 = x0 + per < chunks ? x0 + per : chunks;
    Block w;
    w.clear();
    if (x0 < x1)
        w.run(rows, rt0 < sh.rt, src, x0, x1, kw, a.kw, a.fmt & kQ4gBf16, false, lds, lane);
    q4g_outputs(a, w.y, rt0, tok0, reinterpret_cast<float *>(lds), lane);
}

constexpr int kMaxParts = 8; // of k, over workgroups

// The parts of k added up in order, and the epilogue: eight loads at once an output, bound by that trip to
// memory (16 x 4096 outputs 2 to 4 us).
__global__ void __launch_bounds__(256) q4g_finish_kernel(Q4gLinear a, int64_t first, int64_t count)
{
    const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= first + count)
        return;
    float parts[kMaxParts];
#pragma unroll
    for (int p = 0; p < kMaxParts; p++)
        parts[p] = p < a.parts ? a.part[p * a.m * a.n + i] : 0.0f;
    float v = parts[0];
#pragma unroll
    for (int p = 1; p < kMaxParts; p++)
        v += parts[p];
    v = activate(a.bias ? v + a.bias[i % a.n] : v, a.act);
    if (a.res)
        v += load_as(a.res, i, a.y_dtype);
    store_as(a.y, i, v, a.y_dtype);
}

// f32 rows as three bf16 parts [part][count], eight values a thread: split once, not by every wave that reads
// them (37 x 2592: 2.5 to 4.8 us, launch and memory latency).
__global__ void __launch_bounds__(256) q4g_split_kernel(const uint8_t *x, uint8_t *parts, int64_t first, int64_t eights,
                                                        int64_t count)
{
    const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= eights)
        return;
    const u32x4 *from = reinterpret_cast<const u32x4 *>(x + i * 32);
    u32x4 a, b, c;
    split3(from[0], from[1], a, b, c);
    *reinterpret_cast<u32x4 *>(parts + i * 16) = a;
    *reinterpret_cast<u32x4 *>(parts + count * 2 + i * 16) = b;
    *reinterpret_cast<u32x4 *>(parts + count * 4 + i * 16) = c;
}

// Whether a product takes the waves that fetch their own activations, in one launch and without a
// workspace: up to four rows; up to 16 while the codes are few (us, so and with the rows in LDS: 14336 x 4096, 16
// rows 14.3 and 17.5, f32 22 and 26; 32000 x 4096, 23 and 27, f32 50 and 43), but on short and wide matrices
// with 9 to 16 rows, where four operands a tile are too much (4096 x 14336, 16 rows 20.0 and 15.5); with more
// rows while the codes that all groups of 16 rows read are few (4096 x 4096, 96 rows 18.1 and 19.4, 128 rows 21.5 and 19.1,
// f32 32 rows 12.5 and 15.0, 64 rows 20.6 and 19.3; 2048 x 2048, 256 rows 13.2 and 15.0; 14336 x 4096, 17 rows 20.5
// and 19.8, 64 rows 44 and 28).
bool q4g_small(bool wide, int64_t m, int64_t n, int64_t k)
{
    if (m <= 4)
        return true;
    if (m <= 16)
        return !(m > 8 && n < 8192 && n * k > (int64_t)1 << 25) && n * k <= (int64_t)1 << (wide ? 27 : 28);
    return (m + 15) / 16 <= ((int64_t)3 << (wide ? 24 : 25)) / (n * k);
}

// How another product is split: T activation rows and `tiles` row tiles a wave, kw
// waves and `parts` workgroups along k.
struct Q4gSplit {
    int rows, tiles, kw, parts, sets; // sets of kw waves of a workgroup
};

// Up to 16 rows (8 as well, PK = 2) the weights are read once, and the work is split along k until some 4096
// waves share it, along workgroups too (whose sums a second launch adds up, which more rows make dear).
Q4gSplit q4g_split(bool wide, int64_t m, int64_t n, int64_t k)
{
    const int64_t rt = (n + 15) / 16, ks = (k + 511) / 512;
    Q4gSplit s{m <= 8 || (wide && m <= 16) ? 8 : 16, 1, 1, 1, 8}; // (16 rows of three parts: LDS of two workgroups)
    if (m > 16) {
        s.tiles = 2;
        if (!wide)
            s.rows = m <= 32 ? 32 : 64;
    }
    const int64_t base = 16384 / (s.rows * (wide ? 3 : 1)) / 512 * 512, chunk = base < 512 ? 512 : base;
    const int64_t pieces = chunk / 512, chunks = (k + chunk - 1) / chunk;
    const int64_t sets = (rt + s.tiles - 1) / s.tiles * ((m + s.rows - 1) / s.rows);
    while (2 * s.kw <= pieces && 2 * s.kw <= ks && sets * s.kw < 4096)
        s.kw *= 2;
    s.sets = 8 / s.kw;
    if (m <= 16) {
        while (2 * s.parts <= chunks && s.parts < kMaxParts && sets * s.kw * s.parts < 4096)
            s.parts *= 2;
        return s;
    }
    // More rows: the sets of a workgroup and the parts of k by what their rounds of workgroups cost, in us.  A
    // chunk takes 5.8, 5.3, 5.2, 6.5 us at one, two, four, eight sets of 64 rows and 4.0, 3.5, 3.4, 4.2 of 32 or of
    // three parts, as its loads and the wait for them are most of it; the parts are written, read
    // and added up by another launch (128 rows, 4096 x 4096, one set of all k 49 us, eight 53, four in four parts 20).
    constexpr double kSetCost[9] = {0, 5.8, 5.3, 0, 5.2, 0, 0, 0, 6.5};
    const double unit = s.rows == 64 ? 1.0 : 0.65;
    const int64_t at_once = s.rows == 32 ? 512 : 256;
    double least = 0;
    for (int parts = 1; parts <= kMaxParts && parts <= chunks; parts *= 2)
        for (int w = 8; w >= 1; w /= 2) {
            const int64_t groups = (rt + s.tiles * w - 1) / (s.tiles * w) * ((m + s.rows - 1) / s.rows) * parts;
            const double cost = (double)((groups + at_once - 1) / at_once * ((chunks + parts - 1) / parts)) * unit * kSetCost[w] +
                                (parts > 1 ? 3 + parts * m * n * 2.3e-6 : 0);
            if (least == 0 || cost < least)
                least = cost, s.sets = w, s.parts = parts;
        }
    return s;
}

size_t part_bytes(const Q4gSplit &s, int64_t m, int64_t n)
{
    return s.parts > 1 ? ((size_t)s.parts * m * n * sizeof(float) + 255) / 256 * 256 : 0;
}

template <int TX, int GRP, int RTN, int PK, int D>
hipError_t linear_few(Q4gLinear a, hipStream_t s)
{
    const int64_t rt = ((a.n + 15) / 16 + RTN - 1) / RTN, ks = (a.k + 511) / 512, groups = (a.m + 16 / PK - 1) / (16 / PK);
    int64_t kw = (4096 + rt * groups - 1) / (rt * groups); // some 4096 waves, a piece each at least
    kw = kw < ks ? kw : ks, kw = kw < 8 ? kw : 8;
    // sets a workgroup: one, until there are two workgroups for every CU
    const int64_t rw = rt * groups / 512;
    a.kw = (int)kw, a.rw = (int)(rw < 1 ? 1 : rw < 8 / kw ? rw : 8 / kw);
    const unsigned threads = 64 * a.kw * a.rw;
    hipError_t e = hipSuccess;
    for (int64_t g0 = 0; g0 < groups && e == hipSuccess; g0 += 1 << 12) {
        const int64_t gn = groups - g0 < 1 << 12 ? groups - g0 : 1 << 12;
        a.tok0 = g0 * (16 / PK);
        e = launch_parts((rt + a.rw - 1) / a.rw, kPartThreads / 512, [&](int64_t first, int64_t count) {
            a.row0 = first;
            q4g_few_kernel<TX, GRP, RTN, PK, D><<<dim3((unsigned)count, (unsigned)gn), threads,
                                                 a.kw > 1 ? 8 * RTN * (4 / PK) * 64 * sizeof(float) : 0, s>>>(a);
        });
    }
    return e;
}

template <int TX, int GRP, int RTN, int C, int PK, int WPS>
hipError_t linear_c(Q4gLinear a, const Q4gSplit &split, hipStream_t s)
{
    using Block = Q4gBlock<TX, GRP, RTN, C, PK>;
    a.kw = split.kw, a.rw = split.sets, a.parts = split.parts;
    const int64_t sets = ((a.n + 15) / 16 + RTN * a.rw - 1) / (RTN * a.rw), threads = 64 * a.kw * a.rw;
    const size_t sums = a.kw > 1 ? (size_t)8 * RTN * C * Block::N * 64 * sizeof(float) : 0;
    const size_t x = Block::lds_bytes(a.k), lds = x > sums ? x : sums;
    const int64_t groups = (a.m + Block::T - 1) / Block::T;
    hipError_t e = hipSuccess;
    for (int64_t g0 = 0; g0 < groups && e == hipSuccess; g0 += 1 << 12) {
        const int64_t gn = groups - g0 < 1 << 12 ? groups - g0 : 1 << 12;
        a.tok0 = g0 * Block::T, a.tok_groups = (int)gn;
        // parts of eight sets, so that only the last one's grid reaches past its rows
        e = launch_parts(sets, kPartThreads / (threads * gn) / 8 * 8, [&](int64_t first, int64_t count) {
            a.row0 = first;
            const dim3 grid((unsigned)((count + 7) / 8 * 8 * gn), (unsigned)a.parts);
            q4g_linear_kernel<TX, GRP, RTN, C, PK, WPS><<<grid, (unsigned)threads, lds, s>>>(a);
        });
    }
    if (e != hipSuccess || a.parts == 1)
        return e;
    return launch_parts(a.m * a.n, kPartThreads, [&](int64_t first, int64_t count) {
        q4g_finish_kernel<<<(unsigned)((count + 255) / 256), 256, 0, s>>>(a, first, count);
    });
}

template <int TX, int GRP>
hipError_t linear_more(const Q4gLinear &a, const Q4gSplit &split, hipStream_t s)
{
    if (split.rows == 8)
        return linear_c<TX, GRP, 1, 1, 2, 4>(a, split, s);
    if constexpr (TX == Q4G_X_PARTS3)
        return linear_c<TX, GRP, 2, 1, 1, 2>(a, split, s);
    else
        return split.tiles == 1   ? linear_c<TX, GRP, 1, 1, 1, 4>(a, split, s)
               : split.rows == 32 ? linear_c<TX, GRP, 2, 2, 1, 2>(a, split, s)
                                  : linear_c<TX, GRP, 2, 4, 1, 2>(a, split, s);
}

template <int TX, int GRP>
hipError_t linear_small(const Q4gLinear &a, hipStream_t s)
{
    return a.m <= 4   ? linear_few<TX, GRP, 1, 4, 4>(a, s)
           : a.m <= 8 ? linear_few<TX, GRP, 1, 2, 2>(a, s)
                      : linear_few<TX, GRP, 2, 1, TX == Q4G_X_F32 ? 1 : 2>(a, s);
}

template <int GRP>
hipError_t linear_g(Q4gLinear a, int dtype, uint8_t *ws, hipStream_t s)
{
    if (q4g_small(dtype == QLL_W_F32, a.m, a.n, a.k))
        return dtype == QLL_W_F32    ? linear_small<Q4G_X_F32, GRP>(a, s)
               : dtype == QLL_W_BF16 ? linear_small<Q4G_X_BF16, GRP>(a, s)
                                     : linear_small<Q4G_X_F16, GRP>(a, s);
    const Q4gSplit split = q4g_split(dtype == QLL_W_F32, a.m, a.n, a.k);
    a.part = reinterpret_cast<float *>(ws);
    if (dtype != QLL_W_F32)
        return dtype == QLL_W_BF16 ? linear_more<Q4G_X_BF16, GRP>(a, split, s) : linear_more<Q4G_X_F16, GRP>(a, split, s);
    uint8_t *parts = ws + part_bytes(split, a.m, a.n);
    const hipError_t e = launch_q4g_split(a.x, parts, a.m * a.k, s);
    if (e != hipSuccess)
        return e;
    a.x = parts;
    return linear_more<Q4G_X_PARTS3, GRP>(a, split, s);
}

} // namespace

size_t q4g_packed_bytes(int64_t n, int64_t k, int64_t group, int fmt) { return (size_t)Q4gShape(n, k, group, fmt).bytes; }

hipError_t launch_q4g_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int64_t group, int fmt,
                           uint8_t *wp, int64_t n, int64_t k, hipStream_t s)
{
    return pack(CodeBytes{codes}, ScaleArray{scales, zeros}, group, fmt, wp, n, k, s);
}

hipError_t launch_q4g_from_q4_0(const uint8_t *w, uint8_t *wp, int64_t n, int64_t k, hipStream_t s)
{
    return pack(CodeBlocks{w}, ScaleBlocks{w}, 32, 0, wp, n, k, s);
}

hipError_t launch_q4g_split(const void *x, void *parts, int64_t count, hipStream_t s)
{
    return launch_parts(count / 8, kPartThreads, [&](int64_t first, int64_t n) {
        q4g_split_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(static_cast<const uint8_t *>(x),
                                                                    static_cast<uint8_t *>(parts), first, count / 8, count);
    });
}

size_t q4g_linear_workspace(int64_t m, int64_t n, int64_t k)
{
    size_t need = 0; // of whichever type of rows takes more
    if (!q4g_small(false, m, n, k))
        need = part_bytes(q4g_split(false, m, n, k), m, n);
    if (!q4g_small(true, m, n, k)) {
        const size_t wide = part_bytes(q4g_split(true, m, n, k), m, n) + (size_t)(m * k) * 6;
        need = need > wide ? need : wide;
    }
    return need;
}

hipError_t launch_q4g_linear(const uint8_t *wp, int64_t group, int fmt, const void *x, int dtype, const float *bias,
                             int act, const void *res, void *y, int y_dtype, int64_t m, int64_t n, int64_t k, void *ws,
                             hipStream_t s)
{
    Q4gLinear a{};
    a.wp = wp, a.x = x, a.bias = bias, a.res = res, a.y = y;
    a.m = m, a.n = n, a.k = k, a.fmt = fmt, a.act = act, a.y_dtype = y_dtype;
    a.kw = a.parts = a.tok_groups = 1;
    uint8_t *w = static_cast<uint8_t *>(ws);
    return group == 32 ? linear_g<32>(a, dtype, w, s) : group == 64 ? linear_g<64>(a, dtype, w, s) : linear_g<128>(a, dtype, w, s);
}

} // namespace qll
