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

template <class Codes>
__global__ void __launch_bounds__(256) q4g_pack_codes_kernel(Codes codes, uint8_t *wp, int64_t tile0, int64_t tiles,
                                                             int64_t kt, int64_t n, int64_t k)
{
    const int64_t tile = tile0 + (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    if (tile >= tile0 + tiles)
        return;
    const int lane = threadIdx.x % 64;
    const int64_t row = tile / kt * 16 + lane % 16, t = tile % kt * 128 + lane / 16 * 8;
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (row < n && t + 32 * j < k)
            v[j] = codes.eight(row, t + 32 * j, k);
    *reinterpret_cast<u32x4 *>(wp + tile * 1024 + lane * 16) = v;
}

// Scales (and zeros) of one row and chunk of 512 weights a thread.
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

template <class Scales>
__global__ void __launch_bounds__(256) q4g_pack_scales_kernel(Scales from, uint8_t *scales, uint8_t *zeros,
                                                              int64_t item0, int64_t items, int64_t ks, int64_t n,
                                                              int64_t groups, int group)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= items)
        return;
    const int64_t item = item0 + i, row = item / 16 / ks * 16 + item % 16, chunk = item / 16 % ks;
    const int per = 512 / group;
    uint16_t *s = reinterpret_cast<uint16_t *>(scales) + item * per;
    uint64_t z = 0;
    for (int g = 0; g < per; g++) {
        const int64_t at = chunk * per + g;
        const bool in = row < n && at < groups;
        s[g] = in ? (uint16_t)from.scale(row, at, groups) : (uint16_t)0;
        if (zeros && in)
            z |= (uint64_t)from.zero(row, at, groups) << (4 * g);
    }
    if (zeros)
        for (int b = 0; b < per / 2; b++)
            zeros[item * (per / 2) + b] = (uint8_t)(z >> (8 * b));
}

template <class Codes, class Scales>
hipError_t pack(const Codes &codes, const Scales &from, int64_t group, int fmt, uint8_t *wp, int64_t n, int64_t k,
                hipStream_t s)
{
    const Q4gShape sh(n, k, group, fmt);
    hipError_t e = launch_parts(sh.rt * sh.kt, kPartThreads / 64, [&](int64_t first, int64_t count) {
        q4g_pack_codes_kernel<<<(unsigned)((count + 3) / 4), 256, 0, s>>>(codes, wp, first, count, sh.kt, n, k);
    });
    if (e != hipSuccess)
        return e;
    return launch_parts(sh.rt * sh.ks * 16, kPartThreads, [&](int64_t first, int64_t count) {
        q4g_pack_scales_kernel<<<(unsigned)((count + 255) / 256), 256, 0, s>>>(
            from, wp + sh.scales, (fmt & kQ4gZeros) ? wp + sh.zeros : nullptr, first, count, sh.ks, n, k / group,
            (int)group);
    });
}

// ------------------------------------------------------------ linear layer

struct Q4gLinear {
    const uint8_t *wp;
    const void *x;
    const float *bias;
    const void *res;
    void *y;
    int64_t m, n, k, row0, tok0; // row0, tok0: this launch's first group of row tiles, first activation row
    int fmt, act, y_dtype;
    int kw, rw, tok_groups; // waves along k and along rows of a workgroup; groups of 16 C activation rows
};

// kw waves share RTN row tiles, each a part of k, and add up in LDS; rw such
// sets a workgroup.  Workgroups eight apart land on the same XCD: those of one set of
// rows follow each other there, so that its weights stay in that L2.
template <int TX, int GRP, int RTN, int C, int PK, int D>
__global__ void __launch_bounds__(512) q4g_linear_kernel(Q4gLinear a)
{
    using Wave = Q4gWave<TX, GRP, RTN, C, PK, D>;
    constexpr int kTokens = 16 / PK; // of a column group
    extern __shared__ float part[];  // [rw][kw][RTN * C * N][64]
    const Q4gShape sh(a.n, a.k, GRP, a.fmt);
    const int lane = threadIdx.x % 64, wave = wave_number(), kw = wave % a.kw, rw = wave / a.kw;
    const int64_t b = blockIdx.x, tg = b / 8 % a.tok_groups, rg = b / 8 / a.tok_groups * 8 + b % 8;
    const int64_t rt0 = (a.row0 + rg * a.rw + rw) * RTN;
    const int64_t tok0 = a.tok0 + tg * kTokens * C;
    Wave w;
    w.clear();
    if (rt0 < sh.rt) {
        typename Wave::Rows rows;
#pragma unroll
        for (int r = 0; r < RTN; r++) // past the last tile: the last one again, not stored
            rows.w[r] = Q4gRows(a.wp, sh, rt0 + r < sh.rt ? rt0 + r : sh.rt - 1, GRP, a.fmt);
#pragma unroll
        for (int c = 0; c < C; c++) {
            int64_t t = kTokens * c + Wave::row_of(lane);
            t = tok0 + t < a.m ? t : a.m - 1 - tok0; // rows past the last: its values again, not stored
            rows.at[c] = (uint32_t)(t * a.k * q4g_x_size(TX)); // 32 rows of f32, 64 of 16 bits: below 2^32
        }
        rows.x = static_cast<const uint8_t *>(a.x) + tok0 * a.k * q4g_x_size(TX);
        rows.part = 0, rows.last = (int)a.k - 32, rows.bf16 = a.fmt & kQ4gBf16, rows.lane = lane;
        const int kt = (int)sh.kt, per = (kt + a.kw - 1) / a.kw, t0 = kw * per, t1 = t0 + per < kt ? t0 + per : kt;
        w.run(rows, t0, t1);
    }
    constexpr int kOuts = RTN * C * Wave::N;
    if (a.kw > 1) {
#pragma unroll
        for (int o = 0; o < kOuts; o++)
            part[(wave * kOuts + o) * 64 + lane] = w.y[o / (C * Wave::N)][o / Wave::N % C][o % Wave::N];
        __syncthreads();
    }
#pragma unroll
    for (int o = 0; o < kOuts; o++) {
        if (o % a.kw != kw) // the set's waves take turns
            continue;
        const int r = o / (C * Wave::N), c = o / Wave::N % C, i = o % Wave::N;
        float v = w.y[r][c][i];
        if (a.kw > 1) {
            v = part[(rw * a.kw * kOuts + o) * 64 + lane];
            for (int p = 1; p < a.kw; p++)
                v += part[((rw * a.kw + p) * kOuts + o) * 64 + lane];
        }
        const int64_t j = (rt0 + r) * 16 + lane % 16, t = tok0 + kTokens * c + Wave::out_of(lane, i);
        if (j >= a.n || t >= a.m)
            continue;
        v = activate(a.bias ? v + a.bias[j] : v, a.act);
        if (a.res)
            v += load_as(a.res, t * a.n + j, a.y_dtype);
        store_as(a.y, t * a.n + j, v, a.y_dtype);
    }
}

template <int TX, int GRP, int RTN, int C, int PK, int D>
hipError_t linear_c(Q4gLinear a, int kw, int rw, hipStream_t s)
{
    constexpr int kTokens = 16 / PK * C; // of a workgroup
    a.kw = kw, a.rw = rw;
    const int64_t sets = ((a.n + 15) / 16 + RTN * rw - 1) / (RTN * rw), threads = 64 * kw * rw;
    const size_t lds = kw > 1 ? (size_t)rw * kw * RTN * C * (4 / PK) * 64 * sizeof(float) : 0;
    const int64_t groups = (a.m + kTokens - 1) / kTokens;
    hipError_t e = hipSuccess;
    for (int64_t g0 = 0; g0 < groups && e == hipSuccess; g0 += 1 << 12) {
        const int64_t gn = groups - g0 < 1 << 12 ? groups - g0 : 1 << 12;
        a.tok0 = g0 * kTokens, a.tok_groups = (int)gn;
        // parts of eight sets, so that only the last one's grid reaches past its rows
        e = launch_parts(sets, kPartThreads / (threads * gn) / 8 * 8, [&](int64_t first, int64_t count) {
            a.row0 = first * rw;
            const int64_t blocks = (count + 7) / 8 * 8 * gn;
            q4g_linear_kernel<TX, GRP, RTN, C, PK, D><<<(unsigned)blocks, (unsigned)threads, lds, s>>>(a);
        });
    }
    return e;
}

template <int TX, int GRP>
hipError_t linear_x(const Q4gLinear &a, hipStream_t s)
{
    const int64_t rt = (a.n + 15) / 16, kt = (a.k + 127) / 128;
    auto split = [&](int64_t sets) { // waves along k: enough to fill the chip, two tiles each at least
        int kw = 1;
        while (kw < 8 && sets * kw < 4096 && 2 * kw <= kt)
            kw *= 2;
        return kw;
    };
    const int kw1 = split(rt), rw1 = kw1 < 4 ? 4 / kw1 : 1;
    if (a.m <= 4)
        return linear_c<TX, GRP, 1, 1, 4, 4>(a, kw1, rw1, s);
    if (a.m <= 8)
        return linear_c<TX, GRP, 1, 1, 2, 4>(a, kw1, rw1, s);
    if (a.m <= 16)
        return linear_c<TX, GRP, 1, 1, 1, 2>(a, kw1, rw1, s);
    const int kw = split((rt + 1) / 2 * ((a.m + 31) / 32));
    return linear_c<TX, GRP, 2, 2, 1, 1>(a, kw, kw < 4 ? 4 / kw : 1, s);
}

template <int TX>
hipError_t linear_g(const Q4gLinear &a, int64_t group, hipStream_t s)
{
    return group == 32 ? linear_x<TX, 32>(a, s) : group == 64 ? linear_x<TX, 64>(a, s) : linear_x<TX, 128>(a, s);
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

hipError_t launch_q4g_linear(const uint8_t *wp, int64_t group, int fmt, const void *x, int dtype, const float *bias,
                             int act, const void *res, void *y, int y_dtype, int64_t m, int64_t n, int64_t k,
                             hipStream_t s)
{
    const Q4gLinear a{wp, x, bias, res, y, m, n, k, 0, 0, fmt, act, y_dtype, 1, 1, 1};
    return dtype == QLL_W_F32    ? linear_g<Q4G_X_F32>(a, group, s)
           : dtype == QLL_W_BF16 ? linear_g<Q4G_X_BF16>(a, group, s)
                                 : linear_g<Q4G_X_F16>(a, group, s);
}

} // namespace qll
