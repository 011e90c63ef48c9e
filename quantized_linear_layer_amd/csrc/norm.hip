// Root-mean-square norm of the residual stream straight into the activation
// formats of the linear layers: for every row
//     h   = T(f32(x) + f32(residual))            T: the stream's type
//     v_t = h_t * w_t / rms,   rms = sqrt(mean_t h_t^2 + eps)
// and v quantized to Q8_0 blocks (Fucina reference "Backends", 9.7) or to one
// int8 row with its scale and code sum (Loom "Plan 9 SIMD Forward", "BitNet
// ternary MAD kernel").
//
// A code is round(127 v_t / max |v|) over its block (or row), and rms cancels
// from it:
//     q_t = round(127 p_t / A),   p_t = h_t w_t,   A = max |p|
// so the codes do not wait for the row's sum of squares, and the only thing
// left for the end is the scale, A / (127 rms) (its inverse for int8 rows).
// p is the exact product (two 24-bit significands in f64) and the quotient is
// rounded as f64 has it, so a code depends on nothing but its own block's
// values: not on how the sum of squares was split, nor on the launch shape.
// Vector f64 runs at the rate of f32 here (without packed f32), so this costs
// little: 25 instructions an element, counted, against the 47 that the 7 bytes of a
// bf16 stream with residual leave at 5.8 TB/s (20 for the 3 bytes of one without).
// Measured: 8192 x 4096 f32 with residual to Q8_0 75 us (438 MB, 5.8 TB/s), 4096 x 6912
// bf16 with residual to int8 46 us (198 MB, 4.3 TB/s); one row of 4096 3.0 us.
#include "common.h"

namespace qll {

typedef _Float16 f16x4_n __attribute__((ext_vector_type(4)));

// Four consecutive elements of a stream row as loaded.
template <typename T>
struct Piece4;
template <>
struct Piece4<float> {
    float4 v;
};
template <>
struct Piece4<uint16_t> { // bf16
    ushort4 v;
};
template <>
struct Piece4<_Float16> {
    f16x4_n v;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widen(_Float16 v) { return (float)v; }

// f32 -> T, round to nearest even.
__device__ __forceinline__ void narrow(float f, float &o) { o = f; }
__device__ __forceinline__ void narrow(float f, _Float16 &o) { o = (_Float16)f; }
__device__ __forceinline__ void narrow(float f, uint16_t &o) { o = __builtin_bit_cast(uint16_t, (__bf16)f); }

// V consecutive elements at p (V = 4: aligned to four elements).
template <int V, typename T>
struct Elems {
    T e[V];
};
template <int V, typename T>
__device__ __forceinline__ Elems<V, T> load_elems(const T *p)
{
    Elems<V, T> r;
    if constexpr (V == 4)
        r = __builtin_bit_cast(Elems<V, T>, *reinterpret_cast<const Piece4<T> *>(p));
    else
        r.e[0] = *p;
    return r;
}
template <int V, typename T>
__device__ __forceinline__ void store_elems(T *p, const Elems<V, T> &v)
{
    if constexpr (V == 4)
        *reinterpret_cast<Piece4<T> *>(p) = __builtin_bit_cast(Piece4<T>, v);
    else
        *p = v.e[0];
}

// 127 / a to about one unit in the last place of f64 (a > 0: a product of two
// f32 values, so far inside f64's normal range): the reciprocal instruction's
// estimate and two Newton steps.
__device__ __forceinline__ double code_factor(double a)
{
    double r = __builtin_amdgcn_rcp(a);
    r = fma(fma(-a, r, 1.0), r, r);
    r = fma(fma(-a, r, 1.0), r, r);
    return a > 0.0 ? 127.0 * r : 0.0;
}

// 1 / sqrt(v), v > 0, the same way.
__device__ __forceinline__ double inverse_root(double v)
{
    double r = __builtin_amdgcn_rsq(v);
    r = fma(fma(-v * r, r, 1.0), 0.5 * r, r);
    return fma(fma(-v * r, r, 1.0), 0.5 * r, r);
}

// The codes of V products, round-half-away(127 p / a) as f64 arithmetic has it,
// f = 127 / a.  p f is within 1e-13 of the quotient: adding 1.5 2^52 rounds it to
// the nearest integer, which then stands in the low bits, and only within 1e-6 of
// a border is the division itself needed (values drawn from few significant bits
// do land on borders, and then the quotient is exactly k + 1/2).
template <int V>
__device__ __forceinline__ void norm_codes(const double (&p)[V], double a, double f, int (&q)[V])
{
    constexpr double kMagic = 6755399441055744.0;
    double y[V], worst = 0.0;
#pragma unroll
    for (int e = 0; e < V; e++) {
        y[e] = fma(p[e], f, kMagic);
        worst = fmax(worst, fabs(fma(p[e], f, kMagic - y[e])));
        q[e] = (int)(uint32_t)__builtin_bit_cast(uint64_t, y[e]);
    }
    if (worst > 0.5 - 1e-6) {
#pragma unroll
        for (int e = 0; e < V; e++) {
            const int c = a > 0.0 ? (int)floor(127.0 * fabs(p[e]) / a + 0.5) : 0;
            q[e] = p[e] < 0.0 ? -c : c;
        }
    }
}

__device__ __forceinline__ uint32_t pack4(const int (&q)[4])
{
    const uint32_t lo = __builtin_amdgcn_perm((uint32_t)q[1], (uint32_t)q[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm((uint32_t)q[3], (uint32_t)q[2], 0x04000c0cu);
    return lo | hi;
}

// v as another lane of the same 16 has it: the neighbour (kXor1), the other pair
// of the quad (kXor2), the other quad of eight lanes (kHalf: what holds after the
// two before), the other eight of sixteen (kRow).
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalf = 0x141, kRow = 0x140;
template <int CTRL>
__device__ __forceinline__ double lane_f64(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int LANE>
__device__ __forceinline__ double from_lane_f64(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, LANE);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), LANE);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Over the 64 lanes, in every lane.
__device__ __forceinline__ double wave_sum(double v)
{
    v += lane_f64<kXor1>(v);
    v += lane_f64<kXor2>(v);
    v += lane_f64<kHalf>(v);
    v += lane_f64<kRow>(v);
    return (from_lane_f64<0>(v) + from_lane_f64<16>(v)) + (from_lane_f64<32>(v) + from_lane_f64<48>(v));
}
__device__ __forceinline__ double wave_max(double v)
{
    v = fmax(v, lane_f64<kXor1>(v));
    v = fmax(v, lane_f64<kXor2>(v));
    v = fmax(v, lane_f64<kHalf>(v));
    v = fmax(v, lane_f64<kRow>(v));
    return fmax(fmax(from_lane_f64<0>(v), from_lane_f64<16>(v)), fmax(from_lane_f64<32>(v), from_lane_f64<48>(v)));
}

// Sum (and, with MAX, the largest `mx`) over the TPR threads of a row; `red`:
// one slot per wave.
template <int TPR, bool MAX>
__device__ __forceinline__ void row_reduce(double &sum, double &mx, double (*red)[2])
{
    sum = wave_sum(sum);
    if (MAX)
        mx = wave_max(mx);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            red[wave][0] = sum;
            if (MAX)
                red[wave][1] = mx;
        }
        __syncthreads();
        sum = red[0][0];
        if (MAX)
            mx = red[0][1];
#pragma unroll
        for (int i = 1; i < TPR / 64; i++) {
            sum += red[i][0];
            if (MAX)
                mx = fmax(mx, red[i][1]);
        }
    }
}

// The stream's pieces of one thread: h (stored to hout if that is wanted) and
// the products with the norm's weights.
template <typename T, bool RES, int V>
__device__ __forceinline__ void norm_products(const Elems<V, T> &x, const Elems<V, T> &r, const Elems<V, float> &w,
                                              T *hout, double &ss, double (&p)[V])
{
    Elems<V, T> h = x;
#pragma unroll
    for (int e = 0; e < V; e++) {
        if (RES)
            narrow(widen(x.e[e]) + widen(r.e[e]), h.e[e]);
        const double hd = (double)widen(h.e[e]);
        ss = fma(hd, hd, ss);
        p[e] = hd * (double)w.e[e];
    }
    if (hout)
        store_elems<V>(hout, h);
}

// Codes of four products; the eight lanes that share a Q8_0 block call it
// together, and a is the block's maximum.
__device__ __forceinline__ uint32_t block_codes(const double (&p)[4], double &a)
{
    double mx = fmax(fmax(fabs(p[0]), fabs(p[1])), fmax(fabs(p[2]), fabs(p[3])));
    mx = fmax(mx, lane_f64<kXor1>(mx));
    mx = fmax(mx, lane_f64<kXor2>(mx));
    mx = fmax(mx, lane_f64<kHalf>(mx));
    int q[4];
    norm_codes<4>(p, mx, code_factor(mx), q);
    a = mx;
    return pack4(q);
}

// Pieces whose loads a thread has out at once: the whole row's up to 256 threads
// (4096 x 6912 bf16 into int8 rows with residual: 42 us, 51 with four, 57 with
// two), four with more threads, where eight cost too many registers (1024 x
// 13824: 24 us, 27 with eight).
constexpr int norm_group(int tpr, int p) { return tpr <= 256 || p < 4 ? p : 4; }

// Dword that only promises 2-byte alignment (codes of a Q8_0 block).
typedef uint32_t u32_a2 __attribute__((aligned(2)));

__device__ __forceinline__ void store_codes(uint8_t *blk, int sub, uint32_t c)
{
    *reinterpret_cast<u32_a2 *>(blk + 2 + 4 * sub) = c;
}

// 1 / (127 rms), v = rms^2.  A row with NaN or an infinity in it (v is NaN or
// infinite, and inverse_root takes 0 times it) has a factor of NaN, which reaches the
// scale of every block: a block's maximum drops its NaN, and is 0 where the others
// are zeros.  A row of zeros with eps = 0 has 0.
__device__ __forceinline__ double block_factor(double v) { return v == 0.0 ? 0.0 : inverse_root(v) * (1.0 / 127.0); }

// d of a block with maximum a; scale: block_factor of its row.
__device__ __forceinline__ void store_scale(uint8_t *blk, double a, double scale)
{
    float d = (float)(a * scale);
    // two roundings, as the quantizer's: the compiler would otherwise convert
    // f64 to binary16 in one (and in a long sequence of integer operations)
    asm volatile("" : "+v"(d));
    *reinterpret_cast<uint16_t *>(blk) = float_to_half_bits(d);
}

// 127 rms / a, v = rms^2, as the int8 quantizer keeps it: a row whose scale is not finite,
// or that is all zeros, has scale 0.
__device__ __forceinline__ float row_scale(double v, double a)
{
    const float sc = a > 0.0 ? (float)(code_factor(a) * (v * inverse_root(v))) : 0.0f;
    return __builtin_isfinite(sc) ? sc : 0.0f;
}

// Codes of one piece of an int8 row, stored; returns their sum.
template <int V>
__device__ __forceinline__ int store_i8(int8_t *q8, const double (&p)[V], double a, double f)
{
    int q[V], sum = 0;
    norm_codes<V>(p, a, f, q);
#pragma unroll
    for (int e = 0; e < V; e++)
        sum += q[e];
    if constexpr (V == 4)
        *reinterpret_cast<uint32_t *>(q8) = pack4(q);
    else
        *q8 = (int8_t)q[0];
    return sum;
}

// Sum of the row's codes; sc: its scale.  In a row without one (0) the codes of NaN are
// the low bits of NaN: zero in the byte that is stored, but not in the 32 that are summed.
template <int TPR>
__device__ __forceinline__ int row_sum(int sum, float sc, int *red)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        sum += __shfl_xor(sum, off);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = sum;
        __syncthreads();
        sum = 0;
#pragma unroll
        for (int i = 0; i < TPR / 64; i++)
            sum += red[i];
    }
    return sc > 0.0f ? sum : 0;
}

// Q8_0 output.  TPR threads per row (64: four rows share a workgroup), thread
// t of a row takes the four-element pieces t, t + TPR, ...: eight consecutive
// lanes share a block.  Each piece's codes and block maximum are formed at once
// and held (three registers for four elements) until the row's sum is known.
template <typename T, bool RES, int TPR, int P>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_q8_0_kernel(const T *x, const T *res,
                                                                             const float *__restrict__ w, double eps, double inv_k,
                                                                             T *h, uint8_t *__restrict__ xq,
                                                                             int64_t m, int k)
{
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1; // rows per workgroup
    __shared__ double red[TPR > 64 ? TPR / 64 : 1][2];
    const int t = RPW > 1 ? threadIdx.x % TPR : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * RPW + (RPW > 1 ? threadIdx.x / TPR : 0);
    if (RPW > 1 && row >= m)
        return; // a whole wave: nothing below meets across waves when RPW > 1
    const int np = k / 4;
    const int64_t base = row * k;
    constexpr int G = norm_group(TPR, P);
    double ss = 0.0, a[P];
    uint32_t code[P];
#pragma unroll
    for (int g = 0; g < P; g += G) {
        Elems<4, T> xe[G], re[G];
        Elems<4, float> we[G];
#pragma unroll
        for (int j = 0; j < G; j++) {
            const int i = t + TPR * (g + j);
            const int o = 4 * (i < np ? i : 0); // past the row: its first piece, masked below
            xe[j] = load_elems<4>(x + base + o);
            if (RES)
                re[j] = load_elems<4>(res + base + o);
            we[j] = load_elems<4>(w + o);
        }
#pragma unroll
        for (int j = 0; j < G; j++) {
            const int i = t + TPR * (g + j);
            const bool ok = i < np;
            double s1 = 0.0, p[4];
            norm_products<T, RES, 4>(xe[j], re[j], we[j], h && ok ? h + base + 4 * i : nullptr, s1, p);
            ss += ok ? s1 : 0.0;
            code[g + j] = block_codes(p, a[g + j]);
        }
    }
    double unused = 0.0;
    row_reduce<TPR, false>(ss, unused, red);
    const double scale = block_factor(fma(ss, inv_k, eps));
#pragma unroll
    for (int j = 0; j < P; j++) {
        const int i = t + TPR * j;
        if (i < np) {
            uint8_t *blk = xq + (row * (k / 32) + (i >> 3)) * 34;
            store_codes(blk, i & 7, code[j]);
            if ((i & 7) == 0)
                store_scale(blk, a[j], scale);
        }
    }
}

// int8 rows.  The codes wait for the row's maximum, so h and w are held and
// their products taken again.  V = 4 where k % 4 == 0, else 1.
template <typename T, bool RES, int V, int TPR, int P>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_i8_rows_kernel(
    const T *x, const T *res, const float *__restrict__ w, double eps, double inv_k, T *h, int8_t *__restrict__ xq,
    float *__restrict__ act_scale, int32_t *__restrict__ act_sum, int64_t m, int k)
{
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    __shared__ double red[TPR > 64 ? TPR / 64 : 1][2];
    __shared__ int red_i[TPR > 64 ? TPR / 64 : 1];
    const int t = RPW > 1 ? threadIdx.x % TPR : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * RPW + (RPW > 1 ? threadIdx.x / TPR : 0);
    if (RPW > 1 && row >= m)
        return;
    const int np = k / V;
    const int64_t base = row * k;
    constexpr int G = V == 1 ? P : norm_group(TPR, P);
    Elems<V, T> xe[P];     // x, then h
    Elems<V, float> we[G]; // read again below where there is more than one group
    double ss = 0.0, mx = 0.0;
#pragma unroll
    for (int g = 0; g < P; g += G) {
        Elems<V, T> re[G];
#pragma unroll
        for (int j = 0; j < G; j++) {
            const int i = t + TPR * (g + j);
            const int o = V * (i < np ? i : 0);
            xe[g + j] = load_elems<V>(x + base + o);
            if (RES)
                re[j] = load_elems<V>(res + base + o);
            we[j] = load_elems<V>(w + o);
        }
#pragma unroll
        for (int j = 0; j < G; j++) {
            const int i = t + TPR * (g + j);
            const bool ok = i < np;
            Elems<V, T> &hv = xe[g + j];
#pragma unroll
            for (int e = 0; e < V; e++) {
                if (RES)
                    narrow(widen(hv.e[e]) + widen(re[j].e[e]), hv.e[e]);
                const double hd = ok ? (double)widen(hv.e[e]) : 0.0;
                ss = fma(hd, hd, ss);
                mx = fmax(mx, fabs(hd * (double)we[j].e[e]));
            }
            if (h && ok)
                store_elems<V>(h + base + V * i, hv);
        }
    }
    row_reduce<TPR, true>(ss, mx, red);
    const float sc = row_scale(fma(ss, inv_k, eps), mx);
    const double a = sc > 0.0f ? mx : 0.0, f = code_factor(a);
    int sum = 0;
#pragma unroll
    for (int j = 0; j < P; j++) {
        const int i = t + TPR * j;
        if (i < np) {
            const Elems<V, float> wj = P == G ? we[j % G] : load_elems<V>(w + V * i);
            double p[V];
#pragma unroll
            for (int e = 0; e < V; e++)
                p[e] = (double)widen(xe[j].e[e]) * (double)wj.e[e];
            sum += store_i8<V>(xq + base + V * i, p, a, f);
        }
    }
    sum = row_sum<TPR>(sum, sc, red_i);
    if (t == 0) {
        act_scale[row] = sc;
        act_sum[row] = sum;
    }
}

// Rows too long for registers (over 4096 pieces of four, or 16384 single
// elements): two sweeps, the second over h where it is kept (each thread reads
// back what it wrote) and over the inputs again where it is not.
template <typename T, bool RES, int V, bool Q8>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(const T *x, const T *res, const float *__restrict__ w,
                                                            double eps, double inv_k, T *h, uint8_t *__restrict__ xq,
                                                            float *__restrict__ act_scale,
                                                            int32_t *__restrict__ act_sum, int k)
{
    __shared__ double red[16][2];
    __shared__ int red_i[16];
    const int64_t row = blockIdx.x, base = row * k;
    const int np = k / V;
    double ss = 0.0, mx = 0.0;
    for (int i = threadIdx.x; i < np; i += 1024) {
        Elems<V, T> r;
        if (RES)
            r = load_elems<V>(res + base + (int64_t)V * i);
        double p[V];
        norm_products<T, RES, V>(load_elems<V>(x + base + (int64_t)V * i), r, load_elems<V>(w + (int64_t)V * i),
                                 h ? h + base + (int64_t)V * i : nullptr, ss, p);
        if (!Q8)
#pragma unroll
            for (int e = 0; e < V; e++)
                mx = fmax(mx, fabs(p[e]));
    }
    row_reduce<1024, !Q8>(ss, mx, red);
    const double scale = block_factor(fma(ss, inv_k, eps));
    const float sc = Q8 ? 0.0f : row_scale(fma(ss, inv_k, eps), mx);
    const double a = sc > 0.0f ? mx : 0.0, f = code_factor(a);
    int sum = 0;
    for (int i = threadIdx.x; i < np; i += 1024) {
        const int64_t o = base + (int64_t)V * i;
        const Elems<V, float> we = load_elems<V>(w + (int64_t)V * i);
        double again = 0.0, p[V];
        if (RES && !h) {
            norm_products<T, RES, V>(load_elems<V>(x + o), load_elems<V>(res + o), we, nullptr, again, p);
        } else {
            const Elems<V, T> hv = load_elems<V>((h ? h : x) + o);
            norm_products<T, false, V>(hv, hv, we, nullptr, again, p);
        }
        if constexpr (Q8) { // np is a multiple of 8: the lanes of a block run together
            uint8_t *blk = xq + (row * (k / 32) + (i >> 3)) * 34;
            double ab;
            store_codes(blk, i & 7, block_codes(p, ab));
            if ((i & 7) == 0)
                store_scale(blk, ab, scale);
        } else {
            sum += store_i8<V>(reinterpret_cast<int8_t *>(xq) + o, p, a, f);
        }
    }
    if constexpr (!Q8) {
        sum = row_sum<1024>(sum, sc, red_i);
        if (threadIdx.x == 0) {
            act_scale[row] = sc;
            act_sum[row] = sum;
        }
    }
}

struct NormArgs {
    const void *x, *res;
    const float *w;
    double eps;
    void *h;
    int64_t m;
    int k;
    // outputs
    uint8_t *xq;
    float *act_scale;
    int32_t *act_sum;
};

template <typename T, bool RES, int V, int TPR, int P>
static hipError_t launch_norm(const NormArgs &a, hipStream_t s)
{
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)((a.m + RPW - 1) / RPW)), block(TPR < 256 ? 256 : TPR);
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *h = static_cast<T *>(a.h);
    if (a.act_scale) {
        hipLaunchKernelGGL((rmsnorm_i8_rows_kernel<T, RES, V, TPR, P>), grid, block, 0, s, x, res, a.w, a.eps, 1.0 / (double)a.k, h,
                           reinterpret_cast<int8_t *>(a.xq), a.act_scale, a.act_sum, a.m, a.k);
    } else {
        if constexpr (V == 4)
            hipLaunchKernelGGL((rmsnorm_q8_0_kernel<T, RES, TPR, P>), grid, block, 0, s, x, res, a.w, a.eps, 1.0 / (double)a.k, h, a.xq,
                               a.m, a.k);
    }
    return hipGetLastError();
}

template <typename T, bool RES, int V>
static hipError_t launch_norm_long(const NormArgs &a, hipStream_t s)
{
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *h = static_cast<T *>(a.h);
    const dim3 grid((unsigned)a.m), block(1024);
    if (a.act_scale) {
        hipLaunchKernelGGL((rmsnorm_long_kernel<T, RES, V, false>), grid, block, 0, s, x, res, a.w, a.eps, 1.0 / (double)a.k, h, a.xq,
                           a.act_scale, a.act_sum, a.k);
    } else {
        if constexpr (V == 4)
            hipLaunchKernelGGL((rmsnorm_long_kernel<T, RES, V, true>), grid, block, 0, s, x, res, a.w, a.eps, 1.0 / (double)a.k, h, a.xq,
                               a.act_scale, a.act_sum, a.k);
    }
    return hipGetLastError();
}

// Threads per row.  Rows of at most 256 pieces: one wave each, four rows a
// workgroup.  Longer ones: 1024, the shortest path for a row, where there are
// fewer rows than CUs; otherwise as few as hold the row in eight pieces each,
// since what every wave does once (the reductions, the scale) weighs on few
// pieces and workgroups of 1024 leave a CU to one row.
template <typename T, bool RES, int V>
static hipError_t launch_norm_v(const NormArgs &a, hipStream_t s)
{
    const int np = a.k / V;
    const bool many = a.m >= 256;
    if (np <= 64)
        return launch_norm<T, RES, V, 64, 1>(a, s);
    if (np <= 256)
        return launch_norm<T, RES, V, 64, 4>(a, s);
    if (np <= 1024)
        return many ? launch_norm<T, RES, V, 256, 4>(a, s) : launch_norm<T, RES, V, 1024, 1>(a, s);
    if (np <= 2048)
        return many ? launch_norm<T, RES, V, 256, 8>(a, s) : launch_norm<T, RES, V, 1024, 2>(a, s);
    if (np <= 4096)
        return many ? launch_norm<T, RES, V, 512, 8>(a, s) : launch_norm<T, RES, V, 1024, 4>(a, s);
    if constexpr (V == 1) {
        if (np <= 16384)
            return launch_norm<T, RES, V, 1024, 16>(a, s);
    }
    return launch_norm_long<T, RES, V>(a, s);
}

// Rows of one launch: a grid has fewer than 2^32 threads.
constexpr int64_t kNormMaxRows = (int64_t)1 << 21;

template <typename T>
static hipError_t launch_norm_t(const NormArgs &all, hipStream_t s)
{
    for (int64_t r0 = 0; r0 < all.m; r0 += kNormMaxRows) {
        NormArgs a = all;
        const int64_t at = r0 * all.k;
        a.m = all.m - r0 < kNormMaxRows ? all.m - r0 : kNormMaxRows;
        a.x = static_cast<const T *>(all.x) + at;
        a.res = all.res ? static_cast<const T *>(all.res) + at : nullptr;
        a.h = all.h ? static_cast<T *>(all.h) + at : nullptr;
        if (all.act_scale) {
            a.xq += at;
            a.act_scale += r0;
            a.act_sum += r0;
        } else {
            a.xq += at / 32 * 34;
        }
        hipError_t e;
        if (a.k % 4 == 0)
            e = a.res ? launch_norm_v<T, true, 4>(a, s) : launch_norm_v<T, false, 4>(a, s);
        else
            e = a.res ? launch_norm_v<T, true, 1>(a, s) : launch_norm_v<T, false, 1>(a, s);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

static hipError_t launch_norm_any(int dtype, const NormArgs &a, hipStream_t s)
{
    switch (dtype) {
    case QLL_W_F32: return launch_norm_t<float>(a, s);
    case QLL_W_BF16: return launch_norm_t<uint16_t>(a, s);
    default: return launch_norm_t<_Float16>(a, s);
    }
}

hipError_t launch_rmsnorm_q8_0(const void *x, int dtype, const void *res, const float *w, float eps, void *h,
                               uint8_t *xq, int64_t m, int64_t k, hipStream_t s)
{
    return launch_norm_any(dtype, NormArgs{x, res, w, (double)eps, h, m, (int)k, xq, nullptr, nullptr}, s);
}

hipError_t launch_rmsnorm_i8_rows(const void *x, int dtype, const void *res, const float *w, float eps, void *h,
                                  int8_t *xq, float *act_scale, int32_t *act_sum, int64_t m, int64_t k,
                                  hipStream_t s)
{
    return launch_norm_any(
        dtype, NormArgs{x, res, w, (double)eps, h, m, (int)k, reinterpret_cast<uint8_t *>(xq), act_scale, act_sum}, s);
}

} // namespace qll
