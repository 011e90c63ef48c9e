// The router and the experts of a mixture-of-experts layer for a few tokens:
//     l = x.Wr^T,  the `top` experts of the largest scores with their weights w,
//     y = sum_j w_j * Wd_e.(act(Wg_e.x) * (Wu_e.x)) + residual,  e = ids[j],
// the experts' matrices packed 4-bit weights (q4g.h).
#include "q4g.h"

namespace qll {
namespace {

// ------------------------------------------------------------ router

constexpr int kRouteE = 4, kRouteT = 4; // experts and tokens of one wave

// Logits in 64 bits: an f32 sum's order would decide between two experts whose
// logits lie next to each other.  The products of bf16 and f16 are exact, those of f32
// nearly so.  A wave takes four experts and four tokens over the whole of k.
template <class TX, class TW>
__global__ void __launch_bounds__(256) moe_logits_kernel(const TX *x, const TW *w, double *logits, int64_t m, int64_t e,
                                                         int64_t k)
{
    const int lane = threadIdx.x % 64;
    const int64_t tiles = (e + kRouteE - 1) / kRouteE, at = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
    const int64_t e0 = at % tiles * kRouteE, t0 = at / tiles * kRouteT;
    if (t0 >= m)
        return;
    double acc[kRouteE][kRouteT] = {};
    const TX *xp[kRouteT];
    const TW *wp[kRouteE];
#pragma unroll
    for (int i = 0; i < kRouteT; i++)
        xp[i] = x + (t0 + i < m ? t0 + i : m - 1) * k;
#pragma unroll
    for (int i = 0; i < kRouteE; i++)
        wp[i] = w + (e0 + i < e ? e0 + i : e - 1) * k;
    for (int64_t i = lane; i < k; i += 64) {
        double xv[kRouteT];
#pragma unroll
        for (int t = 0; t < kRouteT; t++)
            xv[t] = (double)(float)xp[t][i];
#pragma unroll
        for (int j = 0; j < kRouteE; j++) {
            const double wv = (double)(float)wp[j][i];
#pragma unroll
            for (int t = 0; t < kRouteT; t++)
                acc[j][t] = fma(wv, xv[t], acc[j][t]);
        }
    }
#pragma unroll
    for (int j = 0; j < kRouteE; j++)
#pragma unroll
        for (int t = 0; t < kRouteT; t++) {
            double v = acc[j][t];
#pragma unroll
            for (int o = 32; o > 0; o >>= 1)
                v += __shfl_xor(v, o);
            if (lane == 0 && e0 + j < e && t0 + t < m)
                logits[(t0 + t) * e + e0 + j] = v;
        }
}

// Order-preserving bits of a double; NaN below every number but above 0, which
// stands for an expert taken already.
__device__ __forceinline__ uint64_t order_bits(double v)
{
    if (v != v)
        return 1;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0); // -0 as +0
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

constexpr int kRoutePer = kMaxExperts / 64; // experts a lane

// One wave a token: scores in 64 bits, then `top` times the largest that is left,
// the lower index first among equal ones.
__global__ void __launch_bounds__(64) moe_top_kernel(const double *logits, const float *bias, int sigmoid, int renorm,
                                                     float scale, int32_t *ids, float *weights, int top, int e)
{
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    double score[kRoutePer];
    uint64_t key[kRoutePer];
    double mx = -__builtin_inf();
#pragma unroll
    for (int i = 0; i < kRoutePer; i++) {
        const int at = i * 64 + lane;
        score[i] = at < e ? logits[t * e + at] : -__builtin_inf();
        mx = fmax(mx, score[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        mx = fmax(mx, __shfl_xor(mx, o));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kRoutePer; i++) {
        const int at = i * 64 + lane;
        const double l = score[i];
        if (i * 64 < e) {
            if (sigmoid)
                score[i] = 1.0 / (1.0 + exp(-l));
            else {
                score[i] = at < e ? exp(l - mx) : 0.0;
                sum += score[i];
            }
        }
        key[i] = at < e ? order_bits(l) : 0;
    }
    if (!sigmoid) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            sum += __shfl_xor(sum, o);
#pragma unroll
        for (int i = 0; i < kRoutePer; i++)
            score[i] /= sum;
    }
    if (bias)
#pragma unroll
        for (int i = 0; i < kRoutePer; i++) {
            const int at = i * 64 + lane;
            if (at < e)
                key[i] = order_bits(score[i] + (double)bias[at]);
        }
    double mine = 0.0, total = 0.0; // lane j holds choice j
    int chosen = 0;
    for (int j = 0; j < top; j++) {
        uint64_t best = 0;
        int at = 0;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < kRoutePer; i++)
            if (key[i] > best)
                best = key[i], at = i * 64 + lane, s = score[i];
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint64_t ob = __shfl_xor((unsigned long long)best, o);
            const int oa = __shfl_xor(at, o);
            const double os = __shfl_xor(s, o);
            if (ob > best || (ob == best && oa < at))
                best = ob, at = oa, s = os;
        }
#pragma unroll
        for (int i = 0; i < kRoutePer; i++)
            if (at == i * 64 + lane)
                key[i] = 0;
        if (lane == j)
            mine = s, chosen = at;
        total += s;
    }
    if (lane < top) {
        ids[t * top + lane] = chosen;
        weights[t * top + lane] = (float)((renorm ? mine / total : mine) * (double)scale);
    }
}

template <class TX, class TW>
hipError_t logits(const void *x, const void *w, double *out, int64_t m, int64_t e, int64_t k, hipStream_t s)
{
    const int64_t tiles = (e + kRouteE - 1) / kRouteE;
    return launch_parts(m, (kPartThreads / 64 / tiles) / kRouteT * kRouteT, [&](int64_t t0, int64_t count) {
        const int64_t waves = tiles * ((count + kRouteT - 1) / kRouteT);
        moe_logits_kernel<TX, TW><<<(unsigned)((waves + 3) / 4), 256, 0, s>>>(
            static_cast<const TX *>(x) + t0 * k, static_cast<const TW *>(w), out + t0 * e, count, e, k);
    });
}

template <class TX>
hipError_t logits_w(const void *x, const void *w, int w_dtype, double *out, int64_t m, int64_t e, int64_t k,
                    hipStream_t s)
{
    return w_dtype == QLL_W_F32    ? logits<TX, float>(x, w, out, m, e, k, s)
           : w_dtype == QLL_W_BF16 ? logits<TX, __bf16>(x, w, out, m, e, k, s)
                                   : logits<TX, _Float16>(x, w, out, m, e, k, s);
}

// ------------------------------------------------------------ experts

// The experts that a group of at most 64 tokens chose, in ascending order, are its
// active ones; active expert a's tokens are numbered in ascending order too.  A token
// that names an expert twice counts once, with the sum of its weights.  The
// gated products of active expert a's token number p stand in row
// (token * top + its first slot of that expert) of h.
struct MoeArgs {
    const uint8_t *wg, *wu, *wd;
    const void *x, *res;
    const int32_t *ids;
    const float *weights;
    void *y;
    float *h;
    int64_t n, k, gu_bytes, d_bytes; // bytes from one expert to the next
    int m, top, e, fmt, act, dtype;
    int kw; // gated products: waves along k
    int parts; // down products: parts of n
};

struct MoeShared { // what a workgroup finds out about the choices first
    int32_t ids[64 * kMaxTop];
    uint32_t active[kMaxExperts / 32];
};

__device__ __forceinline__ void moe_choices(MoeShared &sh, const MoeArgs &a)
{
    for (int i = threadIdx.x; i < kMaxExperts / 32; i += blockDim.x)
        sh.active[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.m * a.top; i += blockDim.x) {
        const int id = a.ids[i];
        sh.ids[i] = id;
        if (id >= 0 && id < a.e)
            atomicOr(&sh.active[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
}

// Active expert number a, or -1.
__device__ __forceinline__ int moe_expert(const MoeShared &sh, int a)
{
    const int lane = threadIdx.x % 64;
    const uint32_t word = lane < kMaxExperts / 32 ? sh.active[lane] : 0;
    int before = __builtin_popcount(word);
    const int own = before;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(before, o);
        if (lane >= o)
            before += v;
    }
    before -= own;
    int id = -1;
    if (a >= before && a < before + own) {
        uint32_t w = word;
        for (int i = before; i < a; i++)
            w &= w - 1;
        id = lane * 32 + __builtin_ctz(w);
    }
    const uint64_t who = __ballot(id >= 0);
    return who ? __shfl(id, __builtin_ctzll(who)) : -1;
}

// This wave's lane t: whether token t chose expert e, its first slot and the sum of its weights.
struct MoeToken {
    uint64_t mask; // tokens that chose it
    int slot;
    float weight;
    __device__ __forceinline__ MoeToken(const MoeShared &sh, const MoeArgs &a, int e, bool weigh)
    {
        const int t = threadIdx.x % 64;
        slot = -1, weight = 0.0f;
        if (t < a.m)
            for (int j = a.top - 1; j >= 0; j--)
                if (sh.ids[t * a.top + j] == e) {
                    slot = j;
                    if (weigh)
                        weight += a.weights[t * a.top + j];
                }
        mask = __ballot(slot >= 0);
    }
    __device__ __forceinline__ int count() const { return __builtin_popcountll(mask); }
    // token number p of the expert (the last one past the end)
    __device__ __forceinline__ int token(int p) const
    {
        const int n = count();
        uint64_t w = mask;
        for (int i = p < n ? p : n - 1; i > 0; i--)
            w &= w - 1;
        return __builtin_ctzll(w);
    }
};

// Gated products of an expert's tokens [p0, p0 + 16 C) on one row tile of gate and up.
template <int TX, int GRP, int C, int I>
__device__ __forceinline__ void moe_gated_tile(const MoeArgs &a, const MoeToken &who, int e, int p0, int64_t rt,
                                               f32x4 *part)
{
    const Q4gShape sh(a.n, a.k, GRP, a.fmt);
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const Q4gRows rows[2] = {Q4gRows(a.wg + e * a.gu_bytes, sh, rt, GRP, a.fmt, lane),
                             Q4gRows(a.wu + e * a.gu_bytes, sh, rt, GRP, a.fmt, lane)};
    const uint8_t *x[C];
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int row = lane % 16, t = who.token(p0 + 16 * c + row / 4 + 4 * (row & 3));
        x[c] = static_cast<const uint8_t *>(a.x) + (t * a.k + 8 * (lane / 16)) * (TX == Q4G_X_F32 ? 4 : 2);
    }
    Q4gWave<TX, GRP, 2, C, I, 1> w;
    w.clear();
    const int64_t per = (sh.kt + a.kw - 1) / a.kw, t0 = wave * per, t1 = t0 + per < sh.kt ? t0 + per : sh.kt;
    w.run(rows, x, t0, t1, a.k);
#pragma unroll
    for (int r = 0; r < 2; r++)
#pragma unroll
        for (int c = 0; c < C; c++)
            part[((wave * 2 + r) * C + c) * 64 + lane] = w.y[r][c];
    __syncthreads();
    const int64_t j = rt * 16 + lane % 16;
    for (int c = wave; c < C; c += a.kw) {
        f32x4 g = part[c * 64 + lane], u = part[(C + c) * 64 + lane];
        for (int o = 1; o < a.kw; o++)
            g += part[(o * 2 * C + c) * 64 + lane], u += part[((o * 2 + 1) * C + c) * 64 + lane];
#pragma unroll
        for (int i = 0; i < I; i++) {
            const int p = p0 + 16 * c + lane / 16 + 4 * i;
            const int t = who.token(p), slot = __shfl(who.slot, t);
            if (p < who.count() && j < a.n)
                a.h[(int64_t)(t * a.top + slot) * a.n + j] = activate(g[i], a.act) * u[i];
        }
    }
    __syncthreads();
}

template <int TX, int GRP>
__global__ void __launch_bounds__(512) moe_gated_kernel(MoeArgs a)
{
    __shared__ MoeShared sh;
    extern __shared__ f32x4 part[];
    moe_choices(sh, a);
    const int e = moe_expert(sh, blockIdx.y);
    if (e < 0)
        return;
    const MoeToken who(sh, a, e, false);
    const int n = who.count();
    if (n <= 4)
        moe_gated_tile<TX, GRP, 1, 1>(a, who, e, 0, blockIdx.x, part);
    else
        for (int p = 0; p < n; p += 16)
            moe_gated_tile<TX, GRP, 1, 4>(a, who, e, p, blockIdx.x, part);
}

// Down products of 16 rows: the waves share out the active experts and the parts
// of n; each adds its weighted products to its own sums, which are then added in order.
template <int GRP, int I>
__device__ __forceinline__ void moe_down_tile(const MoeArgs &a, const MoeToken &who, int e, int p0, int64_t rt,
                                              int64_t t0, int64_t t1, float *sums)
{
    const Q4gShape sh(a.k, a.n, GRP, a.fmt);
    const int lane = threadIdx.x % 64, row = lane % 16;
    const Q4gRows rows[1] = {Q4gRows(a.wd + e * a.d_bytes, sh, rt, GRP, a.fmt, lane)};
    const int t = who.token(p0 + row / 4 + 4 * (row & 3)), slot = __shfl(who.slot, t);
    const uint8_t *x[1] = {reinterpret_cast<const uint8_t *>(a.h + (int64_t)(t * a.top + slot) * a.n + 8 * (lane / 16))};
    Q4gWave<Q4G_X_F32, GRP, 1, 1, I, 1> w;
    w.clear();
    w.run(rows, x, t0, t1, a.n);
#pragma unroll
    for (int i = 0; i < I; i++) {
        const int p = p0 + lane / 16 + 4 * i, to = who.token(p);
        const float weight = __shfl(who.weight, to);
        if (p < who.count())
            sums[to * 16 + row] = fmaf(weight, w.y[0][0][i], sums[to * 16 + row]);
    }
}

template <int GRP>
__global__ void __launch_bounds__(512) moe_down_kernel(MoeArgs a)
{
    __shared__ MoeShared sh;
    extern __shared__ float sums[]; // [waves][m][16]
    const int wave = threadIdx.x / 64, waves = blockDim.x / 64;
    for (int i = threadIdx.x; i < waves * a.m * 16; i += blockDim.x)
        sums[i] = 0.0f;
    moe_choices(sh, a);
    const int64_t rt = blockIdx.x, kt = (a.n + 127) / 128, per = (kt + a.parts - 1) / a.parts;
    for (int item = wave;; item += waves) {
        const int e = moe_expert(sh, item / a.parts);
        if (e < 0)
            break;
        const MoeToken who(sh, a, e, true);
        const int64_t t0 = item % a.parts * per, t1 = t0 + per < kt ? t0 + per : kt;
        const int n = who.count();
        if (n <= 4)
            moe_down_tile<GRP, 1>(a, who, e, 0, rt, t0, t1, sums + wave * a.m * 16);
        else
            for (int p = 0; p < n; p += 16)
                moe_down_tile<GRP, 4>(a, who, e, p, rt, t0, t1, sums + wave * a.m * 16);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.m * 16; i += blockDim.x) {
        float v = sums[i];
        for (int o = 1; o < waves; o++)
            v += sums[o * a.m * 16 + i];
        const int64_t j = rt * 16 + i % 16, at = i / 16 * a.k + j;
        if (j < a.k) {
            if (a.res)
                v += load_as(a.res, at, a.dtype);
            store_as(a.y, at, v, a.dtype);
        }
    }
}

template <int TX, int GRP>
hipError_t experts(MoeArgs a, hipStream_t s)
{
    const int active = a.m * a.top < a.e ? a.m * a.top : a.e;
    const int64_t rt = (a.n + 15) / 16, kt = (a.k + 127) / 128, dt = (a.k + 15) / 16, nt = (a.n + 127) / 128;
    a.kw = kt >= 8 ? 8 : kt >= 4 ? 4 : kt >= 2 ? 2 : 1;
    moe_gated_kernel<TX, GRP><<<dim3((unsigned)rt, (unsigned)active), 64 * a.kw,
                               (size_t)a.kw * 2 * 64 * sizeof(f32x4), s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    a.parts = 1;
    while (a.parts < 16 && active * a.parts < 8 && 4 * a.parts <= nt)
        a.parts *= 2;
    moe_down_kernel<GRP><<<(unsigned)dt, 512, (size_t)8 * a.m * 16 * sizeof(float), s>>>(a);
    return hipGetLastError();
}

template <int TX>
hipError_t experts_g(const MoeArgs &a, int64_t group, hipStream_t s)
{
    return group == 32 ? experts<TX, 32>(a, s) : group == 64 ? experts<TX, 64>(a, s) : experts<TX, 128>(a, s);
}

} // namespace

size_t moe_route_workspace(int64_t m, int64_t e) { return ((size_t)(m * e) * sizeof(double) + 255) / 256 * 256; }

hipError_t launch_moe_route(const void *x, int dtype, const void *w, int w_dtype, const float *bias, int sigmoid,
                            int renorm, float scale, int32_t *ids, float *weights, int64_t top, int64_t m, int64_t e,
                            int64_t k, void *ws, hipStream_t s)
{
    double *l = static_cast<double *>(ws);
    const hipError_t rc = dtype == QLL_W_F32    ? logits_w<float>(x, w, w_dtype, l, m, e, k, s)
                          : dtype == QLL_W_BF16 ? logits_w<__bf16>(x, w, w_dtype, l, m, e, k, s)
                                                : logits_w<_Float16>(x, w, w_dtype, l, m, e, k, s);
    if (rc != hipSuccess)
        return rc;
    return launch_parts(m, kPartThreads / 64, [&](int64_t t0, int64_t count) {
        moe_top_kernel<<<(unsigned)count, 64, 0, s>>>(l + t0 * e, bias, sigmoid, renorm, scale, ids + t0 * top,
                                                      weights + t0 * top, (int)top, (int)e);
    });
}

// Groups of 64 tokens, one after another, in the same workspace.
constexpr int64_t kMoeTokens = 64;

size_t q4g_moe_workspace(int64_t m, int64_t n, int64_t top)
{
    return ((size_t)((m < kMoeTokens ? m : kMoeTokens) * top * n) * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_q4g_moe(const void *x, int dtype, const int32_t *ids, const float *weights, int64_t top,
                          const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, int64_t group, int fmt, int act,
                          const void *res, void *y, int64_t m, int64_t n, int64_t k, int64_t e, void *ws, hipStream_t s)
{
    const int64_t row = k * (dtype == QLL_W_F32 ? 4 : 2);
    for (int64_t t0 = 0; t0 < m; t0 += kMoeTokens) {
        MoeArgs a{};
        a.wg = wg, a.wu = wu, a.wd = wd;
        a.x = static_cast<const uint8_t *>(x) + t0 * row;
        a.res = res ? static_cast<const uint8_t *>(res) + t0 * row : nullptr;
        a.y = static_cast<uint8_t *>(y) + t0 * row;
        a.ids = ids + t0 * top, a.weights = weights + t0 * top;
        a.h = static_cast<float *>(ws);
        a.n = n, a.k = k;
        a.gu_bytes = q4g_packed_bytes(n, k, group, fmt), a.d_bytes = q4g_packed_bytes(k, n, group, fmt);
        a.m = (int)(m - t0 < kMoeTokens ? m - t0 : kMoeTokens), a.top = (int)top, a.e = (int)e;
        a.fmt = fmt, a.act = act, a.dtype = dtype;
        const hipError_t rc = dtype == QLL_W_F32    ? experts_g<Q4G_X_F32>(a, group, s)
                              : dtype == QLL_W_BF16 ? experts_g<Q4G_X_BF16>(a, group, s)
                                                    : experts_g<Q4G_X_F16>(a, group, s);
        if (rc != hipSuccess)
            return rc;
    }
    return hipSuccess;
}

} // namespace qll
