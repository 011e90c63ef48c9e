// The router and the experts of a mixture-of-experts layer for a few tokens:
//     l = x.Wr^T,  the `top` experts of the largest scores with their weights w,
//     y = sum_j w_j * Wd_e.(act(Wg_e.x) * (Wu_e.x)) + residual,  e = ids[j],
// the experts' matrices packed 4-bit weights (q4g.h).
#include "q4g.h"

namespace qll {
namespace {

// ------------------------------------------------------------ router

// Eight consecutive elements as they are loaded, and one of them.
template <class T>
struct RouteEight {
    u32x4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++)
            v[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ __forceinline__ double at(int i) const
    {
        if constexpr (sizeof(T) == 4)
            return (double)__builtin_bit_cast(float, (uint32_t)v[i / 4][i % 4]);
        else
            return (double)(float)__builtin_bit_cast(T, (uint16_t)(v[0][i / 2] >> (16 * (i % 2))));
    }
};

// The sums over a wave's lanes of N values each (N a power of 2, at most 32), in N + 5
// exchanges in place of 6 N: every step halves the values a lane holds.  v[0] becomes the sum
// of the value whose number is returned; the first N lanes hold all of them.
template <int N, int O = 1, int ALL>
__device__ __forceinline__ int route_reduce(double (&v)[ALL])
{
    if constexpr (O == 64)
        return 0;
    else if constexpr (N == 1) {
        v[0] += __shfl_xor(v[0], O);
        return route_reduce<1, 2 * O>(v);
    } else {
        const bool up = threadIdx.x & O;
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
            const double keep = up ? v[i + N / 2] : v[i], give = up ? v[i] : v[i + N / 2];
            v[i] = keep + __shfl_xor(give, O);
        }
        return (up ? N / 2 : 0) + route_reduce<N / 2, 2 * O>(v);
    }
}

// Logits in 64 bits: an f32 sum's order would decide between two experts whose
// logits lie next to each other.  The products are exact in f64 for every type.  A
// workgroup's four waves share the k of TE experts and TT tokens; with VEC (k a multiple of
// eight) a lane takes eight elements of a row at a time.
template <class TX, class TW, int TE, int TT, bool VEC>
__global__ void __launch_bounds__(256) moe_logits_kernel(const TX *x, const TW *w, double *logits, int m, int e, int k)
{
    __shared__ double part[4][TE * TT];
    const int wave = threadIdx.x / 64, tiles = (e + TE - 1) / TE;
    const int e0 = blockIdx.x % tiles * TE, t0 = blockIdx.x / tiles * TT;
    double acc[TE * TT] = {};
    const TX *xp[TT];
    const TW *wp[TE];
#pragma unroll
    for (int i = 0; i < TT; i++)
        xp[i] = x + (int64_t)(t0 + i < m ? t0 + i : m - 1) * k;
#pragma unroll
    for (int i = 0; i < TE; i++)
        wp[i] = w + (int64_t)(e0 + i < e ? e0 + i : e - 1) * k;
    if constexpr (VEC) {
#pragma unroll 2
        for (int at = threadIdx.x * 8; at < k; at += 2048) {
            RouteEight<TX> xv[TT];
            RouteEight<TW> wv[TE];
#pragma unroll
            for (int i = 0; i < TE; i++)
                wv[i].load(wp[i] + at);
#pragma unroll
            for (int i = 0; i < TT; i++)
                xv[i].load(xp[i] + at);
#pragma unroll
            for (int b = 0; b < 8; b++) {
                double xd[TT];
#pragma unroll
                for (int t = 0; t < TT; t++)
                    xd[t] = xv[t].at(b);
#pragma unroll
                for (int j = 0; j < TE; j++) {
                    const double wd = wv[j].at(b);
#pragma unroll
                    for (int t = 0; t < TT; t++)
                        acc[j * TT + t] = fma(wd, xd[t], acc[j * TT + t]);
                }
            }
        }
    } else
        for (int at = threadIdx.x; at < k; at += 256) {
            double xd[TT];
#pragma unroll
            for (int t = 0; t < TT; t++)
                xd[t] = (double)(float)xp[t][at];
#pragma unroll
            for (int j = 0; j < TE; j++) {
                const double wd = (double)(float)wp[j][at];
#pragma unroll
                for (int t = 0; t < TT; t++)
                    acc[j * TT + t] = fma(wd, xd[t], acc[j * TT + t]);
            }
        }
    const int index = route_reduce<TE * TT>(acc);
    if (threadIdx.x % 64 < TE * TT)
        part[wave][index] = acc[0];
    __syncthreads();
    if (threadIdx.x < TE * TT) {
        const int j = e0 + threadIdx.x / TT, t = t0 + threadIdx.x % TT;
        if (j < e && t < m)
            logits[(int64_t)t * e + j] = (part[0][threadIdx.x] + part[1][threadIdx.x]) +
                                         (part[2][threadIdx.x] + part[3][threadIdx.x]);
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

// v of the lane that a DPP control names, 0 where there is none: reductions towards
// lane 63 in six register moves.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp64(uint64_t v)
{
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 15, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 15, false);
    return (uint64_t)hi << 32 | lo;
}
template <class F>
__device__ __forceinline__ uint64_t wave_all(uint64_t v, const F &f) // f(0, v) = v
{
    v = f(dpp64<0x111, 15>(v), v); // row_shr 1, 2, 4, 8: lane 15 of each 16 has its row's
    v = f(dpp64<0x112, 15>(v), v);
    v = f(dpp64<0x114, 15>(v), v);
    v = f(dpp64<0x118, 15>(v), v);
    v = f(dpp64<0x142, 10>(v), v); // row_bcast 15 into rows 1 and 3, 31 into rows 2 and 3
    v = f(dpp64<0x143, 12>(v), v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, 63);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
    return wave_all(v, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ double wave_sum(double v)
{
    return __builtin_bit_cast(double, wave_all(__builtin_bit_cast(uint64_t, v), [](uint64_t a, uint64_t b) {
                                  return __builtin_bit_cast(uint64_t, __builtin_bit_cast(double, a) +
                                                                          __builtin_bit_cast(double, b));
                              }));
}

// One wave a token, PER experts a lane (lane * PER + i): scores in 64 bits, then `top` times the
// largest that is left, the lower index first among equal ones.
template <int PER>
__global__ void __launch_bounds__(64) moe_top_kernel(const double *logits, const float *bias, int sigmoid, int renorm,
                                                     float scale, int32_t *ids, float *weights, int top, int e)
{
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    double score[PER];
    uint64_t key[PER];
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int at = lane * PER + i;
        score[i] = at < e ? logits[t * e + at] : -__builtin_inf();
        key[i] = at < e ? order_bits(score[i]) : 0;
        best = key[i] > best ? key[i] : best;
    }
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; i++)
            score[i] = 1.0 / (1.0 + exp(-score[i]));
    } else {
        const uint64_t b = wave_max(best);
        const double mx = __builtin_bit_cast(double, b >> 63 ? b & 0x7fffffffffffffffull : ~b);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            score[i] = exp(score[i] - mx);
            sum += lane * PER + i < e ? score[i] : 0.0;
        }
        sum = 1.0 / wave_sum(sum);
#pragma unroll
        for (int i = 0; i < PER; i++)
            score[i] *= sum;
    }
    if (bias)
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int at = lane * PER + i;
            if (at < e)
                key[i] = order_bits(score[i] + (double)bias[at]);
        }
    double mine = 0.0, total = 0.0; // lane j holds choice j
    int chosen = 0;
    for (int j = 0; j < top; j++) {
        uint64_t b = 0;
        int at = 0;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (key[i] > b)
                b = key[i], at = i, s = score[i];
        const uint64_t all = wave_max(b);
        const int who = __builtin_ctzll(__ballot(b == all)); // lanes hold ascending experts
        at = __builtin_amdgcn_readlane(at, who);
        const uint64_t sb = __builtin_bit_cast(uint64_t, s);
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)sb, who);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(sb >> 32), who);
        s = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (lane == who && i == at)
                key[i] = 0;
        if (lane == j)
            mine = s, chosen = who * PER + at;
        total += s;
    }
    if (lane < top) {
        ids[t * top + lane] = chosen;
        weights[t * top + lane] = (float)((renorm ? mine / total : mine) * (double)scale);
    }
}

template <class TX, class TW, int TE, int TT>
hipError_t logits_t(const TX *x, const TW *w, double *out, int64_t m, int64_t e, int64_t k, hipStream_t s)
{
    const int64_t tiles = (e + TE - 1) / TE;
    return launch_parts(m, kPartThreads / 256 / tiles / TT * TT, [&](int64_t t0, int64_t count) {
        const unsigned blocks = (unsigned)(tiles * ((count + TT - 1) / TT));
        if (k % 8 == 0)
            moe_logits_kernel<TX, TW, TE, TT, true><<<blocks, 256, 0, s>>>(x + t0 * k, w, out + t0 * e, (int)count,
                                                                          (int)e, (int)k);
        else
            moe_logits_kernel<TX, TW, TE, TT, false><<<blocks, 256, 0, s>>>(x + t0 * k, w, out + t0 * e, (int)count,
                                                                           (int)e, (int)k);
    });
}

// Tiles of one expert and token, two and four, four and eight: larger ones read less,
// smaller ones give more workgroups.
template <class TX, class TW>
hipError_t logits(const void *xv, const void *wv, double *out, int64_t m, int64_t e, int64_t k, hipStream_t s)
{
    const TX *x = static_cast<const TX *>(xv);
    const TW *w = static_cast<const TW *>(wv);
    if (m == 1)
        return logits_t<TX, TW, 1, 1>(x, w, out, m, e, k, s);
    if ((m + 7) / 8 * ((e + 3) / 4) < 256)
        return logits_t<TX, TW, 2, 4>(x, w, out, m, e, k, s);
    return logits_t<TX, TW, 4, 8>(x, w, out, m, e, k, s);
}

template <class TX>
hipError_t logits_w(const void *x, const void *w, int w_dtype, double *out, int64_t m, int64_t e, int64_t k,
                    hipStream_t s)
{
    return w_dtype == QLL_W_F32    ? logits<TX, float>(x, w, out, m, e, k, s)
           : w_dtype == QLL_W_BF16 ? logits<TX, __bf16>(x, w, out, m, e, k, s)
                                   : logits<TX, _Float16>(x, w, out, m, e, k, s);
}

template <int PER>
hipError_t top_e(const double *l, const float *bias, int sigmoid, int renorm, float scale, int32_t *ids, float *weights,
                 int64_t top, int64_t m, int64_t e, hipStream_t s)
{
    return launch_parts(m, kPartThreads / 64, [&](int64_t t0, int64_t count) {
        moe_top_kernel<PER><<<(unsigned)count, 64, 0, s>>>(l + t0 * e, bias, sigmoid, renorm, scale, ids + t0 * top,
                                                          weights + t0 * top, (int)top, (int)e);
    });
}

// ------------------------------------------------------------ experts

constexpr int kMoeTokens = 64; // at most, in one go

// The experts that a group of at most 64 tokens chose, in ascending order, are its
// active ones; active expert a's tokens are numbered in ascending order too.  A token
// that names an expert twice counts once, with the sum of its weights.
struct MoePlan {
    int32_t expert, count; // count 0: no such active expert
    uint32_t row[kMoeTokens]; // per token of the expert: token << 16 | its row in h, token * top + first slot of it
    float weight[kMoeTokens];
};

// The gated products between the two kernels: two bf16 parts of each where the
// stream has 16 bits (what is left out is below 2^-17 of the value, against 2^-9 and 2^-12 of
// the outputs' own rounding), three (all 24 bits) where it is f32.  The parts are what the
// matrix core reads, so the down kernel's waves load them as they stand: splitting
// f32 values there would be done again for every 16 output rows.
struct MoeArgs {
    const uint8_t *wg, *wu, *wd;
    const void *x, *res;
    const int32_t *ids;
    const float *weights;
    void *y;
    uint8_t *h; // [part][m * top][n]
    MoePlan *plan;
    int64_t n, k, gu_bytes, d_bytes; // bytes from one expert to the next
    int m, top, e, fmt, act, dtype;
    int kw;    // gated products: waves along k
    int active, parts; // down products: active experts at most, parts of n
};

struct MoeShared { // what a workgroup finds out about the choices first
    int32_t ids[kMoeTokens * kMaxTop];
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
    for (int o = 1; o < kMaxExperts / 32; o <<= 1) {
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

// An expert's tokens: lane p holds number p (the last one past the end) as token << 16 | row.
struct MoeTokens {
    int count;
    uint32_t row;
    __device__ __forceinline__ uint32_t of(int p) const { return __shfl(row, p < count ? p : count - 1); }
};

__device__ __forceinline__ MoeTokens moe_tokens(const MoeShared &sh, const MoeArgs &a, int e, MoePlan *plan)
{
    const int t = threadIdx.x % 64;
    int slot = -1;
    float weight = 0.0f;
    if (t < a.m)
        for (int j = a.top - 1; j >= 0; j--)
            if (sh.ids[t * a.top + j] == e) {
                slot = j;
                if (plan)
                    weight += a.weights[t * a.top + j];
            }
    const uint64_t mask = __ballot(slot >= 0);
    const int at = __builtin_popcountll(mask & (((uint64_t)1 << t) - 1)), count = __builtin_popcountll(mask);
    const uint32_t mine = (uint32_t)t << 16 | (uint32_t)(t * a.top + slot);
    if (plan && slot >= 0)
        plan->row[at] = mine, plan->weight[at] = weight;
    // token number p stands in the lane of the mask's p-th bit
    uint64_t left = mask;
    for (int i = t < count ? t : count - 1; i > 0; i--)
        left &= left - 1;
    return {count, (uint32_t)__shfl(mine, __builtin_ctzll(left))};
}

__device__ __forceinline__ void store_part(uint8_t *h, int64_t at, float v)
{
    reinterpret_cast<uint16_t *>(h)[at] = (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16);
}

// Gated products of an expert's tokens [p0, p0 + 16 / PK) on one row tile of gate and up a wave.
template <int TX, int GRP, int PK, int D>
__device__ __forceinline__ void moe_gated_tile(const MoeArgs &a, const MoeTokens &who, int e, int p0, int64_t rt,
                                               float *part)
{
    using Wave = Q4gWave<TX, GRP, 2, 1, PK, D>;
    constexpr int N = Wave::N;
    const Q4gShape sh(a.n, a.k, GRP, a.fmt);
    const int lane = opaque_lane(), wave = wave_number(), kw = wave % a.kw, set = wave - kw;
    Wave w;
    w.clear();
    if (rt < sh.rt) {
        typename Wave::Rows rows;
        rows.w[0] = Q4gRows(a.wg + e * a.gu_bytes, sh, rt, GRP, a.fmt);
        rows.w[1] = Q4gRows(a.wu + e * a.gu_bytes, sh, rt, GRP, a.fmt);
        rows.x = static_cast<const uint8_t *>(a.x); // 64 rows of under 2^24 elements: offsets below 2^32
        rows.at[0] = (who.of(p0 + Wave::row_of(lane)) >> 16) * (uint32_t)a.k * q4g_x_size(TX);
        rows.part = 0, rows.last = (int)a.k - 32, rows.bf16 = a.fmt & kQ4gBf16, rows.lane = lane;
        const int kt = (int)sh.kt, per = (kt + a.kw - 1) / a.kw, t0 = kw * per;
        w.run(rows, t0, t0 + per < kt ? t0 + per : kt);
    }
    if (a.kw > 1) {
#pragma unroll
        for (int i = 0; i < N; i++)
            part[(wave * 2 * N + i) * 64 + lane] = w.y[0][0][i], part[((wave * 2 + 1) * N + i) * 64 + lane] = w.y[1][0][i];
        __syncthreads();
    }
    const int64_t j = rt * 16 + lane % 16, whole = (int64_t)a.m * a.top * a.n;
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (i % a.kw != kw) // the set's waves take turns
            continue;
        float g = w.y[0][0][i], u = w.y[1][0][i];
        if (a.kw > 1) {
            g = part[(set * 2 * N + i) * 64 + lane], u = part[((set * 2 + 1) * N + i) * 64 + lane];
            for (int o = 1; o < a.kw; o++)
                g += part[((set + o) * 2 * N + i) * 64 + lane], u += part[(((set + o) * 2 + 1) * N + i) * 64 + lane];
        }
        const int p = p0 + Wave::out_of(lane, i);
        const int64_t at = (int64_t)(who.of(p) & 0xffffu) * a.n + j;
        if (p < who.count && j < a.n) {
            const float v = activate(g, a.act) * u, v1 = below_bf16(v);
            store_part(a.h, at, v);
            if (TX == Q4G_X_F32) {
                store_part(a.h, whole + at, v1);
                store_part(a.h, 2 * whole + at, below_bf16(v1));
            } else
                reinterpret_cast<__bf16 *>(a.h)[whole + at] = (__bf16)v1;
        }
    }
    if (a.kw > 1)
        __syncthreads();
}

template <int TX, int GRP>
__global__ void __launch_bounds__(512, 4) moe_gated_kernel(MoeArgs a)
{
    __shared__ MoeShared sh;
    extern __shared__ float part[];
    moe_choices(sh, a);
    const int e = __builtin_amdgcn_readfirstlane(moe_expert(sh, blockIdx.y));
    MoePlan *plan = blockIdx.x == 0 && threadIdx.x < 64 ? a.plan + blockIdx.y : nullptr; // the down kernel's
    if (e < 0) {
        if (plan && threadIdx.x == 0)
            plan->count = 0;
        return;
    }
    const MoeTokens who = moe_tokens(sh, a, e, plan);
    if (plan && threadIdx.x == 0)
        plan->expert = e, plan->count = who.count;
    const int rw = wave_number() / a.kw, sets = blockDim.x / 64 / a.kw, n = who.count;
    const int64_t tiles = (a.n + 15) / 16, step = (int64_t)gridDim.x * sets;
    for (int64_t rt = (int64_t)blockIdx.x * sets; rt < tiles; rt += step)
        if (n <= 4)
            moe_gated_tile<TX, GRP, 4, 2>(a, who, e, 0, rt + rw, part);
        else if (n <= 8)
            moe_gated_tile<TX, GRP, 2, 1>(a, who, e, 0, rt + rw, part);
        else
            for (int p = 0; p < n; p += 16)
                moe_gated_tile<TX, GRP, 1, 1>(a, who, e, p, rt + rw, part);
}

// Down products of 16 rows and an expert's tokens [p0, p0 + 16 / PK), weighted and added
// to the wave's own sums [m][16].  No two of them are one token's.
template <int TX, int GRP, int PK, int D>
__device__ __forceinline__ void moe_down_tile(const MoeArgs &a, const MoeTokens &who, float weight, int e, int p0,
                                              int64_t rt, int t0, int t1, float *sums)
{
    using Wave = Q4gWave<TX, GRP, 1, 1, PK, D>;
    const Q4gShape sh(a.k, a.n, GRP, a.fmt);
    const int lane = opaque_lane();
    typename Wave::Rows rows;
    rows.w[0] = Q4gRows(a.wd + e * a.d_bytes, sh, rt, GRP, a.fmt);
    rows.x = a.h; // 2048 rows of under 2^20 elements: offsets below 2^32
    rows.at[0] = (who.of(p0 + Wave::row_of(lane)) & 0xffffu) * (uint32_t)a.n * 2;
    rows.part = (int64_t)a.m * a.top * a.n * 2, rows.last = (int)a.n - 32, rows.bf16 = a.fmt & kQ4gBf16, rows.lane = lane;
    Wave w;
    w.clear();
    w.run(rows, t0, t1);
#pragma unroll
    for (int i = 0; i < Wave::N; i++) {
        const int p = p0 + Wave::out_of(lane, i);
        float *to = sums + (who.of(p) >> 16) * 16 + lane % 16;
        const float f = __shfl(weight, p & 63);
        if (p < who.count)
            *to = fmaf(f, w.y[0][0][i], *to);
    }
}

// One workgroup for 16 rows: the waves share out the active experts and the parts
// of n; each adds up its own, then their sums are added in order.
template <int TX, int GRP>
__global__ void __launch_bounds__(1024) moe_down_kernel(MoeArgs a)
{
    extern __shared__ float sums[]; // [waves][m][16]
    const int wave = wave_number(), lane = threadIdx.x % 64, waves = blockDim.x / 64;
    float *own = sums + wave * a.m * 16;
    for (int i = lane; i < a.m * 16; i += 64)
        own[i] = 0.0f;
    const int64_t rt = blockIdx.x;
    const int kt = (int)((a.n + 127) / 128), per = (kt + a.parts - 1) / a.parts;
    for (int item = wave; item < a.active * a.parts; item += waves) {
        const MoePlan &plan = a.plan[item / a.parts];
        const int n = __builtin_amdgcn_readfirstlane(plan.count);
        if (n == 0)
            break;
        const int at = lane < n ? lane : n - 1;
        const MoeTokens who = {n, plan.row[at]};
        const float weight = plan.weight[at];
        const int e = __builtin_amdgcn_readfirstlane(plan.expert);
        const int t0 = item % a.parts * per, t1 = t0 + per < kt ? t0 + per : kt;
        if (n <= 4)
            moe_down_tile<TX, GRP, 4, 2>(a, who, weight, e, 0, rt, t0, t1, own);
        else if (n <= 8)
            moe_down_tile<TX, GRP, 2, 1>(a, who, weight, e, 0, rt, t0, t1, own);
        else
            for (int p = 0; p < n; p += 16)
                moe_down_tile<TX, GRP, 1, 1>(a, who, weight, e, p, rt, t0, t1, own);
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
    a.active = a.m * a.top < a.e ? a.m * a.top : a.e;
    const int64_t rt = (a.n + 15) / 16, kt = (a.k + 127) / 128, dt = (a.k + 15) / 16, nt = (a.n + 127) / 128;
    a.kw = 1;
    while (a.kw < 8 && rt * a.active * a.kw < 4096 && 2 * a.kw <= kt)
        a.kw *= 2;
    const int64_t most = (rt * a.kw + 7) / 8, want = (1024 + a.active - 1) / a.active;
    moe_gated_kernel<TX, GRP><<<dim3((unsigned)(most < want ? most : want), (unsigned)a.active), 512,
                               a.kw > 1 ? (size_t)8 * 2 * 4 * 64 * sizeof(float) : 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    a.parts = 1;
    while (a.parts < 16 && a.active * a.parts < 64 && 4 * a.parts <= nt)
        a.parts *= 2;
    const int items = a.active * a.parts, waves = items < 16 ? items : 16;
    constexpr int TH = TX == Q4G_X_F32 ? Q4G_X_PARTS3 : Q4G_X_PARTS2;
    moe_down_kernel<TH, GRP><<<(unsigned)dt, 64 * waves, (size_t)waves * a.m * 16 * sizeof(float), s>>>(a);
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
    const auto choose = e <= 64 ? top_e<1> : e <= 128 ? top_e<2> : e <= 256 ? top_e<4> : e <= 512 ? top_e<8> : top_e<16>;
    return choose(l, bias, sigmoid, renorm, scale, ids, weights, top, m, e, s);
}

// Groups of 64 tokens, one after another, in the same workspace: plans, then h.
static size_t moe_plan_bytes(int64_t tokens, int64_t top)
{
    const int64_t active = tokens * top < kMaxExperts ? tokens * top : kMaxExperts;
    return ((size_t)active * sizeof(MoePlan) + 255) / 256 * 256;
}

size_t q4g_moe_workspace(int64_t m, int64_t n, int64_t top)
{
    const int64_t tokens = m < kMoeTokens ? m : kMoeTokens;
    return moe_plan_bytes(tokens, top) + ((size_t)(tokens * top * n) * 6 + 255) / 256 * 256;
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
        a.plan = static_cast<MoePlan *>(ws);
        a.n = n, a.k = k;
        a.gu_bytes = q4g_packed_bytes(n, k, group, fmt), a.d_bytes = q4g_packed_bytes(k, n, group, fmt);
        a.m = (int)(m - t0 < kMoeTokens ? m - t0 : kMoeTokens), a.top = (int)top, a.e = (int)e;
        a.h = static_cast<uint8_t *>(ws) + moe_plan_bytes(a.m, top);
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
