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
constexpr int kMoePairs = kMoeTokens * (int)kMaxTop;
constexpr int kMoeEntries = (int)kMaxExperts + kMoePairs / 16;

// Who chose whom, for a group of at most 64 tokens.  An entry is up to 4, 8 or 16 tokens of
// an expert (class 0, 1, 2): an expert with at most four tokens is one entry of class 0, up to eight
// one of class 1, more of them entries of sixteen.  begin[c] is class c's first entry,
// begin[3] their number; entries stand in ascending order of the experts within
// a class.  A token that names an expert twice counts once, with the sum of its weights.
struct MoePlan {
    int32_t begin[4];
    uint32_t entry[kMoeEntries]; // expert | first pair << 10 | pairs << 21
    uint16_t row[kMoePairs];     // per pair: its row in h, token * top + the first slot of that expert
    float weight[kMoePairs];
};

struct MoeEntry {
    int expert, first, count;
    __device__ __forceinline__ explicit MoeEntry(uint32_t v)
        : expert(v & 1023), first(v >> 10 & 2047), count(v >> 21)
    {
    }
    __host__ __device__ static constexpr uint32_t packed(int expert, int first, int count)
    {
        return (uint32_t)expert | (uint32_t)first << 10 | (uint32_t)count << 21;
    }
};
static_assert(kMaxExperts <= 1024 && kMoePairs <= 2048, "the fields of an entry");

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
    int kw; // gated products: waves along k
};

// One workgroup makes the plan; threads are experts, then pairs.
__device__ __forceinline__ void moe_plan(const int32_t *ids, const float *weights, int m, int top, int e, MoePlan &plan)
{
    __shared__ unsigned long long chose[kMaxExperts]; // tokens that named it
    __shared__ unsigned long long sums[16];
    __shared__ int32_t id[kMoePairs];
    __shared__ uint16_t first[kMaxExperts];
    const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64; // 1024 threads
    chose[tid] = 0;
    __syncthreads();
    for (int i = tid; i < m * top; i += 1024) {
        const int v = ids[i];
        id[i] = v;
        if (v >= 0 && v < e)
            atomicOr(&chose[v], 1ull << (i / top));
    }
    __syncthreads();
    const int count = __builtin_popcountll(chose[tid]);
    const int cls = count <= 4 ? 0 : count <= 8 ? 1 : 2, entries = cls < 2 ? count > 0 : (count + 15) / 16;
    // running sums of the pairs and of each class's entries, 16 bits each
    const uint64_t own = (uint64_t)count | (uint64_t)entries << (16 * (cls + 1));
    uint64_t upto = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t v = __shfl_up((unsigned long long)upto, o);
        if (lane >= o)
            upto += v;
    }
    if (lane == 63)
        sums[wave] = upto;
    __syncthreads();
    uint64_t before = upto - own, all = 0;
    for (int w = 0; w < 16; w++) {
        if (w < wave)
            before += sums[w];
        all += sums[w];
    }
    const int c0 = all >> 16 & 0xffff, c1 = all >> 32 & 0xffff, c2 = all >> 48;
    if (tid == 0)
        plan.begin[0] = 0, plan.begin[1] = c0, plan.begin[2] = c0 + c1, plan.begin[3] = c0 + c1 + c2;
    first[tid] = (uint16_t)before;
    const int at = (int)(before >> (16 * (cls + 1)) & 0xffff) + (cls == 0 ? 0 : cls == 1 ? c0 : c0 + c1);
    for (int i = 0; i < entries; i++)
        plan.entry[at + i] = MoeEntry::packed(tid, (int)(before & 0xffff) + 16 * i, min(count - 16 * i, 16));
    __syncthreads();
    for (int i = tid; i < m * top; i += 1024) {
        const int v = id[i], t = i / top;
        bool once = v >= 0 && v < e;
        for (int j = t * top; j < i; j++)
            once = once && id[j] != v;
        if (once) {
            float w = 0.0f;
            for (int j = i; j < (t + 1) * top; j++)
                w += id[j] == v ? weights[j] : 0.0f;
            const int p = first[v] + __builtin_popcountll(chose[v] & ((1ull << t) - 1));
            plan.row[p] = (uint16_t)i;
            plan.weight[p] = w;
        }
    }
}

__global__ void __launch_bounds__(1024) moe_plan_kernel(MoeArgs a) { moe_plan(a.ids, a.weights, a.m, a.top, a.e, *a.plan); }

__device__ __forceinline__ void store_part(uint8_t *h, int64_t at, float v)
{
    reinterpret_cast<uint16_t *>(h)[at] = (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16);
}

// Gated products of an entry's tokens on one row tile of gate and up a wave.  ONE: the
// only token's choice number entry.first, without a plan.
template <int TX, int GRP, int PK, int D, bool ONE>
__device__ __forceinline__ void moe_gated_tile(const MoeArgs &a, const MoeEntry &entry, int64_t rt, float *part)
{
    using Wave = Q4gWave<TX, GRP, 2, 1, PK, D>;
    constexpr int N = Wave::N;
    const Q4gShape sh(a.n, a.k, GRP, a.fmt);
    const int lane = opaque_lane(), wave = wave_number(), kw = wave % a.kw, set = wave - kw;
    const auto row = [&](int p) { // of h; past the last the last one
        return ONE ? entry.first : (int)a.plan->row[entry.first + (p < entry.count ? p : entry.count - 1)];
    };
    Wave w;
    w.clear();
    if (rt < sh.rt) {
        typename Wave::Rows rows;
        rows.w[0] = Q4gRows(a.wg + entry.expert * a.gu_bytes, sh, rt, GRP, a.fmt);
        rows.w[1] = Q4gRows(a.wu + entry.expert * a.gu_bytes, sh, rt, GRP, a.fmt);
        rows.x = static_cast<const uint8_t *>(a.x); // 64 rows of under 2^24 elements: offsets below 2^32
        rows.at[0] = ONE ? 0 : (uint32_t)(row(Wave::row_of(lane)) / a.top) * (uint32_t)a.k * q4g_x_size(TX);
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
        const int p = Wave::out_of(lane, i);
        if (p < entry.count && j < a.n) {
            const int64_t at = row(p) * a.n + j;
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

template <int TX, int GRP, bool ONE>
__global__ void __launch_bounds__(512, 4) moe_gated_kernel(MoeArgs a)
{
    extern __shared__ float part[];
    const int rw = wave_number() / a.kw, sets = blockDim.x / 64 / a.kw, y = blockIdx.y;
    const int64_t tiles = (a.n + 15) / 16, step = (int64_t)gridDim.x * sets;
    if constexpr (ONE) {
        const int id = a.ids[y];
        if (id < 0 || id >= a.e)
            return;
        const MoeEntry entry(MoeEntry::packed(id, y, 1));
        for (int64_t rt = (int64_t)blockIdx.x * sets; rt < tiles; rt += step)
            moe_gated_tile<TX, GRP, 4, 2, true>(a, entry, rt + rw, part);
    } else {
        if (y >= a.plan->begin[3])
            return;
        const MoeEntry entry(__builtin_amdgcn_readfirstlane(a.plan->entry[y]));
        for (int64_t rt = (int64_t)blockIdx.x * sets; rt < tiles; rt += step)
            if (y < a.plan->begin[1])
                moe_gated_tile<TX, GRP, 4, 2, false>(a, entry, rt + rw, part);
            else if (y < a.plan->begin[2])
                moe_gated_tile<TX, GRP, 2, 1, false>(a, entry, rt + rw, part);
            else
                moe_gated_tile<TX, GRP, 1, 1, false>(a, entry, rt + rw, part);
    }
}

// What a workgroup of the down products keeps in LDS.
struct MoeLists {
    float *sums, *weight;  // sums [waves][m][16]
    uint32_t *entry;
    uint16_t *row;
};

// Down products of 16 rows with the entries [e0, e1) of a class.  The tiles of their
// matrices' 16 rows, one entry after another, are one sequence that the waves
// share evenly, each with D tiles in flight across the entries' ends; at such an end it adds its
// weighted products to its own sums [m][16].  No two products of an entry are one token's.
template <int TX, int GRP, int PK, int D>
__device__ __forceinline__ void moe_down_stream(const MoeArgs &a, const MoeLists &l, int e0, int e1, int64_t rt,
                                                int waves)
{
    using Wave = Q4gWave<TX, GRP, 1, 1, PK, D>;
    const Q4gShape sh(a.k, a.n, GRP, a.fmt);
    const int lane = opaque_lane(), wave = wave_number(), kt = (int)sh.kt;
    const int64_t tiles = (int64_t)(e1 - e0) * kt;
    const int64_t f0 = tiles * wave / waves, f1 = tiles * (wave + 1) / waves;
    if (f0 >= f1)
        return;
    float *sums = l.sums + wave * a.m * 16;
    typename Wave::Rows rows;
    rows.x = a.h; // 2048 rows of under 2^20 elements: offsets below 2^32
    rows.part = (int64_t)a.m * a.top * a.n * 2, rows.last = (int)a.n - 32, rows.bf16 = a.fmt & kQ4gBf16, rows.lane = lane;
    Wave w;
    w.clear();
    typename Wave::Stage st[D];
    int le = e0 + (int)(f0 / kt), lt = (int)(f0 % kt), ue = le, ut = lt; // the next tile to load, to use
    const auto enter = [&]() {
        const MoeEntry en(__builtin_amdgcn_readfirstlane(l.entry[le]));
        const int p = Wave::row_of(lane);
        rows.w[0] = Q4gRows(a.wd + en.expert * a.d_bytes, sh, rt, GRP, a.fmt);
        rows.at[0] = l.row[en.first + (p < en.count ? p : en.count - 1)] * (uint32_t)a.n * 2;
    };
    const auto leave = [&]() {
        const MoeEntry en(__builtin_amdgcn_readfirstlane(l.entry[ue]));
#pragma unroll
        for (int i = 0; i < Wave::N; i++) {
            const int p = Wave::out_of(lane, i);
            if (p < en.count) {
                float *to = sums + l.row[en.first + p] / a.top * 16 + lane % 16;
                *to = fmaf(l.weight[en.first + p], w.y[0][0][i], *to);
            }
        }
        w.clear();
    };
    int64_t left = f1 - f0; // tiles to load
    const auto load = [&](typename Wave::Stage &s) {
        Wave::load(s, rows, lt);
        if (--left > 0 && ++lt == kt) { // past the end: the last one again
            lt = 0, le++;
            enter();
        }
    };
    const auto use = [&](const typename Wave::Stage &s) {
        w.use(s, rows.bf16, ut);
        if (++ut == kt) {
            leave();
            ut = 0, ue++;
        }
    };
    enter();
#pragma unroll
    for (int i = 0; i < D; i++)
        load(st[i]);
    int64_t f = f0;
    for (; f + D < f1; f += D) {
#pragma unroll
        for (int i = 0; i < D; i++) {
            use(st[i]);
            __builtin_amdgcn_sched_barrier(0);
            load(st[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int i = 0; i < D; i++) {
        if (f + i < f1)
            use(st[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (ut > 0)
        leave();
}

constexpr int kDownWaves = 16;

// One workgroup for 16 rows, over all entries; the waves' sums are added in order.
template <int TX, int GRP, bool ONE>
__global__ void __launch_bounds__(64 * kDownWaves) moe_down_kernel(MoeArgs a)
{
    extern __shared__ float lds[];
    const int waves = blockDim.x / 64, pairs = a.m * a.top;
    MoeLists l;
    l.sums = lds, l.weight = l.sums + waves * a.m * 16;
    l.entry = reinterpret_cast<uint32_t *>(l.weight + pairs);
    for (int i = threadIdx.x; i < waves * a.m * 16; i += blockDim.x)
        l.sums[i] = 0.0f;
    const int64_t rt = blockIdx.x;
    if constexpr (ONE) { // the only token's choices are the entries, but for padding
        l.row = reinterpret_cast<uint16_t *>(l.entry + pairs);
        const int i = threadIdx.x, id = i < a.top ? a.ids[i] : -1;
        const bool in = id >= 0 && id < a.e;
        const uint64_t who = __ballot(in);
        if (in) {
            const int at = __builtin_popcountll(who & ((1ull << i) - 1));
            l.entry[at] = MoeEntry::packed(id, at, 1);
            l.row[at] = (uint16_t)i, l.weight[at] = a.weights[i];
        }
        __shared__ int count;
        if (i == 0)
            count = __builtin_popcountll(who);
        __syncthreads();
        moe_down_stream<TX, GRP, 4, 4>(a, l, 0, count, rt, waves);
    } else {
        const int c1 = a.plan->begin[1], c2 = a.plan->begin[2], c3 = a.plan->begin[3];
        l.row = reinterpret_cast<uint16_t *>(l.entry + c3);
        for (int i = threadIdx.x; i < c3; i += blockDim.x)
            l.entry[i] = a.plan->entry[i];
        for (int i = threadIdx.x; i < pairs; i += blockDim.x)
            l.row[i] = a.plan->row[i], l.weight[i] = a.plan->weight[i];
        __syncthreads();
        moe_down_stream<TX, GRP, 4, 4>(a, l, 0, c1, rt, waves);
        moe_down_stream<TX, GRP, 2, 2>(a, l, c1, c2, rt, waves);
        moe_down_stream<TX, GRP, 1, 1>(a, l, c2, c3, rt, waves);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.m * 16; i += blockDim.x) {
        float v = l.sums[i];
        for (int o = 1; o < waves; o++)
            v += l.sums[o * a.m * 16 + i];
        const int64_t j = rt * 16 + i % 16, at = i / 16 * a.k + j;
        if (j < a.k) {
            if (a.res)
                v += load_as(a.res, at, a.dtype);
            store_as(a.y, at, v, a.dtype);
        }
    }
}

template <int TX, int GRP, bool ONE>
hipError_t experts(MoeArgs a, hipStream_t s)
{
    const int64_t pairs = (int64_t)a.m * a.top, active = pairs < a.e ? pairs : a.e;
    const int64_t rt = (a.n + 15) / 16, kt = (a.k + 127) / 128, dt = (a.k + 15) / 16, nt = (a.n + 127) / 128;
    a.kw = 1;
    while (a.kw < 8 && rt * active * a.kw < 4096 && 2 * a.kw <= kt)
        a.kw *= 2;
    const int64_t most = (rt * a.kw + 7) / 8, want = (1024 + active - 1) / active;
    const int64_t entries = ONE ? pairs : active + pairs / 16; // at most
    moe_gated_kernel<TX, GRP, ONE><<<dim3((unsigned)(most < want ? most : want), (unsigned)entries), 512,
                                    a.kw > 1 ? (size_t)8 * 2 * 4 * 64 * sizeof(float) : 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t most_waves = a.m > 32 ? 8 : kDownWaves, waves = active * nt < most_waves ? active * nt : most_waves;
    const size_t lds = (size_t)waves * a.m * 64 + pairs * 6 + entries * 4;
    constexpr int TH = TX == Q4G_X_F32 ? Q4G_X_PARTS3 : Q4G_X_PARTS2;
    moe_down_kernel<TH, GRP, ONE><<<(unsigned)dt, (unsigned)(64 * waves), lds, s>>>(a);
    return hipGetLastError();
}

template <int TX>
hipError_t experts_g(const MoeArgs &a, int64_t group, hipStream_t s)
{
    if (a.m == 1)
        return group == 32 ? experts<TX, 32, true>(a, s) : group == 64 ? experts<TX, 64, true>(a, s) : experts<TX, 128, true>(a, s);
    moe_plan_kernel<<<1, 1024, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    return group == 32 ? experts<TX, 32, false>(a, s) : group == 64 ? experts<TX, 64, false>(a, s) : experts<TX, 128, false>(a, s);
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

// Groups of 64 tokens, one after another, in the same workspace: the plan, then h.
constexpr size_t kMoePlanBytes = (sizeof(MoePlan) + 255) / 256 * 256;

size_t q4g_moe_workspace(int64_t m, int64_t n, int64_t top)
{
    const int64_t tokens = m < kMoeTokens ? m : kMoeTokens;
    return kMoePlanBytes + ((size_t)(tokens * top * n) * 6 + 255) / 256 * 256;
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
        a.h = static_cast<uint8_t *>(ws) + kMoePlanBytes;
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
