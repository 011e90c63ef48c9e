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
// eight) a lane takes eight elements of a row at a time.  One token, 128 x 4096 bf16: 2.8 us, a trip to memory and
// the sums over the lanes; 64 tokens, 256 x 4096 f32 11 us (12 TFLOP/s of f64): converting and multiplying in f64,
// and every expert's row loaded again for eight tokens (tiles of 8 x 8: 14.5).
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
// largest that is left, the lower index first among equal ones.  Latency of dependent f64 steps (exp, sums and
// maxima over the lanes, `top` of these one after another): 3.3 us for 8 of 128, 4.1 for 8 of 256, of
// which 1.8 is the launch.
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
    if (renorm && total < 0x1p-900) { // scores that leave f64's range (all chosen ones far below 1): by their logits
        const double l = lane < top ? logits[t * e + chosen] : -__builtin_inf();
        const uint64_t b = wave_max(order_bits(l));
        mine = exp(l - __builtin_bit_cast(double, b >> 63 ? b & 0x7fffffffffffffffull : ~b));
        total = wave_sum(mine);
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
constexpr int kMoeEntries = (int)kMaxExperts + kMoePairs / 8;

// Who chose whom, for a group of at most 64 tokens.  An entry is up to 4, 8 or 16 tokens of
// an expert (class 0, 1, 2): an expert with at most four tokens is one entry of class 0, up to eight
// one of class 1, more of them entries of sixteen (of eight, class 1, where rows come as three
// parts: sixteen such rows take the LDS of two workgroups).  begin[c] is class c's first entry,
// begin[3] their number; entries stand in ascending order of the experts within
// a class.  A token that names an expert twice is one pair.
struct MoePlan {
    int32_t begin[4];
    uint32_t entry[kMoeEntries]; // expert | first pair << 10 | pairs << 21
    uint16_t row[kMoePairs];     // per pair: its row in h, token * top + the first slot of that expert
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

// The gated products between the two: three bf16 parts of each, all 24 bits, where the stream is f32 or
// there are up to four tokens.  Two parts for more tokens of a 16-bit stream: what is left out is up to 2^-17 of the value,
// against 2^-9 and 2^-12 of the outputs' own rounding, and moves one of 350 f16 and of 900 bf16 outputs to the
// neighbouring value.  (A third part costs one to four tokens 1 to 6%, but 2 of 8 experts of 3 x 14336 x 4096 on 32
// tokens 303 us in place of 224, as sixteen such rows do not fit in LDS at once.)  The parts are what the
// matrix core reads, so the down kernel's waves load them as they stand: splitting
// f32 values there would be done again for every 16 output rows.
struct MoeArgs {
    const uint8_t *wg, *wu, *wd;
    const void *x, *res;
    const int32_t *ids;
    const float *weights;
    void *y;
    uint8_t *h; // [part][m * top][n], moe_h_type()
    MoePlan *plan;
    int64_t n, k, gu_bytes, d_bytes; // bytes from one expert to the next
    int m, top, e, fmt, act, dtype;
    int kw;     // waves along k
    float *out; // down products of each choice, [m * top][k]
    uint8_t *x_parts; // f32 rows as three bf16 parts, [part][m][k] (in the same place, before them)
};

// One workgroup makes the plan; threads are experts, then pairs.  Latency of its five steps: 3.8 to 5 us (made by
// the choice's workgroup instead, one for all tokens, both take 10.7 against 4.6 + 4.9).
__device__ __forceinline__ void moe_plan(const int32_t *ids, int m, int top, int e, bool wide, MoePlan &plan)
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
    const int cls = count <= 4 ? 0 : count <= 8 || wide ? 1 : 2, most = 4 << cls, entries = (count + most - 1) / most;
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
        plan.entry[at + i] = MoeEntry::packed(tid, (int)(before & 0xffff) + most * i, min(count - most * i, most));
    __syncthreads();
    for (int i = tid; i < m * top; i += 1024) {
        const int v = id[i], t = i / top;
        bool once = v >= 0 && v < e;
        for (int j = t * top; j < i; j++)
            once = once && id[j] != v;
        if (once) {
            const int p = first[v] + __builtin_popcountll(chose[v] & ((1ull << t) - 1));
            plan.row[p] = (uint16_t)i;
        }
    }
}

__global__ void __launch_bounds__(1024) moe_plan_kernel(MoeArgs a) { moe_plan(a.ids, a.m, a.top, a.e, a.dtype == QLL_W_F32, *a.plan); }

__device__ __forceinline__ void store_part(uint8_t *h, int64_t at, float v)
{
    reinterpret_cast<uint16_t *>(h)[at] = (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16);
}

enum { MOE_ONE, MOE_FEW, MOE_ALL }; // one token; up to four; more
constexpr int moe_h_type(int tx, int kind)
{
    return tx == Q4G_X_F32 || tx == Q4G_X_PARTS3 || kind != MOE_ALL ? Q4G_X_PARTS3 : Q4G_X_PARTS2;
}

// What becomes of an entry's products with one row tile, N a lane.  The waves of a set add up in LDS:
// KW along k.  GATED: gate and up product meet, in a wave (R = 2) or as the set's KW waves on the
// gate matrix and KW on the up matrix (R = 1), and the products' parts go to h.  Otherwise the products
// go to `out` [m * top][k], f32, one row a choice.
template <int TX, bool GATED, int KIND, int R, int N>
__device__ __forceinline__ void moe_outputs(const MoeArgs &a, const MoeEntry &entry, const float (&y)[R][1][N], int64_t rt,
                                            int KW, float *sums, int lane)
{
    const int SW = GATED && R == 1 ? 2 * KW : KW, wave = wave_number(), set = wave - wave % SW;
    if (SW > 1) {
        __syncthreads(); // LDS is read
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int i = 0; i < N; i++)
                sums[((wave * R + r) * N + i) * 64 + lane] = y[r][0][i];
        __syncthreads();
    }
    const int64_t outs = GATED ? a.n : a.k, j = rt * 16 + lane % 16, whole = (int64_t)a.m * a.top * a.n;
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (SW > 1 && i % SW != wave % SW) // the set's waves take turns
            continue;
        float v[2] = {y[0][0][i], y[R - 1][0][i]};
        if (SW > 1)
#pragma unroll
            for (int b = 0; b < (GATED ? 2 : 1); b++) {
                const int from = (R == 1 ? (set + b * KW) : set * R + b) * N + i;
                v[b] = sums[from * 64 + lane];
                for (int o = 1; o < KW; o++)
                    v[b] += sums[(from + o * R * N) * 64 + lane];
            }
        const int p = lane / 16 * N + i;
        if (p >= entry.count || j >= outs)
            continue;
        const int64_t to = (KIND == MOE_ONE ? entry.first : (int)a.plan->row[entry.first + p]) * outs + j;
        if constexpr (GATED) {
            const float h = activate(v[0], a.act) * v[1];
            if constexpr (moe_h_type(TX, KIND) == Q4G_X_PARTS3) {
                const float rest = below_bf16(h);
                store_part(a.h, to, h);
                store_part(a.h, whole + to, rest);
                store_part(a.h, 2 * whole + to, below_bf16(rest));
            } else { // both parts to nearest
                const __bf16 upper = (__bf16)h;
                reinterpret_cast<__bf16 *>(a.h)[to] = upper;
                reinterpret_cast<__bf16 *>(a.h)[whole + to] = (__bf16)(h - (float)upper);
            }
        } else
            a.out[to] = v[0];
    }
}

// An entry's products with every so-manieth set of row tiles, one of gate and one of up, or R of down.
// Offsets into the rows are 32 bits: 64 rows of x of under 2^24 elements, 2048 of h of under 2^20.
template <int TX, int GRP, bool GATED, int KIND>
__device__ __forceinline__ void moe_few(const MoeArgs &a, const MoeEntry &entry, float *sums)
{
    constexpr int R = GATED ? 2 : 1;
    using Wave = Q4gWave<TX, GRP, R, 4, GATED || TX == Q4G_X_PARTS3 ? 2 : 4>;
    const int64_t outs = GATED ? a.n : a.k;
    const int k = (int)(GATED ? a.k : a.n);
    const Q4gShape sh(outs, k, GRP, a.fmt);
    const int lane = opaque_lane(), wave = wave_number(), KW = a.kw, kw = wave % KW, sets = 8 / KW;
    typename Wave::From f;
    int row = entry.first;
    if constexpr (KIND != MOE_ONE) { // past the last token: its row again
        const int p = Wave::row_of(lane);
        row = a.plan->row[entry.first + (p < entry.count ? p : entry.count - 1)];
    }
    f.x = !GATED ? a.h : TX == Q4G_X_PARTS3 ? a.x_parts : static_cast<const uint8_t *>(a.x);
    f.at = (uint32_t)(GATED ? row / a.top : row) * (uint32_t)k * q4g_x_size(TX);
    f.part = (int64_t)a.m * (GATED ? a.k : a.top * a.n) * 2, f.last = k - 32, f.kt = (int)sh.kt;
    const int ks = (int)sh.ks, per = (ks + KW - 1) / KW, p0 = kw * per, p1 = p0 + per < ks ? p0 + per : ks;
    for (int64_t at = (int64_t)blockIdx.x * sets; at < sh.rt; at += (int64_t)gridDim.x * sets) {
        const int64_t rt = at + wave / KW;
        Wave w;
        w.clear();
        if (rt < sh.rt) {
            if constexpr (GATED) {
                f.w[0] = Q4gRows(a.wg + entry.expert * a.gu_bytes, sh, rt, GRP, a.fmt);
                f.w[1] = Q4gRows(a.wu + entry.expert * a.gu_bytes, sh, rt, GRP, a.fmt);
            } else
                f.w[0] = Q4gRows(a.wd + entry.expert * a.d_bytes, sh, rt, GRP, a.fmt);
            w.run(f, p0, p1, a.fmt & kQ4gBf16, lane);
        }
        moe_outputs<TX, GATED, KIND>(a, entry, w.y, rt, KW, sums, lane);
    }
}

// The same for up to 16 / PK tokens, their rows in LDS, gate and up as two sets of waves (both in one
// take up to 170 registers).
template <int TX, int GRP, int PK, bool GATED>
__device__ __forceinline__ void moe_more(const MoeArgs &a, const MoeEntry &entry, uint8_t *lds)
{
    using Block = Q4gBlock<TX, GRP, 1, 1, PK>;
    const int64_t outs = GATED ? a.n : a.k;
    const int k = (int)(GATED ? a.k : a.n);
    const Q4gShape sh(outs, k, GRP, a.fmt);
    const int KW = a.kw < Block::kPieces ? a.kw : Block::kPieces, SW = GATED ? 2 * KW : KW;
    const int lane = opaque_lane(), wave = wave_number(), kw = wave % KW, sets = 8 / SW;
    const uint8_t *matrix = GATED ? (wave / KW % 2 ? a.wu : a.wg) + entry.expert * a.gu_bytes : a.wd + entry.expert * a.d_bytes;
    typename Block::X src;
    src.base = !GATED ? a.h : TX == Q4G_X_PARTS3 ? a.x_parts : static_cast<const uint8_t *>(a.x), src.k = k;
    src.part = (int64_t)a.m * (GATED ? a.k : a.top * a.n) * 2;
    const int p = Block::row_of(lane);
    src.at[0] = ~0u;
    if (p < entry.count) {
        const int row = a.plan->row[entry.first + p];
        src.at[0] = (uint32_t)(GATED ? row / a.top : row) * (uint32_t)k * 2;
    }
    const int chunks = (k + Block::kChunk - 1) / Block::kChunk;
    float *sums = reinterpret_cast<float *>(lds + (chunks == 1 ? Block::lds_bytes(k) : 0));
    bool first = true;
    for (int64_t at = (int64_t)blockIdx.x * sets; at < sh.rt; at += (int64_t)gridDim.x * sets) {
        const int64_t rt = at + wave / SW;
        const Q4gRows rows[1] = {Q4gRows(matrix, sh, rt < sh.rt ? rt : sh.rt - 1, GRP, a.fmt)};
        Block w;
        w.clear();
        if (chunks > 1 && !first)
            __syncthreads(); // LDS is read
        w.run(rows, rt < sh.rt, src, 0, chunks, kw, KW, a.fmt & kQ4gBf16, chunks == 1 && !first, lds, lane);
        first = false;
        moe_outputs<TX, GATED, MOE_ALL>(a, entry, w.y, rt, KW, sums, lane);
    }
}

// The products of entry blockIdx.y.  What bounds them is the experts' weights and the instructions that widen
// them: one bf16 token, two experts of 3 x 14336 x 4096 gate and up in 27 us (122 MB, 4.5 TB/s); 64 tokens, six of 64 experts of
// 3 x 1536 x 4096, 88 to 95 us (418 MB, 4.4 to 4.7 TB/s) and down 53 to 58 (3.6 to 3.9).  37 f32 tokens, three of 23
// experts of 3 x 1440 x 2592, take 42 to 44 us (99 MB, 2.3 TB/s) and 26 to 28: three parts a value are three times the
// matrix instructions (busy 24% of the time) and LDS reads.
template <int TX, int GRP, bool GATED, int KIND>
__global__ void __launch_bounds__(512, 4) moe_entry_kernel(MoeArgs a)
{
    extern __shared__ __attribute__((aligned(16))) uint8_t entry_lds[];
    float *sums = reinterpret_cast<float *>(entry_lds);
    const int y = blockIdx.y;
    if constexpr (KIND == MOE_ONE) {
        const int id = a.ids[y];
        if (id >= 0 && id < a.e)
            moe_few<TX, GRP, GATED, KIND>(a, MoeEntry(MoeEntry::packed(id, y, 1)), sums);
    } else {
        if (y >= a.plan->begin[3])
            return;
        const MoeEntry entry(__builtin_amdgcn_readfirstlane(a.plan->entry[y]));
        if constexpr (KIND == MOE_FEW)
            moe_few<TX, GRP, GATED, KIND>(a, entry, sums);
        else if (y < a.plan->begin[1])
            moe_few<TX, GRP, GATED, KIND>(a, entry, sums);
        else if (y < a.plan->begin[2])
            moe_more<TX, GRP, 2, GATED>(a, entry, entry_lds);
        else if constexpr (TX != Q4G_X_PARTS3)
            moe_more<TX, GRP, 1, GATED>(a, entry, entry_lds);
    }
}

// The weighted sum of a token's choices, in their order, and the residual: four columns a thread.  The
// choices' order makes results repeat, where atomic additions would not.  64 x 6 x 4096: 4.8 us (8 MB, mostly
// latency).
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeArgs a)
{
    const int64_t column = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, j = column < a.k ? column : 0; // whole waves stay
    const int t = blockIdx.y;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const int slot = threadIdx.x % 64; // a lane holds a choice
    const int id = slot < a.top ? a.ids[t * a.top + slot] : -1;
    const float weight = id >= 0 && id < a.e ? a.weights[t * a.top + slot] : 0.0f;
    for (int s0 = 0; s0 < a.top; s0 += 8) { // eight choices' loads at once
        f32x4 p[8];
        float w[8];
#pragma unroll
        for (int b = 0; b < 8; b++) {
            const int other = __builtin_amdgcn_readlane(id, s0 + b); // top <= 32
            w[b] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), s0 + b));
            p[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (other >= 0 && other < a.e) { // the first slot that names it has the product
                const int from = __builtin_ctzll(__ballot(id == other));
                p[b] = *reinterpret_cast<const f32x4 *>(a.out + (int64_t)(t * a.top + from) * a.k + j);
            }
        }
#pragma unroll
        for (int b = 0; b < 8; b++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = fmaf(w[b], p[b][i], v[i]);
    }
    if (column >= a.k)
        return;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float o = a.res ? v[i] + load_as(a.res, t * a.k + j + i, a.dtype) : v[i];
        store_as(a.y, t * a.k + j + i, o, a.dtype);
    }
}

constexpr int kDownWaves = 16;

// One token's down products of 16 rows, weighted and added up.  The pieces of its choices' matrices'
// rows, one choice after another, are one sequence that the waves share evenly, with
// loads in flight across the choices' ends; at such an end a wave adds its weighted products.  Two experts of
// 14336 -> 4096: 20 to 21 us (61 MB, 3.0 TB/s), 16 waves a row tile with 1441 vector instructions each, which take half
// of it, and a third of their time waiting to issue; eight of 1024 -> 2048 7 to 8 us, latency.
template <int TX, int GRP>
__global__ void __launch_bounds__(64 * kDownWaves) moe_down_kernel(MoeArgs a)
{
    using Wave = Q4gWave<TX, GRP, 1, 4, 4>;
    __shared__ float sums[kDownWaves][16], weights[kMaxTop];
    __shared__ int expert[kMaxTop], slot[kMaxTop], count;
    const int waves = blockDim.x / 64, wave = wave_number(), lane = threadIdx.x % 64;
    const int64_t rt = blockIdx.x;
    if (wave == 0) { // the choices but for padding
        const int id = lane < a.top ? a.ids[lane] : -1;
        const bool in = id >= 0 && id < a.e;
        const uint64_t who = __ballot(in);
        if (in) {
            const int at = __builtin_popcountll(who & ((1ull << lane) - 1));
            expert[at] = id, slot[at] = lane, weights[at] = a.weights[lane];
        }
        if (lane == 0)
            count = __builtin_popcountll(who);
    }
    __syncthreads();
    const Q4gShape sh(a.k, a.n, GRP, a.fmt);
    const int ks = (int)sh.ks, pieces = __builtin_amdgcn_readfirstlane(count) * ks; // below 2^5 * 2^11
    const int f0 = pieces * wave / waves, f1 = pieces * (wave + 1) / waves;
    float sum = 0.0f;
    if (f0 < f1) {
        const bool bf16 = a.fmt & kQ4gBf16;
        typename Wave::From f;
        f.x = a.h, f.part = (int64_t)a.top * a.n * 2, f.last = (int)a.n - 32, f.kt = (int)sh.kt;
        const auto enter = [&](int choice) {
            f.w[0] = Q4gRows(a.wd + __builtin_amdgcn_readfirstlane(expert[choice]) * a.d_bytes, sh, rt, GRP, a.fmt);
            f.at = (uint32_t)slot[choice] * (uint32_t)a.n * 2;
        };
        int choice = f0 / ks, p = f0 % ks;
        Wave w;
        w.clear();
        enter(choice);
        w.start(f, p, lane);
        for (int i = f0; i < f1; i++) {
            const bool end = p + 1 == ks;
            const int after = end ? 0 : p + 1;
            if (i + 1 < f1) {
                if (end)
                    enter(choice + 1);
                w.template use_piece<true, false>(f, p, f, after, bf16, lane); // four tiles in flight: f is the next one's
            } else
                w.template use_piece<false, false>(f, p, f, 0, bf16, lane);
            if (end || i + 1 == f1) {
                sum = fmaf(weights[choice], w.y[0][0][0], sum);
                w.clear();
                choice++;
            }
            p = after;
        }
    }
    if (lane < 16)
        sums[wave][lane] = sum;
    __syncthreads();
    const int64_t j = rt * 16 + threadIdx.x;
    if (threadIdx.x < 16 && j < a.k) {
        float v = sums[0][lane];
        for (int o = 1; o < waves; o++)
            v += sums[o][lane];
        if (a.res)
            v += load_as(a.res, j, a.dtype);
        store_as(a.y, j, v, a.dtype);
    }
}

// Room that a token's down products take in a column, 4 bytes a choice, and before them its f32 value as
// parts, 6 bytes.
int64_t moe_column_bytes(int64_t top) { return (int64_t)sizeof(float) * (top < 2 ? 2 : top); }

// Room for these of up to 64 tokens: 32768 columns, 32 MiB at most; one token needs none.
int64_t moe_out_bytes(int64_t m, int64_t top)
{
    const int64_t all = m == 1 ? 0 : m * 32768 * moe_column_bytes(top);
    return all < (int64_t)32 << 20 ? all : (int64_t)32 << 20;
}

// Tokens that go at once: 64, or as many as have that room.
int64_t moe_group(int64_t m, int64_t top, int64_t k)
{
    const int64_t tokens = m < kMoeTokens ? m : kMoeTokens, room = moe_out_bytes(tokens, top);
    const int64_t each = k * moe_column_bytes(top);
    return room / each < 2 ? 1 : room / each < tokens ? room / each : tokens;
}

// Entries' products as one launch of up to some 4096 workgroups: mostly one set of row tiles each, whose
// ends overlap with others' work (1024 with several each: down products 5% slower).
template <int TX, int GRP, bool GATED, int KIND>
hipError_t entries(MoeArgs a, int64_t active, int64_t count, hipStream_t s)
{
    const int64_t outs = GATED ? a.n : a.k, k = GATED ? a.k : a.n, ks = (k + 511) / 512, tiles = (outs + 15) / 16;
    // Waves along k, at most (a class whose chunks have fewer pieces takes fewer), until there are so many in all: 4
    // tokens, 6 of 64 experts of 3 x 1536 x 4096 86 -> 75 us against 2048 gated, 2 of 8 of 3 x 14336 x 4096 157 -> 147
    // against 4096 down, where 16 and more tokens lose by more (180 -> 203).
    const int64_t waves = GATED ? 3000 : KIND == MOE_FEW ? 8192 : 4096;
    a.kw = 1;
    while (a.kw < 8 && 2 * a.kw <= ks && tiles * active * a.kw < waves)
        a.kw *= 2;
    const int64_t most = (tiles * a.kw + 7) / 8, want = (4096 + active - 1) / active;
    int64_t lds = (GATED ? 2 : 1) * 8 * 64 * sizeof(float);
    if constexpr (KIND == MOE_ALL) { // whichever of the classes takes most
        using B2 = Q4gBlock<TX, GRP, 1, 1, 2>;
        using B1 = Q4gBlock<TX, GRP, 1, 1, 1>;
        const int64_t x1 = a.m <= 8 || TX == Q4G_X_PARTS3 ? 0 : B1::lds_bytes(k);
        lds = 4 * lds + (B2::lds_bytes(k) > x1 ? B2::lds_bytes(k) : x1);
    }
    moe_entry_kernel<TX, GRP, GATED, KIND><<<dim3((unsigned)(most < want ? most : want), (unsigned)count), 512,
                                            (size_t)lds, s>>>(a);
    return hipGetLastError();
}

// TX: the rows as the kernels take them, which for more than four f32 rows is as parts.
template <int TX, int GRP, int KIND>
hipError_t experts(const MoeArgs &a, hipStream_t s)
{
    constexpr int TH = moe_h_type(TX, KIND);
    const int64_t pairs = (int64_t)a.m * a.top, active = pairs < a.e ? pairs : a.e;
    const int64_t count = KIND == MOE_ONE ? pairs : active + pairs / (TX == Q4G_X_PARTS3 ? 8 : 16); // of entries, at most
    hipError_t e = entries<TX, GRP, true, KIND>(a, active, count, s);
    if (e != hipSuccess)
        return e;
    if constexpr (KIND == MOE_ONE) {
        const int64_t dt = (a.k + 15) / 16, pieces = active * ((a.n + 511) / 512), waves = pieces < kDownWaves ? pieces : kDownWaves;
        moe_down_kernel<TH, GRP><<<(unsigned)dt, (unsigned)(64 * waves), 0, s>>>(a);
    } else {
        e = entries<TH, GRP, false, KIND>(a, active, count, s);
        if (e != hipSuccess)
            return e;
        moe_combine_kernel<<<dim3((unsigned)((a.k + 1023) / 1024), (unsigned)a.m), 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int TX, int GRP>
hipError_t experts_k(const MoeArgs &a, hipStream_t s)
{
    if (a.m == 1)
        return experts<TX, GRP, MOE_ONE>(a, s);
    if (a.m <= 4)
        return experts<TX, GRP, MOE_FEW>(a, s);
    if constexpr (TX == Q4G_X_F32) {
        const hipError_t e = launch_q4g_split(a.x, a.x_parts, a.m * a.k, s);
        return e != hipSuccess ? e : experts<Q4G_X_PARTS3, GRP, MOE_ALL>(a, s);
    } else
        return experts<TX, GRP, MOE_ALL>(a, s);
}

template <int TX>
hipError_t experts_g(const MoeArgs &a, int64_t group, hipStream_t s)
{
    if (a.m > 1) {
        moe_plan_kernel<<<1, 1024, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return group == 32 ? experts_k<TX, 32>(a, s) : group == 64 ? experts_k<TX, 64>(a, s) : experts_k<TX, 128>(a, s);
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

// Groups of tokens, one after another, in the same workspace: the plan, the down products, h.
constexpr size_t kMoePlanBytes = (sizeof(MoePlan) + 255) / 256 * 256;

size_t q4g_moe_workspace(int64_t m, int64_t n, int64_t top)
{
    const int64_t tokens = m < kMoeTokens ? m : kMoeTokens;
    return kMoePlanBytes + (size_t)moe_out_bytes(tokens, top) + ((size_t)(tokens * top * n) * 6 + 255) / 256 * 256;
}

hipError_t launch_q4g_moe(const void *x, int dtype, const int32_t *ids, const float *weights, int64_t top,
                          const uint8_t *wg, const uint8_t *wu, const uint8_t *wd, int64_t group, int fmt, int act,
                          const void *res, void *y, int64_t m, int64_t n, int64_t k, int64_t e, void *ws, hipStream_t s)
{
    const int64_t row = k * (dtype == QLL_W_F32 ? 4 : 2);
    const int64_t group_of = moe_group(m, top, k), room = moe_out_bytes(m < kMoeTokens ? m : kMoeTokens, top);
    for (int64_t t0 = 0; t0 < m; t0 += group_of) {
        MoeArgs a{};
        a.wg = wg, a.wu = wu, a.wd = wd;
        a.x = static_cast<const uint8_t *>(x) + t0 * row;
        a.res = res ? static_cast<const uint8_t *>(res) + t0 * row : nullptr;
        a.y = static_cast<uint8_t *>(y) + t0 * row;
        a.ids = ids + t0 * top, a.weights = weights + t0 * top;
        a.plan = static_cast<MoePlan *>(ws);
        a.n = n, a.k = k;
        a.gu_bytes = q4g_packed_bytes(n, k, group, fmt), a.d_bytes = q4g_packed_bytes(k, n, group, fmt);
        a.m = (int)(m - t0 < group_of ? m - t0 : group_of), a.top = (int)top, a.e = (int)e;
        a.out = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kMoePlanBytes);
        a.x_parts = reinterpret_cast<uint8_t *>(a.out);
        a.h = a.x_parts + room;
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
