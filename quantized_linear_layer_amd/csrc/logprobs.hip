// Token log probabilities off the logits of the vocabulary projection: for
// every row x[0 .. v) with M = max x and S = sum exp(x_j - M)
//     log p_j  = x_j - M - log S
//     entropy  = log S - sum (x_j - M) exp(x_j - M) / S
// the log probabilities of given tokens, the entropy, and the `top` most
// probable tokens in the order (value descending, index ascending).
//
// Each logit is read once, as a stream: a workgroup takes a segment of a row
// (the whole of it where there are rows enough), its lanes add each step's
// logits to their own sums while the next steps' are on their way to LDS, and
// every wave keeps a list of its best so far there.  Segments of a row are joined by a
// second launch (the given tokens' logits are read by index).
//
// Sums run against a reference that is a logit of the lane, x - M first and
// log2(e) after it: finite for logits of any size, so a row masked by the
// type's lowest value is an ordinary row.  The reference moves only when a
// logit passes it by more than kLpSlack, far from f32's range.
//
// Selection.  In its first step every wave publishes the j-th of its 64 lane
// maxima, found bit by bit from ballots, with j = top / waves rounded up: the
// least of the published ones is a bound for the workgroup, since `top` elements
// or more are no worse (the lanes ahead of it hold one each).  Whatever beats
// the bound is appended to the wave's list, and a list that fills up is cut back
// to its `top` best, whose last is the wave's new bound.  Elements compare as
// 64-bit keys (value, then index), so ties neither flood the list nor depend on
// the order of arrival.  After steps 4, 16, ... the waves publish again.  A step
// is tested by its pieces' maxima, which the sums need anyway; in a long row
// most steps have no candidate.
//
// Many rows are bound by the reads: 512 x 128256 f32 (263 MB) 50 us without
// alternatives, 58 with five, 61 with twenty.  A single row is bound by latency, a step's loads
// and the search for a bound, then the same again to join: 6.7 + 6.1 us.
#include "common.h"

namespace qll {

constexpr int kLpCap = 192; // entries of a wave's list
constexpr float kLpSlack = 16.0f, kLog2e = 1.44269504f;

__device__ __forceinline__ float lp_widen(float v) { return v; }
__device__ __forceinline__ float lp_widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float lp_widen(_Float16 v) { return (float)v; }

// 16 bytes of a row.
template <typename T>
struct LpPiece {
    static constexpr int V = 16 / (int)sizeof(T);
    T e[V];
};

// A bigger key is a better element: the value's bits in unsigned order (-0 as
// +0), then the lower index.
__device__ __forceinline__ uint32_t order_bits(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ (uint32_t)((int32_t)u >> 31) ^ (u >> 31 << 31 ^ 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t order_key(float x, int i)
{
    return (uint64_t)order_bits(x + 0.0f) << 32 | (uint32_t)~i;
}

// The key of a list entry {value bits, index}.
__device__ __forceinline__ uint64_t list_key(uint64_t o)
{
    return order_key(__uint_as_float((uint32_t)o), (int)(uint32_t)(o >> 32));
}

__device__ __forceinline__ int lanes_before(uint64_t mask)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// LDS written by lanes of this wave is read by others of it next.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The largest order bits that at least k of the 64 lanes reach.
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t ob, int k)
{
    uint32_t tb = 0;
#pragma unroll 4
    for (int b = 31; b >= 0; b--) {
        const uint32_t c = tb | 1u << b;
        tb = __popcll(__ballot(ob >= c)) >= k ? c : tb;
    }
    return tb;
}

// The value just below v; NaN below -inf, so that !(x <= below(v)) is x >= v for
// every x.  Below +0 (and -0, which order_key takes for it) is the least
// negative value.
__device__ __forceinline__ float below(float v)
{
    const uint32_t ob = order_bits(v + 0.0f);
    return order_value(ob - (ob == 0x80000000u ? 2u : 1u));
}

// Keys that waves publish to each other in LDS: any value read is a bound, so no
// barrier goes with the later ones.
#define QLL_LDS_L __attribute__((address_space(3)))
template <typename V>
__device__ __forceinline__ V shared_load(const V *p)
{
    return __hip_atomic_load((const QLL_LDS_L V *)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
template <typename V>
__device__ __forceinline__ void shared_store(V *p, V v)
{
    __hip_atomic_store((QLL_LDS_L V *)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// A wave's best elements: every element that beats the bound (tv, tlo) is in
// list[0 .. n) or behind k others that are.  All members are uniform.
struct WaveTop {
    uint64_t *list; // [kLpCap] in LDS: {value bits, index}, index high
    int k, n;
    float tv;     // an element is taken if its value is above tv,
    uint32_t tlo; // or equal to it with ~index above tlo

    // The wave's key that j of its elements reach, to shared.
    template <int NW, int E, class IDX>
    static __device__ __forceinline__ void publish(const float (&x)[E], float mx, int j, const IDX &idx,
                                                   uint64_t *shared)
    {
        const uint32_t ob = order_bits(mx + 0.0f), tb = kth_of_lanes(ob, j);
        const float t = order_value(tb);
        // j lanes: those above t and the first of the lanes that have an element
        // equal to it; among elements equal to t, those up to the last of these
        // lanes' first ones are enough.  (Lanes without a logit count as -inf:
        // where that leaves too few, every element equal to t passes.)
        uint32_t mine = 0;
        bool seen = false;
#pragma unroll
        for (int e = 0; e < E; e++) {
            const bool here = x[e] == t;
            mine = here && !seen ? (uint32_t)idx(e) : mine;
            seen |= here;
        }
        const int need = j - __popcll(__ballot(ob > tb));
        const uint64_t equal = __ballot(ob == tb && seen);
        uint32_t last = ob == tb && seen && lanes_before(equal) < need ? mine : 0u;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            last = max(last, (uint32_t)__shfl_xor((int)last, off));
        if (__popcll(equal) < need)
            last = 0x7fffffff;
        if ((threadIdx.x & 63) == 0)
            shared_store(shared + (threadIdx.x >> 6), (uint64_t)tb << 32 | (~last - 1u));
    }

    // The bound from the first E elements a lane, mx the largest of each lane;
    // the workgroup's NW waves call it together.
    template <int NW, int E, class IDX>
    __device__ __forceinline__ void init(const float (&x)[E], float mx, const IDX &idx, uint64_t *shared)
    {
        publish<NW>(x, mx, (k + NW - 1) / NW, idx, shared);
        __syncthreads();
        const uint32_t none = order_bits(-INFINITY);
        uint64_t b = ~0ull, most = 0;
        int some = 0; // waves with enough logits that are not masked
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const uint64_t o = shared_load(shared + w);
            some += (uint32_t)(o >> 32) != none;
            b = o < b ? o : b;
            most = o > most ? o : most;
        }
        const bool masked = some < NW && some > 0, equal = (uint32_t)(b >> 32) == (uint32_t)(most >> 32);
        if (masked || equal) {
            // A row's last segment, or masked logits: the waves that have enough of
            // them find k among themselves, if they can.  Equal logits in all waves
            // (or nothing left): the least index is the last wave's, so one wave's own k
            // are the better bound.
            const int j = masked ? (k + some - 1) / some : k;
            __syncthreads();
            publish<NW>(x, mx, j, idx, shared);
            __syncthreads();
            uint64_t least = ~0ull;
            int found = 0;
#pragma unroll
            for (int w = 0; w < NW; w++) {
                const uint64_t o = shared_load(shared + w);
                if ((uint32_t)(o >> 32) != none) {
                    found += j;
                    least = o < least ? o : least;
                }
                b = j >= k && o > b ? o : b;
            }
            b = masked && found >= k && least > b ? least : b;
        }
        tv = order_value(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)));
        tlo = __builtin_amdgcn_readfirstlane((uint32_t)b);
        n = 0;
    }

    // Appends, from E elements a lane in pieces of V with maxima pm, those that
    // are above ts, or (TIES) that beat the bound and are not at or below ts.
    // What does not fit the list is only counted.
    template <bool TIES, int V, int E, class IDX>
    __device__ __forceinline__ void append(const float (&x)[E], const float (&pm)[E / V], float ts, const IDX &idx)
    {
#pragma unroll
        for (int p = 0; p < E / V; p++) {
            if (__ballot(!(pm[p] <= ts)) == 0)
                continue;
#pragma unroll
            for (int j = p * V; j < p * V + V; j++) {
                bool take = x[j] > ts;
                if constexpr (TIES)
                    take = !(x[j] <= ts) && (x[j] > tv || (x[j] == tv && ~(uint32_t)idx(j) > tlo));
                const uint64_t q = __ballot(take);
                if (q == 0)
                    continue;
                const int to = n + lanes_before(q);
                if (take && to < kLpCap)
                    list[to] = (uint64_t)(uint32_t)idx(j) << 32 | __float_as_uint(x[j]);
                n += __popcll(q);
            }
        }
    }

    // Where a step has more candidates than the list has room for, the list is
    // first cut to its k best, then those that fit give a tighter bound, and the
    // step is gone through again (this keeps the search for a bound, which is long,
    // in one place of the code).  With k entries before the step, 192 - k of its
    // candidates fit and at most k of them stay above the bound, so every time
    // through at least 64 fewer are left.  (With 128 entries before it and k = 64,
    // the 64 that fit could all stay, and the search went on forever.)
    template <int V, int E, class IDX>
    __device__ __forceinline__ void add(const float (&x)[E], const float (&pm)[E / V], float ts, bool ties,
                                        const IDX &idx)
    {
        bool over;
        do {
            const int n0 = n;
            if (ties)
                append<true, V>(x, pm, ts, idx);
            else
                append<false, V>(x, pm, ts, idx);
            over = n > kLpCap;
            const bool shorten = over && n0 > k;
            if (shorten)
                n = n0;
            if (shorten || n > kLpCap - 64)
                cut(!over || shorten);
            if (over) {
                n = shorten ? n : n0;
                // the bound lies among this step's elements now: values equal to
                // it are told apart by index
                ts = fmaxf(ts, below(tv));
                ties = true;
            }
        } while (over);
    }

    // The bound at the k-th best of the list, n > k (of its first kLpCap, if it
    // ran over); with `keep`, the list is cut to those.
    __device__ __forceinline__ void cut(bool keep)
    {
        constexpr int R = kLpCap / 64;
        const int lane = threadIdx.x & 63;
        wave_sync();
        uint32_t hi[R], lo[R];
#pragma unroll
        for (int i = 0; i < R; i++) {
            const uint64_t o = list[64 * i + lane], key = list_key(o);
            hi[i] = 64 * i + lane < n ? (uint32_t)(key >> 32) : 0u;
            lo[i] = (uint32_t)key;
        }
        uint32_t tb = 0;
#pragma unroll 1
        for (int b = 31; b >= 0; b--) {
            const uint32_t c = tb | 1u << b;
            int count = 0;
#pragma unroll
            for (int i = 0; i < R; i++)
                count += __popcll(__ballot(hi[i] >= c));
            tb = count >= k ? c : tb;
        }
        int above = 0, equal = 0;
#pragma unroll
        for (int i = 0; i < R; i++) {
            above += __popcll(__ballot(hi[i] > tb));
            equal += __popcll(__ballot(hi[i] == tb));
        }
        uint32_t tl = 0;
        if (above + equal > k) // ties at the border: by index
#pragma unroll 1
            for (int b = 31; b >= 0; b--) {
                const uint32_t c = tl | 1u << b;
                int count = above;
#pragma unroll
                for (int i = 0; i < R; i++)
                    count += __popcll(__ballot(hi[i] == tb && lo[i] >= c));
                tl = count >= k ? c : tl;
            }
        tv = order_value(tb);
        // (an element of the step that is gone through again may be the k-th itself)
        tlo = keep ? tl : tl - (tl != 0);
        if (!keep)
            return;
        n = 0;
#pragma unroll
        for (int i = 0; i < R; i++) {
            const bool stays = hi[i] > tb || (hi[i] == tb && lo[i] >= tl);
            const uint64_t q = __ballot(stays);
            if (stays)
                list[n + lanes_before(q)] = (uint64_t)~lo[i] << 32 | __float_as_uint(order_value(hi[i]));
            n += __popcll(q);
        }
        wave_sync();
    }
};

template <int NW>
struct LpTop {
    uint64_t list[NW][kLpCap];
    uint64_t shared[NW]; // each wave's published key of the first step
    float bound[NW];     // and of later ones a value that only better elements are above
    int total;

    // Before the first step, which has a barrier.
    __device__ __forceinline__ void clear()
    {
        if (threadIdx.x < NW)
            bound[threadIdx.x] = -INFINITY;
        if (threadIdx.x == 0)
            total = 0;
    }
    __device__ __forceinline__ float least_bound() const
    {
        float r = shared_load(&bound[0]);
#pragma unroll
        for (int w = 1; w < NW; w++)
            r = fminf(r, shared_load(&bound[w]));
        return r;
    }
};

// Where the lists are merged (the stages' LDS, once they are done with).
template <int NW>
struct LpMerge {
    uint64_t all[NW * 64];
    int rank[NW * 64];
};

// The k best of the NW waves' lists, out(rank, value, index) once for each rank
// below k; where NaN has left fewer, the remaining ranks get (-inf, pad + rank).
// What the waves' bounds still admit is gathered and ranked by counting.
template <int NW, class OUT>
__device__ __forceinline__ void merge_top(WaveTop &w, LpTop<NW> &s, LpMerge<NW> &g, int pad, const OUT &out)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    g.rank[threadIdx.x] = 0;
    if (w.n > 64)
        w.cut(true);
    wave_sync();
    const float t = s.least_bound();
    const uint64_t key = list_key(w.list[lane]);
    const bool stays = lane < w.n && !(order_value((uint32_t)(key >> 32)) <= t && t != -INFINITY);
    const uint64_t q = __ballot(stays);
    int to = 0;
    if (lane == 0)
        to = atomicAdd(&s.total, __popcll(q));
    to = __builtin_amdgcn_readfirstlane(to);
    if (stays)
        g.all[to + lanes_before(q)] = key;
    __syncthreads();
    const int total = s.total;
    for (int c = 0; c < total; c += 64) {
        const uint64_t own = c + lane < total ? g.all[c + lane] : ~0ull;
        int r = 0;
#pragma unroll 4
        for (int i = wave; i < total; i += NW)
            r += g.all[i] > own;
        if (r != 0)
            atomicAdd(&g.rank[c + lane], r);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < total; c += 64 * NW)
        if (g.rank[c] < w.k)
            out(g.rank[c], order_value((uint32_t)(g.all[c] >> 32)), (int)~(uint32_t)g.all[c]);
    if (total + (int)threadIdx.x < w.k)
        out(total + threadIdx.x, -INFINITY, pad + total + (int)threadIdx.x);
}

// Part of a row: a reference m (-inf: no logit but masked ones), s = sum 2^a and
// t = sum a 2^a with a = log2(e) (x - m).
struct LpStat {
    double s, t;
    float m, unused;
};

// A lane's running sums: a step's logits are summed in f32, the steps in f64 (a
// lane of a long row adds thousands of terms; two conversions and two additions
// for eight or sixteen logits).
struct LaneSum {
    float m;
    double s, t;

    template <int E>
    __device__ __forceinline__ void add(const float (&x)[E], float mx)
    {
        if (__ballot(mx > m + kLpSlack) != 0) { // uniform; the first logits of a lane among them
            if (mx > m) {
                const float d = fmaxf((m - mx) * kLog2e, -200.0f), w = __builtin_amdgcn_exp2f(d);
                t = (t + s * (double)d) * (double)w;
                s *= (double)w;
                m = mx;
            }
        }
        // a lane of masked logits (-inf) counts against 0.  The floor of -200
        // (far below where 2^a is 0) keeps 0 * inf out of t; NaN stays in s.
        const float ref = m == -INFINITY ? 0.0f : m;
        float ps = 0.0f, pt = 0.0f;
#pragma unroll
        for (int j = 0; j < E; j++) {
            const float a = (x[j] - ref) * kLog2e, e = __builtin_amdgcn_exp2f(a);
            ps += e;
            pt = fmaf(e, fmaxf(a, -200.0f), pt);
        }
        s += (double)ps;
        t += (double)pt;
    }

    // The wave's sums, in every lane.
    __device__ __forceinline__ LpStat wave() const
    {
        float wm = m;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            wm = fmaxf(wm, __shfl_xor(wm, off));
        const float d = (m - (wm == -INFINITY ? 0.0f : wm)) * kLog2e, w = __builtin_amdgcn_exp2f(d);
        double ws = s * (double)w, wt = (t + s * (double)fmaxf(d, -200.0f)) * (double)w;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            ws += __shfl_xor(ws, off);
            wt += __shfl_xor(wt, off);
        }
        return LpStat{ws, wt, wm, 0.0f};
    }
};

// A row's sums joined in f64 (t in natural units).
struct RowSum {
    double s, t;
    __device__ __forceinline__ void add(const LpStat &q, float m)
    {
        if (q.m == -INFINITY) { // 0, or NaN
            s += q.s;
            return;
        }
        const float d = (q.m - m) * kLog2e, w = __builtin_amdgcn_exp2f(d);
        s += (double)w * q.s;
        if (w != 0.0f)
            t += (double)w * (q.t + q.s * (double)d) * 0.6931471805599453;
    }
};

// What a call asks for.
struct LpOut {
    const int32_t *tokens;
    int64_t nt;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprob;
    int top, v;

    // The same for rows r0, r0 + 1, ... as rows 0, 1, ...
    LpOut rows(int64_t r0) const
    {
        LpOut o = *this;
        o.tokens = nt > 0 ? tokens + r0 * nt : nullptr;
        o.logprob = nt > 0 ? logprob + r0 * nt : nullptr;
        o.entropy = entropy ? entropy + r0 : nullptr;
        o.top_ids = top > 0 ? top_ids + r0 * top : nullptr;
        o.top_logprob = top > 0 ? top_logprob + r0 * top : nullptr;
        return o;
    }
};

// log p from a row's reference and sums; NaN in a row with nothing left (m is
// -inf, the sum 0).
struct RowLog {
    double m, log_s;
    __device__ __forceinline__ float operator()(float x) const { return (float)(((double)x - m) - log_s); }
};

template <typename T>
__device__ __forceinline__ float lp_given(const T *xr, int32_t id, int v)
{
    return id >= 0 && id < v ? lp_widen(xr[id]) : __builtin_nanf("");
}

// Entropy and given tokens of a row by TH threads; x0: the logit of this
// thread's first given token.
template <int TH, typename T>
__device__ __forceinline__ RowLog row_outputs(const LpOut &o, const T *xr, int64_t row, float m, const RowSum &sum,
                                              float x0)
{
    const RowLog log_p{(double)m, log(sum.s)};
    if (o.entropy && threadIdx.x == 0)
        o.entropy[row] = (float)(log_p.log_s - sum.t / sum.s);
    if ((int64_t)threadIdx.x < o.nt)
        o.logprob[row * o.nt + threadIdx.x] = log_p(x0);
    for (int64_t i = threadIdx.x + TH; i < o.nt; i += TH)
        o.logprob[row * o.nt + i] = log_p(lp_given(xr, o.tokens[row * o.nt + i], o.v));
    return log_p;
}

// Workspace of one row: a stat a segment and wave, then `top` keys a segment.
struct LpWs {
    LpStat *stat;  // [m][segments * kLpWaves]
    uint64_t *key; // [m][segments * top]
};

constexpr int kLpWaves = 4, kLpRowWaves = 8;
// Logits a thread and step.  A whole row takes two pieces: four cost registers
// (the selection is spelled out for every logit), one makes the work between
// steps count (512 x 128256, 5 alternatives: f32 57 us with two, 59 with four;
// bf16 47 with two, 50 with one).  Segments take eight logits, so that a single
// row spreads over twice the workgroups in 16 bits (1 x 128256 bf16: 12.2 against
// 15.0 us with sixteen).
template <typename T, bool ROW>
constexpr int lp_elems() { return ROW ? 2 * LpPiece<T>::V : 8; }

// Wait until at most N vector-memory operations of this wave are outstanding.
template <int N>
__device__ __forceinline__ void lp_wait()
{
    static_assert(N < 16, "vmcnt field");
    __builtin_amdgcn_s_waitcnt(N | (0xf << 8) | (0x7 << 4)); // lgkmcnt, expcnt: no wait
    asm volatile("" ::: "memory");
}

// A wave's stream of steps: E logits a lane and step in P pieces of 16 bytes,
// thread t's piece p of a step at element V (t + TH p), through S stages in LDS.
// A row's last piece is read from where it ends with the row (its first logits
// are then another thread's and count for nothing), and pieces past the end read
// that one, so every load is in bounds and unconditional.  The row must hold V
// logits.
template <typename T, int E, int TH>
struct LpStream {
    static constexpr int V = LpPiece<T>::V, P = E / V, S = 8 / P, kBytes = S * P * 1024;
    const T *row;
    uint32_t lds; // this wave's stages
    int first, end;

    __device__ __forceinline__ int place(int st, int p) const
    {
        return first + st * (TH * E) + V * ((int)threadIdx.x + TH * p);
    }

    __device__ __forceinline__ void load(int st) const
    {
#pragma unroll
        for (int p = 0; p < P; p++)
            lds_dma16(row, (uint32_t)sizeof(T) * (uint32_t)min(place(st, p), end - V),
                      lds + (uint32_t)((st % S) * P + p) * 1024u);
    }

    // Step st into x, after it has landed; then the step S ahead is requested
    // into its stage.
    __device__ __forceinline__ void take(int st, float (&x)[E]) const
    {
        lp_wait<(S - 1) * P>();
        const QLL_LDS_L char *at =
            (const QLL_LDS_L char *)(uintptr_t)(lds + (uint32_t)(st % S) * (P * 1024u) + 16u * (threadIdx.x & 63));
        u32x4 raw[P];
#pragma unroll
        for (int p = 0; p < P; p++)
            raw[p] = *reinterpret_cast<const QLL_LDS_L u32x4 *>(at + 1024 * p);
#pragma unroll
        for (int p = 0; p < P; p++)
            asm volatile("" : "+v"(raw[p])); // the reads are done before their stage is written again
        __builtin_amdgcn_s_waitcnt(0xf | (0x3 << 14) | (0x7 << 4)); // lgkmcnt(0)
        load(st + S);
#pragma unroll
        for (int p = 0; p < P; p++) {
            const LpPiece<T> q = __builtin_bit_cast(LpPiece<T>, raw[p]);
#pragma unroll
            for (int e = 0; e < V; e++)
                x[p * V + e] = lp_widen(q.e[e]);
        }
    }

    __device__ __forceinline__ bool whole(int st) const { return first + (st + 1) * (TH * E) <= end; }

    // Index of element j of step st, and whether it counts.
    __device__ __forceinline__ int index(int st, int j) const { return min(place(st, j / V), end - V) + j % V; }
    __device__ __forceinline__ bool counts(int st, int j) const { return index(st, j) >= place(st, j / V); }
};

// The pieces' maxima and the lane's (-inf at least).
template <int V, int E>
__device__ __forceinline__ float piece_maxima(const float (&x)[E], float (&pm)[E / V])
{
    float mx = -INFINITY;
#pragma unroll
    for (int p = 0; p < E / V; p++) {
        pm[p] = x[p * V];
#pragma unroll
        for (int e = 1; e < V; e++)
            pm[p] = fmaxf(pm[p], x[p * V + e]);
        mx = fmaxf(mx, pm[p]);
    }
    return mx;
}

// NW waves per workgroup.  ROW: a workgroup per
// row, which ends in the outputs; otherwise per segment of `steps` steps, which
// ends in the workspace.
template <typename T, int NW, bool ROW>
__global__ __launch_bounds__(64 * NW, 4) void logprob_kernel(const T *__restrict__ logits, LpWs ws, LpOut o,
                                                             int segments, int steps)
{
    constexpr int TH = 64 * NW, E = lp_elems<T, ROW>();
    typedef LpStream<T, E, TH> Stream;
    __shared__ __attribute__((aligned(16))) char stages[NW][Stream::kBytes];
    static_assert(sizeof(stages) >= sizeof(LpMerge<NW>), "the merge fits in the stages");
    LpMerge<NW> &merge = *reinterpret_cast<LpMerge<NW> *>(&stages[0][0]);
    __shared__ LpTop<NW> s;
    __shared__ LpStat stats[NW];
    const int64_t row = ROW ? (int64_t)blockIdx.x : blockIdx.x / segments;
    const int seg = ROW ? 0 : blockIdx.x % segments, v = o.v;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T *xr = logits + row * v;
    Stream in;
    in.row = xr;
    in.lds = (uint32_t)(uintptr_t)(const QLL_LDS_L char *)&stages[wave][0];
    in.first = seg * steps * (TH * E);
    in.end = min(v, in.first + steps * (TH * E));
    const int n_steps = (in.end - in.first + TH * E - 1) / (TH * E);
#pragma unroll
    for (int st = 0; st < Stream::S; st++)
        in.load(st);
    float x0 = 0.0f;
    if (ROW && (int64_t)threadIdx.x < o.nt)
        x0 = lp_given(xr, o.tokens[row * o.nt + threadIdx.x], v);
    s.clear();
    LaneSum sum{-INFINITY, 0.0, 0.0};
    WaveTop best{s.list[wave], o.top, 0, 0.0f, 0u};
    float lane_max = -INFINITY;
    int publish = 4; // the number of steps done at which to publish next
    float ts = -INFINITY;
    for (int st = 0; st < n_steps; st++) {
        float x[E], pm[Stream::P];
        in.take(st, x);
        const bool whole = in.whole(st); // uniform
        if (!whole)
#pragma unroll
            for (int j = 0; j < E; j++)
                x[j] = in.counts(st, j) ? x[j] : -INFINITY;
        float mx = piece_maxima<Stream::V>(x, pm);
        sum.add(x, mx);
        if (o.top == 0) // uniform
            continue;
        if (!whole) { // what does not count is not chosen either
#pragma unroll
            for (int j = 0; j < E; j++)
                x[j] = in.counts(st, j) ? x[j] : __builtin_nanf("");
            mx = piece_maxima<Stream::V>(x, pm);
        }
        // opaque, or the compiler forms every logit's index and comparisons in
        // every step
        int own = in.place(st, 0);
        asm volatile("" : "+v"(own));
        const auto idx = [&](int j) {
            return min(own + Stream::V * TH * (j / Stream::V), in.end - Stream::V) + j % Stream::V;
        };
        // A later step's elements that equal the wave's own bound lose to what it
        // stands for, all of a lower index; to another wave's later bound they may
        // not, which is why that is published as the value below it.
        if (st == 0) {
            best.template init<NW>(x, mx, idx, s.shared);
            ts = below(best.tv);
        } else if ((st & 3) == 1) {
            ts = s.least_bound();
        }
        if (st > 0)
            ts = fmaxf(ts, best.tv);
        if (__ballot(!(mx <= ts)) != 0) {
            // where the lanes nearly all have a candidate (rising logits), k of them
            // bound the step itself
            if (st > 0 && __popcll(__ballot(mx > ts)) >= max(o.top, 32))
                ts = fmaxf(ts, below(order_value(kth_of_lanes(order_bits(mx + 0.0f), o.top))));
            asm volatile("" : "+v"(own), "+v"(ts));
            best.template add<Stream::V>(x, pm, ts, st == 0, idx);
        }
        lane_max = fmaxf(lane_max, mx);
        if (st + 1 == publish || (st + 1 == n_steps && st > 0)) {
            const uint32_t b = kth_of_lanes(order_bits(lane_max + 0.0f), (o.top + NW - 1) / NW);
            const float t = order_value(b);
            if ((threadIdx.x & 63) == 0)
                shared_store(&s.bound[wave], t == -INFINITY ? t : below(t));
            publish *= 4;
        }
    }
    lp_wait<0>(); // no load may still be writing this workgroup's LDS when it ends
    const LpStat st = sum.wave();
    if constexpr (ROW) {
        if ((threadIdx.x & 63) == 0)
            stats[wave] = st;
        __syncthreads();
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; w++)
            m = fmaxf(m, stats[w].m);
        RowSum sums{0.0, 0.0};
#pragma unroll
        for (int w = 0; w < NW; w++)
            sums.add(stats[w], m);
        const RowLog log_p = row_outputs<TH>(o, xr, row, m, sums, x0);
        if (o.top > 0)
            merge_top(best, s, merge, 0x40000000, [&](int r, float val, int i) {
                o.top_ids[row * o.top + r] = i < v ? i : v - 1; // (only a row with NaN runs out of logits)
                o.top_logprob[row * o.top + r] = log_p(val);
            });
    } else {
        if ((threadIdx.x & 63) == 0)
            ws.stat[(row * segments + seg) * NW + wave] = st;
        __syncthreads(); // the waves' last bounds; the stages are free
        if (o.top > 0)
            merge_top(best, s, merge, 0x40000000 + 64 * seg, [&](int r, float val, int i) {
                ws.key[(row * segments + seg) * o.top + r] = order_key(val, i);
            });
    }
}

// Rows shorter than a piece (at most seven logits): a thread per row, in f64.
template <typename T>
__global__ __launch_bounds__(64) void logprob_tiny_kernel(const T *__restrict__ logits, LpOut o, int64_t m)
{
    const int64_t row = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (row >= m)
        return;
    const T *xr = logits + row * o.v;
    float big = -INFINITY;
    for (int j = 0; j < o.v; j++)
        big = fmaxf(big, lp_widen(xr[j]));
    RowSum sum{0.0, 0.0};
    for (int j = 0; j < o.v; j++) {
        const double d = (double)lp_widen(xr[j]) - (double)big, e = exp(d);
        sum.s += e;
        sum.t += e != 0.0 ? d * e : 0.0;
    }
    const RowLog log_p{(double)big, log(sum.s)};
    if (o.entropy)
        o.entropy[row] = (float)(log_p.log_s - sum.t / sum.s);
    for (int64_t i = 0; i < o.nt; i++)
        o.logprob[row * o.nt + i] = log_p(lp_given(xr, o.tokens[row * o.nt + i], o.v));
    uint64_t last = ~0ull;
    for (int r = 0; r < o.top; r++) {
        uint64_t best = 0;
        for (int j = 0; j < o.v; j++) {
            const float x = lp_widen(xr[j]);
            const uint64_t key = order_key(x == x ? x : -INFINITY, j);
            best = key < last && key > best ? key : best;
        }
        o.top_ids[row * o.top + r] = (int)~(uint32_t)best;
        o.top_logprob[row * o.top + r] = log_p(order_value((uint32_t)(best >> 32)));
        last = best;
    }
}

// One workgroup per row joins its segments, in an order fixed by their numbers.
// Everything that it reads is requested first.  JE: list keys a thread holds
// (0: no alternatives are asked for), `turn` places further in each 256 keys, so
// that a thread's keys have ranks spread evenly over 0 .. top - 1 and its best is one
// of the first in some segment: that makes the lanes' maxima a close bound (1 x
// 128256 f32, 64 alternatives: 8.5 us, 18 with turn 0).
template <typename T, int JE>
__global__ __launch_bounds__(64 * kLpWaves) void logprob_join_kernel(const T *__restrict__ logits, LpWs ws, LpOut o,
                                                                     int segments, int turn)
{
    constexpr int NW = kLpWaves, TH = 64 * NW, R = JE ? JE : 1;
    __shared__ LpTop<NW> s;
    __shared__ LpMerge<NW> merge;
    __shared__ float red_m[NW];
    __shared__ RowSum red[NW];
    s.clear();
    const int64_t row = blockIdx.x;
    const T *xr = logits + row * o.v;
    const int n = segments * NW, nk = segments * o.top, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LpStat *st = ws.stat + row * n;
    LpStat first{0.0, 0.0, -INFINITY, 0.0f};
    if ((int)threadIdx.x < n)
        first = st[threadIdx.x];
    float x0 = 0.0f;
    if ((int64_t)threadIdx.x < o.nt)
        x0 = lp_given(xr, o.tokens[row * o.nt + threadIdx.x], o.v);
    uint64_t key[R];
    if constexpr (JE > 0) {
#pragma unroll
        for (int j = 0; j < JE; j++) {
            const int i = ((int)threadIdx.x + turn * j) % TH + TH * j;
            key[j] = i < nk ? ws.key[row * nk + i] : order_key(-INFINITY, 0x50000000 + i);
        }
    }
    float m = first.m;
    for (int i = threadIdx.x + TH; i < n; i += TH)
        m = fmaxf(m, st[i].m);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        m = fmaxf(m, __shfl_xor(m, off));
    if (lane == 0)
        red_m[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; w++)
        m = fmaxf(m, red_m[w]);
    RowSum sums{0.0, 0.0};
    sums.add(first, m);
    for (int i = threadIdx.x + TH; i < n; i += TH)
        sums.add(st[i], m);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        sums.s += __shfl_xor(sums.s, off);
        sums.t += __shfl_xor(sums.t, off);
    }
    if (lane == 0)
        red[wave] = sums;
    __syncthreads();
    sums = red[0];
#pragma unroll
    for (int w = 1; w < NW; w++) {
        sums.s += red[w].s;
        sums.t += red[w].t;
    }
    const RowLog log_p = row_outputs<TH>(o, xr, row, m, sums, x0);
    if constexpr (JE > 0) {
        float x[R], pm[R], mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < R; j++) {
            x[j] = pm[j] = order_value((uint32_t)(key[j] >> 32));
            mx = fmaxf(mx, x[j]);
        }
        const auto idx = [&](int j) { return (int)~(uint32_t)key[j]; };
        WaveTop best{s.list[wave], o.top, 0, 0.0f, 0u};
        best.template init<NW>(x, mx, idx, s.shared);
        best.template add<1>(x, pm, below(best.tv), true, idx);
        merge_top(best, s, merge, 0x60000000, [&](int r, float val, int i) {
            o.top_ids[row * o.top + r] = i < o.v ? i : o.v - 1;
            o.top_logprob[row * o.top + r] = log_p(val);
        });
    }
}

// How a call is split: a workgroup per row from 256 rows (one for each CU; at
// 256 / 128 rows of 128256 f32 logits 38 / 35 us against 39 / 30 in segments) or
// where a row is one step; otherwise segments of at least one step, as many as
// it takes for about 1024 workgroups (512 measured 0 to 10% slower, workgroups of
// eight waves up to 40%).
constexpr int kLpGroups = 1024;
constexpr int64_t kLpMaxRows = (int64_t)1 << 22; // whole rows of one launch: a grid has fewer than 2^32 threads
struct LpPlan {
    bool row;
    int segments, steps;
};

template <typename T>
static LpPlan lp_plan(int64_t m, int64_t v)
{
    const int64_t row_step = lp_elems<T, true>() * 64 * kLpRowWaves, step = lp_elems<T, false>() * 64 * kLpWaves;
    const int64_t row_steps = (v + row_step - 1) / row_step;
    if (m >= 256 || row_steps == 1)
        return LpPlan{true, 1, (int)row_steps};
    const int64_t all = (v + step - 1) / step;
    int64_t seg = (kLpGroups + m - 1) / m;
    if (seg > all)
        seg = all;
    if (seg > 128) // the join holds 128 * 64 keys
        seg = 128;
    const int64_t steps = (all + seg - 1) / seg;
    return LpPlan{false, (int)((all + steps - 1) / steps), (int)steps};
}

// For logits of any type.
size_t token_logprobs_workspace(int64_t m, int64_t v, int64_t top)
{
    const size_t each = kLpWaves * sizeof(LpStat) + (size_t)top * sizeof(uint64_t);
    const LpPlan plans[] = {lp_plan<float>(m, v), lp_plan<uint16_t>(m, v)};
    size_t need = 256;
    for (const LpPlan &p : plans) {
        const size_t bytes = ((size_t)m * p.segments * each + 255) / 256 * 256;
        if (!p.row && bytes > need)
            need = bytes;
    }
    return need;
}

template <typename T>
static hipError_t launch_logprobs(const T *x, const LpOut &o, int64_t m, void *wsp, hipStream_t s)
{
    const LpPlan p = lp_plan<T>(m, o.v);
    LpWs ws;
    ws.stat = static_cast<LpStat *>(wsp);
    ws.key = reinterpret_cast<uint64_t *>(ws.stat + m * p.segments * kLpWaves);
    if (p.row) {
        for (int64_t r0 = 0; r0 < m; r0 += kLpMaxRows) {
            const int64_t rows = m - r0 < kLpMaxRows ? m - r0 : kLpMaxRows;
            const T *xr = x + r0 * o.v;
            const LpOut part = o.rows(r0);
            if (o.v < LpPiece<T>::V)
                hipLaunchKernelGGL(logprob_tiny_kernel<T>, dim3((unsigned)((rows + 63) / 64)), dim3(64), 0, s, xr, part,
                                   rows);
            else
                hipLaunchKernelGGL((logprob_kernel<T, kLpRowWaves, true>), dim3((unsigned)rows),
                                   dim3(64 * kLpRowWaves), 0, s, xr, ws, part, 1, p.steps);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
        return hipSuccess;
    }
    const dim3 grid((unsigned)(m * p.segments)); // m < 256
    const dim3 block(64 * kLpWaves);
    hipLaunchKernelGGL((logprob_kernel<T, kLpWaves, false>), grid, block, 0, s, x, ws, o, p.segments, p.steps);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int nk = p.segments * o.top;
    // so that from one of a thread's keys to its next the rank moves on by about
    // 256 / segments, which its nk / 256 keys make into one turn through the ranks
    const int threads = 64 * kLpWaves, apart = threads / p.segments - threads;
    const int turn = o.top > 0 ? (apart % o.top + o.top) % o.top : 0;
    const auto join = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)m), block, 0, s, x, ws, o, p.segments, turn);
    };
    if (nk == 0)
        join(logprob_join_kernel<T, 0>);
    else if (nk <= 64 * kLpWaves * 2)
        join(logprob_join_kernel<T, 2>);
    else if (nk <= 64 * kLpWaves * 8)
        join(logprob_join_kernel<T, 8>);
    else if (nk <= 64 * kLpWaves * 16)
        join(logprob_join_kernel<T, 16>);
    else
        join(logprob_join_kernel<T, 32>);
    return hipGetLastError();
}

hipError_t launch_token_logprobs(const void *logits, int dtype, const int32_t *tokens, int64_t nt, float *logprob,
                                 float *entropy, int64_t top, int32_t *top_ids, float *top_logprob, int64_t m,
                                 int64_t v, void *ws, hipStream_t s)
{
    const LpOut o{tokens, nt, logprob, entropy, top_ids, top_logprob, (int)top, (int)v};
    switch (dtype) {
    case QLL_W_F32: return launch_logprobs(static_cast<const float *>(logits), o, m, ws, s);
    case QLL_W_BF16: return launch_logprobs(static_cast<const uint16_t *>(logits), o, m, ws, s);
    default: return launch_logprobs(static_cast<const _Float16 *>(logits), o, m, ws, s);
    }
}

} // namespace qll
