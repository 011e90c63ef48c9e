// Token log probabilities off the logits of the vocabulary projection: for
// every row x[0 .. v) with M = max x and S = sum exp(x_j - M),
//     log p_j  = x_j - M - log S
//     entropy  = log S - sum (x_j - M) exp(x_j - M) / S
// the log probabilities of given tokens, the entropy, and the `top` most
// probable tokens in the order (value descending, index ascending).
//
// Each logit is read once.  A workgroup takes a chunk of a row into registers
// and reduces it there to its sums and its own `top` best; a second launch
// joins a row's chunks (the given tokens' logits are read there by index).
// Large batches are bound by the read and by the vector ALU about equally:
// 4 bytes a logit at 5 TB/s leave 30 operations, and the sums and the selection
// take about 20.
//
// Selection.  The wave's 64 lane maxima are ranked; the top-th of them, T, is a
// lower bound on the wave's top-th element (the lanes ahead of it hold one
// element each that is no worse), and the best of the waves' bounds is one for
// the chunk.  Elements at least as good as T, typically a few more than `top`,
// are gathered in LDS and ranked by counting.  Equal values compare by index, so
// rows of ties do not flood the list; rows made so that they do (many good
// elements on the same lanes) fall back to `top` rounds of an argmax.
#include "common.h"

namespace qll {

constexpr int kLpThreads = 256, kLpWaves = kLpThreads / 64;
constexpr int kLpCap = 512; // gathered elements ranked by counting
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

__device__ __forceinline__ float lp_widen(float v) { return v; }
__device__ __forceinline__ float lp_widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float lp_widen(_Float16 v) { return (float)v; }

// 16 bytes of a row whose length need not be a multiple of anything: only the
// element's own alignment is promised.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
struct LpPiece {
    static constexpr int V = 16 / (int)sizeof(T);
    T e[V];
};
__device__ __forceinline__ LpPiece<float> lp_load(const float *p)
{
    return __builtin_bit_cast(LpPiece<float>, *reinterpret_cast<const u32x4_a4 *>(p));
}
template <typename T>
__device__ __forceinline__ LpPiece<T> lp_load(const T *p)
{
    return __builtin_bit_cast(LpPiece<T>, *reinterpret_cast<const u32x4_a2 *>(p));
}

// Element a of value x ahead of element b of value y.
__device__ __forceinline__ bool ahead(float x, int a, float y, int b) { return x > y || (x == y && a < b); }

struct LpTop {
    float tv[kLpWaves];
    int ti[kLpWaves];
    int count;
    float cv[kLpCap];
    int ci[kLpCap];
};

// The k best (1 <= k <= 64) of the workgroup's kLpThreads * E elements,
// out(rank, value, index) once for each rank below k.  mx: the lane's largest
// element (-inf at least).  Indices are distinct; NaN is never chosen, and where
// too few elements are left the remaining ranks get (-inf, pad + rank).
template <int E, class IDX, class OUT>
__device__ __forceinline__ void block_top(const float (&x)[E], float mx, const IDX &idx, int k, int pad, LpTop &s,
                                          const OUT &out)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x == 0)
        s.count = 0;
    int rank = 0;
#pragma unroll
    for (int l = 0; l < 64; l++) {
        const float o = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mx), l));
        rank += o > mx || (o == mx && l < lane);
    }
    const int lk = __builtin_ctzll(__ballot(rank == k - 1));
    float t = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mx), lk));
    // the bound's index: the last of the first k lanes' own (an element that
    // equals t and comes after it is behind k others)
    int first = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < E; j++)
        first = min(first, x[j] == t ? idx(j) : 0x7fffffff);
    int ti = rank < k && mx == t ? first : -1;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        ti = max(ti, __shfl_xor(ti, off));
    if (lane == 0) {
        s.tv[wave] = t;
        s.ti[wave] = ti;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLpWaves; w++)
        if (ahead(s.tv[w], s.ti[w], t, ti)) {
            t = s.tv[w];
            ti = s.ti[w];
        }
#pragma unroll
    for (int j = 0; j < E; j++)
        if (x[j] >= t && (x[j] > t || idx(j) <= ti)) {
            const int at = atomicAdd(&s.count, 1);
            if (at < kLpCap) {
                s.cv[at] = x[j];
                s.ci[at] = idx(j);
            }
        }
    __syncthreads();
    const int n = s.count;
    if (n <= kLpCap) {
        for (int i = threadIdx.x; i < n; i += kLpThreads) {
            const float v = s.cv[i];
            const int a = s.ci[i];
            int r = 0;
            for (int q = 0; q < n; q++)
                r += ahead(s.cv[q], s.ci[q], v, a);
            if (r < k)
                out(r, v, a);
        }
        for (int r = n + threadIdx.x; r < k; r += kLpThreads)
            out(r, -INFINITY, pad + r);
        return;
    }
    float lv = INFINITY; // the last one chosen
    int li = -1;
    for (int r = 0; r < k; r++) {
        float bv = -INFINITY;
        int bi = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < E; j++)
            if (ahead(lv, li, x[j], idx(j)) && ahead(x[j], idx(j), bv, bi)) {
                bv = x[j];
                bi = idx(j);
            }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const float ov = __shfl_xor(bv, off);
            const int oi = __shfl_xor(bi, off);
            if (ahead(ov, oi, bv, bi)) {
                bv = ov;
                bi = oi;
            }
        }
        __syncthreads(); // the last round's values have been read
        if (lane == 0) {
            s.tv[wave] = bv;
            s.ti[wave] = bi;
        }
        __syncthreads();
        lv = s.tv[0];
        li = s.ti[0];
#pragma unroll
        for (int w = 1; w < kLpWaves; w++)
            if (ahead(s.tv[w], s.ti[w], lv, li)) {
                lv = s.tv[w];
                li = s.ti[w];
            }
        if (threadIdx.x == 0)
            out(r, lv, li);
    }
}

// One wave's part of a row: its largest logit m, s = sum exp(x - m) and
// t = sum log2(e) (x - m) exp(x - m).
struct LpStat {
    float m, s, t, unused;
};

// Workspace of one row: kLpWaves stats a chunk, then `top` values and `top`
// indices a chunk.
struct LpWs {
    LpStat *stat; // [m][chunks * kLpWaves]
    float *cv;    // [m][chunks * top]
    int *ci;      // [m][chunks * top]
};

template <typename T, int E>
__global__ __launch_bounds__(kLpThreads) void logprob_chunk_kernel(const T *__restrict__ logits, LpWs ws, int v,
                                                                   int chunks, int top)
{
    typedef LpPiece<T> Piece;
    constexpr int V = Piece::V, P = E / V;
    __shared__ LpTop s;
    const int64_t row = blockIdx.x / chunks;
    const int ch = blockIdx.x % chunks, base = ch * (kLpThreads * E);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T *xr = logits + row * v + base;
    // this thread's elements: pieces threadIdx.x + 256 p of V logits
    const auto at = [&](int j) { return V * ((int)threadIdx.x + kLpThreads * (j / V)) + j % V; };
    const auto idx = [&](int j) { return base + at(j); };
    float x[E];
    if (base + kLpThreads * E <= v) { // uniform
        Piece raw[P];
#pragma unroll
        for (int p = 0; p < P; p++)
            raw[p] = lp_load(xr + at(p * V));
#pragma unroll
        for (int j = 0; j < E; j++)
            x[j] = lp_widen(raw[j / V].e[j % V]);
    } else { // a row's last chunk; past the row: -inf with an index no logit has
#pragma unroll
        for (int j = 0; j < E; j++)
            x[j] = idx(j) < v ? lp_widen(xr[at(j)]) : -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < E; j++)
        mx = fmaxf(mx, x[j]);
    // sums against the lane's own maximum, then brought to the wave's; a lane
    // of masked logits (-inf) counts against 0.  The floor of -200 (far below
    // where exp is 0) keeps 0 * inf out of t; NaN stays in s.
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, t = 0.0f;
#pragma unroll
    for (int j = 0; j < E; j++) {
        const float a = (x[j] - ref) * kLog2e, e = __builtin_amdgcn_exp2f(a);
        sum += e;
        t = fmaf(e, fmaxf(a, -200.0f), t);
    }
    float wm = mx;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        wm = fmaxf(wm, __shfl_xor(wm, off));
    const float wref = wm == -INFINITY ? 0.0f : wm;
    const float d = (mx - wref) * kLog2e, scale = __builtin_amdgcn_exp2f(d);
    sum *= scale;
    t = fmaf(sum, fmaxf(d, -200.0f), t * scale);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        sum += __shfl_xor(sum, off);
        t += __shfl_xor(t, off);
    }
    if (lane == 0)
        ws.stat[(row * chunks + ch) * kLpWaves + wave] = LpStat{wm, sum, t, 0.0f};
    if (top > 0) { // uniform
        const int64_t o = (row * chunks + ch) * top;
        block_top<E>(x, mx, idx, top, 0x40000000 + ch * 64, s, [&](int r, float val, int i) {
            ws.cv[o + r] = val;
            ws.ci[o + r] = i;
        });
    }
}

template <int JE, typename T>
__device__ __forceinline__ void lp_join_top(const LpWs &ws, int64_t row, int n, int top, double m, double log_s, int v,
                                            int32_t *ids, float *lps, LpTop &s)
{
    float x[JE], mx = -INFINITY;
    int id[JE];
#pragma unroll
    for (int j = 0; j < JE; j++) {
        const int i = threadIdx.x + kLpThreads * j;
        x[j] = i < n ? ws.cv[row * n + i] : -INFINITY;
        id[j] = i < n ? ws.ci[row * n + i] : 0x50000000 + i;
        mx = fmaxf(mx, x[j]);
    }
    block_top<JE>(x, mx, [&](int j) { return id[j]; }, top, 0x60000000, s, [&](int r, float val, int i) {
        ids[row * top + r] = i < v ? i : v - 1; // (only a row with NaN runs out of logits)
        lps[row * top + r] = (float)((double)val - m - log_s);
    });
}

// One workgroup per row: the sums joined in f64, in an order fixed by the chunk
// numbers, then the given tokens, the entropy and the best of the chunks' best.
template <typename T>
__global__ __launch_bounds__(kLpThreads) void logprob_join_kernel(const T *__restrict__ logits, LpWs ws, int v,
                                                                  int chunks, const int32_t *__restrict__ tokens,
                                                                  int64_t nt, float *__restrict__ logprob,
                                                                  float *__restrict__ entropy, int top,
                                                                  int32_t *__restrict__ top_ids,
                                                                  float *__restrict__ top_logprob)
{
    __shared__ LpTop s;
    __shared__ float red_m[kLpWaves];
    __shared__ double red[kLpWaves][2];
    const int64_t row = blockIdx.x;
    const int n = chunks * kLpWaves, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const LpStat *st = ws.stat + row * n;
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kLpThreads)
        mx = fmaxf(mx, st[i].m);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        mx = fmaxf(mx, __shfl_xor(mx, off));
    if (lane == 0)
        red_m[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLpWaves; w++)
        mx = fmaxf(mx, red_m[w]);
    double sum = 0.0, t = 0.0; // t in natural units
    for (int i = threadIdx.x; i < n; i += kLpThreads) {
        const LpStat q = st[i];
        if (q.m == -INFINITY) {
            sum += q.s; // 0, or NaN
            continue;
        }
        const float d = q.m - mx;
        const double w = (double)expf(d) * (double)q.s;
        sum += w;
        if (w != 0.0)
            t += (double)expf(d) * (double)kLn2 * (double)q.t + w * (double)d;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        sum += __shfl_xor(sum, off);
        t += __shfl_xor(t, off);
    }
    if (lane == 0) {
        red[wave][0] = sum;
        red[wave][1] = t;
    }
    __syncthreads();
    sum = red[0][0];
    t = red[0][1];
#pragma unroll
    for (int w = 1; w < kLpWaves; w++) {
        sum += red[w][0];
        t += red[w][1];
    }
    // a row with nothing left has M = -inf and S = 0: everything NaN
    const double m = mx, log_s = log(sum);
    if (entropy && threadIdx.x == 0)
        entropy[row] = (float)(log_s - t / sum);
    for (int64_t i = threadIdx.x; i < nt; i += kLpThreads) {
        const int32_t id = tokens[row * nt + i];
        logprob[row * nt + i] = id >= 0 && id < v ? (float)((double)lp_widen(logits[row * v + id]) - m - log_s)
                                                  : __builtin_nanf("");
    }
    if (top > 0) {
        const int nc = chunks * top;
        if (nc <= kLpThreads * 2)
            lp_join_top<2, T>(ws, row, nc, top, m, log_s, v, top_ids, top_logprob, s);
        else if (nc <= kLpThreads * 8)
            lp_join_top<8, T>(ws, row, nc, top, m, log_s, v, top_ids, top_logprob, s);
        else
            lp_join_top<32, T>(ws, row, nc, top, m, log_s, v, top_ids, top_logprob, s);
    }
}

// Logits a thread holds: 32, or 8 where the long chunks would leave most of the
// chip idle (fewer than 256 workgroups) and the join can take the short ones'
// lists (at most 8192 entries; 128 chunks of 8192 logits at the largest v).
static int lp_elems(int64_t m, int64_t v, int64_t top)
{
    const int64_t longs = (v + 32 * kLpThreads - 1) / (32 * kLpThreads);
    const int64_t shorts = (v + 8 * kLpThreads - 1) / (8 * kLpThreads);
    return m * longs < 256 && shorts * top <= 32 * kLpThreads ? 8 : 32;
}

static int lp_chunks(int64_t v, int e) { return (int)((v + e * kLpThreads - 1) / (e * kLpThreads)); }

size_t token_logprobs_workspace(int64_t m, int64_t v, int64_t top)
{
    const size_t c = (size_t)m * (size_t)lp_chunks(v, lp_elems(m, v, top));
    return (c * (kLpWaves * sizeof(LpStat) + (size_t)top * 8) + 255) / 256 * 256;
}

template <typename T>
static hipError_t launch_logprobs(const void *logits, const int32_t *tokens, int64_t nt, float *logprob,
                                  float *entropy, int64_t top, int32_t *top_ids, float *top_logprob, int64_t m,
                                  int64_t v, void *wsp, hipStream_t s)
{
    const int e = lp_elems(m, v, top), chunks = lp_chunks(v, e);
    if (m * chunks > 0x7fffffff)
        return hipErrorInvalidConfiguration;
    LpWs ws;
    ws.stat = static_cast<LpStat *>(wsp);
    ws.cv = reinterpret_cast<float *>(ws.stat + m * chunks * kLpWaves);
    ws.ci = reinterpret_cast<int *>(ws.cv + m * chunks * top);
    const T *x = static_cast<const T *>(logits);
    const dim3 grid((unsigned)(m * chunks)), block(kLpThreads);
    if (e == 8)
        hipLaunchKernelGGL((logprob_chunk_kernel<T, 8>), grid, block, 0, s, x, ws, (int)v, chunks, (int)top);
    else
        hipLaunchKernelGGL((logprob_chunk_kernel<T, 32>), grid, block, 0, s, x, ws, (int)v, chunks, (int)top);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    hipLaunchKernelGGL(logprob_join_kernel<T>, dim3((unsigned)m), block, 0, s, x, ws, (int)v, chunks, tokens, nt,
                       logprob, entropy, (int)top, top_ids, top_logprob);
    return hipGetLastError();
}

hipError_t launch_token_logprobs(const void *logits, int dtype, const int32_t *tokens, int64_t nt, float *logprob,
                                 float *entropy, int64_t top, int32_t *top_ids, float *top_logprob, int64_t m,
                                 int64_t v, void *ws, hipStream_t s)
{
    switch (dtype) {
    case QLL_W_F32:
        return launch_logprobs<float>(logits, tokens, nt, logprob, entropy, top, top_ids, top_logprob, m, v, ws, s);
    case QLL_W_BF16:
        return launch_logprobs<uint16_t>(logits, tokens, nt, logprob, entropy, top, top_ids, top_logprob, m, v, ws, s);
    default:
        return launch_logprobs<_Float16>(logits, tokens, nt, logprob, entropy, top, top_ids, top_logprob, m, v, ws, s);
    }
}

} // namespace qll
