// Stores of a wave's 2 x 2 matrix-core tiles (32 x 32 outputs each), shared by
// the direct and the repacked prefill GEMM.
#pragma once

#include "common.h"

namespace qll {

// acc[i][j][v] of lane l is twice the output at row
// row0 + 32 i + 8 (v / 4) + 4 (l / 32) + v % 4 (the scale tiles are
// 2 d_x d_w).  Plain and linear: column col0 + 32 j + l % 32.  Gated: column
// col0 + l % 32, j = 0 the gate's product and j = 1 the up projection's.
// The values a linear epilogue reads (a row of 32 residual values per
// register, as wide as the stores) are requested for a whole tile before any
// of them is used.
template <class EP, typename V16>
__device__ __forceinline__ void q4_tile_store(const EP &ep, V16 (&acc)[2][2], float *y, int64_t m, int64_t n,
                                              int64_t row0, int64_t col0, int lane)
{
    const auto row_of = [&](int i, int v) { return row0 + 32 * i + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3); };
    if constexpr (EP::kGated) {
        const int64_t col = col0 + (lane & 31);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            V16 g, u;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                g[v] = 0.5f * acc[i][0][v];
                u[v] = 0.5f * acc[i][1][v];
            }
            if (ep.raw) { // uniform
#pragma unroll
                for (int v = 0; v < 16; v++)
                    if (row_of(i, v) < m && col < n) {
                        y[row_of(i, v) * n + col] = g[v];
                        y[(m + row_of(i, v)) * n + col] = u[v];
                    }
                continue;
            }
            activate16(g, ep.act);
#pragma unroll
            for (int v = 0; v < 16; v++)
                if (row_of(i, v) < m && col < n)
                    y[row_of(i, v) * n + col] = g[v] * u[v];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int64_t col = col0 + 32 * j + (lane & 31);
                if constexpr (EP::kLinear) {
                    const float b = ep.bias && col < n ? ep.bias[col] : 0.0f;
                    V16 t, r;
#pragma unroll
                    for (int v = 0; v < 16; v++) {
                        t[v] = 0.5f * acc[i][j][v] + b;
                        r[v] = ep.res && row_of(i, v) < m && col < n ? ep.res[row_of(i, v) * n + col] : 0.0f;
                    }
                    activate16(t, ep.act);
#pragma unroll
                    for (int v = 0; v < 16; v++)
                        if (row_of(i, v) < m && col < n)
                            y[row_of(i, v) * n + col] = t[v] + r[v];
                } else {
#pragma unroll
                    for (int v = 0; v < 16; v++)
                        if (row_of(i, v) < m && col < n)
                            y[row_of(i, v) * n + col] = 0.5f * acc[i][j][v];
                }
            }
    }
}

} // namespace qll
