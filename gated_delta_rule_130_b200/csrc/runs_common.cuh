// What the kernels of decode_runs.cu and decode_runs_tc.cu share.
#pragma once

#include "kernels.h"
#include "vec.cuh"

namespace gdn {

constexpr int kRunTokens = 8;  // tokens taken at once

// The decay and the write strength of a token as the recurrence uses them; with logits
// alpha = exp(-softplus(x)) = 1 / (1 + e^x).
__device__ __forceinline__ float2 decay_pair(float la, float be, unsigned flags) {
    if (flags & kFlagGateLogits) return make_float2(sigmoid(-la), sigmoid(be));
    return make_float2(expf(la), be);
}

// x of row p, eight floats 16 bytes aligned.
__device__ __forceinline__ void load8(const float *p, float (&x)[kRunTokens]) {
#pragma unroll
    for (int i = 0; i < kRunTokens; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + i);
        x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
}
// The product of al[l] over from <= l < to.
__device__ __forceinline__ float decay_between(const float (&al)[kRunTokens], int from, int to) {
    float d = 1.f;
#pragma unroll
    for (int l = 0; l < kRunTokens; ++l) d *= l >= from && l < to ? al[l] : 1.f;
    return d;
}

// One warp: tm[0] = T = (I + A)^-1 diag(beta), tm[1] = M = P T, on and below the diagonal of
// their first m rows, from A (below it) and P (on and below it).  Lane j of eight solves
// for column j by substitution; above the diagonal A and P are not looked at, and no
// row takes anything from a later token's, so a later token's NaN stays with it.
__device__ __forceinline__ void solve_tokens(const float (&sA)[kRunTokens][kRunTokens],
                                             const float (&sP)[kRunTokens][kRunTokens],
                                             const float *be, int m, int lane,
                                             float (&tm)[2][kRunTokens][kRunTokens]) {
    constexpr int n = kRunTokens;
    const int j = lane % n;
    float x[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        float row[n];
        load8(sA[i], row);
        float even = i == j ? 1.f : 0.f, odd = 0.f;
#pragma unroll
        for (int l = 0; l < i; ++l) (l % 2 ? odd : even) -= row[l] * x[l];
        x[i] = even + odd;
    }
    const float b = j < m ? be[j] : 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // rows lane / 8 and lane / 8 + 4
        const int i = lane / n + 4 * half;
        float row[n], p = 0.f, xi = 0.f;
        load8(sP[i], row);
#pragma unroll
        for (int l = 0; l < n; ++l) {
            p += (l <= i ? row[l] : 0.f) * (l <= i ? x[l] : 0.f);
            xi = l == i ? x[l] : xi;
        }
        if (j <= i && i < m) {
            tm[0][i][j] = b * xi;
            tm[1][i][j] = b * p;
        }
    }
}

}  // namespace gdn
