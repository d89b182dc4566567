// The recurrent form over a pool of states: each sequence of a packed batch
// advances its own state, states[slot], by a run of a few tokens (one token of a
// decode batch, a draft to be verified, the tail of a prompt).
//
// Up to 8 tokens are taken at once.  With S the state before them, gamma_i the
// product of the decays up to token i, Gamma_ij the product of those after j up
// to i, one value channel (row) S_r of the state gives
//     a_i = S_r . k_i,  b_i = S_r . q_i                     (all i, one pass over S_r)
//     u_i = beta_i (v_i - gamma_i a_i - sum_{j<i} Gamma_ij (k_i.k_j) u_j)
//     o_i = gamma_i b_i + sum_{j<=i} Gamma_ij (q_i.k_j) u_j
//     S_r <- gamma_m S_r + sum_j Gamma_mj u_j k_j
// which is the token recurrence S_t = alpha_t S_{t-1} + u_t k_t^T unrolled.  With
// A_ij = beta_i Gamma_ij k_i.k_j (j < i), T = (I + A)^-1 diag(beta), P_ij = Gamma_ij
// q_i.k_j (j <= i), M = P T and r = v - gamma a, that is u = T r and o = gamma b + M r:
// T and M are one 8 x 8 matrix each for all rows of a head, so a row costs 3
// multiply-adds per element and token (2 where the state is not written back) and
// no row waits for one token after the other.  The Gammas are products of the decays,
// never quotients, so a decay of 0 (log alpha = -inf) is exact.
//
// A warp holds its rows in registers, LW lanes per row with V float4 each; k and q
// stand in shared memory as float32, already normalised.  Everything is float32: the
// state is carried over thousands of steps.
#include "common.cuh"
#include "kernels.h"

namespace gdn {

namespace {

constexpr int kTok = 8;       // tokens taken at once
constexpr int kMaxWarps = 8;  // per block

// Sums of NV values per lane over LW neighbouring lanes: while lanes and values
// last, each step hands half of the values to the partner lane; afterwards lane l
// of its group holds the sums of the values [first, first + n), n = max(1, NV / LW).
template <int NV, int LW>
__device__ __forceinline__ int reduce_scatter(float (&x)[NV], int lane) {
    int first = 0;
    int n = NV;
#pragma unroll
    for (int off = LW / 2; off > 0; off >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool upper = lane & off;
#pragma unroll
            for (int i = 0; i < NV / 2; ++i)
                if (i < n) {
                    const float give = upper ? x[i] : x[i + n];
                    const float keep = upper ? x[i + n] : x[i];
                    x[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            if (upper) first += n;
        } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], off);
        }
    }
    return first;
}

template <bool VEC>
__device__ __forceinline__ float4 load_state(const float *row, int c, int Dk) {
    if (VEC) return c < Dk ? *reinterpret_cast<const float4 *>(row + c) : make_float4(0, 0, 0, 0);
    float4 s;
    s.x = c < Dk ? row[c] : 0.f;
    s.y = c + 1 < Dk ? row[c + 1] : 0.f;
    s.z = c + 2 < Dk ? row[c + 2] : 0.f;
    s.w = c + 3 < Dk ? row[c + 3] : 0.f;
    return s;
}
template <bool VEC>
__device__ __forceinline__ void store_state(float *row, int c, int Dk, float4 s) {
    if (VEC) {
        if (c < Dk) *reinterpret_cast<float4 *>(row + c) = s;
        return;
    }
    if (c < Dk) row[c] = s.x;
    if (c + 1 < Dk) row[c + 1] = s.y;
    if (c + 2 < Dk) row[c + 2] = s.z;
    if (c + 3 < Dk) row[c + 3] = s.w;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// LW lanes share a row, V float4 each; R rows per lane group, so ROWS rows per warp.
constexpr int R = 4;
template <int LW> constexpr int kRows = R * (32 / LW);

template <typename T, int LW, int V, bool VEC>
__global__ void __launch_bounds__(32 * kMaxWarps, 3)
decode_runs_kernel(RunsArgs a, int row_blocks) {
    constexpr int ROWS = kRows<LW>;
    constexpr int PD = LW * V * 4;       // padded Dk
    constexpr int E = (PD + 31) / 32;    // a lane's elements of k where a warp holds a token
    __shared__ __align__(16) float sk[kTok][PD], sq[kTok][PD], sv[kTok][kMaxWarps * ROWS];
    // tm[0]: T with u = T r, tm[1]: M with o = gamma b + M r  (r = v - gamma a)
    __shared__ float sA[kTok][kTok], sP[kTok][kTok], tm[2][kTok][kTok];
    __shared__ float al[kTok], be[kTok], gam[kTok], tail[kTok];
    __shared__ __align__(16) float ra[kMaxWarps][ROWS][kTok], rb_[kMaxWarps][ROWS][kTok];
    __shared__ __align__(16) float su[kMaxWarps][kTok][ROWS];

    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
    const int rb = blockIdx.x % row_blocks;
    const int nh = blockIdx.x / row_blocks;
    const int n = nh / a.Hv, h = nh % a.Hv;
    const int t0 = a.cu ? a.cu[n] : n, t1 = a.cu ? a.cu[n + 1] : n + 1;
    const int slot = a.slots ? a.slots[n] : n;
    if (t0 < 0 || t1 > a.total || t0 >= t1) return;  // empty, or offsets that are none
    bool run = slot >= 0 && slot < a.n_slots;
    const int row0 = rb * warps * ROWS;
    const T *vp = static_cast<const T *>(a.v);
    T *op = static_cast<T *>(a.o);

    const int sub = lane % LW, grp = lane / LW;
    const int wrow = row0 + warp * ROWS;  // the warp's first row
    float *state = a.states + ((long long)(run ? slot : 0) * a.Hv + h) * a.Dv * a.Dk;
    float4 s[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int row = wrow + grp * R + r;
            s[r][v] = run && row < a.Dv
                          ? load_state<VEC>(state + (long long)row * a.Dk, 4 * (v * LW + sub), a.Dk)
                          : make_float4(0, 0, 0, 0);
        }
    const int hk = h / (a.Hv / a.Hk);

    for (int c0 = t0; c0 < t1; c0 += kTok) {
        const int m = min(kTok, t1 - c0);
        // a warp per token: k and q (normalised), v of the block's rows, the gates
        for (int j = warp; j < m && run; j += warps) {
            const long long t = c0 + j;
            const T *kr = static_cast<const T *>(a.k) + t * a.k_stride + (long long)hk * a.Dk;
            const T *qr = a.q ? static_cast<const T *>(a.q) + t * a.q_stride + (long long)hk * a.Dk
                              : nullptr;
            const T *vr = vp + t * a.v_stride + (long long)h * a.Dv;
            float x[E], y[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = lane + 32 * i;
                x[i] = c < a.Dk ? to_f32(kr[c]) : 0.f;
                y[i] = qr && c < a.Dk ? to_f32(qr[c]) : 0.f;
            }
            const float g0 = a.log_alpha[t * a.la_stride + h], g1 = a.beta[t * a.be_stride + h];
            for (int i = lane; i < warps * ROWS; i += 32)
                sv[j][i] = row0 + i < a.Dv ? to_f32(vr[row0 + i]) : 0.f;
            float kn = 0.f, qn = 0.f, kq = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                kn += x[i] * x[i];
                qn += y[i] * y[i];
                kq += x[i] * y[i];
            }
            float rk = 1.f, rq = 1.f;
            if (a.flags & kFlagL2Norm) {
                rk = rsqrtf(warp_sum(kn) + kNormEps);
                rq = rsqrtf(warp_sum(qn) + kNormEps);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int c = lane + 32 * i;
                if (c < PD) {
                    sk[j][c] = rk * x[i];
                    sq[j][c] = rq * y[i];
                }
            }
            if (m == 1) kq = warp_sum(kq);
            if (lane == 0) {
                const float2 gp = gate_pair(g0, g1, a.flags);
                const float alpha = expf(gp.x);
                al[j] = alpha;
                be[j] = gp.y;
                if (m == 1) {
                    gam[0] = alpha;
                    tail[0] = 1.f;
                    tm[0][0][0] = gp.y;
                    tm[1][0][0] = gp.y * (rk * rq * kq);
                }
            }
        }
        if (c0 == t0) {
            // of the sequences with tokens that name one slot the first has it
            int taken = 0;
            if (run && a.update && a.slots)
                for (int i = tid; i < n; i += blockDim.x)
                    if (a.slots[i] == slot) taken |= !a.cu || a.cu[i] < a.cu[i + 1];
            if (__syncthreads_or(taken)) run = false;
            if (!run) {  // a row of padding: its outputs are zero, nothing else is touched
                if (op)
                    for (int t = t0; t < t1; ++t)
                        for (int i = tid; i < warps * ROWS && row0 + i < a.Dv; i += blockDim.x)
                            op[((long long)t * a.Hv + h) * a.Dv + row0 + i] = from_f32<T>(0.f);
                return;
            }
        } else {
            __syncthreads();
        }
        if (m > 1) {
            // a warp per token i: A_ij = beta_i Gamma_ij k_i.k_j (j < i) and
            // P_ij = Gamma_ij q_i.k_j (j <= i)
            for (int i = warp; i < m; i += warps) {
                float x[2 * kTok];
#pragma unroll
                for (int j = 0; j < 2 * kTok; ++j) x[j] = 0.f;
#pragma unroll
                for (int c = 0; c < E; ++c) {
                    const int at = lane + 32 * c;
                    if (at < PD) {
                        const float ki = sk[i][at], qi = sq[i][at];
#pragma unroll
                        for (int j = 0; j < kTok; ++j)
                            if (j <= i) {
                                const float kj = sk[j][at];
                                x[j] += ki * kj;
                                x[kTok + j] += qi * kj;
                            }
                    }
                }
                const int w = reduce_scatter<2 * kTok, 32>(x, lane), j = w % kTok;
                float dec = 1.f;
                for (int l = j + 1; l <= i; ++l) dec *= al[l];
                if (lane % 2 == 0 && j <= i) {
                    if (w < kTok) sA[i][j] = be[i] * dec * x[0];
                    else sP[i][j] = dec * x[0];
                }
                if (lane == 0) {
                    float g = 1.f;
                    for (int l = 0; l <= i; ++l) g *= al[l];
                    gam[i] = g;
                    g = 1.f;
                    for (int l = i + 1; l < m; ++l) g *= al[l];
                    tail[i] = g;
                }
            }
            __syncthreads();
            if (warp == 0) {  // column j of T = (I + A)^-1 diag(beta), then of M = P T
                const int j = lane % kTok;
                float x[kTok];
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    x[i] = i == j ? 1.f : 0.f;
#pragma unroll
                    for (int l = 0; l < i; ++l)
                        if (i < m && l >= j) x[i] -= sA[i][l] * x[l];
                }
                const float b = j < m ? be[j] : 0.f;
                for (int i = lane / kTok; i < m; i += 32 / kTok) {
                    float p = 0.f, xi = 0.f;
#pragma unroll
                    for (int l = 0; l < kTok; ++l)
                        if (l >= j && l <= i) {
                            p += sP[i][l] * x[l];
                            if (l == i) xi = x[l];
                        }
                    if (j <= i) {
                        tm[0][i][j] = b * xi;
                        tm[1][i][j] = b * p;
                    }
                }
            }
        }
        // the rows' products with k and q
        for (int j = 0; j < m; ++j) {
            float2 x2[2 * R];
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) x2[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sk[j][4 * (v * LW + sub)]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&sq[j][4 * (v * LW + sub)]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 lo = make_float2(s[r][v].x, s[r][v].y);
                    const float2 hi = make_float2(s[r][v].z, s[r][v].w);
                    x2[r] = __ffma2_rn(lo, make_float2(k4.x, k4.y), x2[r]);
                    x2[r] = __ffma2_rn(hi, make_float2(k4.z, k4.w), x2[r]);
                    x2[R + r] = __ffma2_rn(lo, make_float2(q4.x, q4.y), x2[R + r]);
                    x2[R + r] = __ffma2_rn(hi, make_float2(q4.z, q4.w), x2[R + r]);
                }
            }
            float x[2 * R];
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) x[i] = x2[i].x + x2[i].y;
            const int first = reduce_scatter<2 * R, LW>(x, lane);
            constexpr int NK = 2 * R > LW ? 2 * R / LW : 1;  // sums left in a lane
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int w = first + i;
                (w < R ? ra[warp][grp * R + w][j] : rb_[warp][grp * R + w - R][j]) = x[i];
            }
        }
        if (m > 1) __syncthreads();
        else __syncwarp();
        // each row's r, then its outputs and corrections
        for (int i = lane; i < ROWS * kTok; i += 32) {
            const int row = i / kTok, j = i % kTok;
            if (j < m) ra[warp][row][j] = sv[j][warp * ROWS + row] - gam[j] * ra[warp][row][j];
        }
        __syncwarp();
        for (int at = lane; at < ROWS * kTok; at += 32) {
            const int row = at / kTok, i = at % kTok;
            if (i < m) {
                float u = 0.f, out = gam[i] * rb_[warp][row][i];
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (j <= i) {
                        const float r = ra[warp][row][j];
                        u += tm[0][i][j] * r;
                        out += tm[1][i][j] * r;
                    }
                su[warp][i][row] = tail[i] * u;
                if (op && wrow + row < a.Dv)
                    op[((long long)(c0 + i) * a.Hv + h) * a.Dv + wrow + row] = from_f32<T>(out);
            }
        }
        __syncwarp();
        if (a.update || c0 + kTok < t1) {
            const float g1 = gam[m - 1];
            const float2 g = make_float2(g1, g1);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 lo = __fmul2_rn(make_float2(s[r][v].x, s[r][v].y), g);
                    const float2 hi = __fmul2_rn(make_float2(s[r][v].z, s[r][v].w), g);
                    s[r][v] = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            for (int j = 0; j < m; ++j) {
                const float4 u4 = *reinterpret_cast<const float4 *>(&su[warp][j][grp * R]);
                const float u[R] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(&sk[j][4 * (v * LW + sub)]);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float2 uu = make_float2(u[r], u[r]);
                        const float2 lo = __ffma2_rn(uu, make_float2(k4.x, k4.y),
                                                     make_float2(s[r][v].x, s[r][v].y));
                        const float2 hi = __ffma2_rn(uu, make_float2(k4.z, k4.w),
                                                     make_float2(s[r][v].z, s[r][v].w));
                        s[r][v] = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
            }
        }
        if (c0 + kTok < t1) __syncthreads();  // the tokens' shared arrays are written again
    }
    if (!a.update) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int row = wrow + grp * R + r;
            if (row < a.Dv)
                store_state<VEC>(state + (long long)row * a.Dk, 4 * (v * LW + sub), a.Dk, s[r][v]);
        }
}

template <typename T, int LW, int V>
cudaError_t launch(const RunsArgs &a, cudaStream_t st) {
    constexpr int ROWS = kRows<LW>;
    const int warps = min(kMaxWarps, (a.Dv + ROWS - 1) / ROWS);
    const int row_blocks = (a.Dv + warps * ROWS - 1) / (warps * ROWS);
    const unsigned blocks = (unsigned)((long long)a.N * a.Hv * row_blocks);
    if (a.Dk % 4 == 0)
        decode_runs_kernel<T, LW, V, true><<<blocks, 32 * warps, 0, st>>>(a, row_blocks);
    else
        decode_runs_kernel<T, LW, V, false><<<blocks, 32 * warps, 0, st>>>(a, row_blocks);
    return cudaPeekAtLastError();
}

template <typename T>
cudaError_t launch_t(const RunsArgs &a, cudaStream_t st) {
    if (a.Dk <= 16) return launch<T, 4, 1>(a, st);
    if (a.Dk <= 32) return launch<T, 4, 2>(a, st);
    if (a.Dk <= 64) return launch<T, 8, 2>(a, st);
    if (a.Dk <= 128) return launch<T, 16, 2>(a, st);
    return launch<T, 32, 2>(a, st);
}

}  // namespace

cudaError_t launch_decode_runs(const RunsArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace gdn
