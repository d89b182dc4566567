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
// which is the token recurrence S_t = alpha_t S_{t-1} + u_t k_t^T unrolled, so a
// row costs 3 multiply-adds per element and token (2 where the state is not
// written back) and its sums over the key channels of several tokens do not wait
// for one another.  The Gammas are products of the decays, never quotients, so a
// decay of 0 (log alpha = -inf) is exact.
//
// A warp holds 8 rows (4 for Dk > 128) in registers, LW lanes per row with V
// float4 each; k and q stand in shared memory as float32, already normalised.
// Everything is float32: the state is carried over thousands of steps.
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

template <typename T, int LW, int V, bool VEC>
__global__ void __launch_bounds__(32 * kMaxWarps)
decode_runs_kernel(RunsArgs a, int row_blocks) {
    constexpr int R = V == 1 ? 8 : 4;   // rows per lane group
    constexpr int G = 32 / LW;          // lane groups per warp
    constexpr int ROWS = R * G;         // rows per warp
    constexpr int PD = LW * V * 4;      // padded Dk
    __shared__ __align__(16) float sk[kTok][PD], sq[kTok][PD];
    __shared__ float kk[kTok][kTok], qk[kTok][kTok];        // i >= j
    __shared__ float al[kTok], be[kTok], gam[kTok], tail[kTok];
    __shared__ float da[kMaxWarps][kTok][ROWS], db[kMaxWarps][kTok][ROWS];

    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
    const int rb = blockIdx.x % row_blocks;
    const int nh = blockIdx.x / row_blocks;
    const int n = nh / a.Hv, h = nh % a.Hv;
    const int t0 = a.cu ? a.cu[n] : n, t1 = a.cu ? a.cu[n + 1] : n + 1;
    if (t0 < 0 || t1 > a.total || t0 >= t1) return;  // empty, or offsets that are none
    const int slot = a.slots ? a.slots[n] : n;
    bool run = slot >= 0 && slot < a.n_slots;
    const int row0 = rb * warps * ROWS;
    const T *qp = static_cast<const T *>(a.q), *kp = static_cast<const T *>(a.k);
    const T *vp = static_cast<const T *>(a.v);
    T *op = static_cast<T *>(a.o);

    // of the sequences with tokens that name one slot the first has it
    int taken = 0;
    if (run && a.update && a.slots)
        for (int i = tid; i < n; i += blockDim.x)
            if (a.slots[i] == slot) taken |= !a.cu || a.cu[i] < a.cu[i + 1];

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
    if (__syncthreads_or(taken)) run = false;
    if (!run) {  // a row of padding: its outputs are zero, nothing else is touched
        if (op)
            for (int t = t0; t < t1; ++t)
                for (int i = tid; i < warps * ROWS && row0 + i < a.Dv; i += blockDim.x)
                    op[((long long)t * a.Hv + h) * a.Dv + row0 + i] = from_f32<T>(0.f);
        return;
    }
    const int hk = h / (a.Hv / a.Hk);

    for (int c0 = t0; c0 < t1; c0 += kTok) {
        const int m = min(kTok, t1 - c0);
        // k, q (normalised) and the gates of the m tokens
        for (int j = warp; j < m; j += warps) {
            const long long t = c0 + j;
            const T *kr = kp + t * a.k_stride + (long long)hk * a.Dk;
            const T *qr = qp ? qp + t * a.q_stride + (long long)hk * a.Dk : nullptr;
            float x[(PD + 31) / 32], y[(PD + 31) / 32], kn = 0.f, qn = 0.f;
#pragma unroll
            for (int i = 0; i < (PD + 31) / 32; ++i) {
                const int c = lane + 32 * i;
                x[i] = c < a.Dk ? to_f32(kr[c]) : 0.f;
                y[i] = qr && c < a.Dk ? to_f32(qr[c]) : 0.f;
                kn += x[i] * x[i];
                qn += y[i] * y[i];
            }
            float rk = 1.f, rq = 1.f;
            if (a.flags & kFlagL2Norm) {
                rk = rsqrtf(warp_sum(kn) + kNormEps);
                rq = rsqrtf(warp_sum(qn) + kNormEps);
            }
#pragma unroll
            for (int i = 0; i < (PD + 31) / 32; ++i) {
                const int c = lane + 32 * i;
                if (c < PD) {
                    sk[j][c] = rk * x[i];
                    sq[j][c] = rq * y[i];
                }
            }
            if (lane == 0) {
                const float2 gp = gate_pair(a.log_alpha[t * a.la_stride + h],
                                            a.beta[t * a.be_stride + h], a.flags);
                al[j] = expf(gp.x);
                be[j] = gp.y;
            }
        }
        __syncthreads();
        // the tokens' products with one another; thread 0: the decays up to and from each
        for (int p = warp; p < m * m; p += warps) {
            const int i = p / m, j = p % m;  // j < i: k_i.k_j, else q_j.k_i (i <= j)
            const float *x = j < i ? sk[i] : sq[j], *y = j < i ? sk[j] : sk[i];
            float d = 0.f;
#pragma unroll
            for (int c = lane; c < PD; c += 32) d += x[c] * y[c];
            d = warp_sum(d);
            if (lane == 0) (j < i ? kk[i][j] : qk[j][i]) = d;
        }
        if (tid == 0) {
            float g = 1.f;
            for (int i = 0; i < m; ++i) gam[i] = g *= al[i];
            g = 1.f;
            for (int i = m - 1; i >= 0; --i) {
                tail[i] = g;
                g *= al[i];
            }
        }
        // the rows' products with k and q
        for (int j = 0; j < m; ++j) {
            float x[2 * R];
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) x[i] = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sk[j][4 * (v * LW + sub)]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&sq[j][4 * (v * LW + sub)]);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    x[r] += s[r][v].x * k4.x + s[r][v].y * k4.y + s[r][v].z * k4.z + s[r][v].w * k4.w;
                    x[R + r] += s[r][v].x * q4.x + s[r][v].y * q4.y + s[r][v].z * q4.z + s[r][v].w * q4.w;
                }
            }
            const int first = reduce_scatter<2 * R, LW>(x, lane);
            constexpr int NK = 2 * R > LW ? 2 * R / LW : 1;  // sums left in a lane
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int w = first + i;
                (w < R ? da[warp][j][grp * R + w] : db[warp][j][grp * R + w - R]) = x[i];
            }
        }
        __syncthreads();
        // each row's corrections u (left in da) and outputs
        for (int i = lane; i < ROWS; i += 32) {
            const int row = wrow + i;
            float u[kTok];
            if (row < a.Dv) {
#pragma unroll
                for (int t = 0; t < kTok; ++t)
                    if (t < m) {
                        const long long tok = c0 + t;
                        float acc = to_f32(vp[tok * a.v_stride + (long long)h * a.Dv + row]) -
                                    gam[t] * da[warp][t][i];
                        float out = gam[t] * db[warp][t][i];
                        float dec = al[t];
#pragma unroll
                        for (int j = kTok - 1; j >= 0; --j)
                            if (j < t) {
                                acc -= dec * kk[t][j] * u[j];
                                out += dec * qk[t][j] * u[j];
                                dec *= al[j];
                            }
                        u[t] = be[t] * acc;
                        if (op)
                            op[(tok * a.Hv + h) * a.Dv + row] = from_f32<T>(out + qk[t][t] * u[t]);
                        da[warp][t][i] = tail[t] * u[t];
                    }
            } else {
                for (int t = 0; t < m; ++t) da[warp][t][i] = 0.f;
            }
        }
        __syncwarp();
        if (a.update || c0 + kTok < t1) {
            const float g = gam[m - 1];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[r][v].x *= g; s[r][v].y *= g; s[r][v].z *= g; s[r][v].w *= g;
                }
            for (int j = 0; j < m; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(&sk[j][4 * (v * LW + sub)]);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float u = da[warp][j][grp * R + r];
                        s[r][v].x += u * k4.x; s[r][v].y += u * k4.y;
                        s[r][v].z += u * k4.z; s[r][v].w += u * k4.w;
                    }
                }
        }
        __syncthreads();  // the tokens' shared arrays are written again
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
    constexpr int ROWS = (V == 1 ? 8 : 4) * (32 / LW);
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
    if (a.Dk <= 32) return launch<T, 8, 1>(a, st);
    if (a.Dk <= 64) return launch<T, 16, 1>(a, st);
    if (a.Dk <= 128) return launch<T, 32, 1>(a, st);
    return launch<T, 32, 2>(a, st);
}

}  // namespace

cudaError_t launch_decode_runs(const RunsArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<float>(a, st);
}

}  // namespace gdn
