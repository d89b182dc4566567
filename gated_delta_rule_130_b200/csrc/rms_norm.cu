// Root-mean-square norm of rows of D elements,
//     h = x (+ residual, rounded to x's type: the residual stream is held in it),
//     y = h rstd w (silu(gate)),   rstd = 1 / sqrt(mean h^2 + eps),
// y in x's type or in 8 bits (e4m3) with a scale = max|y| / 448 per row or per 128
// columns; and its gradients, with n = h rstd, dn = dy (silu(gate)):
//     dx = rstd (w dn) - h rstd^3 mean(w dn h) (+ d_res),  dw = sum over rows of dn n,
//     dgate = dy n w silu'(gate).
// rstd is formed again in the backward: its sum runs beside that of w dn h.
//
// Both directions read and write each element once and are bound by HBM.  A row is
// held in the registers of TPR threads (part of a warp, a warp or a block) as IT
// vectors of 16 bytes each; sums are float32.
//
// On B200, bf16: 16384 rows of 2048 with residual to e4m3 39.1 us (235 MB, 0.92 of the
// measured copy rate); 262144 gated rows of 128 35.9 us (201 MB, 0.86); gradients of
// 16384 x 2048 with d_res 54 us (268 MB, 0.76, 4 us of it the sum over the blocks), of
// the gated rows 68 us (336 MB, 0.75).
#include <cuda_fp8.h>

#include "kernels.h"
#include "vec.cuh"

namespace gdn {

namespace {

constexpr float kE4M3Max = 448.f;
constexpr float kTinyMax = 1e-30f;  // smallest maximum that a scale is made from

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

template <int LANES, bool MAX>
__device__ __forceinline__ float lanes_reduce(float x) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, off);
        x = MAX ? max_nan(x, y) : x + y;
    }
    return x;
}

// Sum (maximum) over the TPR threads of a row; TPR above 32: over the block, by way
// of `part` (one float per warp; the caller has a barrier between two uses).
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float x, float *part) {
    x = lanes_reduce<(TPR < 32 ? TPR : 32), MAX>(x);
    if (TPR > 32) {
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
        __syncthreads();
        x = part[0];
        for (int i = 1; i < (int)blockDim.x / 32; ++i) x = MAX ? max_nan(x, part[i]) : x + part[i];
    }
    return x;
}

__device__ __forceinline__ float quant_inverse(float top, float *scale) {
    top = max_nan(fmaf(top, 0.f, top), kTinyMax);  // an infinity becomes NaN
    *scale = top * (1.f / kE4M3Max);
    return kE4M3Max / top;
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&x)[VEC], float inv) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(x[0] * inv, __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}

// Where row r begins: its token and its elements before it in the token.
struct Row {
    long long token, in;
    __device__ __forceinline__ Row(const NormArgs &a, int r) : token(r), in(0) {
        if (a.H > 1) {
            token = (unsigned)r / (unsigned)a.H;
            in = (long long)(r - (int)token * a.H) * a.D;
        }
    }
    template <typename T>
    __device__ __forceinline__ const T *of(const void *p, long long stride) const {
        return static_cast<const T *>(p) + token * stride + in;
    }
};

enum Quant { kNoQuant, kRowQuant, kGroupQuant };

// A row in registers: D <= VEC * TPR * IT, D a multiple of VEC.
template <typename T, int VEC, int TPR, int IT, int Q>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 256)
rms_fwd(NormArgs a) {
    constexpr int RPB = TPR > 32 ? 1 : 256 / TPR;  // rows per block
    __shared__ float part[2][32];
    const int sub = threadIdx.x % TPR;
    const int r = blockIdx.x * RPB + threadIdx.x / TPR;
    const int width = r < a.rows ? a.D : 0;  // 0: a row behind the last one
    const int row = r < a.rows ? r : 0;
    const Row at(a, row);
    const T *x = at.of<T>(a.x, a.x_stride);
    const long long out = (long long)row * a.D;

    Raw<T, VEC> h[IT], g[IT];
    {
        Raw<T, VEC> b[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + sub) * VEC;
            if (c < width) h[i] = load_raw<T, VEC>(x + c);
        }
        if (a.residual) {
            const T *res = at.of<T>(a.residual, a.res_stride);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = (i * TPR + sub) * VEC;
                if (c < width) b[i] = load_raw<T, VEC>(res + c);
            }
        }
        if (a.gate) {
            const T *gate = at.of<T>(a.gate, a.gate_stride);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = (i * TPR + sub) * VEC;
                if (c < width) g[i] = load_raw<T, VEC>(gate + c);
            }
        }
        if (a.residual) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = (i * TPR + sub) * VEC;
                float u[VEC], v[VEC];
                widen(h[i], u);
                widen(b[i], v);
                add_vec<VEC>(u, v);
                h[i] = pack(u, h[i]);
                if (a.h && c < width)
                    *reinterpret_cast<Raw<T, VEC> *>(static_cast<T *>(a.h) + out + c) = h[i];
            }
        } else if (a.h) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = (i * TPR + sub) * VEC;
                if (c < width)
                    *reinterpret_cast<Raw<T, VEC> *>(static_cast<T *>(a.h) + out + c) = h[i];
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        float u[VEC], q[VEC] = {};
        widen(h[i], u);
        fma_vec<VEC>(u, u, q);
        if ((i * TPR + sub) * VEC < width)
#pragma unroll
            for (int e = 0; e < VEC; ++e) ss += q[e];
    }
    const float rstd = rsqrtf(row_reduce<TPR, false>(ss, part[0]) / a.D + a.eps);
    float y[Q == kRowQuant ? IT : 1][VEC], top = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + sub) * VEC;
        float(&v)[VEC] = y[Q == kRowQuant ? i : 0];
        if (c < width) {
            float w[VEC];
            widen(h[i], v);
            load_param<T, VEC>(a.weight, c, a.weight_f32, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] *= rstd * w[e];
            if (a.gate) {
                float gg[VEC], sig[VEC];
                widen(g[i], gg);
                fast_sigmoid<VEC>(gg, sig);
                mul_vec<VEC>(gg, sig);
                mul_vec<VEC>(v, gg);
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = 0.f;
        }
        if (Q == kNoQuant) {
            if (c < width) store_vec(static_cast<T *>(a.y) + out + c, v);
            continue;
        }
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) t = max_nan(t, fabsf(v[e]));
        if (Q == kRowQuant) {
            top = max_nan(top, t);
        } else {  // 128 columns: 128 / VEC neighbouring lanes (TPR is no smaller)
            constexpr int LANES = 128 / VEC < TPR ? 128 / VEC : TPR;
            float scale;
            const float inv = quant_inverse(lanes_reduce<(LANES < 32 ? LANES : 32), true>(t), &scale);
            if (c < width) {
                store_e4m3<VEC>(static_cast<uint8_t *>(a.y) + out + c, v, inv);
                if (c % 128 == 0) a.scale[(out + c) / 128] = scale;
            }
        }
    }
    if (Q == kRowQuant) {
        float scale;
        const float inv = quant_inverse(row_reduce<TPR, true>(top, part[1]), &scale);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + sub) * VEC;
            if (c < width) {
                store_e4m3<VEC>(static_cast<uint8_t *>(a.y) + out + c, y[Q == kRowQuant ? i : 0], inv);
                if (c == 0) a.scale[row] = scale;
            }
        }
    }
}

constexpr int kAnyThreads = 256;

// Any D and any alignment: a block per row, element by element, reading again what
// does not fit in registers.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads)
rms_fwd_any(NormArgs a) {
    __shared__ float part[2][32];
    const int row = blockIdx.x;
    const Row at(a, row);
    const T *x = at.of<T>(a.x, a.x_stride);
    const T *res = a.residual ? at.of<T>(a.residual, a.res_stride) : nullptr;
    const T *gate = a.gate ? at.of<T>(a.gate, a.gate_stride) : nullptr;
    const long long out = (long long)row * a.D;
    // h may take the place of x or of the residual, y that of x: once a.h is
    // written, h is read from there
    float ss = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kAnyThreads) {
        float h = to_f32(x[c]);
        if (res) h = to_f32(from_f32<T>(h + to_f32(res[c])));
        if (a.h) static_cast<T *>(a.h)[out + c] = from_f32<T>(h);
        ss += h * h;
    }
    const float rstd = rsqrtf(row_reduce<kAnyThreads, false>(ss, part[0]) / a.D + a.eps);
    const T *hp = a.h ? static_cast<const T *>(a.h) + out : x;
    auto value = [&](int c) {
        float w[1];
        load_param<T, 1>(a.weight, c, a.weight_f32, w);
        float y = to_f32(hp[c]) * (rstd * w[0]);
        if (gate) {
            const float g = to_f32(gate[c]);
            y *= g * fast_sigmoid(g);
        }
        return y;
    };
    if (!a.group) {
        for (int c = threadIdx.x; c < a.D; c += kAnyThreads)
            static_cast<T *>(a.y)[out + c] = from_f32<T>(value(c));
        return;
    }
    uint8_t *y = static_cast<uint8_t *>(a.y) + out;
    if (a.group == a.D) {
        float top = 0.f, scale;
        for (int c = threadIdx.x; c < a.D; c += kAnyThreads) top = max_nan(top, fabsf(value(c)));
        const float inv = quant_inverse(row_reduce<kAnyThreads, true>(top, part[1]), &scale);
        for (int c = threadIdx.x; c < a.D; c += kAnyThreads) {
            const float v[1] = {value(c)};
            store_e4m3<1>(y + c, v, inv);
        }
        if (threadIdx.x == 0) a.scale[row] = scale;
        return;
    }
    const int lane = threadIdx.x % 32;
    for (int c0 = threadIdx.x / 32 * 128; c0 < a.D; c0 += kAnyThreads / 32 * 128) {
        float v[4][1], top = 0.f, scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i][0] = value(c0 + lane + 32 * i);  // D is a multiple of 128 here
            top = max_nan(top, fabsf(v[i][0]));
        }
        const float inv = quant_inverse(lanes_reduce<32, true>(top), &scale);
#pragma unroll
        for (int i = 0; i < 4; ++i) store_e4m3<1>(y + c0 + lane + 32 * i, v[i], inv);
        if (lane == 0) a.scale[(out + c0) / 128] = scale;
    }
}

// Backward, a row in registers; each block takes the rows blockIdx.x * RPB + ... in
// steps of the grid, the next row's loads being issued before this row's sums, keeps
// its columns' sums for dw in registers and leaves them in partial[blockIdx.x].
// The grid is the blocks that fit at once, 148 times this many: more than one round of
// blocks leaves SMs idle in the last.  On 16384 x 2048 bf16 with d_res: 128 threads to a
// row with the next row in registers, 3 blocks per SM of 152 registers and a grid of 592
// took 92.7 us, 4 of 128 registers 62.8 us, the ring with 5 blocks 55.1 us.
template <int TPR, int IT> constexpr int kBwdPerSM =
    TPR > 256 ? 1 : TPR == 256 ? 2 : TPR == 128 ? 5 : IT == 1 ? 3 : 2;
constexpr int kMostBwdBlocks = 148 * 6;

// A row's vectors of x, dy, d_res and gate: in registers (the next row's beside this
// row's) or, 128 threads to a row, in a ring of shared memory that the rows come into
// asynchronously, S - 1 ahead, each thread's own part by itself.
template <typename T, int VEC, int TPR, int IT, bool GATE>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 256, kBwdPerSM<TPR, IT>)
rms_bwd(NormArgs a) {
    constexpr int RPB = TPR > 32 ? 1 : 256 / TPR;
    constexpr bool RING = TPR == 128;
    constexpr bool KEEP = GATE && IT == 1;  // what the gate gives is kept, not formed again
    constexpr int S = 2, NT = GATE ? 4 : 3;
    __shared__ float part[2][32][2];
    __shared__ float cols[TPR > 32 ? 1 : VEC * TPR * IT];
    __shared__ __align__(16) Raw<T, VEC> ring[RING ? S : 1][RING ? NT : 1][RING ? IT : 1]
                                             [RING ? TPR : 1];
    Raw<T, VEC> held[RING ? 1 : 2][RING ? 1 : NT][RING ? 1 : IT];
    const int sub = threadIdx.x % TPR;
    float dw[IT][VEC];
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
    const int step = gridDim.x * RPB;
    int r = blockIdx.x * RPB + threadIdx.x / TPR, turn = 0, slot = 0;
    // row r into slot `to` of the ring (or the second of the registers)
    const auto fetch = [&](int row, int to) {
        if (row < a.rows) {
            const Row at(a, row);
            const T *p[4] = {at.of<T>(a.x, a.x_stride), at.of<T>(a.dy, a.dy_stride),
                             a.d_res ? at.of<T>(a.d_res, a.dres_stride) : nullptr,
                             GATE ? at.of<T>(a.gate, a.gate_stride) : nullptr};
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (p[n])
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        const int c = (i * TPR + sub) * VEC;
                        if (c < a.D) {
                            if constexpr (RING) copy_async<T, VEC>(&ring[to][n][i][sub], p[n] + c);
                            else held[1][n][i] = load_raw<T, VEC>(p[n] + c);
                        }
                    }
        }
        if constexpr (RING) copy_commit();
    };
    const auto in = [&](int n, int i) {
        if constexpr (RING) return ring[slot][n][i][sub];
        else return held[0][n][i];
    };
    const auto advance = [&] {
        if constexpr (!RING)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < IT; ++i) held[0][n][i] = held[1][n][i];
    };
    if constexpr (RING) {
#pragma unroll
        for (int k = 0; k < S - 1; ++k) fetch(r < a.rows - k * step ? r + k * step : a.rows, k);
    } else {
        fetch(r, 0);
        advance();
    }
    for (int r0 = blockIdx.x * RPB; r0 < a.rows; r0 += step, r += step, turn ^= 1) {
        const int width = r < a.rows ? a.D : 0;
        if constexpr (RING) {
            copy_wait<S - 2>();  // this row has come
            fetch(r < a.rows - (S - 1) * step ? r + (S - 1) * step : a.rows, slot ? slot - 1 : S - 1);
        } else {
            fetch(r < a.rows - step ? r + step : a.rows, 1);
        }
        const long long out = (long long)r * a.D;
        float h[IT][VEC], t[IT][VEC];  // t: w dn
        float dg[1][VEC], dn[1][VEC];
        float p[VEC] = {}, q[VEC] = {}, ss = 0.f, sd = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + sub) * VEC;
            if (c < width) {
                float w[VEC];
                widen(in(0, i), h[i]);
                widen(in(1, i), t[i]);
                load_param<T, VEC>(a.weight, c, a.weight_f32, w);
                if constexpr (GATE) {
                    float g[VEC], sig[VEC];
                    widen(in(3, i), g);
                    fast_sigmoid<VEC>(g, sig);
                    if constexpr (KEEP) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            // dy w silu'(g), which waits for rstd
                            dg[0][e] = t[i][e] * w[e] * sig[e] * (1.f + g[e] * (1.f - sig[e]));
                        }
                    }
                    mul_vec<VEC>(g, sig);
                    mul_vec<VEC>(t[i], g);
                    if constexpr (KEEP) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) dn[0][e] = t[i][e];
                    }
                }
                mul_vec<VEC>(t[i], w);
                fma_vec<VEC>(h[i], h[i], p);
                fma_vec<VEC>(t[i], h[i], q);
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            ss += p[e];
            sd += q[e];
        }
        ss = lanes_reduce<(TPR < 32 ? TPR : 32), false>(ss);
        sd = lanes_reduce<(TPR < 32 ? TPR : 32), false>(sd);
        if (TPR > 32) {
            if (threadIdx.x % 32 == 0) {
                part[turn][threadIdx.x / 32][0] = ss;
                part[turn][threadIdx.x / 32][1] = sd;
            }
            __syncthreads();  // two rows' parts in turn: one barrier per row is enough
            ss = sd = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) {
                ss += part[turn][i][0];
                sd += part[turn][i][1];
            }
        }
        const float rstd = rsqrtf(ss / a.D + a.eps);
        const float back = -(sd / a.D * rstd * rstd * rstd);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + sub) * VEC;
            if (c < width) {
                float dx[VEC], d[VEC];
                if constexpr (KEEP) {
                    float out_g[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        out_g[e] = dg[0][e] * (h[i][e] * rstd);
                        d[e] = dn[0][e];
                    }
                    store_vec(static_cast<T *>(a.dgate) + out + c, out_g);
                } else {
                    widen(in(1, i), d);
                }
                if constexpr (GATE && !KEEP) {
                    float g[VEC], w[VEC], sig[VEC], out_g[VEC];
                    widen(in(3, i), g);
                    load_param<T, VEC>(a.weight, c, a.weight_f32, w);
                    fast_sigmoid<VEC>(g, sig);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        out_g[e] = d[e] * (h[i][e] * rstd) * w[e] * sig[e] * (1.f + g[e] * (1.f - sig[e]));
                        d[e] *= g[e] * sig[e];
                    }
                    store_vec(static_cast<T *>(a.dgate) + out + c, out_g);
                }
                if (a.d_res) {
                    widen(in(2, i), dx);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) dx[e] = 0.f;
                }
                float backs[VEC], rstds[VEC], n[VEC] = {};
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    backs[e] = back;
                    rstds[e] = rstd;
                }
                fma_vec<VEC>(h[i], backs, dx);
                fma_vec<VEC>(t[i], rstds, dx);
                fma_vec<VEC>(h[i], rstds, n);
                fma_vec<VEC>(d, n, dw[i]);
                store_vec(static_cast<T *>(a.dx) + out + c, dx);
            }
        }
        advance();
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    float *mine = a.partial + (long long)blockIdx.x * a.D;
    if (TPR > 32) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * TPR + sub) * VEC;
            if (c < a.D)
#pragma unroll
                for (int e = 0; e < VEC; ++e) mine[c + e] = dw[i][e];
        }
    } else {  // the block's row groups one after another, so that the sum has one order
        for (int k = 0; k < RPB; ++k) {
            if ((int)threadIdx.x / TPR == k)
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int c = (i * TPR + sub) * VEC;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) cols[c + e] = dw[i][e] + (k ? cols[c + e] : 0.f);
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.D; c += blockDim.x) mine[c] = cols[c];
    }
}

// Backward for any D and alignment; the sums for dw of a block's rows go straight to
// partial[blockIdx.x], each column always by the same thread.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads)
rms_bwd_any(NormArgs a) {
    __shared__ float part[2][32];
    float *mine = a.partial + (long long)blockIdx.x * a.D;
    for (int c = threadIdx.x; c < a.D; c += kAnyThreads) mine[c] = 0.f;
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const Row at(a, row);
        const T *x = at.of<T>(a.x, a.x_stride), *dy = at.of<T>(a.dy, a.dy_stride);
        const T *gate = a.gate ? at.of<T>(a.gate, a.gate_stride) : nullptr;
        const T *dres = a.d_res ? at.of<T>(a.d_res, a.dres_stride) : nullptr;
        const long long out = (long long)row * a.D;
        float ss = 0.f, sd = 0.f, w[1];
        for (int c = threadIdx.x; c < a.D; c += kAnyThreads) {
            const float h = to_f32(x[c]);
            float dn = to_f32(dy[c]);
            if (gate) {
                const float g = to_f32(gate[c]);
                dn *= g * fast_sigmoid(g);
            }
            load_param<T, 1>(a.weight, c, a.weight_f32, w);
            ss += h * h;
            sd += w[0] * dn * h;
        }
        ss = row_reduce<kAnyThreads, false>(ss, part[0]);
        sd = row_reduce<kAnyThreads, false>(sd, part[1]);
        const float rstd = rsqrtf(ss / a.D + a.eps);
        const float back = sd / a.D * rstd * rstd * rstd;
        for (int c = threadIdx.x; c < a.D; c += kAnyThreads) {
            const float h = to_f32(x[c]);
            float dn = to_f32(dy[c]);
            load_param<T, 1>(a.weight, c, a.weight_f32, w);
            if (gate) {
                const float g = to_f32(gate[c]), sig = fast_sigmoid(g);
                static_cast<T *>(a.dgate)[out + c] =
                    from_f32<T>(dn * (h * rstd) * w[0] * sig * (1.f + g * (1.f - sig)));
                dn *= g * sig;
            }
            float dx = rstd * (w[0] * dn) - h * back;
            if (dres) dx += to_f32(dres[c]);
            static_cast<T *>(a.dx)[out + c] = from_f32<T>(dx);
            mine[c] += dn * (h * rstd);
        }
        __syncthreads();  // `part` is written again
    }
}

// dw[c] = sum over the blocks' partial sums, always in the same order: a block takes 8
// columns (a sector of each row), 128 threads to a column.
constexpr int kSumCols = 8;
__global__ void __launch_bounds__(1024)
rms_bwd_sum(const float *partial, float *dw, int blocks, int D) {
    __shared__ float part[32][kSumCols];
    const int col = threadIdx.x % kSumCols, c = blockIdx.x * kSumCols + col;
    float s = 0.f;
    if (c < D)
#pragma unroll 8
        for (int b = threadIdx.x / kSumCols; b < blocks; b += 1024 / kSumCols)
            s += partial[(long long)b * D + c];
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (threadIdx.x % 32 < kSumCols) part[threadIdx.x / 32][col] = s;
    __syncthreads();
    if (threadIdx.x >= kSumCols || c >= D) return;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) s += part[w][col];
    dw[c] = s;
}

// Partial sums a workspace has room for.
int bwd_blocks(int rows) { return rows < kMostBwdBlocks ? rows : kMostBwdBlocks; }

bool aligned(const void *p, long long stride, int elem) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * elem % 16 == 0;
}
bool vectors_fit(const NormArgs &a, int elem) {
    return (long long)a.D * elem % 16 == 0 && aligned(a.x, a.x_stride, elem) &&
           aligned(a.residual, a.res_stride, elem) && aligned(a.gate, a.gate_stride, elem) &&
           aligned(a.dy, a.dy_stride, elem) && aligned(a.d_res, a.dres_stride, elem);
}

template <typename T, int VEC, int TPR, int IT>
void run_fwd(const NormArgs &a, cudaStream_t st) {
    constexpr int rpb = TPR > 32 ? 1 : 256 / TPR, threads = TPR > 32 ? TPR : 256;
    const int blocks = (a.rows + rpb - 1) / rpb;
    if (!a.group) rms_fwd<T, VEC, TPR, IT, kNoQuant><<<blocks, threads, 0, st>>>(a);
    else if (a.group == a.D) rms_fwd<T, VEC, TPR, IT, kRowQuant><<<blocks, threads, 0, st>>>(a);
    else rms_fwd<T, VEC, TPR, IT, kGroupQuant><<<blocks, threads, 0, st>>>(a);
}
template <typename T, int VEC, int TPR, int IT>
void run_bwd(const NormArgs &a, cudaStream_t st) {
    constexpr int rpb = TPR > 32 ? 1 : 256 / TPR, threads = TPR > 32 ? TPR : 256;
    const int need = (a.rows + rpb - 1) / rpb, most = 148 * kBwdPerSM<TPR, IT>;
    const int blocks = need < most ? need : most;
    if (a.gate) rms_bwd<T, VEC, TPR, IT, true><<<blocks, threads, 0, st>>>(a);
    else rms_bwd<T, VEC, TPR, IT, false><<<blocks, threads, 0, st>>>(a);
    rms_bwd_sum<<<(a.D + kSumCols - 1) / kSumCols, 1024, 0, st>>>(a.partial, a.dw, blocks, a.D);
}

// Threads and vectors per row, from sweeps on bf16 rows (us; plain / with residual and
// e4m3): 16384 rows of 2048: 64 threads of 4 vectors 24.9 / 38.2, 128 of 2 26.7 / 40.2,
// 256 of 1 35.6 / 50.7, a warp of 8 44.5 / 41.0; 1184 rows: 3.7 / 4.1 and 3.1 / 4.2 for
// the first two, which meet near 4736 rows.  16384 rows of 1024: 64 of 2 12.7 / 20.7,
// 32 of 4 13.3 / 21.8, 128 of 1 16.4 / 25.3; of 8192: 256 of 4 106.6 / 152.5, 512 of 2
// 141.0 / 188.6.
constexpr int kManyRows = 148 * 32;

template <typename T, int VEC>
cudaError_t fwd_t(const NormArgs &a, cudaStream_t st) {
    const int nv = a.D / VEC;  // vectors per row
    if (!vectors_fit(a, sizeof(T)) || nv > 4096) {
        rms_fwd_any<T><<<a.rows, kAnyThreads, 0, st>>>(a);
    } else if (nv <= 4) {
        run_fwd<T, VEC, 4, 1>(a, st);
    } else if (nv <= 8) {
        run_fwd<T, VEC, 4, 2>(a, st);
    } else if (nv <= 16) {  // two vectors per thread: 35.6 us on 262144 gated rows of 128,
        run_fwd<T, VEC, 8, 2>(a, st);  // one 38.1 us, four 36.6 us
    } else if (nv <= 32) {
        run_fwd<T, VEC, 16, 2>(a, st);
    } else if (nv <= 64) {
        run_fwd<T, VEC, 32, 2>(a, st);
    } else if (nv <= 128) {
        run_fwd<T, VEC, 64, 2>(a, st);
    } else if (nv <= 256 && a.rows >= kManyRows) {
        run_fwd<T, VEC, 64, 4>(a, st);
    } else if (nv <= 256) {
        run_fwd<T, VEC, 128, 2>(a, st);
    } else if (nv <= 512 && a.rows >= kManyRows) {
        run_fwd<T, VEC, 128, 4>(a, st);
    } else if (nv <= 512) {
        run_fwd<T, VEC, 256, 2>(a, st);
    } else if (nv <= 1024) {
        run_fwd<T, VEC, 256, 4>(a, st);
    } else if (nv <= 2048) {
        run_fwd<T, VEC, 512, 4>(a, st);
    } else {
        run_fwd<T, VEC, 1024, 4>(a, st);
    }
    return cudaPeekAtLastError();
}

template <typename T, int VEC>
cudaError_t bwd_t(const NormArgs &a, cudaStream_t st) {
    const int nv = a.D / VEC;
    if (!vectors_fit(a, sizeof(T)) || nv > 2048) {
        const int blocks = bwd_blocks(a.rows);
        rms_bwd_any<T><<<blocks, kAnyThreads, 0, st>>>(a);
        rms_bwd_sum<<<(a.D + kSumCols - 1) / kSumCols, 1024, 0, st>>>(a.partial, a.dw, blocks, a.D);
    } else if (nv <= 4) {
        run_bwd<T, VEC, 4, 1>(a, st);
    } else if (nv <= 8) {
        run_bwd<T, VEC, 8, 1>(a, st);
    } else if (nv <= 16) {
        run_bwd<T, VEC, 16, 1>(a, st);
    } else if (nv <= 32) {
        run_bwd<T, VEC, 32, 1>(a, st);
    } else if (nv <= 64) {
        run_bwd<T, VEC, 32, 2>(a, st);
    } else if (nv <= 128) {
        run_bwd<T, VEC, 128, 1>(a, st);
    } else if (nv <= 256) {
        run_bwd<T, VEC, 128, 2>(a, st);
    } else if (nv <= 512) {
        run_bwd<T, VEC, 256, 2>(a, st);
    } else if (nv <= 1024) {
        run_bwd<T, VEC, 512, 2>(a, st);
    } else {
        run_bwd<T, VEC, 1024, 2>(a, st);
    }
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_rms_norm_fwd(const NormArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? fwd_t<__nv_bfloat16, 8>(a, st) : fwd_t<float, 4>(a, st);
}

size_t rms_norm_bwd_bytes(int rows, int D) {
    return (size_t)bwd_blocks(rows) * D * sizeof(float);
}

cudaError_t launch_rms_norm_bwd(const NormArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? bwd_t<__nv_bfloat16, 8>(a, st) : bwd_t<float, 4>(a, st);
}

}  // namespace gdn
