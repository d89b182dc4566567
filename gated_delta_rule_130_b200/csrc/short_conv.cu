// The short causal depthwise convolution in front of the rule,
//     z[t, c] = bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c],   y = silu(z) or z,
// W in 2..4, over sequences packed along the tokens; the inputs before a sequence
// come from its slot of a pool of the last W - 1 inputs (which then takes the
// sequence's own last ones) or are zero.  Backward, for sequences from zero:
//     dz = dy silu'(z) or dy,   dx[t] = sum_j w[W - 1 - j] dz[t + j] (same sequence),
//     dw[c, j] = sum_t dz[t] x[t - (W - 1) + j],   dbias = sum_t dz[t].
//
// Both directions are bound by HBM: x is read and y written once (backward: dy, x and
// dx).  A thread owns 16 bytes' worth of channels (forward) and walks a tile of
// tokens with the last W inputs in registers; the W - 1 inputs before a tile are read
// again.  Sums are float32; dw is summed per tile and then over the tiles, in one
// order.
#include "kernels.h"
#include "vec.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 128;

// Warp-collective: the last n in [0, N) with cu[n] <= t, which is the sequence of
// token t where cu[n + 1] > t.  32 offsets are looked at in each step; whatever
// cu holds, n stays in range.
__device__ __forceinline__ int seq_of(const int *cu, int N, int t, int lane) {
    int lo = 0, len = N;
    while (len > 1) {
        const int step = (len + 31) / 32, i = lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < len && cu[lo + i] <= t);
        const int c = le ? 31 - __clz(le) : 0;
        lo += c * step;
        len = min(step, len - c * step);
    }
    return lo;
}

// What a lane knows of token t0 + lane (or t0 - (W - 1) + lane): its sequence's span.
struct Span {
    int n, start, end;  // start >= end: not in a sequence
};
__device__ __forceinline__ Span span_of(const ConvArgs &a, int t, int lo, int hi) {
    Span s{0, 0, 0};
    if (t < 0 || t >= a.total) return s;
    if (!a.cu) return Span{t, t, t + 1};
    while (lo < hi) {  // the last n in [lo, hi] with cu[n] <= t
        const int mid = (lo + hi + 1) / 2;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    s = Span{lo, a.cu[lo], a.cu[lo + 1]};
    if (s.start < 0 || s.start > t || s.end <= t || s.end > a.total) s.start = s.end = 0;
    return s;
}

// The array that holds channel c, and c's place in it.
__device__ __forceinline__ int part_of(const ConvArgs &a, int c) {
    int p = 0;
    if (a.parts > 1 && c >= a.begin[1]) p = 1;
    if (a.parts > 2 && c >= a.begin[2]) p = 2;
    return p;
}

template <typename T, int VEC, int W>
__device__ __forceinline__ void load_weights(const ConvArgs &a, int c, float (&w)[W][VEC],
                                             float (&b)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float x[1];
            load_param<T, 1>(a.weight, (long long)(c + e) * W + j, a.weight_f32, x);
            w[j][e] = x[0];
        }
        b[e] = 0.f;
        if (a.bias) {
            float x[1];
            load_param<T, 1>(a.bias, c + e, a.weight_f32, x);
            b[e] = x[0];
        }
    }
}

// Forward.  A block: kThreads * VEC channels and the tokens [t0, t0 + TT).  The
// block that holds a sequence's first token also takes the sequence's next W - 2
// tokens, where they lie behind its tile, and no other block does: so the held inputs
// of a slot are read and written by one thread only.
template <typename T, int VEC, int W, int TT>
__global__ void __launch_bounds__(kThreads)
conv_fwd(ConvArgs a, unsigned ctiles) {
    static_assert(TT + W - 2 <= 32, "a lane per token");
    const int lane = threadIdx.x % 32;
    const int c = (int)((blockIdx.x % ctiles * kThreads + threadIdx.x) * VEC);
    const int t0 = (int)(blockIdx.x / ctiles * TT), t1 = min(t0 + TT, a.total);
    // lane i: token t0 + i, its sequence and whether this block takes it
    const int far = min(t1 + W - 2, a.total) - 1;
    int lo = 0, hi = 0;
    if (a.cu) {
        lo = seq_of(a.cu, a.N, t0, lane);
        hi = seq_of(a.cu, a.N, far, lane);
    }
    const int t_mine = t0 + lane;
    Span sp = span_of(a, t_mine <= far ? t_mine : -1, lo, hi);
    int slot = -1;
    bool mine = sp.start < sp.end;
    if (mine) {
        const bool heads_here = sp.start >= t0 && sp.start < t1;
        mine = t_mine - sp.start < W - 1 ? heads_here : t_mine < t1;
        if (a.states) {
            slot = a.slots ? a.slots[sp.n] : sp.n;
            if (slot >= a.n_slots) slot = -1;
        }
    }
    // of the sequences with tokens that name one slot the first has it
    bool padding = a.states && slot < 0;
    if (a.states && a.slots) {
        unsigned todo = __ballot_sync(0xffffffffu, mine && !padding);
        while (todo) {
            const int i = __ffs(todo) - 1;
            const int n = __shfl_sync(0xffffffffu, sp.n, i);
            const int want = __shfl_sync(0xffffffffu, slot, i);
            int taken = 0;
            for (int k = lane; k < n; k += 32)
                if (a.slots[k] == want) taken |= !a.cu || a.cu[k] < a.cu[k + 1];
            taken = __any_sync(0xffffffffu, taken);
            if (sp.n == n) padding |= taken;
            todo &= ~__ballot_sync(0xffffffffu, sp.n == n);
        }
    }
    const int flags = (mine ? 1 : 0) | (padding ? 2 : 0);

    const bool live = c < a.C;
    const int cc = live ? c : 0;
    const T *x = static_cast<const T *>(a.x) + cc;
    const int p = part_of(a, cc);
    T *y = static_cast<T *>(a.part[p]) + (cc - a.begin[p]);
    float w[W][VEC], b[VEC];
    load_weights<T, VEC, W>(a, cc, w, b);
    float win[W][VEC];  // the inputs t - (W - 1) .. t
    int at = -1;        // the token that win ends with
    for (int i = 0; i < TT + W - 2; ++i) {
        const int t = t0 + i;
        const int f = __shfl_sync(0xffffffffu, flags, i);
        const int start = __shfl_sync(0xffffffffu, sp.start, i);
        const int end = __shfl_sync(0xffffffffu, sp.end, i);
        const int sl = __shfl_sync(0xffffffffu, slot, i);
        if (!(f & 1) || !live) continue;
        if (f & 2) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[W - 1][e] = 0.f;
            store_vec(y + t * a.part_stride[p], win[W - 1]);
            continue;
        }
        T *held = a.states ? static_cast<T *>(a.states) + (long long)sl * (W - 1) * a.C + cc : nullptr;
        if (at == t - 1 && t > start) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) win[j][e] = win[j + 1][e];
        } else {  // a new sequence, or the tile begins inside one
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const int s = t - (W - 1) + j;
                if (s >= start) {
                    load_vec<T, VEC>(x + s * a.x_stride, win[j]);
                } else if (held) {
                    load_vec<T, VEC>(held + (long long)(W - 1 + s - start) * a.C, win[j]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
                }
            }
        }
        load_vec<T, VEC>(x + t * a.x_stride, win[W - 1]);
        at = t;
        float out[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float z = b[e];
#pragma unroll
            for (int j = 0; j < W; ++j) z += w[j][e] * win[j][e];
            out[e] = a.silu ? z * fast_sigmoid(z) : z;
        }
        store_vec(y + t * a.part_stride[p], out);
        // with the last token that needs them the held inputs give way to the
        // sequence's last ones (win still holds the older ones of a short sequence)
        if (held && t == min(start + W - 2, end - 1)) {
            const int len = end - start;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                float v[VEC];
                if (len >= W - 1) {
                    load_vec<T, VEC>(x + (end - (W - 1) + j) * a.x_stride, v);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[e] = win[j + 1][e];
                }
                store_vec(held + (long long)j * a.C, v);
            }
        }
    }
}

constexpr int kBwdTokens = 128;  // tokens per block

// Backward.  A block: kThreads * VEC channels and the tokens [t0, t0 + kBwdTokens): their
// dx (dz of the W - 1 tokens behind the tile is formed again) and their share of dw.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
conv_bwd(ConvArgs a, unsigned ctiles) {
    const int lane = threadIdx.x % 32;
    const int c = (int)((blockIdx.x % ctiles * kThreads + threadIdx.x) * VEC);
    const int tile = (int)(blockIdx.x / ctiles);
    const int t0 = tile * kBwdTokens, t1 = min(t0 + kBwdTokens, a.total);
    const bool live = c < a.C;
    const int cc = live ? c : 0;
    const T *x = static_cast<const T *>(a.x) + cc;
    const int p = part_of(a, cc);
    const T *dy = static_cast<const T *>(a.part[p]) + (cc - a.begin[p]);
    T *dx = static_cast<T *>(a.dx) + cc;
    float w[W][VEC], b[VEC], dw[W][VEC], db[VEC];
    load_weights<T, VEC, W>(a, cc, w, b);
    float win[W][VEC], acc[W][VEC];  // acc[j]: dx of token t - (W - 1) + j so far
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) win[j][e] = acc[j][e] = dw[j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) db[e] = 0.f;
    int n = a.cu ? seq_of(a.cu, a.N, t0, lane) : t0;
    Span sp = span_of(a, t0, n, n);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {  // the inputs before the tile
        const int s = t0 - (W - 1) + j;
        if (live && s >= 0) load_vec<T, VEC>(x + s * a.x_stride, win[j + 1]);
    }
    for (int t = t0; t < t1 + W - 1; ++t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                win[j][e] = win[j + 1][e];
                acc[j][e] = acc[j + 1][e];
            }
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[W - 1][e] = 0.f;
        if (t < a.total && t >= sp.end) {  // the next sequence
            if (a.cu) {
                if (n + 1 < a.N && a.cu[n + 1] <= t && a.cu[n + 2] > t) ++n;
                else n = seq_of(a.cu, a.N, t, lane);
                sp = span_of(a, t, n, n);
            } else {
                sp = Span{t, t, t + 1};
            }
        }
        if (t < a.total && sp.start < sp.end && live) {
            float d[VEC];
            load_vec<T, VEC>(x + t * a.x_stride, win[W - 1]);
            load_vec<T, VEC>(dy + t * a.part_stride[p], d);
            float in[W][VEC];  // the inputs of t's sequence only
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    in[j][e] = t - (W - 1) + j >= sp.start ? win[j][e] : 0.f;
            if (a.silu) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float z = b[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) z += w[j][e] * in[j][e];
                    const float sig = fast_sigmoid(z);
                    d[e] *= sig * (1.f + z * (1.f - sig));
                }
            }
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (t - (W - 1) + j >= sp.start)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[j][e] += w[j][e] * d[e];
            if (t < t1) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    db[e] += d[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[j][e] += d[e] * in[j][e];
                }
            }
        }
        const int done = t - (W - 1);
        if (live && done >= t0 && done < t1) store_vec(dx + (long long)done * a.C, acc[0]);
    }
    if (!live) return;
    float *mine = a.partial + (long long)tile * a.C * (W + 1);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) mine[(long long)j * a.C + c + e] = dw[j][e];
#pragma unroll
    for (int e = 0; e < VEC; ++e) mine[(long long)W * a.C + c + e] = db[e];
}

// dw[c, j] and db[c] = sums over the tiles' partial sums, always in the same order.
__global__ void __launch_bounds__(256)
conv_bwd_sum(const float *partial, float *dw, float *db, int tiles, int C, int W) {
    const int i = blockIdx.x * 256 + threadIdx.x;  // j * C + c
    if (i >= (W + (db ? 1 : 0)) * C) return;
    float s = 0.f;
    for (int k = 0; k < tiles; ++k) s += partial[(long long)k * C * (W + 1) + i];
    const int j = i / C, c = i % C;
    if (j < W) dw[(long long)c * W + j] = s;
    else db[c] = s;
}

template <typename T>
bool vectors_fit(const ConvArgs &a) {
    const auto fits = [](const void *p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * (int)sizeof(T) % 16 == 0;
    };
    bool ok = fits(a.x, a.x_stride) && fits(a.states, a.C) && fits(a.dx, a.C);
    for (int p = 0; p < a.parts; ++p)
        ok = ok && fits(a.part[p], a.part_stride[p]) && a.begin[p] * sizeof(T) % 16 == 0;
    return ok && a.C * sizeof(T) % 16 == 0;
}

template <typename T, int VEC, int W>
cudaError_t fwd_w(const ConvArgs &a, cudaStream_t st) {
    const unsigned bx = (a.C + kThreads * VEC - 1) / (kThreads * VEC);
    if ((long long)bx * a.total <= 148 * 16) {
        conv_fwd<T, VEC, W, 1><<<bx * a.total, kThreads, 0, st>>>(a, bx);
    } else {
        conv_fwd<T, VEC, W, 16><<<bx * ((a.total + 15) / 16), kThreads, 0, st>>>(a, bx);
    }
    return cudaPeekAtLastError();
}

template <typename T, int VEC, int W>
cudaError_t bwd_w(const ConvArgs &a, cudaStream_t st) {
    const int tiles = (a.total + kBwdTokens - 1) / kBwdTokens;
    const unsigned bx = (a.C + kThreads * VEC - 1) / (kThreads * VEC);
    conv_bwd<T, VEC, W><<<bx * tiles, kThreads, 0, st>>>(a, bx);
    const int sums = (W + (a.db ? 1 : 0)) * a.C;
    conv_bwd_sum<<<(sums + 255) / 256, 256, 0, st>>>(a.partial, a.dw, a.db, tiles, a.C, W);
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_short_conv_fwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
#define GDN_CONV(T, VEC)                                 \
    switch (a.W) {                                       \
        case 2: return fwd_w<T, VEC, 2>(a, st);          \
        case 3: return fwd_w<T, VEC, 3>(a, st);          \
        default: return fwd_w<T, VEC, 4>(a, st);         \
    }
    if (bf16) {
        if (vectors_fit<__nv_bfloat16>(a)) GDN_CONV(__nv_bfloat16, 8)
        GDN_CONV(__nv_bfloat16, 1)
    }
    if (vectors_fit<float>(a)) GDN_CONV(float, 4)
    GDN_CONV(float, 1)
#undef GDN_CONV
}

size_t short_conv_bwd_bytes(int total, int C, int W) {
    return (size_t)((total + kBwdTokens - 1) / kBwdTokens) * C * (W + 1) * sizeof(float);
}

cudaError_t launch_short_conv_bwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
#define GDN_CONV(T, VEC)                                 \
    switch (a.W) {                                       \
        case 2: return bwd_w<T, VEC, 2>(a, st);          \
        case 3: return bwd_w<T, VEC, 3>(a, st);          \
        default: return bwd_w<T, VEC, 4>(a, st);         \
    }
    if (bf16) {
        if (vectors_fit<__nv_bfloat16>(a)) GDN_CONV(__nv_bfloat16, 8)
        GDN_CONV(__nv_bfloat16, 1)
    }
    if (vectors_fit<float>(a)) GDN_CONV(float, 4)
    GDN_CONV(float, 1)
#undef GDN_CONV
}

}  // namespace gdn
