// The short causal depthwise convolution in front of the rule,
//     z[t, c] = bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c],   y = silu(z) or z,
// W in 2..4, over sequences packed along the tokens; the inputs before a sequence
// come from its slot of a pool of the last W - 1 inputs (which then takes the
// sequence's own last ones) or are zero.  A token's sequence is found by bisection of the
// offsets: where they decrease, valid sequences may be left out (nothing outside the arrays is
// touched, and a slot still belongs to one sequence).  Backward, for sequences from zero:
//     dz = dy silu'(z) or dy,   dx[t] = sum_j w[W - 1 - j] dz[t + j] (same sequence),
//     dw[c, j] = sum_t dz[t] x[t - (W - 1) + j],   dbias = sum_t dz[t].
//
// Both directions are bound by HBM: x is read and y written once (backward: dy, x and
// dx).  A thread owns four neighbouring channels and walks a tile of tokens with the
// last W inputs in registers, the rows of the next tokens on their way; the W - 1 rows
// before a tile are read again.  Sums are float32; dw is summed per tile and then over
// the tiles, in one order.
//
// On B200, bf16, W = 4, 12 sequences of 16384 tokens, 6144 channels: forward 74.5 us (403
// MB, 0.82 of the measured copy rate), backward 119 us (604 MB, 0.77; 120 registers leave
// 16 warps per SM, and it issues 23 instructions per element); one token each of 256
// sequences 10.9 us (25 MB: three rounds of blocks that wait for offsets, slot and held
// inputs in turn).
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

// The sequence of token t, known to lie in [lo, hi].
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

// w[j][e] = weight[c + e, j]: VEC * W consecutive parameters, in vectors where VEC > 1.
template <typename P, int VEC, int W>
__device__ __forceinline__ void load_taps(const P *p, float (&w)[W][VEC]) {
    constexpr int V = VEC > 1 ? 4 : 1;
#pragma unroll
    for (int i = 0; i < VEC * W / V; ++i) {
        float x[V];
        load_vec<P, V>(p + i * V, x);
#pragma unroll
        for (int e = 0; e < V; ++e) w[(i * V + e) % W][(i * V + e) / W] = x[e];
    }
}
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_weights(const ConvArgs &a, int c, float (&w)[W][VEC],
                                             float (&b)[VEC]) {
    if (a.weight_f32) load_taps<float, VEC, W>(static_cast<const float *>(a.weight) + (long long)c * W, w);
    else load_taps<T, VEC, W>(static_cast<const T *>(a.weight) + (long long)c * W, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) b[e] = 0.f;
    if (a.bias) {
        if (a.weight_f32) load_vec<float, VEC>(static_cast<const float *>(a.bias) + c, b);
        else load_vec<T, VEC>(static_cast<const T *>(a.bias) + c, b);
    }
}

// y = silu(z) in place of z
template <int VEC> __device__ __forceinline__ void silu_vec(float (&z)[VEC]) {
    float s[VEC];
    fast_sigmoid<VEC>(z, s);
    mul_vec<VEC>(z, s);
}
// d *= silu'(z) = sig (1 + z - z sig)
template <int VEC>
__device__ __forceinline__ void silu_grad_vec(const float (&z)[VEC], float (&d)[VEC]) {
    float s[VEC], n[VEC], t[VEC];
    fast_sigmoid<VEC>(z, s);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        n[e] = -s[e];
        t[e] = z[e];
    }
    fma_vec<VEC>(n, z, t);  // z - z sig
    mul_vec<VEC>(d, s);
    fma_vec<VEC>(d, t, d);
}

// Forward.  A block: kThreads * VEC channels and the tokens [t0, t0 + tile).  The block that
// holds a sequence's first token also takes the sequence's next W - 2 tokens, where
// they lie behind its tile, and no other block does: so the held inputs of a slot are
// read and written by one thread only.
constexpr int kMine = 1, kPadding = 2, kFirst = 4, kHold = 8;
constexpr int kMaxTile = 256;  // tokens per block

// Of the sequences with tokens that name one slot the first has it.  A block asks for all
// sequences of its tile in one pass over the slots before them: a table in shared memory
// holds, for each slot that the tile names, the first token that does; a place is the
// token's index in the tile, kTaken with it once an earlier sequence has named the slot.
// (The slots before each sequence one after the other: a token each of 4096 sequences of
// 6144 channels 228 us, so 91 us; without slots 81 us.)
constexpr int kPlaces = 2 * kMaxTile, kFree = -1, kTaken = 1 << 16;
struct SlotTable {
    int place[kPlaces], slot[kMaxTile + 2];  // slot: of each token, -1: none or padding

    // Where `want` stands, or the free place that ends its search.
    __device__ __forceinline__ int find(int want) const {
        int i = (int)((unsigned)want * 2654435761u % kPlaces);
        while (place[i] != kFree && slot[place[i] & (kTaken - 1)] != want) i = (i + 1) % kPlaces;
        return i;
    }
    // Token i names its slot.
    __device__ __forceinline__ void insert(int i) {
        const int want = slot[i];
        for (int at = (int)((unsigned)want * 2654435761u % kPlaces);; at = (at + 1) % kPlaces) {
            const int old = atomicCAS(&place[at], kFree, i);
            if (old == kFree) return;
            if (slot[old] == want) {
                atomicMin(&place[at], i);
                return;
            }
        }
    }
};

// The rows of x come through a ring of shared memory, each thread's own channels by
// itself, S - 1 groups of B rows ahead.
// Three groups in the ring and 7 blocks per SM took 73.2 us on 16384 x 6144, 6 blocks
// 74.6; four groups and 6 or 5 blocks, of which 4 ran at once, 85.7 and 88.6.
template <typename T, int VEC> constexpr int kFwdPerSM = VEC * sizeof(T) > 8 ? 5 : 7;

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads, kFwdPerSM<T, VEC>)
conv_fwd(ConvArgs a, unsigned ctiles, int tile) {
    constexpr int B = 8, S = VEC * sizeof(T) > 8 ? 2 : 3;
    __shared__ __align__(16) Raw<T, VEC> ring[S][B][kThreads];
    // of the tile's tokens and those behind it: the sequence (-1: none), the flags
    __shared__ int seq[kMaxTile + W - 2];
    __shared__ __align__(8) unsigned char flag[(kMaxTile + W - 2 + 7) / 8 * 8];
    // the table lies in the ring's last group, which is empty until the tokens are begun, if
    // it is large enough (more shared memory would take L1 from the copies: 85.4 us)
    constexpr bool kInRing = sizeof(ring[0]) >= sizeof(SlotTable);
    __shared__ __align__(16) unsigned char own_table[kInRing ? 16 : sizeof(SlotTable)];
    SlotTable &table = *reinterpret_cast<SlotTable *>(kInRing ? static_cast<void *>(ring[S - 1]) : own_table);
    const int tid = threadIdx.x, lane = tid % 32;
    const int c = (int)((blockIdx.x % ctiles * kThreads + tid) * VEC);
    const int t0 = (int)(blockIdx.x / ctiles) * tile, t1 = min(t0 + tile, a.total);
    const int stop = min(t1 + W - 2, a.total);
    const bool live = c < a.C;
    const int cc = live ? c : 0;
    const T *x = static_cast<const T *>(a.x) + cc;

    // the rows are on their way while the sequences are found
    const T *xa = x + (long long)t0 * a.x_stride;  // the row copied next
    int copied = t0;
    const auto copy_group = [&](int slot) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (copied + i < stop) copy_async<T, VEC>(&ring[slot][i][tid], xa);
            xa += a.x_stride;
        }
        copied += B;
        copy_commit();
    };
#pragma unroll
    for (int g = 0; g < S - 1; ++g) copy_group(g);
    float win[W - 1][VEC];  // the inputs before the token
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int s = t0 - (W - 1) + j;
        if (s >= 0) load_vec<T, VEC>(x + s * a.x_stride, win[j]);
    }
    float w[W][VEC], b[VEC];
    load_weights<T, VEC, W>(a, cc, w, b);

    int lo = 0, hi = 0;
    if (a.cu) {
        lo = seq_of(a.cu, a.N, t0, lane);
        hi = seq_of(a.cu, a.N, stop - 1, lane);
    }
    const bool named = a.states && a.slots;
    for (int i = tid; i < stop - t0; i += kThreads) {
        const int t = t0 + i;
        const Span sp = span_of(a, t, lo, hi);
        const bool in = sp.start < sp.end;
        int f = 0, slot = -1;
        if (in) {
            const int pos = t - sp.start;
            const bool head = sp.start >= t0 && sp.start < t1;
            if (pos < W - 1 ? head : t < t1) f |= kMine;
            if (pos == 0) f |= kFirst;
            if (a.states) {
                slot = a.slots ? a.slots[sp.n] : sp.n;
                if (slot < 0 || slot >= a.n_slots) {
                    f |= kPadding;
                    slot = -1;
                } else if (t == min(sp.start + W - 2, sp.end - 1)) {
                    f |= kHold;  // with the last token that needs them the held inputs give way
                }
            }
        }
        seq[i] = in ? sp.n : -1;
        flag[i] = f;
        if (named) table.slot[i] = slot;
    }
    if (tid < 8 && stop - t0 + tid < (int)sizeof(flag)) flag[stop - t0 + tid] = 0;
    if (named)
        for (int i = tid; i < kPlaces; i += kThreads) table.place[i] = kFree;
    __syncthreads();
    if (named) {
        for (int i = tid; i < stop - t0; i += kThreads)
            if (table.slot[i] >= 0 && (i == 0 || seq[i - 1] != seq[i])) table.insert(i);
        __syncthreads();
        const int last = a.cu ? hi : stop - 1;  // the tile's last sequence
        for (int m = 4 * tid; m < last; m += 4 * kThreads) {
            int s[4];
            load_slots(a.slots, m, last, s);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (s[k] < 0) continue;
                const int at = table.find(s[k]), held_by = table.place[at];
                if (held_by >= 0 && held_by < kTaken && m + k < seq[held_by] &&
                    has_tokens(a.cu, a.total, m + k))
                    atomicOr(&table.place[at], kTaken);
            }
        }
        __syncthreads();
        for (int i = tid; i < stop - t0; i += kThreads)
            if (table.slot[i] >= 0) {
                const int held_by = table.place[table.find(table.slot[i])];
                if (held_by >= kTaken || seq[held_by] != seq[i]) flag[i] |= kPadding;
            }
        __syncthreads();
    }
    if (!live) return;
    int count = t1 - t0;
    for (int i = t1 - t0; i < stop - t0; ++i)
        if (flag[i] & kMine) count = i + 1;

    const int p = part_of(a, cc);
    T *y = static_cast<T *>(a.part[p]) + (cc - a.begin[p]) + t0 * a.part_stride[p];
    int slot = 0;
    for (int i0 = 0; i0 < count; i0 += B, slot = slot + 1 == S ? 0 : slot + 1) {
        copy_wait<S - 2>();  // this group's rows have come
        copy_group(slot ? slot - 1 : S - 1);
        if (*reinterpret_cast<const unsigned long long *>(&flag[i0]) ==
            0x0101010101010101ull * kMine) {
            // eight tokens inside one sequence: no case to tell apart
            float in[W - 1 + B][VEC];
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) in[j][e] = win[j][e];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                widen(ring[slot][i][tid], in[W - 1 + i]);
                float z[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) z[e] = b[e];
#pragma unroll
                for (int j = 0; j < W; ++j) fma_vec<VEC>(w[j], in[i + j], z);
                if (a.silu) silu_vec<VEC>(z);
                store_vec(y, z);
                y += a.part_stride[p];
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) win[j][e] = in[B + j][e];
            continue;
        }
#pragma unroll 1
        for (int i = 0; i < B && i0 + i < count; ++i) {
            const int f = flag[i0 + i];
            T *held = nullptr;
            int start = 0, end = 0;
            if (f & (kFirst | kHold)) {
                const int n = seq[i0 + i];
                start = a.cu ? a.cu[n] : n;
                end = a.cu ? a.cu[n + 1] : n + 1;
                if (a.states && !(f & kPadding))
                    held = static_cast<T *>(a.states) +
                           (long long)(a.slots ? a.slots[n] : n) * (W - 1) * a.C + cc;
                if (f & kFirst) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        if (held) {
                            load_vec<T, VEC>(held + (long long)j * a.C, win[j]);
                        } else {
#pragma unroll
                            for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
                        }
                    }
                }
            }
            float now[VEC], z[VEC];
            widen(ring[slot][i][tid], now);
#pragma unroll
            for (int e = 0; e < VEC; ++e) z[e] = b[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) fma_vec<VEC>(w[j], win[j], z);
            fma_vec<VEC>(w[W - 1], now, z);
            if (f & kMine) {
                if (a.silu) silu_vec<VEC>(z);
                if (f & kPadding) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) z[e] = 0.f;
                }
                store_vec(y, z);
            }
            y += a.part_stride[p];
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) win[j][e] = j + 1 < W - 1 ? win[j + 1][e] : now[e];
            if (held && (f & kMine) && (f & kHold)) {
                // the sequence's last inputs; win has them where it is that short
                const bool is_short = end - start < W - 1;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    float v[VEC];
                    if (is_short) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) v[e] = win[j][e];
                    } else {
                        load_vec<T, VEC>(x + (end - (W - 1) + j) * a.x_stride, v);
                    }
                    store_vec(held + (long long)j * a.C, v);
                }
            }
        }
    }
}

// Forward of few tokens (a decode batch), where latency counts: a block takes
// kThreads * VEC channels of one token t, each warp for itself and without a barrier.
// The token that begins a sequence brings the sequence's next W - 2 tokens with it.
// One token each of 256 sequences, 6144 channels: 10.7 us, with the tiles above 14.6 us;
// one sequence of 512 tokens: 12.0 and 6.5 us.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
conv_few(ConvArgs a, unsigned ctiles) {
    const int lane = threadIdx.x % 32;
    const int c = (int)((blockIdx.x % ctiles * kThreads + threadIdx.x) * VEC);
    const int t = (int)(blockIdx.x / ctiles);
    const bool live = c < a.C;
    const int cc = live ? c : 0;
    const T *x = static_cast<const T *>(a.x) + cc;
    float now[VEC], w[W][VEC], b[VEC];
    load_vec<T, VEC>(x + t * a.x_stride, now);
    load_weights<T, VEC, W>(a, cc, w, b);

    int n = t, start = t, end = t + 1, slot = -1;
    if (a.cu) {
        n = (int)((long long)t * a.N / a.total);  // right where the sequences are equally long
        start = a.cu[n];
        end = a.cu[n + 1];
    }
    if (a.states) slot = a.slots ? a.slots[n] : n;
    if (start > t || end <= t) {
        n = seq_of(a.cu, a.N, t, lane);
        start = a.cu[n];
        end = a.cu[n + 1];
        if (a.states) slot = a.slots ? a.slots[n] : n;
    }
    if (start < 0 || start > t || end <= t || end > a.total) return;  // in no sequence
    const int pos = t - start;
    if (pos > 0 && pos < W - 1) return;  // taken with the sequence's first token
    if (slot >= a.n_slots) slot = -1;
    const bool padding = a.states && slot < 0;
    T *held = a.states && !padding
                  ? static_cast<T *>(a.states) + (long long)slot * (W - 1) * a.C + cc : nullptr;
    float win[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (pos) {
            load_vec<T, VEC>(x + (t - (W - 1) + j) * a.x_stride, win[j]);
        } else if (held) {
            load_vec<T, VEC>(held + (long long)j * a.C, win[j]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
        }
    }
    // of the sequences with tokens that name one slot the first has it
    bool zero = padding;
    if (held && a.slots) {
        zero = __any_sync(0xffffffffu, slot_taken(a.slots, a.cu, a.total, n, slot, lane, 32));
    }
    if (!live) return;
    const int p = part_of(a, cc);
    T *y = static_cast<T *>(a.part[p]) + (cc - a.begin[p]) + t * a.part_stride[p];
    const int last = pos ? t : min(t + W - 2, end - 1);
    for (int s = t;; ++s) {
        float z[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) z[e] = b[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) fma_vec<VEC>(w[j], win[j], z);
        fma_vec<VEC>(w[W - 1], now, z);
        if (a.silu) silu_vec<VEC>(z);
        if (zero)
#pragma unroll
            for (int e = 0; e < VEC; ++e) z[e] = 0.f;
        store_vec(y, z);
        y += a.part_stride[p];
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[j][e] = j + 1 < W - 1 ? win[j + 1][e] : now[e];
        if (s == last) break;
        load_vec<T, VEC>(x + (s + 1) * a.x_stride, now);
    }
    if (pos || !held || zero) return;
    // the sequence's last inputs; win has them where it is that short
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        if (end - start >= W - 1) load_vec<T, VEC>(x + (end - (W - 1) + j) * a.x_stride, win[j]);
        store_vec(held + (long long)j * a.C, win[j]);
    }
}

// Blocks of the backward per SM: 4 of 120 registers a thread (5 of 96 spill, and took
// 163.5 us on 16384 x 6144 where these take 119.0 us).
constexpr int kBwdPerSM = 4, kMaxBwdTile = 512;

// Backward.  A block: kThreads * VEC channels and the tokens [t0, t0 + tile): their dx
// (dz of the W - 1 tokens behind the tile is formed again) and their share of dw.
// The rows of x and dy come through a ring of shared memory, each thread's own
// channels by itself, S - 1 groups of B rows ahead.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads, kBwdPerSM)
conv_bwd(ConvArgs a, unsigned ctiles, int tile) {
    constexpr int B = 4, S = VEC * sizeof(T) > 8 ? 2 : 4;
    __shared__ __align__(16) Raw<T, VEC> ring[2][S][B][kThreads];
    const int tid = threadIdx.x;
    // of each token of the tile and behind it: how many inputs of its sequence lie
    // before it (W - 1 at most), -1 where it is in none
    __shared__ __align__(4) signed char before[kMaxBwdTile + W - 1];
    const int lane = threadIdx.x % 32;
    const int c = (int)((blockIdx.x % ctiles * kThreads + threadIdx.x) * VEC);
    const int t0 = (int)(blockIdx.x / ctiles) * tile, t1 = min(t0 + tile, a.total);
    const int stop = min(t1 + W - 1, a.total);  // tokens whose dz is formed
    const bool live = c < a.C;
    const int cc = live ? c : 0;
    const T *x = static_cast<const T *>(a.x) + cc;
    const int p = part_of(a, cc);
    const T *dy = static_cast<const T *>(a.part[p]) + (cc - a.begin[p]);
    const long long dy_stride = a.part_stride[p];

    float win[W - 1][VEC];  // the inputs before the token
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int s = t0 - (W - 1) + j;
#pragma unroll
        for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
        if (s >= 0) load_vec<T, VEC>(x + s * a.x_stride, win[j]);
    }
    const T *xa = x + (long long)t0 * a.x_stride;  // the rows copied next
    const T *da = dy + (long long)t0 * dy_stride;
    int copied = t0;
    const auto copy_group = [&](int slot) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (copied + i < stop) {
                copy_async<T, VEC>(&ring[0][slot][i][tid], xa);
                copy_async<T, VEC>(&ring[1][slot][i][tid], da);
            }
            xa += a.x_stride;
            da += dy_stride;
        }
        copied += B;
        copy_commit();
    };
#pragma unroll
    for (int g = 0; g < S - 1; ++g) copy_group(g);
    {
        int lo = 0, hi = 0;
        if (a.cu) {
            lo = seq_of(a.cu, a.N, t0, lane);
            hi = seq_of(a.cu, a.N, stop - 1, lane);
        }
        for (int t = t0 + threadIdx.x; t < stop; t += kThreads) {
            const Span sp = span_of(a, t, lo, hi);
            before[t - t0] = sp.start < sp.end ? min(t - sp.start, W - 1) : -1;
        }
    }
    float w[W][VEC], b[VEC], dw[W][VEC], db[VEC], acc[W - 1][VEC];
    load_weights<T, VEC, W>(a, cc, w, b);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (j < W - 1) acc[j][e] = 0.f;
            dw[j][e] = 0.f;
        }
#pragma unroll
    for (int e = 0; e < VEC; ++e) db[e] = 0.f;
    __syncthreads();
    if (!live) return;
    // acc[j]: dx of token t - (W - 1) + j so far; it leaves with the last token that
    // reads the input
    T *dx = static_cast<T *>(a.dx) + cc + (t0 - (W - 1)) * (long long)a.C;
    int slot = 0;
    for (int i0 = t0; i0 < t1 + W - 1; i0 += B, slot = slot + 1 == S ? 0 : slot + 1) {
        copy_wait<S - 2>();  // this group's rows have come
        copy_group(slot ? slot - 1 : S - 1);
        if (i0 >= t0 + W - 1 && i0 + B <= t1 &&
            *reinterpret_cast<const unsigned *>(&before[i0 - t0]) == 0x01010101u * (W - 1)) {
            // four tokens inside one sequence and the tile: no case to tell apart
            float in[W - 1 + B][VEC], out[W - 1 + B][VEC];
#pragma unroll
            for (int j = 0; j < W - 1 + B; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (j < W - 1) in[j][e] = win[j][e];
                    out[j][e] = j < W - 1 ? acc[j][e] : 0.f;
                }
#pragma unroll
            for (int i = 0; i < B; ++i) {
                float d[VEC];
                widen(ring[0][slot][i][tid], in[W - 1 + i]);
                widen(ring[1][slot][i][tid], d);
                if (a.silu) {
                    float z[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) z[e] = b[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) fma_vec<VEC>(w[j], in[i + j], z);
                    silu_grad_vec<VEC>(z, d);
                }
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    fma_vec<VEC>(w[j], d, out[i + j]);
                    fma_vec<VEC>(d, in[i + j], dw[j]);
                }
                add_vec<VEC>(db, d);
                store_vec(dx, out[i]);
                dx += a.C;
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    win[j][e] = in[B + j][e];
                    acc[j][e] = out[B + j][e];
                }
        } else {
#pragma unroll 1
            for (int i = 0; i < B; ++i) {
                const int t = i0 + i;
                const int have = t < stop ? before[t - t0] : -1;
                float out[W][VEC];
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[j][e] = j < W - 1 ? acc[j][e] : 0.f;
                if (have >= 0) {
                    float in[W][VEC], d[VEC], now[VEC];
                    widen(ring[0][slot][i][tid], now);
                    widen(ring[1][slot][i][tid], d);
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)  // the sequence's own inputs only
                            in[j][e] = W - 1 - j > have ? 0.f : j < W - 1 ? win[j][e] : now[e];
                    if (a.silu) {
                        float z[VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) z[e] = b[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) fma_vec<VEC>(w[j], in[j], z);
                        silu_grad_vec<VEC>(z, d);
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        if (W - 1 - j <= have) fma_vec<VEC>(w[j], d, out[j]);
                    if (t < t1) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) db[e] += d[e];
#pragma unroll
                        for (int j = 0; j < W; ++j) fma_vec<VEC>(d, in[j], dw[j]);
                    }
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            win[j][e] = j + 1 < W - 1 ? win[j + 1][e] : now[e];
                }
                const int done = t - (W - 1);
                if (done >= t0 && done < t1) store_vec(dx, out[0]);
                dx += a.C;
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[j][e] = out[j + 1][e];
            }
        }
    }
    float *mine = a.partial + (long long)(blockIdx.x / ctiles) * a.C * (W + 1);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) mine[(long long)j * a.C + c + e] = dw[j][e];
#pragma unroll
    for (int e = 0; e < VEC; ++e) mine[(long long)W * a.C + c + e] = db[e];
}

// dw[c, j] and db[c] = sums over the tiles' partial sums, always in the same order:
// eight threads take every eighth tile each.
__global__ void __launch_bounds__(256)
conv_bwd_sum(const float *partial, float *dw, float *db, int tiles, int C, int W) {
    __shared__ float part[8][33];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const long long i = (long long)blockIdx.x * 32 + tx;  // j * C + c
    const bool in = i < (long long)(W + (db ? 1 : 0)) * C;
    float s = 0.f;
    if (in)
#pragma unroll 4
        for (int k = ty; k < tiles; k += 8) s += partial[(long long)k * C * (W + 1) + i];
    part[ty][tx] = s;
    __syncthreads();
    if (ty || !in) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) s += part[k][tx];
    const int j = (int)(i / C), c = (int)(i % C);
    if (j < W) dw[(long long)c * W + j] = s;
    else db[c] = s;
}

template <typename T, int VEC>
bool vectors_fit(const ConvArgs &a) {
    constexpr size_t bytes = VEC * sizeof(T);
    const auto fits = [](const void *p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * sizeof(T) % bytes == 0;
    };
    bool ok = a.C % VEC == 0 && fits(a.x, a.x_stride) && fits(a.states, a.C) && fits(a.dx, a.C);
    for (int p = 0; p < a.parts; ++p)
        ok = ok && fits(a.part[p], a.part_stride[p]) && a.begin[p] % VEC == 0;
    return ok;
}

unsigned channel_tiles(int C, int vec) { return (C + kThreads * vec - 1) / (kThreads * vec); }

// Tokens per block such that `per_sm` blocks per SM take them all at once, at least 8.
int tile_of(int total, unsigned ctiles, int per_sm, int most) {
    const int rows = 148 * per_sm / (int)ctiles > 1 ? 148 * per_sm / (int)ctiles : 1;
    const int tile = ((total + rows - 1) / rows + 7) / 8 * 8;
    return tile > most ? most : tile;
}

template <typename T, int VEC, int W>
cudaError_t fwd_w(const ConvArgs &a, cudaStream_t st) {
    const unsigned ct = channel_tiles(a.C, VEC);
    // (each warp of conv_few looks at the slots for itself: a token each of 4096 sequences of
    // 512 channels 20.6 us, with the tiles 16.4 us; of 1024 sequences 6.6 and 6.4 us)
    if ((long long)ct * a.total <= 148 * 32 && !(a.slots && a.N > 1024)) {
        conv_few<T, VEC, W><<<ct * a.total, kThreads, 0, st>>>(a, ct);
    } else {
        const int tile = tile_of(a.total, ct, kFwdPerSM<T, VEC>, kMaxTile);
        conv_fwd<T, VEC, W><<<ct * ((a.total + tile - 1) / tile), kThreads, 0, st>>>(a, ct, tile);
    }
    return cudaPeekAtLastError();
}

// The backward's tile.  Sized for vectors of 4 channels whatever
// the call's alignment and type are, so that the workspace depends on the sizes alone.
int bwd_tile(int total, int C) { return tile_of(total, channel_tiles(C, 4), kBwdPerSM, kMaxBwdTile); }

template <typename T, int VEC, int W>
cudaError_t bwd_w(const ConvArgs &a, cudaStream_t st) {
    const int tile = bwd_tile(a.total, a.C), tiles = (a.total + tile - 1) / tile;
    const unsigned ct = channel_tiles(a.C, VEC);
    conv_bwd<T, VEC, W><<<ct * tiles, kThreads, 0, st>>>(a, ct, tile);
    const long long sums = (long long)(W + (a.db ? 1 : 0)) * a.C;
    conv_bwd_sum<<<(unsigned)((sums + 31) / 32), 256, 0, st>>>(a.partial, a.dw, a.db, tiles, a.C, W);
    return cudaPeekAtLastError();
}

#define GDN_CONV(F, T, VEC)                   \
    switch (a.W) {                            \
        case 2: return F<T, VEC, 2>(a, st);   \
        case 3: return F<T, VEC, 3>(a, st);   \
        default: return F<T, VEC, 4>(a, st);  \
    }

}  // namespace

cudaError_t launch_short_conv_fwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
    if (bf16) {
        if (vectors_fit<__nv_bfloat16, 4>(a)) GDN_CONV(fwd_w, __nv_bfloat16, 4)
        GDN_CONV(fwd_w, __nv_bfloat16, 1)
    }
    if (vectors_fit<float, 4>(a)) GDN_CONV(fwd_w, float, 4)
    GDN_CONV(fwd_w, float, 1)
}

size_t short_conv_bwd_bytes(int total, int C, int W) {
    const int tile = bwd_tile(total, C);
    return (size_t)((total + tile - 1) / tile) * C * (W + 1) * sizeof(float);
}

cudaError_t launch_short_conv_bwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
    if (bf16) {
        if (vectors_fit<__nv_bfloat16, 4>(a)) GDN_CONV(bwd_w, __nv_bfloat16, 4)
        GDN_CONV(bwd_w, __nv_bfloat16, 1)
    }
    if (vectors_fit<float, 4>(a)) GDN_CONV(bwd_w, float, 4)
    GDN_CONV(bwd_w, float, 1)
}

#undef GDN_CONV

}  // namespace gdn
