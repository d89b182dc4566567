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
// A warp holds its rows in registers, LW lanes per row with V float4 each.  Everything
// is float32: the state is carried over thousands of steps.
//
// Two kernels.  Token by token, for batches of short runs (decode): bound by HBM, the
// state being read and written once; one token each of 256 sequences of 16 heads of
// 128 x 128, 541 MB: 91.7 us on B200, 0.90 of the measured copy rate.  Up to 8 tokens at
// once, for longer runs: bound by the issue of its products' reductions and by the
// barriers between its phases; 8 tokens of 256 sequences of 16 heads in float32: 182 us
// (token by token 412 us).  bf16 runs of Dk = 64 or 128 go to decode_runs_tc.cu.  Where
// the two meet, us for 1 / 2 / 3 tokens of 256 sequences of 16 heads of 128 x 128:
// float32 token by token 90 / 129 / 177, up to 8 at once 107 / 116 / 124; bf16 89 / 133 /
// 185 and about 120 for any number.
//
// Token by token each warp looks for its slot among the earlier sequences' by itself; for
// 1024 sequences of 16 heads that is 341 us instead of 328, for 4096 1483 instead of 1283.
// Shared by the block it needs a barrier between the loads and the products: 348 and 1395
// us, and 96 instead of 91 at 256.
#include "runs_common.cuh"

namespace gdn {

namespace {

constexpr int kTok = kRunTokens;
constexpr int kMaxWarps = 8;  // per block
constexpr int kTokenBlocks = 5, kChunkBlocks = 3;  // blocks per SM

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

// How a row of Dk key channels is read: element by element, by float4, or by float4
// with Dk known to fill the lanes (no element of a row needs a test).
enum Rows { kAny, kVec, kFull };

template <int K>
__device__ __forceinline__ float4 load_state(const float *row, int c, int Dk) {
    if (K == kFull) return *reinterpret_cast<const float4 *>(row + c);
    if (K == kVec) return c < Dk ? *reinterpret_cast<const float4 *>(row + c) : make_float4(0, 0, 0, 0);
    float4 s;
    s.x = c < Dk ? row[c] : 0.f;
    s.y = c + 1 < Dk ? row[c + 1] : 0.f;
    s.z = c + 2 < Dk ? row[c + 2] : 0.f;
    s.w = c + 3 < Dk ? row[c + 3] : 0.f;
    return s;
}
template <int K>
__device__ __forceinline__ void store_state(float *row, int c, int Dk, float4 s) {
    if (K != kAny) {
        if (K == kFull || c < Dk) *reinterpret_cast<float4 *>(row + c) = s;
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

// Elements c .. c + 3 of a row of k or q, widened; 0 from Dk on.
template <int K, typename T>
__device__ __forceinline__ float4 load_key(const T *row, int c, int Dk, bool aligned) {
    if (K != kAny && aligned)
        return K == kFull || c < Dk ? load4(row + c) : make_float4(0, 0, 0, 0);
    return make_float4(c < Dk ? to_f32(row[c]) : 0.f, c + 1 < Dk ? to_f32(row[c + 1]) : 0.f,
                       c + 2 < Dk ? to_f32(row[c + 2]) : 0.f, c + 3 < Dk ? to_f32(row[c + 3]) : 0.f);
}

__device__ __forceinline__ float2 lo2(const float4 &x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(const float4 &x) { return make_float2(x.z, x.w); }

// LW lanes share a row, V float4 each; R rows per lane group, so this many per warp.
template <int LW, int R> constexpr int kRows = R * (32 / LW);

// acc[r] += s_r . k, acc[R + r] += s_r . q over the elements of one float4 per row.
template <int R, int V>
__device__ __forceinline__ void row_dots(const float4 (&s)[R][V], int v, const float4 &k4,
                                         const float4 &q4, float2 (&acc)[2 * R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        acc[r] = __ffma2_rn(lo2(s[r][v]), lo2(k4), acc[r]);
        acc[r] = __ffma2_rn(hi2(s[r][v]), hi2(k4), acc[r]);
        acc[R + r] = __ffma2_rn(lo2(s[r][v]), lo2(q4), acc[R + r]);
        acc[R + r] = __ffma2_rn(hi2(s[r][v]), hi2(q4), acc[R + r]);
    }
}

// s_r <- g s_r
template <int R, int V>
__device__ __forceinline__ void scale_rows(float4 (&s)[R][V], float g) {
    const float2 g2 = make_float2(g, g);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 lo = __fmul2_rn(lo2(s[r][v]), g2), hi = __fmul2_rn(hi2(s[r][v]), g2);
            s[r][v] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
}
// s_r <- s_r + u_r k, one float4 per row.
template <int R, int V>
__device__ __forceinline__ void add_rows(float4 (&s)[R][V], int v, const float (&u)[R],
                                         const float4 &k4) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float2 uu = make_float2(u[r], u[r]);
        const float2 lo = __ffma2_rn(uu, lo2(k4), lo2(s[r][v]));
        const float2 hi = __ffma2_rn(uu, hi2(k4), hi2(s[r][v]));
        s[r][v] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
}

// A warp's rows of the state from wrow on, zero from Dv on.
template <int LW, int R, int V, int K>
__device__ __forceinline__ void load_rows(const RunsArgs &a, const float *state, int wrow, int lane,
                                          bool run, float4 (&s)[R][V]) {
    const int Dk = K == kFull ? LW * V * 4 : a.Dk;
    const float *p = state + (long long)(wrow + lane / LW * R) * Dk;
    const bool all = run && wrow + kRows<LW, R> <= a.Dv;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[r][v] = all || (run && wrow + lane / LW * R + r < a.Dv)
                          ? load_state<K>(p + r * Dk, 4 * (v * LW + lane % LW), Dk)
                          : make_float4(0, 0, 0, 0);
}
template <int LW, int R, int V, int K>
__device__ __forceinline__ void store_rows(const RunsArgs &a, float *state, int wrow, int lane,
                                           const float4 (&s)[R][V]) {
    const int Dk = K == kFull ? LW * V * 4 : a.Dk;
    float *p = state + (long long)(wrow + lane / LW * R) * Dk;
    if (wrow + kRows<LW, R> <= a.Dv) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v)
                store_state<K>(p + r * Dk, 4 * (v * LW + lane % LW), Dk, s[r][v]);
        return;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (wrow + lane / LW * R + r < a.Dv)
                store_state<K>(p + r * Dk, 4 * (v * LW + lane % LW), Dk, s[r][v]);
}

// Token by token: every warp for itself, k, q and their norms in registers and no
// barrier, so that a run of one token costs little beyond the loads and stores of
// the state.  A block: `tiles` times warps * ROWS value channels of one value head of
// one sequence.
template <typename T, int LW, int R, int V, int K>
__global__ void __launch_bounds__(32 * kMaxWarps, kTokenBlocks)
decode_tokens_kernel(RunsArgs a, int row_blocks, int tiles) {
    constexpr int ROWS = kRows<LW, R>, NK = 2 * R > LW ? 2 * R / LW : 1;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int sub = lane % LW;
    const int nh = blockIdx.x / row_blocks;
    const int n = nh / a.Hv, h = nh % a.Hv;
    const int t0 = a.cu ? a.cu[n] : n, t1 = a.cu ? a.cu[n + 1] : n + 1;
    const int slot = a.slots ? a.slots[n] : n;
    if (t0 < 0 || t1 > a.total || t0 >= t1) return;  // empty, or offsets that are none
    bool run = slot >= 0 && slot < a.n_slots;
    const int row0 = blockIdx.x % row_blocks * tiles * warps * ROWS;
    float *state = a.states + ((long long)(run ? slot : 0) * a.Hv + h) * a.Dv * a.Dk;
    const int hk = h / (a.Hv / a.Hk);
    const T *kr = static_cast<const T *>(a.k) + (long long)hk * a.Dk;
    const T *qr = a.q ? static_cast<const T *>(a.q) + (long long)hk * a.Dk : nullptr;
    const T *vr = static_cast<const T *>(a.v) + (long long)h * a.Dv;
    T *op = a.o ? static_cast<T *>(a.o) + (long long)h * a.Dv : nullptr;
    const bool aligned = a.k_stride % 4 == 0 && a.q_stride % 4 == 0;
    const bool unit = a.flags & kFlagL2Norm;

    // a lane ends up with NK of a row group's sums: its rows' S.k in the lower half of
    // the lanes, their S.q in the upper half
    const int first = LW >= 2 * R ? sub / (LW / (2 * R)) : sub * NK;
    float4 k4[V], q4[V];
    float kq = 0.f, rk = 1.f, rq = 1.f, alpha = 0.f, beta = 0.f;
    for (int tile = 0; tile < tiles; ++tile) {
        const int wrow = row0 + (tile * warps + warp) * ROWS;
        if (wrow >= a.Dv) return;
        float4 s[R][V];
        load_rows<LW, R, V, K>(a, state, wrow, lane, run, s);
        const int grow = wrow + lane / LW * R;  // the lane group's first row
        for (int t = t0; t < t1; ++t) {
            float vv[NK];
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                const int row = grow + (first + i) % R;
                vv[i] = run && row < a.Dv ? to_f32(vr[t * a.v_stride + row]) : 0.f;
            }
            if (run && (tile == 0 || t1 - t0 > 1)) {  // tiles share the token of a run of one
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    k4[v] = load_key<K>(kr + t * a.k_stride, 4 * (v * LW + sub), a.Dk, aligned);
                    q4[v] = qr ? load_key<K>(qr + t * a.q_stride, 4 * (v * LW + sub), a.Dk, aligned)
                               : make_float4(0, 0, 0, 0);
                }
                const float g0 = a.log_alpha[t * a.la_stride + h], g1 = a.beta[t * a.be_stride + h];
                if (t == t0 && tile == 0 && a.update && a.slots &&
                    __any_sync(0xffffffffu, slot_taken(a.slots, a.cu, a.total, n, slot, lane, 32)))
                    run = false;
                float kk = 0.f, qq = 0.f;
                kq = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    kk += k4[v].x * k4[v].x + k4[v].y * k4[v].y + k4[v].z * k4[v].z + k4[v].w * k4[v].w;
                    qq += q4[v].x * q4[v].x + q4[v].y * q4[v].y + q4[v].z * q4[v].z + q4[v].w * q4[v].w;
                    kq += k4[v].x * q4[v].x + k4[v].y * q4[v].y + k4[v].z * q4[v].z + k4[v].w * q4[v].w;
                }
#pragma unroll
                for (int off = LW / 2; off > 0; off >>= 1) {
                    kq += __shfl_xor_sync(0xffffffffu, kq, off);
                    if (unit) {
                        kk += __shfl_xor_sync(0xffffffffu, kk, off);
                        qq += __shfl_xor_sync(0xffffffffu, qq, off);
                    }
                }
                if (unit) {
                    rk = rsqrtf(kk + kNormEps);
                    rq = rsqrtf(qq + kNormEps);
                }
                const float2 gp = decay_pair(g0, g1, a.flags);
                alpha = gp.x;
                beta = gp.y;
            }
            if (!run) {  // a row of padding: its outputs are zero, nothing else is touched
                if (op)
                    for (int i = lane; i < ROWS && wrow + i < a.Dv; i += 32)
                        op[(long long)t * a.Hv * a.Dv + wrow + i] = from_f32<T>(0.f);
                continue;
            }
            float2 acc[2 * R];
            float x[2 * R], un[NK];
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) row_dots<R, V>(s, v, k4[v], q4[v], acc);
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) x[i] = acc[i].x + acc[i].y;
            reduce_scatter<2 * R, LW>(x, lane);
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                // u = beta (v - alpha S.k), in the lanes that hold S.k, for the others too
                un[i] = __shfl_sync(0xffffffffu, beta * (vv[i] - alpha * rk * x[i]), sub % (LW / 2),
                                    LW);
                const int row = grow + (first + i) % R;
                if (op && first + i >= R && row < a.Dv)
                    op[(long long)t * a.Hv * a.Dv + row] =
                        from_f32<T>(rq * (alpha * x[i] + un[i] * rk * kq));
            }
            if (!a.update && t + 1 == t1) break;
            float u[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
                u[r] = rk * __shfl_sync(0xffffffffu, un[r % NK],
                                        r / NK * (LW >= 2 * R ? LW / (2 * R) : 1), LW);
            scale_rows<R, V>(s, alpha);
#pragma unroll
            for (int v = 0; v < V; ++v) add_rows<R, V>(s, v, u, k4[v]);
        }
        if (run && a.update) store_rows<LW, R, V, K>(a, state, wrow, lane, s);
    }
}

// Up to 8 tokens at once; a block as above.  k and q stand in shared memory as float32,
// already normalised; a warp per token forms its products with the earlier ones, one
// warp solves for T and M while the others go on to S . k and S . q.
template <typename T, int LW, int R, int V, int K>
__global__ void __launch_bounds__(32 * kMaxWarps, kChunkBlocks)
decode_chunks_kernel(RunsArgs a, int row_blocks, int tiles) {
    constexpr int ROWS = kRows<LW, R>;
    constexpr int PD = LW * V * 4;       // padded Dk
    constexpr int E = (PD + 31) / 32;    // a lane's elements of k where a warp holds a token
    constexpr int VI = ROWS * kTok / 32;  // a lane's share of a warp's rows and tokens
    __shared__ __align__(16) float sk[kTok][PD], sq[kTok][PD];
    // tm[0]: T with u = T r, tm[1]: M with o = gamma b + M r  (r = v - gamma a)
    __shared__ __align__(16) float sA[kTok][kTok], sP[kTok][kTok], al[kTok];
    __shared__ float tm[2][kTok][kTok], be[kTok], gam[kTok], tail[kTok];
    // per warp and token, a row per column: a then r, b, the corrections
    __shared__ __align__(16) float ra[kMaxWarps][kTok][ROWS], rb_[kMaxWarps][kTok][ROWS];
    __shared__ __align__(16) float su[kMaxWarps][kTok][ROWS];

    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
    const int rb = blockIdx.x % row_blocks;
    const int nh = blockIdx.x / row_blocks;
    const int n = nh / a.Hv, h = nh % a.Hv;
    const int t0 = a.cu ? a.cu[n] : n, t1 = a.cu ? a.cu[n + 1] : n + 1;
    const int slot = a.slots ? a.slots[n] : n;
    if (t0 < 0 || t1 > a.total || t0 >= t1) return;  // empty, or offsets that are none
    bool run = slot >= 0 && slot < a.n_slots;
    const int row0 = rb * tiles * warps * ROWS;
    float *state = a.states + ((long long)(run ? slot : 0) * a.Hv + h) * a.Dv * a.Dk;
    const T *vp = static_cast<const T *>(a.v) + (long long)h * a.Dv;
    T *op = a.o ? static_cast<T *>(a.o) + (long long)h * a.Dv : nullptr;
    const int sub = lane % LW, grp = lane / LW;
    const int hk = h / (a.Hv / a.Hk);
    float4 s[R][V];
    load_rows<LW, R, V, K>(a, state, row0 + warp * ROWS, lane, run, s);

    for (int tile = 0; tile < tiles; ++tile) {
        const int wrow = row0 + (tile * warps + warp) * ROWS;  // the warp's first row
        if (row0 + tile * warps * ROWS >= a.Dv) break;
        if (tile) load_rows<LW, R, V, K>(a, state, wrow, lane, true, s);
        for (int c0 = t0; c0 < t1; c0 += kTok) {
            const int m = min(kTok, t1 - c0);
            float vv[VI];  // v of the warp's rows, needed last
#pragma unroll
            for (int i = 0; i < VI; ++i) {
                const int j = (lane + 32 * i) / ROWS, row = (lane + 32 * i) % ROWS;
                vv[i] = run && j < m && wrow + row < a.Dv
                            ? to_f32(vp[(c0 + j) * a.v_stride + wrow + row]) : 0.f;
            }
            // a run of one chunk keeps its tokens' arrays for all row tiles
            if (tile == 0 || t1 - t0 > kTok) {
                if (tile || c0 > t0) __syncthreads();  // the arrays are written again
                // a warp per token: k and q (normalised), the gates
                for (int j = warp; j < m && run; j += warps) {
                    const long long t = c0 + j;
                    const T *kr = static_cast<const T *>(a.k) + t * a.k_stride + (long long)hk * a.Dk;
                    const T *qr = a.q ? static_cast<const T *>(a.q) + t * a.q_stride +
                                            (long long)hk * a.Dk
                                      : nullptr;
                    float x[E], y[E];
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const int c = lane + 32 * i;
                        x[i] = c < a.Dk ? to_f32(kr[c]) : 0.f;
                        y[i] = qr && c < a.Dk ? to_f32(qr[c]) : 0.f;
                    }
                    const float g0 = a.log_alpha[t * a.la_stride + h];
                    const float g1 = a.beta[t * a.be_stride + h];
                    float rk = 1.f, rq = 1.f;
                    if (a.flags & kFlagL2Norm) {
                        float kn = 0.f, qn = 0.f;
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            kn += x[i] * x[i];
                            qn += y[i] * y[i];
                        }
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
                    if (lane == 0) {
                        const float2 gp = decay_pair(g0, g1, a.flags);
                        al[j] = gp.x;
                        be[j] = gp.y;
                    }
                }
                if (tile == 0 && c0 == t0) {
                    // of the sequences with tokens that name one slot the first has it
                    const int taken =
                        run && a.update && a.slots
                            ? slot_taken(a.slots, a.cu, a.total, n, slot, tid, blockDim.x) : 0;
                    if (__syncthreads_or(taken)) run = false;
                    if (!run) {  // a row of padding: its outputs are zero, nothing else is touched
                        if (op)
                            for (int t = t0; t < t1; ++t)
                                for (int i = tid; i < tiles * warps * ROWS && row0 + i < a.Dv;
                                     i += blockDim.x)
                                    op[(long long)t * a.Hv * a.Dv + row0 + i] = from_f32<T>(0.f);
                        return;
                    }
                } else {
                    __syncthreads();
                }
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
                    float dk[kTok];
                    load8(al, dk);
                    const float dec = decay_between(dk, j + 1, i + 1);  // Gamma_ij
                    if (lane == 0) gam[i] = decay_between(dk, 0, i + 1);
                    if (lane == 1) tail[i] = decay_between(dk, i + 1, m);
                    if (lane % 2 == 0 && j <= i) {
                        if (w < kTok) sA[i][j] = be[i] * dec * x[0];
                        else sP[i][j] = dec * x[0];
                    }
                }
                __syncthreads();
                if (warp == 0) solve_tokens(sA, sP, be, m, lane, tm);
            }
            // the rows' products with k and q
            for (int j = 0; j < m; ++j) {
                float2 acc[2 * R];
                float x[2 * R];
#pragma unroll
                for (int i = 0; i < 2 * R; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(&sk[j][4 * (v * LW + sub)]);
                    const float4 q4 = *reinterpret_cast<const float4 *>(&sq[j][4 * (v * LW + sub)]);
                    row_dots<R, V>(s, v, k4, q4, acc);
                }
#pragma unroll
                for (int i = 0; i < 2 * R; ++i) x[i] = acc[i].x + acc[i].y;
                const int first = reduce_scatter<2 * R, LW>(x, lane);
                constexpr int NK = 2 * R > LW ? 2 * R / LW : 1;  // sums left in a lane
#pragma unroll
                for (int i = 0; i < NK; ++i) {
                    const int w = first + i;
                    (w < R ? ra[warp][j][grp * R + w] : rb_[warp][j][grp * R + w - R]) = x[i];
                }
            }
            if (tile == 0 || t1 - t0 > kTok) __syncthreads();  // T and M are there
            else __syncwarp();
            // each row's r, then its outputs and corrections
#pragma unroll
            for (int i = 0; i < VI; ++i) {
                const int j = (lane + 32 * i) / ROWS, row = (lane + 32 * i) % ROWS;
                if (j < m) ra[warp][j][row] = vv[i] - gam[j] * ra[warp][j][row];
            }
            __syncwarp();
            for (int at = lane; at < ROWS * m; at += 32) {
                const int i = at / ROWS, row = at % ROWS;
                float u = 0.f, out = gam[i] * rb_[warp][i][row];
                for (int j = 0; j <= i; ++j) {
                    const float r = ra[warp][j][row];
                    u += tm[0][i][j] * r;
                    out += tm[1][i][j] * r;
                }
                su[warp][i][row] = tail[i] * u;
                if (op && wrow + row < a.Dv)
                    op[(long long)(c0 + i) * a.Hv * a.Dv + wrow + row] = from_f32<T>(out);
            }
            __syncwarp();
            if (a.update || c0 + kTok < t1) {
                scale_rows<R, V>(s, gam[m - 1]);
                for (int j = 0; j < m; ++j) {
                    float u[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) u[r] = su[warp][j][grp * R + r];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float4 k4 = *reinterpret_cast<const float4 *>(&sk[j][4 * (v * LW + sub)]);
                        add_rows<R, V>(s, v, u, k4);
                    }
                }
            }
            __syncwarp();
        }
        if (a.update) store_rows<LW, R, V, K>(a, state, wrow, lane, s);
    }
}

// How a launch covers the value channels: warps per block, row tiles per block, blocks
// per (sequence, head).  Few heads: their rows are shared out over more blocks, up to
// two per SM.
struct Cover {
    int warps, tiles, row_blocks;
    unsigned blocks;
};
Cover cover(const RunsArgs &a, int rows) {
    Cover c;
    c.warps = min(kMaxWarps, (a.Dv + rows - 1) / rows);
    c.tiles = (a.Dv + c.warps * rows - 1) / (c.warps * rows);
    c.row_blocks = 1;
    while (c.tiles > 1 && (long long)a.N * a.Hv * c.row_blocks < 148 * 2) {
        c.tiles = (c.tiles + 1) / 2;
        c.row_blocks = (a.Dv + c.tiles * c.warps * rows - 1) / (c.tiles * c.warps * rows);
    }
    c.blocks = (unsigned)((long long)a.N * a.Hv * c.row_blocks);
    return c;
}

// About two tokens per sequence or more on average: up to 8 tokens at once, else token by
// token.  The figures for many sequences are above.  The host knows the sizes alone, not the
// offsets: of a buffer of `total` rows any number from N on may belong to sequences.  For few
// sequences the 4 sets the border where either mistake costs about the same.  In us, token by
// token and at once, bf16, 16 heads of 128 x 128: one sequence of 1 token 3.6 and 6.7, of 3
// 6.7 and 6.9, of 4 8.3 and 6.8, of 5 9.7 and 6.9 (float32 1 token 3.7 and 6.0, 5 tokens 7.4
// and 7.1); 4 sequences of 1 token 4.7 and 7.1, of 2 6.3 and 7.2; 7 sequences of 1 token 5.6
// and 7.2, of 2 8.0 and 7.3; 8 sequences of 1 token 5.9 and 7.3, of 2 8.2 and 7.1.  So a
// sequence of 4 or 5 tokens in a buffer of its own size loses 3 us at most, a single token in
// a buffer of 6 rows or more as much.  The average also knows nothing of a mixed batch: one
// run of 400 tokens among 511 of one token goes token by token and takes 2913 us, at once it
// would be 276 (float32 1976 and 691), as two calls 352.
bool many_tokens(const RunsArgs &a) {
    return a.total >= 2ll * a.N - a.N / 8 + (a.N < 8 ? 4 : 1);
}

template <typename T, int K>
cudaError_t launch_t(const RunsArgs &a, cudaStream_t st) {
#define GDN_RUNS(KERNEL, LW, R, V)                                                          \
    do {                                                                                    \
        const Cover c = cover(a, kRows<LW, R>);                                             \
        KERNEL<T, LW, R, V, K><<<c.blocks, 32 * c.warps, 0, st>>>(a, c.row_blocks, c.tiles); \
    } while (0)
    if (!many_tokens(a)) {
        // (a row over as many lanes as it has float4, four rows per lane group: 92.9 us on
        // 256 sequences of 16 heads of 128 x 128; 16 lanes of two float4 and two rows
        // 101.6 us, 8 lanes of four 129.8 us)
        if (a.Dk <= 16) GDN_RUNS(decode_tokens_kernel, 4, 4, 1);
        else if (a.Dk <= 32) GDN_RUNS(decode_tokens_kernel, 8, 4, 1);
        else if (a.Dk <= 64) GDN_RUNS(decode_tokens_kernel, 16, 4, 1);
        else if (a.Dk <= 128) GDN_RUNS(decode_tokens_kernel, 32, 4, 1);
        else GDN_RUNS(decode_tokens_kernel, 32, 2, 2);
    } else {
        // (two float4 per lane and four rows per lane group: 8 float32 tokens of 256
        // sequences of 16 heads of 128 x 128 182 us, four float4 and two rows 196 us; of
        // 4 heads of 256 x 256 157 and 172 us)
        if (a.Dk <= 16) GDN_RUNS(decode_chunks_kernel, 4, 4, 1);
        else if (a.Dk <= 32) GDN_RUNS(decode_chunks_kernel, 8, 4, 1);
        else if (a.Dk <= 64) GDN_RUNS(decode_chunks_kernel, 8, 4, 2);
        else if (a.Dk <= 128) GDN_RUNS(decode_chunks_kernel, 16, 4, 2);
        else GDN_RUNS(decode_chunks_kernel, 32, 4, 2);
    }
#undef GDN_RUNS
    return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_decode_runs(const RunsArgs &a, bool bf16, cudaStream_t st) {
    if (bf16 && many_tokens(a) && runs_tc_supported(a)) return launch_decode_runs_tc(a, st);
    const bool full = a.Dk == 16 || a.Dk == 32 || a.Dk == 64 || a.Dk == 128 || a.Dk == 256;
    if (a.Dk % 4) return bf16 ? launch_t<__nv_bfloat16, kAny>(a, st) : launch_t<float, kAny>(a, st);
    if (!full) return bf16 ? launch_t<__nv_bfloat16, kVec>(a, st) : launch_t<float, kVec>(a, st);
    return bf16 ? launch_t<__nv_bfloat16, kFull>(a, st) : launch_t<float, kFull>(a, st);
}

}  // namespace gdn
