// decode_runs for runs of several bf16 tokens, Dk = 64 or 128: the same 8 tokens at
// once as decode_runs.cu (the formulas stand there), their products by mma.sync.
//
// A warp holds 16 rows of the state in registers, as float32.  A float32 x is the
// exact sum of three bf16 numbers, its mantissa's upper, middle and lower 8 bits, so
// S . k is three products of bf16 matrices with float32 sums: as good as in float32,
// k and q being bf16 as they came (the factors 1 / |k|, 1 / |q| are applied to the
// sums).  Likewise S + u k^T with u in three parts.  One warp forms the tokens'
// products with one another, their norms and the 8 x 8 matrices T and M of the head.
//
// The key channels stand in shared memory in the order 0 1 4 5 8 9 12 13 2 3 6 7 10 11
// 14 15 of each 16, so that a lane's float4 of a row (channels 4t .. 4t + 3) is its part
// of both the state's fragments: as left operand in S . k and as accumulator in the
// update.  8 x 8 token products are far too small for a tcgen05 tile of 64 or 128 rows
// with its round trip through tensor memory.
//
// 64 runs of 1 to 8 tokens against 32 value heads of 128 x 128 (read only, 135 MB): 42.7
// us on B200, 0.48 of the measured copy rate (in float32 arithmetic 61.5 us); 8 tokens of
// 256 sequences of 16 heads, states written, 571 MB: 122.5 us, 0.71.  Two blocks of 128
// registers a thread per SM; what bounds it is the chain of one part of the work -
// offsets and slot, k and q, the tokens' products and the substitution on one warp, the
// outputs - with only 16 warps to hide it.  The tokens' loads go ahead of the state's:
// behind them they came 2 us later (49.4 us).  Tried and slower, against 49.4: every warp
// forming T and M for itself (55.6), a ninth warp for them (67), blocks of 4 warps (50.4),
// 3 blocks of 80 registers (56.5), blocks that stay and copy the next part's rows and
// tokens ahead (58.8: the copies' issue waits as long as the loads did), the next round's
// rows fetched into L2 (49.6).  Against 42.4: blocks that stay, the next part's rows by one
// bulk copy of 64 KB (57.8, one per SM without spills 65.4: twice the instructions, and the
// barriers' waits stay).  A kernel for read-only runs alone, 3 blocks of 80 registers that hold
// three of the eight steps of a row at a time, took 40.8 (and 78.7 instead of 85.2 at 256
// sequences of 16 heads), but spills where such a run is longer than 8 tokens; the split
// into three parts and its products are then what it waits for (one part alone: 34).
//
// An infinity does not split into three parts: it meets their zeros and differences and comes
// out as NaN.  One in the state or in v gives NaN in its row, one in q in its token's outputs,
// one in k from its token on, where the recurrence might give an infinity.
#include "runs_common.cuh"

namespace gdn {

namespace {

constexpr int kTok = kRunTokens, kWarps = 8;

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *row) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(row));
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], const void *row) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(row));
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// c += a b, 16 x 16 times 16 x 8.
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a b, 16 x 8 times 8 x 8.
__device__ __forceinline__ void mma8(float &c0, float &c1, float &c2, float &c3, uint32_t a0,
                                     uint32_t a1, uint32_t b) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3) : "r"(a0), "r"(a1), "r"(b));
}

// The upper halves of x (low) and y (high): two bf16, cut off.
__device__ __forceinline__ uint32_t upper2(float x, float y) {
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
// x, y -> three bf16 pairs whose sum is x, y (to 2^-24 of each, and below 2^-110).
__device__ __forceinline__ void split3(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = upper2(x, y);
        if (i < 2) {
            const float2 rest = __fadd2_rn(
                make_float2(x, y), make_float2(-__uint_as_float(__float_as_uint(x) & 0xffff0000u),
                                               -__uint_as_float(__float_as_uint(y) & 0xffff0000u)));
            x = rest.x;
            y = rest.y;
        }
    }
}

// A block: 16 rows per warp of one value head of one sequence.
template <int KS>
__global__ void __launch_bounds__(32 * kWarps, 2)
decode_chunks_tc_kernel(RunsArgs a, int row_blocks) {
    constexpr int DK = 16 * KS, LD = DK + 8;  // rows 16 bytes apart in their banks
    __shared__ __align__(16) __nv_bfloat16 tok[2][kTok][LD];  // k, q, channels as said above
    // decay and write strength per token
    __shared__ __align__(16) float al[kTok], be[kTok];
    // formed by warp 0
    struct __align__(16) Own {
        float A[kTok][kTok], P[kTok][kTok], tm[2][kTok][kTok];  // tm: T and M
        float nk[kTok], nq[kTok];                // 1 / |k|, 1 / |q|
        float ga[kTok], gb[kTok], cf[kTok];      // gamma / |k|, gamma / |q|, the decays behind / |k|
    };
    __shared__ Own my;
    __shared__ float gall;  // the product of the decays

    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int g = lane / 4, t = lane % 4;
    const int nh = blockIdx.x / row_blocks;
    const int n = nh / a.Hv, h = nh % a.Hv;
    const int t0 = a.cu ? a.cu[n] : n, t1 = a.cu ? a.cu[n + 1] : n + 1;
    const int slot = a.slots ? a.slots[n] : n;
    if (t0 < 0 || t1 > a.total || t0 >= t1) return;  // empty, or offsets that are none
    bool run = slot >= 0 && slot < a.n_slots;
    const int rows = blockDim.x / 2;  // 16 per warp
    const int row0 = blockIdx.x % row_blocks * rows;
    const int hk = h / (a.Hv / a.Hk);
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.k) + (long long)hk * DK;
    const __nv_bfloat16 *qp = a.q ? static_cast<const __nv_bfloat16 *>(a.q) + (long long)hk * DK : nullptr;
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(a.v) + (long long)h * a.Dv;
    __nv_bfloat16 *op = a.o ? static_cast<__nv_bfloat16 *>(a.o) + (long long)h * a.Dv : nullptr;
    const int r0 = row0 + warp * 16 + g, r1 = r0 + 8;  // this lane's rows
    const bool in0 = r0 < a.Dv, in1 = r1 < a.Dv;
    float *state = a.states + ((long long)(run ? slot : 0) * a.Hv + h) * a.Dv * DK + 4 * t;
    // piece i of the tokens from c0 on: 8 channels of a token's k or q
    const auto load_piece = [&](int c0, int i) {
        const int j = i / (2 * KS) % kTok, q = i / (2 * KS * kTok);
        if (c0 + j >= t1 || (q && !qp)) return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4 *>(
            (q ? qp + (c0 + j) * a.q_stride : kp + (c0 + j) * a.k_stride) + 8 * (i % (2 * KS)));
    };
    // v of this lane's rows and tokens
    const auto load_v = [&](int c0, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * t + i % 2;
            v[i] = run && c0 + j < t1 && (i < 2 ? in0 : in1)
                       ? to_f32(vp[(c0 + j) * a.v_stride + (i < 2 ? r0 : r1)]) : 0.f;
        }
    };
    // the first tokens' loads go ahead of the state's, which the tokens' products do not
    // wait for
    uint4 piece = make_uint4(0, 0, 0, 0);
    float v[4], g0 = 0.f, g1 = 0.f;
    if (run) {
        piece = load_piece(t0, tid);
        if (tid < kTok && t0 + tid < t1) {
            g0 = a.log_alpha[(t0 + tid) * a.la_stride + h];
            g1 = a.beta[(t0 + tid) * a.be_stride + h];
        }
    }
    load_v(t0, v);
    float4 s[2][KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        s[0][k] = run && in0 ? *reinterpret_cast<const float4 *>(state + r0 * DK + 16 * k)
                             : make_float4(0, 0, 0, 0);
        s[1][k] = run && in1 ? *reinterpret_cast<const float4 *>(state + r1 * DK + 16 * k)
                             : make_float4(0, 0, 0, 0);
    }

    for (int c0 = t0; c0 < t1; c0 += kTok) {
        const int m = min(kTok, t1 - c0);
        if (c0 > t0) {
            load_v(c0, v);
            __syncthreads();  // the arrays are written again
        }
        for (int i = tid; i < 2 * kTok * 2 * KS && run; i += blockDim.x) {
            const int j = i / (2 * KS) % kTok, at = i % (2 * KS), q = i / (2 * KS * kTok);
            const uint4 x = c0 == t0 && i == tid ? piece : load_piece(c0, i);
            uint32_t *to = reinterpret_cast<uint32_t *>(&tok[q][j][16 * (at / 2)]) + 2 * (at % 2);
            to[0] = x.x;
            to[4] = x.y;
            to[1] = x.z;
            to[5] = x.w;
        }
        if (tid < kTok && run) {
            if (c0 > t0 && tid < m) {
                g0 = a.log_alpha[(c0 + tid) * a.la_stride + h];
                g1 = a.beta[(c0 + tid) * a.be_stride + h];
            }
            const float2 gp = tid < m ? decay_pair(g0, g1, a.flags) : make_float2(1.f, 0.f);
            al[tid] = gp.x;
            be[tid] = gp.y;
        }
        if (c0 == t0) {
            // of the sequences with tokens that name one slot the first has it
            const int taken = run && a.update && a.slots
                                  ? slot_taken(a.slots, a.cu, a.total, n, slot, tid, blockDim.x) : 0;
            if (__syncthreads_or(taken)) run = false;
            if (!run) {  // a row of padding: its outputs are zero, nothing else is touched
                if (op)
                    for (int j = t0; j < t1; ++j)
                        for (int i = tid; i < rows && row0 + i < a.Dv; i += blockDim.x)
                            op[(long long)j * a.Hv * a.Dv + row0 + i] = from_f32<__nv_bfloat16>(0.f);
                return;
            }
        } else {
            __syncthreads();
        }
        // a lane's row of the tokens' tiles: k or q, first or second 8 of 16 channels
        const __nv_bfloat16 *tile = &tok[lane / 16][lane % 8][lane / 8 % 2 * 8];
        if (warp == 0) {
            float ck[4] = {}, cq[4] = {};  // [k; q] k^T, [k; q] q^T
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b[4];  // k first, k second, q first, q second
                ldmatrix4(b, tile + 16 * k);
                const uint32_t left[4] = {b[0], b[2], b[1], b[3]};
                mma16(ck, left, b[0], b[1]);
                mma16(cq, left, b[2], b[3]);
            }
            if (g / 2 == t) {
                my.nk[g] = a.flags & kFlagL2Norm ? rsqrtf((g % 2 ? ck[1] : ck[0]) + kNormEps) : 1.f;
                my.nq[g] = a.flags & kFlagL2Norm ? rsqrtf((g % 2 ? cq[3] : cq[2]) + kNormEps) : 1.f;
            }
            float dk[kTok];
            load8(al, dk);
            __syncwarp();
            const float nkg = my.nk[g], nqg = my.nq[g];
            // Gamma_gj and A_gj, P_gj of j = 2t + 1, then of 2t
            float dec = decay_between(dk, 2 * t + 2, g + 1);
#pragma unroll
            for (int e = 1; e >= 0; --e) {
                const int j = 2 * t + e;
                const float f = my.nk[j] * dec;
                my.A[g][j] = be[g] * nkg * f * ck[e];
                my.P[g][j] = nqg * f * ck[2 + e];
                if (e && j <= g) dec *= al[j];
            }
            // the decays up to token g (t = 0), behind it (t = 1), all (t = 2)
            const float run_of = decay_between(dk, t == 1 ? g + 1 : 0, t == 0 ? g + 1 : kTok);
            if (t == 0) {
                my.ga[g] = run_of * nkg;
                my.gb[g] = run_of * nqg;
            } else if (t == 1) {
                my.cf[g] = run_of * nkg;
            }
            if (lane == 2) gall = run_of;
            __syncwarp();
            solve_tokens(my.A, my.P, be, m, lane, my.tm);
        }
        // the rows' products with k and q, the state's three parts apart
        float ak[2][4] = {}, aq[2][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t b[4], p[4][3];
            ldmatrix4(b, tile + 16 * k);
            split3(s[0][k].x, s[0][k].y, p[0]);
            split3(s[1][k].x, s[1][k].y, p[1]);
            split3(s[0][k].z, s[0][k].w, p[2]);
            split3(s[1][k].z, s[1][k].w, p[3]);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const uint32_t left[4] = {p[0][i], p[1][i], p[2][i], p[3][i]};
                mma16(ak[i > 0], left, b[0], b[1]);
                mma16(aq[i > 0], left, b[2], b[3]);
            }
        }
        __syncthreads();  // T and M are there
        // r of this lane's rows and tokens, then of its rows and all tokens
        float r[4], all[2][kTok];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = v[i] - my.ga[2 * t + i % 2] * (ak[0][i] + ak[1][i]);
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
            all[0][j] = __shfl_sync(0xffffffffu, r[j % 2], lane / 4 * 4 + j / 2);
            all[1][j] = __shfl_sync(0xffffffffu, r[2 + j % 2], lane / 4 * 4 + j / 2);
        }
        const bool write = a.update || c0 + kTok < t1;
        float u[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * t + e;
            float T[kTok], M[kTok];
#pragma unroll
            for (int j = 0; j < kTok; j += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&my.tm[0][i][j]);
                const float4 y = *reinterpret_cast<const float4 *>(&my.tm[1][i][j]);
                T[j] = x.x; T[j + 1] = x.y; T[j + 2] = x.z; T[j + 3] = x.w;
                M[j] = y.x; M[j + 1] = y.y; M[j + 2] = y.z; M[j + 3] = y.w;
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float uu = 0.f, out = my.gb[i] * (aq[0][2 * w + e] + aq[1][2 * w + e]);
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (j <= i) {  // what a later token holds stays out
                        uu += T[j] * all[w][j];
                        out += M[j] * all[w][j];
                    }
                u[2 * w + e] = i < m ? my.cf[i] * uu : 0.f;
                if (op && i < m && (w ? in1 : in0))
                    op[(long long)(c0 + i) * a.Hv * a.Dv + (w ? r1 : r0)] = from_f32<__nv_bfloat16>(out);
            }
        }
        if (write) {
            uint32_t p0[3], p1[3];
            split3(u[0], u[1], p0);
            split3(u[2], u[3], p1);
            const float2 g2 = make_float2(gall, gall);
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t b[4];  // 8 channels each: first, second of k, first, second of k + 1
                ldmatrix4_trans(b, &tok[0][lane % 8][16 * k + lane / 8 * 8]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4 &x = s[0][k + e], &y = s[1][k + e];
                    const float2 xl = __fmul2_rn(make_float2(x.x, x.y), g2);
                    const float2 xh = __fmul2_rn(make_float2(x.z, x.w), g2);
                    const float2 yl = __fmul2_rn(make_float2(y.x, y.y), g2);
                    const float2 yh = __fmul2_rn(make_float2(y.z, y.w), g2);
                    x = make_float4(xl.x, xl.y, xh.x, xh.y);
                    y = make_float4(yl.x, yl.y, yh.x, yh.y);
#pragma unroll
                    for (int i = 2; i >= 0; --i) {  // the small parts first
                        mma8(x.x, x.y, y.x, y.y, p0[i], p1[i], b[2 * e]);
                        mma8(x.z, x.w, y.z, y.w, p0[i], p1[i], b[2 * e + 1]);
                    }
                }
            }
        }
    }
    if (!a.update) return;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        if (in0) *reinterpret_cast<float4 *>(state + r0 * DK + 16 * k) = s[0][k];
        if (in1) *reinterpret_cast<float4 *>(state + r1 * DK + 16 * k) = s[1][k];
    }
}

}  // namespace

bool runs_tc_supported(const RunsArgs &a) {
    return (a.Dk == 64 || a.Dk == 128) && a.k_stride % 8 == 0 && a.q_stride % 8 == 0;
}

cudaError_t launch_decode_runs_tc(const RunsArgs &a, cudaStream_t st) {
    const int warps = a.Dv > 16 * (kWarps - 1) ? kWarps : (a.Dv + 15) / 16;
    const int row_blocks = (a.Dv + 16 * warps - 1) / (16 * warps);
    const unsigned blocks = (unsigned)((long long)a.N * a.Hv * row_blocks);
    if (a.Dk == 64) decode_chunks_tc_kernel<4><<<blocks, 32 * warps, 0, st>>>(a, row_blocks);
    else decode_chunks_tc_kernel<8><<<blocks, 32 * warps, 0, st>>>(a, row_blocks);
    return cudaPeekAtLastError();
}

}  // namespace gdn
