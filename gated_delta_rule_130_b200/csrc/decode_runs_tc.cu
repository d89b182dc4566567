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
// with its round trip through tensor memory; what bounds the kernel is the issue of the
// splitting (9 instructions per two elements) beside the state's loads.
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
    __shared__ __align__(16) float tm[2][kTok][kTok];  // T and M, rows of later tokens
    __shared__ float sA[kTok][kTok], sP[kTok][kTok];
    // per token: decay, write strength, 1 / |k|, 1 / |q|; gamma / |k|, gamma / |q|, and
    // the decays behind it / |k|; last: gamma of all
    __shared__ float al[kTok], be[kTok], nk[kTok], nq[kTok], ga[kTok], gb[kTok], cf[kTok], gall;

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
        float v[4];  // v of this lane's rows and tokens, needed last
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * t + i % 2;
            v[i] = run && j < m && (i < 2 ? in0 : in1)
                       ? to_f32(vp[(c0 + j) * a.v_stride + (i < 2 ? r0 : r1)]) : 0.f;
        }
        if (c0 > t0) __syncthreads();  // the arrays are written again
        for (int i = tid; i < 2 * kTok * 2 * KS && run; i += blockDim.x) {  // 8 channels each
            const int j = i / (2 * KS) % kTok, piece = i % (2 * KS), q = i / (2 * KS * kTok);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (j < m && (!q || qp))
                x = *reinterpret_cast<const uint4 *>(
                    (q ? qp + (c0 + j) * a.q_stride : kp + (c0 + j) * a.k_stride) + 8 * piece);
            uint32_t *to = reinterpret_cast<uint32_t *>(&tok[q][j][16 * (piece / 2)]) + 2 * (piece % 2);
            to[0] = x.x;
            to[4] = x.y;
            to[1] = x.z;
            to[5] = x.w;
        }
        if (tid < kTok && run) {
            float2 gp = make_float2(1.f, 0.f);
            if (tid < m)
                gp = decay_pair(a.log_alpha[(c0 + tid) * a.la_stride + h],
                                a.beta[(c0 + tid) * a.be_stride + h], a.flags);
            al[tid] = gp.x;
            be[tid] = gp.y;
        }
        if (c0 == t0) {
            // of the sequences with tokens that name one slot the first has it
            const int taken = run && a.update && a.slots
                                  ? slot_taken(a, n, slot, tid, blockDim.x) : 0;
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
                nk[g] = a.flags & kFlagL2Norm ? rsqrtf((g % 2 ? ck[1] : ck[0]) + kNormEps) : 1.f;
                nq[g] = a.flags & kFlagL2Norm ? rsqrtf((g % 2 ? cq[3] : cq[2]) + kNormEps) : 1.f;
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // A_gj and P_gj, j = 2t + e
                const int j = 2 * t + e;
                float dec = nk[j];
#pragma unroll
                for (int l = 1; l < kTok; ++l)
                    if (l > j && l <= g) dec *= al[l];
                if (j < g) sA[g][j] = be[g] * nk[g] * dec * ck[e];
                if (j <= g) sP[g][j] = nq[g] * dec * ck[2 + e];
            }
            if (lane < kTok) {
                float x = 1.f, y = 1.f;
#pragma unroll
                for (int l = 0; l < kTok; ++l) {
                    if (l <= lane) x *= al[l];
                    else y *= al[l];  // 1 behind the last token
                }
                ga[lane] = x * nk[lane];
                gb[lane] = x * nq[lane];
                cf[lane] = y * nk[lane];
                if (lane == kTok - 1) gall = x;
            }
            __syncwarp();
            // column j of T = (I + A)^-1 diag(beta), then of M = P T
            const int j = lane % kTok;
            float x[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                x[i] = i == j ? 1.f : 0.f;
#pragma unroll
                for (int l = 0; l < i; ++l)
                    if (l >= j) x[i] -= sA[i][l] * x[l];
            }
            const float b = be[j];
            for (int i = g / 2; i < kTok; i += 4) {
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
        // the rows' products with k and q, the state's three parts apart
        float ak[3][4] = {}, aq[3][4] = {};
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
                mma16(ak[i], left, b[0], b[1]);
                mma16(aq[i], left, b[2], b[3]);
            }
        }
        __syncthreads();  // T and M are there
        // r of this lane's rows and tokens, then of its rows and all tokens
        float r[4], all[2][kTok];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = v[i] - ga[2 * t + i % 2] * (ak[0][i] + (ak[1][i] + ak[2][i]));
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
                const float4 x = *reinterpret_cast<const float4 *>(&tm[0][i][j]);
                const float4 y = *reinterpret_cast<const float4 *>(&tm[1][i][j]);
                T[j] = x.x; T[j + 1] = x.y; T[j + 2] = x.z; T[j + 3] = x.w;
                M[j] = y.x; M[j + 1] = y.y; M[j + 2] = y.z; M[j + 3] = y.w;
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float uu = 0.f, out = gb[i] * (aq[0][2 * w + e] + (aq[1][2 * w + e] + aq[2][2 * w + e]));
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (j <= i) {  // what a later token holds stays out
                        uu += T[j] * all[w][j];
                        out += M[j] * all[w][j];
                    }
                u[2 * w + e] = i < m ? cf[i] * uu : 0.f;
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
