// C-ABI entry points of the operators around the rule (declared in include/gdn.h):
// argument checks on the host, then dispatch to the kernels.  Nothing is launched
// when a check fails, and the library allocates nothing.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/gdn.h"
#include "kernels.h"

namespace {

constexpr int kMaxSeqs = 65535, kMaxTokens = 1 << 30, kMaxHeads = 65535, kMaxNormD = 1 << 20, kMaxChannels = 1 << 24;
// (rows - 1) * stride + width, in bytes, stays inside size_t for 2^31 rows
constexpr long long kMaxStride = 1ll << 30, kMaxBlocks = 0x7fffffffll, kMaxPool = 1ll << 40;

// Bytes [p, p + n) that a call reads or writes.
struct Span {
    const void *p;
    size_t n;
};
bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}
// A strided tensor: `rows` rows of `width` elements, `stride` apart.
Span strided(const void *p, long long rows, long long stride, long long width, size_t elem) {
    return Span{p, rows ? (size_t)((rows - 1) * stride + width) * elem : 0};
}
bool stride_ok(long long stride, long long width) { return stride >= width && stride <= kMaxStride; }
bool dtype_ok(gdn_dtype_t d) { return d == GDN_F32 || d == GDN_BF16; }
size_t size_of(gdn_dtype_t d) { return d == GDN_BF16 ? 2 : 4; }
gdn_status_t status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Offsets and slots of a packed batch.
gdn_status_t check_seqs(const int *slots, const int *cu, int N, int total) {
    if (N < 0 || total < 0) return GDN_ERR_INVALID_ARG;
    if (N > kMaxSeqs || total > kMaxTokens) return GDN_ERR_UNSUPPORTED;
    if (!cu && N != total) return GDN_ERR_INVALID_ARG;
    if ((slots && !aligned(slots, 16)) || (cu && !aligned(cu, 16))) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}
Span ints(const int *p, long long n) { return Span{p, (size_t)n * sizeof(int)}; }

// The arrays that share the channels of a convolution's y or dy.
gdn_status_t check_parts(const void *const *part, const long long *strides, const int *begin,
                         int parts, int C) {
    if (parts < 1 || parts > gdn::kConvParts || !part || !strides || !begin)
        return GDN_ERR_INVALID_ARG;
    if (begin[0] != 0 || begin[parts] != C) return GDN_ERR_INVALID_ARG;
    for (int p = 0; p < parts; ++p) {
        if (begin[p] < 0 || begin[p + 1] <= begin[p] || begin[p + 1] > C || !part[p] ||
            !aligned(part[p], 16) || !stride_ok(strides[p], begin[p + 1] - begin[p]))
            return GDN_ERR_INVALID_ARG;
    }
    return GDN_OK;
}

gdn_status_t check_conv(const int *slots, const int *cu, int N, int total, int C, int W,
                        long long x_stride, gdn_dtype_t dtype, gdn_dtype_t param_dtype) {
    if (C <= 0 || W <= 0 || !dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
    if (param_dtype != GDN_F32 && param_dtype != dtype) return GDN_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || C > kMaxChannels) return GDN_ERR_UNSUPPORTED;
    if (total > 0 && ((long long)C + 127) / 128 * total > kMaxBlocks) return GDN_ERR_UNSUPPORTED;
    if (!stride_ok(x_stride, C)) return GDN_ERR_INVALID_ARG;
    return check_seqs(slots, cu, N, total);
}

gdn_status_t check_norm(int tokens, int heads, int D, float eps, gdn_dtype_t dtype,
                        gdn_dtype_t param_dtype) {
    if (tokens < 0 || heads < 0 || D <= 0 || !dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
    if (param_dtype != GDN_F32 && param_dtype != dtype) return GDN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || isinf(eps)) return GDN_ERR_INVALID_ARG;
    if (D > kMaxNormD || (long long)tokens * heads > kMaxTokens) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_decode_runs(const void *q, const void *k, const void *v, const float *log_alpha,
                             const float *beta, float *states, const int *slots,
                             const int *cu_seqlens, void *o, int N, int total, int Hk, int Hv,
                             int Dk, int Dv, int n_slots, long long q_stride, long long k_stride,
                             long long v_stride, long long log_alpha_stride, long long beta_stride,
                             gdn_dtype_t dtype, unsigned flags, void *stream) {
    if (Hk < 0 || Hv < 0 || Dk <= 0 || Dv <= 0 || n_slots < 0 || !dtype_ok(dtype))
        return GDN_ERR_INVALID_ARG;
    if (flags & ~(GDN_FLAG_L2NORM_QK | GDN_FLAG_GATE_LOGITS | GDN_FLAG_READ_ONLY))
        return GDN_ERR_INVALID_ARG;
    if (Dk > 256 || Dv > 512 || Hv > kMaxHeads) return GDN_ERR_UNSUPPORTED;
    const gdn_status_t seqs = check_seqs(slots, cu_seqlens, N, total);
    if (seqs != GDN_OK) return seqs;
    if ((long long)N * Hv * Dv > kMaxBlocks || (long long)n_slots * Hv > kMaxPool) return GDN_ERR_UNSUPPORTED;
    if (N == 0 || total == 0 || Hv == 0) return GDN_OK;
    if (Hk == 0 || Hv % Hk) return GDN_ERR_INVALID_ARG;
    if (!k || !v || !log_alpha || !beta || !states || (o && !q)) return GDN_ERR_INVALID_ARG;
    if (!stride_ok(k_stride, (long long)Hk * Dk) || !stride_ok(v_stride, (long long)Hv * Dv) ||
        (q && !stride_ok(q_stride, (long long)Hk * Dk)) || !stride_ok(log_alpha_stride, Hv) ||
        !stride_ok(beta_stride, Hv))
        return GDN_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)states, (const void *)o})
        if (p && !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(log_alpha, 4) || !aligned(beta, 4)) return GDN_ERR_INVALID_ARG;
    const size_t esz = size_of(dtype);
    const Span in[] = {strided(q, total, q_stride, (long long)Hk * Dk, esz),
                       strided(k, total, k_stride, (long long)Hk * Dk, esz),
                       strided(v, total, v_stride, (long long)Hv * Dv, esz),
                       strided(log_alpha, total, log_alpha_stride, Hv, 4),
                       strided(beta, total, beta_stride, Hv, 4),
                       ints(slots, N), ints(cu_seqlens, (long long)N + 1)};
    const Span out{o, (size_t)total * Hv * Dv * esz};
    const Span pool{states, (size_t)n_slots * Hv * Dv * Dk * sizeof(float)};
    for (const Span &s : in)
        if (overlap(s, out) || (!(flags & GDN_FLAG_READ_ONLY) && overlap(s, pool)))
            return GDN_ERR_INVALID_ARG;
    if (overlap(out, pool)) return GDN_ERR_INVALID_ARG;
    gdn::RunsArgs a{q, k, v, log_alpha, beta, states, slots, cu_seqlens, o, N, total, Hk, Hv, Dk,
                    Dv, n_slots, q_stride, k_stride, v_stride, log_alpha_stride, beta_stride,
                    flags & ~GDN_FLAG_READ_ONLY, !(flags & GDN_FLAG_READ_ONLY)};
    return status(gdn::launch_decode_runs(a, dtype == GDN_BF16, static_cast<cudaStream_t>(stream)));
}

gdn_status_t gdn_short_conv_fwd(const void *x, const void *weight, const void *bias, void *states,
                                const int *slots, const int *cu_seqlens, void *const *y,
                                const long long *part_strides, const int *part_begin, int parts,
                                int N, int total, int C, int W, int n_slots, long long x_stride,
                                int silu, gdn_dtype_t dtype, gdn_dtype_t param_dtype,
                                void *stream) {
    gdn_status_t st = check_conv(slots, cu_seqlens, N, total, C, W, x_stride, dtype, param_dtype);
    if (st != GDN_OK) return st;
    if (n_slots < 0) return GDN_ERR_INVALID_ARG;
    if (N == 0 || total == 0) return GDN_OK;
    st = check_parts(y, part_strides, part_begin, parts, C);
    if (st != GDN_OK) return st;
    if (!x || !weight) return GDN_ERR_INVALID_ARG;
    for (const void *p : {x, weight, bias, (const void *)states})
        if (p && !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    const size_t esz = size_of(dtype), psz = size_of(param_dtype);
    const Span pool{states, (size_t)n_slots * (W - 1) * C * esz};
    const Span in[] = {strided(x, total, x_stride, C, esz), Span{weight, (size_t)C * W * psz},
                       Span{bias, (size_t)C * psz}, ints(slots, N),
                       ints(cu_seqlens, (long long)N + 1)};
    gdn::ConvArgs a{};
    for (int p = 0; p < parts; ++p) {
        const Span out = strided(y[p], total, part_strides[p], part_begin[p + 1] - part_begin[p], esz);
        for (const Span &s : in)
            if (overlap(s, out)) return GDN_ERR_INVALID_ARG;
        if (overlap(out, pool)) return GDN_ERR_INVALID_ARG;
        // parts may be column slices of one array: the same stride, side by side
        for (int r = 0; r < p; ++r) {
            const Span other =
                strided(y[r], total, part_strides[r], part_begin[r + 1] - part_begin[r], esz);
            if (!overlap(out, other)) continue;
            const long long d = (static_cast<const char *>(y[p]) - static_cast<const char *>(y[r])) /
                                (long long)esz;
            const long long wr = part_begin[r + 1] - part_begin[r];
            const long long wp = part_begin[p + 1] - part_begin[p];
            const long long s = part_strides[p];
            const bool apart = part_strides[r] == s &&
                               ((d >= wr && d + wp <= s) || (-d >= wp && -d + wr <= s));
            if (!apart) return GDN_ERR_INVALID_ARG;
        }
        a.part[p] = y[p];
        a.part_stride[p] = part_strides[p];
    }
    for (const Span &s : in)
        if (overlap(s, pool)) return GDN_ERR_INVALID_ARG;
    for (int p = 0; p <= parts; ++p) a.begin[p] = part_begin[p];
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.states = states;
    a.slots = states ? slots : nullptr;
    a.cu = cu_seqlens;
    a.N = N;
    a.total = total;
    a.C = C;
    a.W = W;
    a.n_slots = n_slots;
    a.parts = parts;
    a.x_stride = x_stride;
    a.weight_f32 = param_dtype == GDN_F32;
    a.silu = silu != 0;
    return status(gdn::launch_short_conv_fwd(a, dtype == GDN_BF16, static_cast<cudaStream_t>(stream)));
}

size_t gdn_short_conv_bwd_workspace_size(int total, int C, int W) {
    if (total <= 0 || total > kMaxTokens || C <= 0 || C > kMaxChannels || W < 2 || W > 4) return 0;
    return gdn::short_conv_bwd_bytes(total, C, W);
}

gdn_status_t gdn_short_conv_bwd(const void *const *dy, const long long *part_strides,
                                const int *part_begin, int parts, const void *x,
                                const void *weight, const void *bias, const int *cu_seqlens,
                                void *dx, float *dweight, float *dbias, int N, int total, int C,
                                int W, long long x_stride, int silu, gdn_dtype_t dtype,
                                gdn_dtype_t param_dtype, void *workspace, size_t workspace_bytes,
                                void *stream) {
    gdn_status_t st = check_conv(nullptr, cu_seqlens, N, total, C, W, x_stride, dtype, param_dtype);
    if (st != GDN_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!dweight || !aligned(dweight, 16) || (dbias && !aligned(dbias, 16)))
        return GDN_ERR_INVALID_ARG;
    const size_t esz = size_of(dtype), psz = size_of(param_dtype);
    const Span dws{dweight, (size_t)C * W * sizeof(float)}, dbs{dbias, (size_t)C * sizeof(float)};
    const Span dxs{dx, (size_t)total * C * esz};
    if (overlap(dws, dbs)) return GDN_ERR_INVALID_ARG;
    if (total == 0 || N == 0) {  // no tokens in a sequence: every gradient is zero
        if (total && (!dx || !aligned(dx, 16) || overlap(dxs, dws) || overlap(dxs, dbs)))
            return GDN_ERR_INVALID_ARG;
        cudaError_t e = cudaMemsetAsync(dweight, 0, dws.n, cs);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, dbs.n, cs);
        if (e == cudaSuccess && total) e = cudaMemsetAsync(dx, 0, dxs.n, cs);
        return status(e);
    }
    st = check_parts(dy, part_strides, part_begin, parts, C);
    if (st != GDN_OK) return st;
    if (!x || !weight || !dx || !workspace) return GDN_ERR_INVALID_ARG;
    for (const void *p : {x, weight, bias, (const void *)dx, (const void *)workspace})
        if (p && !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn::short_conv_bwd_bytes(total, C, W);
    if (workspace_bytes < need) return GDN_ERR_INVALID_ARG;
    const Span ws{workspace, need};
    const Span out[] = {dxs, dws, dbs, ws};
    Span in[4 + gdn::kConvParts] = {strided(x, total, x_stride, C, esz),
                                    Span{weight, (size_t)C * W * psz}, Span{bias, (size_t)C * psz},
                                    ints(cu_seqlens, (long long)N + 1)};
    gdn::ConvArgs a{};
    for (int p = 0; p < parts; ++p) {
        in[4 + p] = strided(dy[p], total, part_strides[p], part_begin[p + 1] - part_begin[p], esz);
        a.part[p] = const_cast<void *>(dy[p]);
        a.part_stride[p] = part_strides[p];
    }
    for (int i = 0; i < 4; ++i) {
        for (int k = 0; k < 4 + parts; ++k)
            if (overlap(out[i], in[k])) return GDN_ERR_INVALID_ARG;
        for (int k = i + 1; k < 4; ++k)
            if (overlap(out[i], out[k])) return GDN_ERR_INVALID_ARG;
    }
    for (int p = 0; p <= parts; ++p) a.begin[p] = part_begin[p];
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.cu = cu_seqlens;
    a.dx = dx;
    a.dw = dweight;
    a.db = dbias;
    a.partial = static_cast<float *>(workspace);
    a.N = N;
    a.total = total;
    a.C = C;
    a.W = W;
    a.parts = parts;
    a.x_stride = x_stride;
    a.weight_f32 = param_dtype == GDN_F32;
    a.silu = silu != 0;
    return status(gdn::launch_short_conv_bwd(a, dtype == GDN_BF16, cs));
}

gdn_status_t gdn_rms_norm_fwd(const void *x, const void *weight, const void *residual,
                              const void *gate, void *y, float *scale, void *h_out, int tokens,
                              int heads, int D, int quant_group, long long x_stride,
                              long long residual_stride, long long gate_stride, float eps,
                              gdn_dtype_t dtype, gdn_dtype_t param_dtype, void *stream) {
    const gdn_status_t st = check_norm(tokens, heads, D, eps, dtype, param_dtype);
    if (st != GDN_OK) return st;
    if (quant_group < 0) return GDN_ERR_INVALID_ARG;
    if (quant_group && quant_group != D && !(quant_group == 128 && D % 128 == 0))
        return GDN_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0) return GDN_OK;
    if (!x || !weight || !y || (quant_group && !scale)) return GDN_ERR_INVALID_ARG;
    const long long width = (long long)heads * D;
    if (!stride_ok(x_stride, width) || (residual && !stride_ok(residual_stride, width)) ||
        (gate && !stride_ok(gate_stride, width)))
        return GDN_ERR_INVALID_ARG;
    for (const void *p : {x, weight, residual, gate, (const void *)y, (const void *)scale,
                          (const void *)h_out})
        if (p && !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    const size_t esz = size_of(dtype), n = (size_t)tokens * width;
    const Span xs = strided(x, tokens, x_stride, width, esz);
    const Span rs = strided(residual, tokens, residual_stride, width, esz);
    const Span gs = strided(gate, tokens, gate_stride, width, esz);
    const Span wsp{weight, (size_t)D * size_of(param_dtype)};
    const Span ys{y, n * (quant_group ? 1 : esz)}, hs{h_out, n * esz};
    const Span ss{quant_group ? scale : nullptr, quant_group ? n / quant_group * sizeof(float) : 0};
    // in place: each element is read and written by one thread
    const bool y_is_x = !quant_group && y == x && x_stride == width && !residual && !h_out;
    const bool h_is_x = h_out && h_out == x && x_stride == width;
    const bool h_is_r = h_out && h_out == residual && residual_stride == width;
    if ((!y_is_x && overlap(ys, xs)) || overlap(ys, rs) || overlap(ys, gs) || overlap(ys, wsp) ||
        overlap(ys, hs) || overlap(ys, ss) || (!h_is_x && overlap(hs, xs)) ||
        (!h_is_r && overlap(hs, rs)) || overlap(hs, gs) || overlap(hs, wsp) || overlap(hs, ss) ||
        overlap(ss, xs) || overlap(ss, rs) || overlap(ss, gs) || overlap(ss, wsp))
        return GDN_ERR_INVALID_ARG;
    gdn::NormArgs a{};
    a.x = x;
    a.weight = weight;
    a.residual = residual;
    a.gate = gate;
    a.y = y;
    a.h = h_out;
    a.scale = scale;
    a.rows = tokens * heads;
    a.H = heads;
    a.D = D;
    a.group = quant_group;
    a.x_stride = x_stride;
    a.res_stride = residual_stride;
    a.gate_stride = gate_stride;
    a.eps = eps;
    a.weight_f32 = param_dtype == GDN_F32;
    return status(gdn::launch_rms_norm_fwd(a, dtype == GDN_BF16, static_cast<cudaStream_t>(stream)));
}

size_t gdn_rms_norm_bwd_workspace_size(int tokens, int heads, int D) {
    if (check_norm(tokens, heads, D, 0.f, GDN_F32, GDN_F32) != GDN_OK || !tokens || !heads) return 0;
    return gdn::rms_norm_bwd_bytes(tokens * heads, D);
}

gdn_status_t gdn_rms_norm_bwd(const void *dy, const void *x, const void *weight, const void *gate,
                              const void *d_res, void *dx, float *dweight, void *dgate, int tokens,
                              int heads, int D, long long dy_stride, long long x_stride,
                              long long gate_stride, long long d_res_stride, float eps,
                              gdn_dtype_t dtype, gdn_dtype_t param_dtype, void *workspace,
                              size_t workspace_bytes, void *stream) {
    const gdn_status_t st = check_norm(tokens, heads, D, eps, dtype, param_dtype);
    if (st != GDN_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!dweight || !aligned(dweight, 16)) return GDN_ERR_INVALID_ARG;
    if (tokens == 0 || heads == 0)
        return status(cudaMemsetAsync(dweight, 0, (size_t)D * sizeof(float), cs));
    if (!dy || !x || !weight || !dx || !workspace || !gate != !dgate) return GDN_ERR_INVALID_ARG;
    const long long width = (long long)heads * D;
    if (!stride_ok(dy_stride, width) || !stride_ok(x_stride, width) ||
        (gate && !stride_ok(gate_stride, width)) || (d_res && !stride_ok(d_res_stride, width)))
        return GDN_ERR_INVALID_ARG;
    for (const void *p : {dy, x, weight, gate, d_res, (const void *)dx, (const void *)dgate,
                          (const void *)workspace})
        if (p && !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    const size_t esz = size_of(dtype), n = (size_t)tokens * width;
    const size_t need = gdn::rms_norm_bwd_bytes(tokens * heads, D);
    if (workspace_bytes < need) return GDN_ERR_INVALID_ARG;
    const Span in[] = {strided(dy, tokens, dy_stride, width, esz),
                       strided(x, tokens, x_stride, width, esz),
                       Span{weight, (size_t)D * size_of(param_dtype)},
                       strided(gate, tokens, gate_stride, width, esz),
                       strided(d_res, tokens, d_res_stride, width, esz)};
    const Span out[] = {Span{dx, n * esz}, Span{dweight, (size_t)D * sizeof(float)},
                        Span{dgate, n * esz}, Span{workspace, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s)) return GDN_ERR_INVALID_ARG;
        for (int k = i + 1; k < 4; ++k)
            if (overlap(out[i], out[k])) return GDN_ERR_INVALID_ARG;
    }
    gdn::NormArgs a{};
    a.x = x;
    a.weight = weight;
    a.gate = gate;
    a.dy = dy;
    a.d_res = d_res;
    a.dx = dx;
    a.dgate = dgate;
    a.dw = dweight;
    a.partial = static_cast<float *>(workspace);
    a.rows = tokens * heads;
    a.H = heads;
    a.D = D;
    a.x_stride = x_stride;
    a.gate_stride = gate_stride;
    a.dy_stride = dy_stride;
    a.dres_stride = d_res_stride;
    a.eps = eps;
    a.weight_f32 = param_dtype == GDN_F32;
    return status(gdn::launch_rms_norm_bwd(a, dtype == GDN_BF16, cs));
}

}  // extern "C"
