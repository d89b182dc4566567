"""Float64 forms of the operators around the rule, token by token on the CPU, and the
bounds that the kernels' results are held to.

Bounds.  A result rounded to a type is off by at most half a step of it, u = eps / 2
(bf16 2^-8, float32 2^-24), relative to its value.  Before that everything is float32;
a sum of n terms in a tree of lanes and a short chain per lane is off by at most about
(n / lanes + log2(lanes) + 2) u32 of the sum of its terms' magnitudes.  ``close`` holds
every element to  u |ref| + c u32 scale,  scale being the sum of magnitudes behind it and c
the number of float32 roundings on the longest way to it.
"""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U32 = 2.0 ** -24
EPS = 1e-6


def close(x, ref, scale, roundings):
    """Whether x (a kernel's) is within u |ref| + roundings u32 scale of ref, elementwise, NaN
    and infinities being where ref has them."""
    x, ref, u = x.detach().cpu(), ref.double().cpu(), U[x.dtype]
    assert x.shape == ref.shape, (x.shape, ref.shape)
    x = x.double()
    same = (x == ref) | (x.isnan() & ref.isnan())
    off = (x - ref).abs()
    bound = u * ref.abs() * 1.001 + roundings * U32 * torch.as_tensor(scale, dtype=torch.float64).cpu()
    bad = ~(same | (off <= bound))
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{x[tuple(i)]} for {ref[tuple(i)]}; worst {float((off / bound.clamp_min(1e-300))[bad].max()):.3g} bounds")
    return True


def spans(cu, total):
    """The sequences' (n, start, end) that offsets describe."""
    if cu is None:
        return [(n, n, n + 1) for n in range(total)]
    return [(n, a, b) for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])) if 0 <= a < b <= total]


def live(seqs, slots, n_slots, update=True):
    """{n: slot} of the sequences that run: a slot in range and, where states are written,
    named by no earlier sequence."""
    got = {}
    for n, a, b in seqs:
        s = n if slots is None else slots[n]
        if 0 <= s < n_slots and not (update and slots is not None and s in got.values()):
            got[n] = s
    return got


def runs(q, k, v, la, be, states, slots, cu, out, update=True, l2norm=False, logits=False):
    """(o, states, scale of o, scale of the states) of decode_runs in float64."""
    q, k, v, la, be = (t.double().cpu() for t in (q, k, v, la, be))
    S, o = states.double().cpu().clone(), out.double().cpu().clone()
    total, Hv = v.shape[0], v.shape[1]
    group = Hv // k.shape[1]
    if l2norm:
        q = q / (q.pow(2).sum(-1, keepdim=True) + EPS).sqrt()
        k = k / (k.pow(2).sum(-1, keepdim=True) + EPS).sqrt()
    if logits:
        la, be = -(la.clamp_min(0) + torch.log1p(torch.exp(-la.abs()))), torch.sigmoid(be)
    os, Ss = torch.zeros_like(o), torch.zeros_like(S)
    seqs = spans(cu, total)
    names = live(seqs, slots, S.shape[0], update)
    for n, a, b in seqs:
        if n not in names:
            o[a:b] = 0
            continue
        for h in range(Hv):
            X = S[names[n], h].clone()
            M = X.abs()  # magnitudes behind the elements of X
            for t in range(a, b):
                kk, qq, al = k[t, h // group], q[t, h // group], torch.exp(la[t, h])
                X = al * X
                M = al * M
                u = be[t, h] * (v[t, h] - X @ kk)
                m = be[t, h].abs() * (v[t, h].abs() + M @ kk.abs())
                X = X + torch.outer(u, kk)
                M = M + torch.outer(m, kk.abs())
                o[t, h] = X @ qq
                os[t, h] = M @ qq.abs()
            if update:
                S[names[n], h], Ss[names[n], h] = X, M
    return o, S, os, Ss


def conv(x, w, bias, cu, states, slots, silu):
    """(y, states, scale) of short_conv_fwd in float64; y is None-like 0 outside sequences and
    `covered` says which rows belong to one."""
    x64, w64 = x.double().cpu(), w.double().cpu()
    total, C = x64.shape
    W = w64.shape[1]
    y, sc = torch.zeros(total, C, dtype=torch.float64), torch.zeros(total, C, dtype=torch.float64)
    covered = torch.zeros(total, dtype=torch.bool)
    S = states.double().cpu().clone() if states is not None else None
    seqs = spans(cu, total)
    names = live(seqs, slots, S.shape[0]) if S is not None else {n: None for n, _, _ in seqs}
    for n, a, b in seqs:
        covered[a:b] = True
        if n not in names:
            continue
        head = S[names[n]] if S is not None else torch.zeros(W - 1, C, dtype=torch.float64)
        p = torch.cat([head, x64[a:b]])
        win = p.unfold(0, W, 1)
        z, m = (win * w64).sum(-1), (win.abs() * w64.abs()).sum(-1)
        if bias is not None:
            z, m = z + bias.double().cpu(), m + bias.double().cpu().abs()
        y[a:b], sc[a:b] = (z * torch.sigmoid(z) if silu else z), m
        if S is not None:
            S[names[n]] = p[-(W - 1):]
    return y, S, sc, covered


def conv_grads(dy, x, w, bias, cu, silu):
    """(dx, dw, db) and their scales, by hand from the formulas, in float64."""
    x, w, dy = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    total, C = x.shape
    W = w.shape[1]
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros(C, dtype=torch.float64)
    sx, sw, sb = dx.clone(), dw.clone(), db.clone()
    for n, a, b in spans(cu, total):
        p = torch.cat([torch.zeros(W - 1, C, dtype=torch.float64), x[a:b]])
        win = p.unfold(0, W, 1)
        d = dy[a:b].clone()
        m = d.abs()
        if silu:
            z = (win * w).sum(-1) + (bias.double().cpu() if bias is not None else 0)
            zm = (win.abs() * w.abs()).sum(-1) + 1
            sig = torch.sigmoid(z)
            d = d * sig * (1 + z * (1 - sig))
            m = m * (1 + zm)
        g, gm = torch.zeros_like(p), torch.zeros_like(p)
        for j in range(W):
            g[j:j + b - a] += w[:, j] * d
            gm[j:j + b - a] += w[:, j].abs() * m
            dw[:, j] += (p[j:j + b - a] * d).sum(0)
            sw[:, j] += (p[j:j + b - a].abs() * m).sum(0)
        dx[a:b], sx[a:b] = g[W - 1:], gm[W - 1:]
        db += d.sum(0)
        sb += m.sum(0)
    return dx, dw, db, sx, sw, sb


def norm(x, w, residual, gate, eps):
    """(y, h) of rms_norm_fwd in float64, h rounded to x's type as the operator defines it."""
    h = x if residual is None else (x.double().cpu() + residual.double().cpu()).to(x.dtype)
    f = h.double().cpu()
    y = f / (f.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()
    if gate is not None:
        g = gate.double().cpu()
        y = y * (g * torch.sigmoid(g))
    return y, h


def norm_grads(dy, x, w, gate, d_res, eps):
    """(dx, dw, dgate) in float64 from the formulas, and the scales of the three.  silu'(g) =
    sig (1 + g (1 - sig)) has a zero near g = -1.278, where 1 and g (1 - sig) cancel: a
    rounding of either is u32 of 1 + |g| (1 - sig), not of their sum, so dgate's scale
    has that factor in its place."""
    x, w, dy = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    rstd = 1 / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n, dn, dgate, sg = x * rstd, dy, None, None
    if gate is not None:
        g = gate.double().cpu()
        sig = torch.sigmoid(g)
        dgate = dy * n * w * sig * (1 + g * (1 - sig))
        sg = (dy * n * w).abs() * sig * (1 + g.abs() * (1 - sig))
        dn = dy * g * sig
    dx = rstd * (w * dn) - x * rstd.pow(3) * (w * dn * x).mean(-1, keepdim=True)
    sx = rstd * ((w * dn).abs() + n.abs() * (w * dn * n).abs().mean(-1, keepdim=True))
    if d_res is not None:
        dx = dx + d_res.double().cpu()
        sx = sx + d_res.double().cpu().abs()
    lead = tuple(range(x.dim() - 1))
    return dx, (dn * n).sum(lead), dgate, sx, (dn * n).abs().sum(lead), sg
