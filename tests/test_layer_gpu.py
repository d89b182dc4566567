"""The operators around the rule together, as a layer uses them: norm with the residual's
addition -> projection -> short convolution -> the rule -> gated norm.  A packed prompt
batch goes through chunk_fwd_varlen and is continued from the pools by decode_runs,
token by token and in runs; the whole is held to a float64 form of the layer over the
whole sequences.  The layer's gradient, through chunk_bwd, is held to automatic
differentiation of that form.  The projections stand for the user's own."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

# Each kernel's float32 result is within 1e-5 of float64 in relative L2 (the tolerance of
# the rule's own tests; the convolution's and norms' are 1e-6 and less), the layer
# chains five, and a norm passes a relative error on once.
TOL = 5e-5
H, D, M = 2, 16, 48  # heads, channels of a head, width of the stream
C = 3 * H * D


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_130_b200 import binding
    return binding


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    return dict(norm=1 + 0.2 * rnd(M), qkv=rnd(M, C) / M ** 0.5, conv=0.5 * rnd(C, 4), bias=0.2 * rnd(C),
                decay=rnd(M, H) / M ** 0.5, write=rnd(M, H) / M ** 0.5, gate=rnd(M, H * D) / M ** 0.5,
                out=1 + 0.2 * rnd(D))


def rel(x, ref):
    return float((x.double().cpu() - ref).norm() / ref.norm())


def reference(x, r, p, unit):
    """One sequence in float64, from x, r [T, M]: (gated output [T, H, D], final state)."""
    h = x + r
    y = h / (h.pow(2).mean(-1, keepdim=True) + R.EPS).sqrt() * p["norm"]
    z = torch.cat([y.new_zeros(3, C), y @ p["qkv"]]).unfold(0, 4, 1)
    z = (z * p["conv"]).sum(-1) + p["bias"]
    q, k, v = (z * torch.sigmoid(z)).view(-1, 3, H, D).unbind(1)
    if unit:
        q, k = (a / (a.pow(2).sum(-1, keepdim=True) + R.EPS).sqrt() for a in (q, k))
    else:
        k = 0.3 * k
    alpha, beta = torch.sigmoid(-(y @ p["decay"])), torch.sigmoid(y @ p["write"])
    S, o = y.new_zeros(H, D, D), []
    for t in range(len(x)):
        S = alpha[t, :, None, None] * S
        u = beta[t, :, None] * (v[t] - torch.einsum("hij,hj->hi", S, k[t]))
        S = S + torch.einsum("hi,hj->hij", u, k[t])
        o.append(torch.einsum("hij,hj->hi", S, q[t]))
    o, g = torch.stack(o), (y @ p["gate"]).view(-1, H, D)
    n = o / (o.pow(2).mean(-1, keepdim=True) + R.EPS).sqrt() * p["out"]
    return n * g * torch.sigmoid(g), S


def test_prompt_then_tokens_then_runs(gdn):
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    p, g = weights(1), torch.Generator().manual_seed(2)
    lens, later = [20, 3, 37], 9                      # prompts, tokens that follow each
    xs = [torch.randn(2, n + later, M, generator=g) for n in lens]
    w = {n: t.cuda() for n, t in p.items()}
    conv_pool, pool = torch.zeros(6, 3, C).cuda(), torch.zeros(6, H, D, D).cuda()
    slots = dev([4, 0, 2])

    def before(x, r):
        y, _, h = gdn.rms_norm_fwd(x.cuda(), w["norm"], residual=r.cuda())
        assert torch.equal(h.cpu(), x + r)
        qkv = torch.cat([y @ w["qkv"], y @ w["gate"]], 1)  # one projection, sliced below
        return y, qkv[:, :C], qkv[:, C:].unflatten(1, (H, D)), y @ w["decay"], y @ w["write"]

    cu = [0, 20, 23, 60]
    y, qkv, gate, decay, write = before(torch.cat([x[0, :n] for x, n in zip(xs, lens)]),
                                        torch.cat([x[1, :n] for x, n in zip(xs, lens)]))
    q, k, v = gdn.short_conv_fwd(qkv, w["conv"], w["bias"], cu_seqlens=dev(cu), states=conv_pool,
                                 slots=slots, splits=[H * D] * 3)
    o, S = gdn.chunk_fwd_varlen(q.view(-1, H, D), k.view(-1, H, D), v.view(-1, H, D), decay, write, cu,
                                l2norm_qk=True, gate_logits=True, chunk=16)
    pool[slots.long()] = S
    out = [list(gdn.rms_norm_fwd(o, w["out"], gate=gate)[0].split(lens))]
    for n in (1, 1, 1, 4, 2):                         # single tokens, then runs
        at = sum(len(step[0]) for step in out[1:])
        take = lambda i: torch.cat([x[i, m + at:m + at + n] for x, m in zip(xs, lens)])
        y, qkv, gate, decay, write = before(take(0), take(1))
        cu = dev([0, n, 2 * n, 3 * n])
        qkv = gdn.short_conv_fwd(qkv, w["conv"], w["bias"], cu_seqlens=cu, states=conv_pool, slots=slots)
        q, k, v = qkv.view(-1, 3, H, D).unbind(1)
        draft = gdn.decode_runs(q, k, v, decay, write, pool, slots=slots, cu_seqlens=cu, update=False,
                                l2norm_qk=True, gate_logits=True)
        o = gdn.decode_runs(q, k, v, decay, write, pool, slots=slots, cu_seqlens=cu,
                            l2norm_qk=True, gate_logits=True)
        assert torch.equal(draft, o)
        out.append(list(gdn.rms_norm_fwd(o, w["out"], gate=gate)[0].split(n)))
    torch.cuda.synchronize()
    p64 = {n: t.double() for n, t in p.items()}
    for i, x in enumerate(xs):
        ref, S = reference(x[0].double(), x[1].double(), p64, True)
        assert rel(torch.cat([step[i] for step in out]), ref) <= TOL
        assert rel(pool[int(slots[i])], S) <= TOL
    assert (pool[[1, 3, 5]] == 0).all() and (conv_pool[[1, 3, 5]] == 0).all()


def test_gradient_of_the_layer(gdn):
    p, g, T = weights(3), torch.Generator().manual_seed(4), 45
    x, r, dout = (torch.randn(s, generator=g) for s in ((T, M), (T, M), (T, H, D)))
    w = {n: t.cuda() for n, t in p.items()}
    # forward
    y, _, h = gdn.rms_norm_fwd(x.cuda(), w["norm"], residual=r.cuda())
    z, gate = y @ w["qkv"], (y @ w["gate"]).view(T, H, D)
    la = -torch.nn.functional.softplus(y @ w["decay"])
    be = torch.sigmoid(y @ w["write"])
    q, k, v = (t.view(1, T, H, D) for t in gdn.short_conv_fwd(z, w["conv"], w["bias"], cu_seqlens=torch.tensor(
        [0, T], dtype=torch.int32, device="cuda"), splits=[H * D] * 3))
    k = 0.3 * k
    o, _ = gdn.chunk_fwd(q, k, v, la[None], be[None], chunk=16)
    # backward
    do, dw_out, dgate = gdn.rms_norm_bwd(dout.cuda(), o[0], w["out"], gate=gate)
    dq, dk, dv, dla, dbe, _ = gdn.chunk_bwd(q, k, v, la[None], be[None], None, do[None], chunk=16)
    dz, dconv, dbias = gdn.short_conv_bwd(tuple(t.view(T, H * D) for t in (dq, 0.3 * dk, dv)), z, w["conv"],
                                          w["bias"], cu_seqlens=torch.tensor([0, T], dtype=torch.int32,
                                                                            device="cuda"))
    ddecay = dla[0] * -torch.sigmoid(y @ w["decay"])
    dwrite = dbe[0] * be * (1 - be)
    dy = dz @ w["qkv"].T + dgate.flatten(1) @ w["gate"].T + ddecay @ w["decay"].T + dwrite @ w["write"].T
    dx, dw_norm, _ = gdn.rms_norm_bwd(dy, h, w["norm"])
    torch.cuda.synchronize()
    # the float64 form, differentiated
    p64 = {n: t.double().requires_grad_() for n, t in p.items()}
    x64, r64 = x.double().requires_grad_(), r.double().requires_grad_()
    ref, _ = reference(x64, r64, p64, False)
    (ref * dout.double()).sum().backward()
    got = {"norm": dw_norm, "out": dw_out, "conv": dconv, "bias": dbias, "qkv": y.T @ dz,
           "gate": y.T @ dgate.flatten(1), "decay": y.T @ ddecay, "write": y.T @ dwrite}
    assert rel(dx, x64.grad) <= TOL and torch.equal(x64.grad, r64.grad)
    for n, t in got.items():
        assert rel(t, p64[n].grad) <= TOL, n
