"""Cases of the operators around the gated delta rule: the recurrent form over a
pool of states (``decode_runs``), the short causal convolution in front of the
rule (``short_conv_fwd``, ``short_conv_bwd``) and the root-mean-square norm
before the layer and, gated, behind the rule (``rms_norm_fwd``, ``rms_norm_bwd``).

``run`` computes a case in its plain form, elementary torch operations in 32
bits, or, where ``own`` is true, by the library's kernels.  ``exact`` computes it
in 64 bits from the operators' definitions.
"""
import math
import random

import torch

own = False

EPS = 1e-6        # of the root-mean-square norm and of the L2 normalisation of q and k
E4M3_MAX = 448.0  # largest finite float8_e4m3fn value
TINY = 1e-30      # smallest group maximum that an 8-bit scale is made from


def listed():
    return [
        # A decode batch at the repository's decode shape: 256 sequences, one token each, their
        # states anywhere in a pool of 320, q, k, v as they come out of one projection.
        dict(name="step 256 sequences", op="runs", dtype="bf16", n=256, live=256, slots=320, run=1,
             hk=16, hv=16, dk=128, dv=128, update=True, mix=1),
        # One user alone: what a single token waits for.
        dict(name="step 1 sequence", op="runs", dtype="bf16", n=1, live=1, slots=8, run=1,
             hk=16, hv=16, dk=128, dv=128, update=True, mix=2),
        # Drafts of 1 to 8 tokens checked against the states without moving them; two value
        # heads share a key head.
        dict(name="verify runs of 8", op="runs", dtype="bf16", n=64, live=61, slots=96, run=8,
             hk=16, hv=32, dk=128, dv=128, update=False, mix=3),
        # The tails of prompts in float32 at odd head sizes, with padding rows in the batch.
        dict(name="tails float32", op="runs", dtype="f32", n=37, live=33, slots=50, run=13,
             hk=3, hv=6, dk=72, dv=40, update=True, mix=4),
        # q, k and v of a packed prompt batch (the repository's 12 sequences of 16384 tokens,
        # 16 heads of 128): one convolution over the fused projection's 3 x 2048 channels.
        dict(name="conv 16384 x 6144", op="conv", dtype="bf16", n=12, live=12, slots=16,
             total=16384, c=6144, w=4, bias=False, parts=3, mix=5),
        # The same layer's decode batch: one token of each of 256 sequences.
        dict(name="conv step 256 x 6144", op="conv", dtype="bf16", n=256, live=250, slots=320,
             total=256, c=6144, w=4, bias=False, parts=3, mix=6),
        # Its gradients in training on packed sequences.
        dict(name="conv backward 16384 x 6144", op="conv_bwd", dtype="bf16", n=12, total=16384,
             c=6144, w=4, bias=True, parts=3, mix=7),
        # The layer's input: the residual added, the norm written in 8 bits with a scale a token.
        dict(name="norm 16384 x 2048 8 bits", op="norm", dtype="bf16", rows=16384, heads=1, d=2048,
             residual=True, gate=False, quant="row"),
        # The same for one token of one user.
        dict(name="norm 1 x 2048", op="norm", dtype="bf16", rows=1, heads=1, d=2048,
             residual=True, gate=False, quant=""),
        # Its gradients, with the gradient that arrives over the residual.
        dict(name="norm backward 16384 x 2048", op="norm_bwd", dtype="bf16", rows=16384, heads=1,
             d=2048, residual=True, gate=False),
        # The rule's output of the headline's token count: 16 heads of 128, gated.
        dict(name="gated norm 16384 x 16 x 128", op="norm", dtype="bf16", rows=16384, heads=16,
             d=128, residual=False, gate=True, quant=""),
        # Its gradients, in float32 at an odd size.
        dict(name="gated norm backward f32", op="norm_bwd", dtype="f32", rows=2047, heads=6, d=200,
             residual=False, gate=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["runs", "runs", "conv", "conv_bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    mix = rng.randrange(1, 1 << 20)
    if op == "runs":
        dk, dv = rng.choice([16, 24, 64, 72, 96, 128, 200, 256]), rng.choice([16, 40, 64, 128, 256])
        hk, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4])
        most = max(1, 256 * 16 * 128 * 128 // (hk * group * dk * dv))
        n = _log_int(rng, 1, min(512, most))
        live = max(1, n - rng.choice([0, 0, n // 8]))
        return dict(op="runs", dtype=dtype, n=n, live=live, slots=n + rng.randrange(0, 9),
                    run=rng.choice([1, 1, 2, 3, 5, 8, 16]), hk=hk, hv=hk * group, dk=dk, dv=dv,
                    update=rng.random() < 0.7, mix=mix)
    if op in ("conv", "conv_bwd"):
        size = 2 if dtype == "bf16" else 4
        c = rng.choice([48, 96, 384, 1000, 1536, 2049, 4096, 6144])
        parts = rng.choice([1, 3]) if c % 3 == 0 else 1
        total = _log_int(rng, 1, min(20000, 16384 * 6144 * 2 // (c * size)))
        n = _log_int(rng, 1, min(total, 300))
        case = dict(op=op, dtype=dtype, n=n, total=total, c=c, w=rng.choice([2, 3, 4, 4]),
                    bias=rng.random() < 0.5, parts=parts, mix=mix)
        if op == "conv":
            case.update(live=max(1, n - rng.choice([0, n // 8])), slots=n + rng.randrange(0, 9))
        return case
    size = 2 if dtype == "bf16" else 4
    gate = rng.random() < 0.5
    heads = rng.choice([1, 3, 8, 16, 32]) if gate else 1
    d = rng.choice([32, 64, 96, 128, 200, 256, 512]) if gate else rng.choice(
        [128, 640, 1001, 1536, 2048, 4096, 5120, 8192])
    rows = _log_int(rng, 1, min(40000, 16384 * 2048 * 2 // (heads * d * size)))
    case = dict(op=op, dtype=dtype, rows=rows, heads=heads, d=d, gate=gate,
                residual=not gate and rng.random() < 0.7)
    if op == "norm":
        case["quant"] = rng.choice(["", "row", "group"]) if d % 128 == 0 else rng.choice(["", "row"])
    return case


def _lens(case):
    """Tokens of each sequence of a packed batch, from the case alone."""
    r, n = random.Random(case["mix"]), case["n"]
    if case["op"] == "runs":
        return [case["run"]] + [r.randint(1, case["run"]) for _ in range(n - 1)]
    w = [math.exp(4 * r.random()) for _ in range(n)]  # a few long prompts, many short ones
    spare = case["total"] - n
    lens = [1 + int(spare * x / sum(w)) for x in w]
    lens[0] += case["total"] - sum(lens)
    return lens


def _plan(case):
    """cu_seqlens and the sequences' slots on the device: `live` sequences with a slot of
    their own, the others (padding of a batch of fixed size) with slot -1."""
    lens, r = _lens(case), random.Random(case["mix"] + 1)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    p = dict(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), total=cu[-1], longest=max(lens))
    if "live" in case:
        places = r.sample(range(case["slots"]), case["n"])
        slots = [s if i < case["live"] else -1 for i, s in enumerate(places)]
        p["slots"] = torch.tensor(slots, dtype=torch.int32, device="cuda")
    return p


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def rnd(*shape, scale=1.0, dtype=None):
        return (scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype or t)

    s = dict(case=case)
    op = case["op"]
    if op == "runs":
        s.update(_plan(case))
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        rows = s["total"] + 3  # a buffer of fixed size, with rows behind the last sequence
        qkv = rnd(rows, 2 * hk * dk + hv * dv)
        s["q"] = qkv[:, :hk * dk].unflatten(1, (hk, dk))
        s["k"] = qkv[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
        s["v"] = qkv[:, 2 * hk * dk:].unflatten(1, (hv, dv))
        s["decay"] = rnd(rows, hv, dtype=torch.float32)   # logits: log alpha = -softplus(x)
        s["write"] = rnd(rows, hv, dtype=torch.float32)   # beta = sigmoid(y)
        s["states"] = rnd(case["slots"], hv, dv, dk, scale=0.1, dtype=torch.float32)
        s["out"] = torch.zeros(rows, hv, dv, dtype=t, device="cuda")
    elif op in ("conv", "conv_bwd"):
        s.update(_plan(case))
        c, w = case["c"], case["w"]
        s["x"] = rnd(case["total"], c)
        s["weight"] = rnd(c, w, scale=0.5)
        s["bias"] = rnd(c, scale=0.2) if case["bias"] else None
        s["splits"] = [c // case["parts"]] * case["parts"]
        if op == "conv":
            s["states"] = rnd(case["slots"], w - 1, c)
        else:
            s["dy"] = tuple(rnd(case["total"], n) for n in s["splits"])
    else:
        shape = (case["rows"], case["heads"], case["d"])
        s["x"] = rnd(*shape, scale=2.0)
        s["weight"] = (1 + 0.1 * torch.randn(case["d"], generator=gen, device="cuda")).to(t)
        s["gate"] = rnd(*shape) if case["gate"] else None
        s["extra"] = rnd(*shape) if case["residual"] else None  # residual, or its gradient
        if op == "norm_bwd":
            s["dy"] = rnd(*shape)
    return s


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "runs":
        lens = _lens(case)[:case["live"]]
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        state = 4 * len(lens) * hv * dk * dv * (2 if case["update"] else 1)
        token = size * (2 * hk * dk + 2 * hv * dv) + 8 * hv
        return dict(bytes=state + sum(lens) * token, flops=7 * sum(lens) * hv * dk * dv)
    if op == "conv":
        held = 2 * case["live"] * (case["w"] - 1) * case["c"] * size
        n = case["total"] * case["c"]
        return dict(bytes=2 * n * size + held + case["c"] * case["w"] * size,
                    flops=(2 * case["w"] + 4) * n)
    if op == "conv_bwd":
        n = case["total"] * case["c"]
        return dict(bytes=3 * n * size + case["c"] * case["w"] * (size + 4),
                    flops=(6 * case["w"] + 10) * n)
    n = case["rows"] * case["heads"] * case["d"]
    rows = case["rows"] * case["heads"]
    if op == "norm":
        reads = 1 + bool(case["residual"]) + bool(case["gate"])
        out = 1 if case["quant"] else size
        groups = {"": 0, "row": rows, "group": n // 128}[case["quant"]]
        return dict(bytes=n * (size * reads + out + (size if case["residual"] else 0)) + 4 * groups,
                    flops=n * (6 + 6 * bool(case["gate"])))
    moved = 3 + bool(case["residual"]) + 2 * bool(case["gate"])
    return dict(bytes=n * size * moved + 4 * case["d"], flops=n * (12 + 12 * bool(case["gate"])))


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from gated_delta_rule_130_b200 import binding as gdn

    case, op = s["case"], s["case"]["op"]
    if op == "runs":
        gdn.decode_runs(s["q"], s["k"], s["v"], s["decay"], s["write"], s["states"],
                        slots=s["slots"], cu_seqlens=s["cu"], out=s["out"],
                        update=case["update"], l2norm_qk=True, gate_logits=True)
        return (s["out"], s["states"]) if case["update"] else (s["out"],)
    if op == "conv":
        y = gdn.short_conv_fwd(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"],
                               states=s["states"], slots=s["slots"], splits=s["splits"])
        return (*y, s["states"])
    if op == "conv_bwd":
        dx, dw, db = gdn.short_conv_bwd(s["dy"], s["x"], s["weight"], s["bias"],
                                        cu_seqlens=s["cu"])
        return (dx, dw) if db is None else (dx, dw, db)
    if op == "norm":
        y, scale, h = gdn.rms_norm_fwd(s["x"], s["weight"], residual=s["extra"], gate=s["gate"],
                                       eps=EPS, quant=case["quant"] or None)
        return tuple(a for a in (y, scale, h) if a is not None)
    dx, dw, dgate = gdn.rms_norm_bwd(s["dy"], s["x"], s["weight"], gate=s["gate"],
                                     d_res=s["extra"], eps=EPS)
    return (dx, dw) if dgate is None else (dx, dw, dgate)


# ---------------------------------------------------------------- the plain forms

def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _softplus(x):
    return x.clamp_min(0) + torch.log1p(torch.exp(-x.abs()))


def _plain_runs(s):
    """The runs as one padded batch of at most 16 tokens each.  With g the running sum of
    log alpha and G_ij = exp(g_i - g_j), the corrections u solve the unit lower triangular
    system (I + A) u = beta (v - e^g S k), A_ij = beta_i G_ij k_i.k_j for j < i, and A^16 = 0
    gives its inverse as (I - A)(I + A^2)(I + A^4)(I + A^8)."""
    case, cu, slots = s["case"], s["cu"].long(), s["slots"].long()
    L, group = s["longest"], case["hv"] // case["hk"]
    at = torch.arange(L, device="cuda")
    idx = cu[:-1, None] + at                                        # [N, L]
    real = (idx < cu[1:, None]) & (slots >= 0)[:, None]
    idx = torch.where(real, idx, 0)
    heads = torch.arange(case["hv"], device="cuda") // group

    def rows(x):  # [rows, H, D] -> [N, H, L, D]
        return torch.where(real[:, :, None, None], x[idx].float(), 0).transpose(1, 2)

    q, k, v = _unit(rows(s["q"])), _unit(rows(s["k"])), rows(s["v"])
    q, k = q[:, heads], k[:, heads]
    la = torch.where(real[:, :, None], -_softplus(s["decay"][idx]), 0).transpose(1, 2)
    be = torch.where(real[:, :, None], 1 / (1 + torch.exp(-s["write"][idx])), 0).transpose(1, 2)
    S = s["states"][slots.clamp_min(0)]                             # [N, H, Dv, Dk]
    g = la.cumsum(-1)
    decay, below = torch.exp(g[..., None]), at[:, None] > at[None, :]
    G = torch.exp(torch.where(at[:, None] >= at[None, :], g[..., :, None] - g[..., None, :], -torch.inf))
    A = torch.where(below, be[..., None] * G * (k @ k.transpose(-1, -2)), 0)
    u = be[..., None] * (v - decay * (k @ S.transpose(-1, -2)))
    A2 = A @ A
    A4 = A2 @ A2
    A8 = A4 @ A4
    u = u + A8 @ u
    u = u + A4 @ u
    u = u + A2 @ u
    u = u - A @ u
    o = decay * (q @ S.transpose(-1, -2)) + (G * (q @ k.transpose(-1, -2))) @ u
    out = s["out"]
    covered = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(cu[1:], covered, right=True)
    out[:s["total"]] = torch.where((slots[seq] >= 0)[:, None, None],
                                   o.transpose(1, 2)[seq, covered - cu[seq]], 0).to(out.dtype)
    if not case["update"]:
        return (out,)
    last = torch.exp(g[..., -1:] - g)[..., None]
    S = torch.exp(g[..., -1])[..., None, None] * S + u.transpose(-1, -2) @ (last * k)
    n = case["live"]
    s["states"].index_copy_(0, slots[:n], S[:n])
    return out, s["states"]


def _before(s, x, j):
    """x of j tokens earlier in the same sequence; where the sequence had not begun, the row
    of its held inputs (zero for a sequence without)."""
    case, cu = s["case"], s["cu"].long()
    t = torch.arange(case["total"], device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    pos = t - cu[seq] - j
    inside = x[(t - j).clamp_min(0)]
    if "states" not in s:
        return torch.where((pos >= 0)[:, None], inside, 0)
    slot = s["slots"].long()[seq]
    held = s["states"][slot.clamp_min(0), (case["w"] - 1 + pos).clamp(0, case["w"] - 2)]
    return torch.where((pos >= 0)[:, None], inside, torch.where((slot >= 0)[:, None], held, 0))


def _plain_conv(s):
    case, w = s["case"], s["weight"].float()
    W, cu, slots, x = case["w"], s["cu"].long(), s["slots"].long(), s["x"]
    z = sum(w[:, W - 1 - j] * _before(s, x, j).float() for j in range(W))
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = z / (1 + torch.exp(-z))
    seq = torch.searchsorted(cu[1:], torch.arange(case["total"], device="cuda"), right=True)
    y = torch.where((slots[seq] >= 0)[:, None], y, 0).to(x.dtype)
    # the last W - 1 inputs of each sequence, older held ones where it is shorter
    n, old = case["live"], torch.arange(W - 1, device="cuda")
    at = cu[1:n + 1, None] - (W - 1) + old
    length = (cu[1:n + 1] - cu[:n])[:, None]
    kept = s["states"][slots[:n, None], (old + length).clamp_max(W - 2)]
    s["states"][slots[:n]] = torch.where((at >= cu[:n, None])[..., None], x[at.clamp_min(0)], kept)
    return (*(p.contiguous() for p in y.split(s["splits"], 1)), s["states"])


def _plain_conv_bwd(s):
    case, w, x = s["case"], s["weight"].float(), s["x"]
    W, cu = case["w"], s["cu"].long()
    z = sum(w[:, W - 1 - j] * _before(s, x, j).float() for j in range(W))
    if s["bias"] is not None:
        z = z + s["bias"].float()
    sig = 1 / (1 + torch.exp(-z))
    dz = torch.cat(s["dy"], 1).float() * (sig * (1 + z * (1 - sig)))
    t = torch.arange(case["total"], device="cuda")
    end = cu[1:][torch.searchsorted(cu[1:], t, right=True)]

    def after(j):  # dz of j tokens later in the same sequence
        return torch.where((t + j < end)[:, None], dz[(t + j).clamp_max(case["total"] - 1)], 0)

    dx = sum(w[:, W - 1 - j] * after(j) for j in range(W)).to(x.dtype)
    dw = torch.stack([(dz * _before(s, x, W - 1 - j).float()).sum(0) for j in range(W)], 1)
    return (dx, dw) if s["bias"] is None else (dx, dw, dz.sum(0))


def _plain_norm(s):
    case, x = s["case"], s["x"]
    h = x if s["extra"] is None else (x.float() + s["extra"].float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["gate"] is not None:
        g = s["gate"].float()
        y = y * (g / (1 + torch.exp(-g)))
    out = []
    if case["quant"]:
        grouped = y.unflatten(-1, (-1, 128 if case["quant"] == "group" else case["d"]))
        top = grouped.abs().amax(-1, keepdim=True).clamp_min(TINY)
        out.append((grouped * (E4M3_MAX / top)).to(torch.float8_e4m3fn).flatten(-2))
        out.append((top / E4M3_MAX).squeeze(-1))
    else:
        out.append(y.to(x.dtype))
    return (*out, h) if s["extra"] is not None else tuple(out)


def _plain_norm_bwd(s):
    x, w, dy = s["x"].float(), s["weight"].float(), s["dy"].float()
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n, dn = x * rstd, dy
    if s["gate"] is not None:
        g = s["gate"].float()
        sig = 1 / (1 + torch.exp(-g))
        dn = dy * (g * sig)
        dgate = (dy * n * w * sig * (1 + g * (1 - sig))).to(s["x"].dtype)
    dx = rstd * (w * dn - n * (w * dn * n).mean(-1, keepdim=True))
    if s["extra"] is not None:
        dx = dx + s["extra"].float()
    out = (dx.to(s["x"].dtype), (dn * n).sum((0, 1)))
    return out if s["gate"] is None else (*out, dgate)


def run(s):
    if own:
        return _own(s)
    return {"runs": _plain_runs, "conv": _plain_conv, "conv_bwd": _plain_conv_bwd,
            "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[s["case"]["op"]](s)


# ---------------------------------------------------------------- in 64 bits

def _exact_runs(s):
    """Token by token, as the rule is written."""
    case, cu, slots = s["case"], s["cu"].tolist(), s["slots"].tolist()
    group = case["hv"] // case["hk"]
    heads = torch.arange(case["hv"], device="cuda") // group
    live = [n for n in range(case["n"]) if slots[n] >= 0]
    where = torch.tensor([slots[n] for n in live], device="cuda")
    S, out = s["states"].double()[where], s["out"].double()
    for t in range(s["longest"]):
        has = [i for i, n in enumerate(live) if cu[n] + t < cu[n + 1]]
        if not has:
            break
        i = torch.tensor(has, device="cuda")
        row = torch.tensor([cu[live[j]] + t for j in has], device="cuda")
        q, k, v = (s[name][row].double() for name in ("q", "k", "v"))
        q = (q / (q.pow(2).sum(-1, keepdim=True) + EPS).sqrt())[:, heads]
        k = (k / (k.pow(2).sum(-1, keepdim=True) + EPS).sqrt())[:, heads]
        alpha = torch.sigmoid(-s["decay"][row].double())[..., None]   # exp(-softplus(x))
        beta = torch.sigmoid(s["write"][row].double())[..., None]
        now = alpha[..., None] * S[i]
        miss = beta * (v - torch.einsum("nhij,nhj->nhi", now, k))
        now = now + torch.einsum("nhi,nhj->nhij", miss, k)
        S[i] = now
        out[row] = torch.einsum("nhij,nhj->nhi", now, q)
    if not case["update"]:
        return (out,)
    states = s["states"].double()
    states[where] = S
    return out, states


def _exact_conv_rows(s, slot_of):
    """z of the convolution in 64 bits, sequence by sequence; the padded inputs too."""
    case, cu = s["case"], s["cu"].tolist()
    W, w = case["w"], s["weight"].double()
    z = torch.zeros(case["total"], case["c"], dtype=torch.float64, device="cuda")
    padded = []
    for n in range(case["n"]):
        x = s["x"][cu[n]:cu[n + 1]].double()
        slot = slot_of(n)
        head = s["states"][slot].double() if slot is not None else x.new_zeros(W - 1, case["c"])
        x = torch.cat([head, x])
        z[cu[n]:cu[n + 1]] = torch.einsum("tcw,cw->tc", x.unfold(0, W, 1), w)
        padded.append(x)
    return (z if s["bias"] is None else z + s["bias"].double()), padded


def _exact_conv(s):
    case, cu, slots = s["case"], s["cu"].tolist(), s["slots"].tolist()
    z, padded = _exact_conv_rows(s, lambda n: slots[n] if slots[n] >= 0 else None)
    y, states = z * torch.sigmoid(z), s["states"].double()
    for n in range(case["n"]):
        if slots[n] >= 0:
            states[slots[n]] = padded[n][-(case["w"] - 1):]
        else:
            y[cu[n]:cu[n + 1]] = 0
    return (*y.split(s["splits"], 1), states)


def _exact_conv_bwd(s):
    case, cu = s["case"], s["cu"].tolist()
    W, w = case["w"], s["weight"].double()
    z, padded = _exact_conv_rows(s, lambda n: None)
    sig = torch.sigmoid(z)
    dz = torch.cat([d.double() for d in s["dy"]], 1) * (sig + z * sig * (1 - sig))
    dx, dw = torch.empty_like(dz), torch.zeros_like(w)
    for n in range(case["n"]):
        d, m = dz[cu[n]:cu[n + 1]], cu[n + 1] - cu[n]
        grad = torch.zeros_like(padded[n])
        for j in range(W):
            grad[j:j + m] += w[:, j] * d
            dw[:, j] += (padded[n][j:j + m] * d).sum(0)
        dx[cu[n]:cu[n + 1]] = grad[W - 1:]
    return (dx, dw) if s["bias"] is None else (dx, dw, dz.sum(0))


def _exact_norm(s):
    case = s["case"]
    h = s["x"].double()
    if s["extra"] is not None:  # the residual stream is held in the inputs' type
        h = (h + s["extra"].double()).to(s["x"].dtype).double()
    y = h / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["weight"].double()
    if s["gate"] is not None:
        g = s["gate"].double()
        y = y * g * torch.sigmoid(g)
    out = [y]
    if case["quant"]:
        size = 128 if case["quant"] == "group" else case["d"]
        parts = y.reshape(*y.shape[:-1], case["d"] // size, size)
        scale = parts.abs().amax(-1) / E4M3_MAX
        out = [(parts / scale[..., None]).reshape(y.shape), scale]
    return (*out, h) if s["extra"] is not None else tuple(out)


def _exact_norm_bwd(s):
    x, w, dy = s["x"].double(), s["weight"].double(), s["dy"].double()
    ms = x.pow(2).mean(-1, keepdim=True) + EPS
    unit = x / ms.sqrt()
    dunit = dy * w
    if s["gate"] is not None:
        g = s["gate"].double()
        sig = torch.sigmoid(g)
        dgate = dy * unit * w * (sig + g * sig * (1 - sig))
        dy = dy * g * sig
        dunit = dunit * g * sig
    dx = dunit / ms.sqrt() - x * (dunit * x).mean(-1, keepdim=True) / ms.pow(1.5)
    if s["extra"] is not None:
        dx = dx + s["extra"].double()
    dw = (dy * unit).flatten(0, 1).sum(0)
    return (dx, dw) if s["gate"] is None else (dx, dw, dgate)


def exact(case, seed):
    s = prepare(case, seed)
    return {"runs": _exact_runs, "conv": _exact_conv, "conv_bwd": _exact_conv_bwd,
            "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}[case["op"]](s)
