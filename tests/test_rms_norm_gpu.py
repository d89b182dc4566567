"""The root-mean-square norm (with residual, gate, 8-bit output) and its gradients against
float64."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_130_b200 import binding
    return binding


def draw(shape, dtype, seed, param=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    d = dict(x=2 * rnd(*shape), res=rnd(*shape), gate=2 * rnd(*shape), dy=rnd(*shape),
             dres=rnd(*shape))
    d = {n: t.to(dtype).cuda() for n, t in d.items()}
    d["w"] = (1 + 0.3 * rnd(shape[-1])).to(param or dtype).cuda()
    return d


def roundings(D):
    # the sum of squares: at most 32 terms per lane (D / 256 where a row is read element
    # by element), 10 levels; half of it, as it stands under a root; five products and
    # the gate's fast functions
    return max(32, D / 256) / 2 + 48


SHAPES = [(1, 1), (5, 7), (3, 32), (4, 3, 64), (9, 96), (2, 2, 5, 128), (6, 200), (7, 512), (3, 640),
          (2, 1001), (5, 1024), (4, 2048), (2, 2056), (3, 4096), (2, 5120), (3, 8192), (1, 12290),
          (2, 16384), (1, 32768), (1, 65536)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(gdn, shape, dtype):
    d = draw(shape, dtype, shape[-1])
    for res, gate in ((None, None), (d["res"], None), (None, d["gate"]), (d["res"], d["gate"])):
        y, scale, h = gdn.rms_norm_fwd(d["x"], d["w"], residual=res, gate=gate, eps=EPS)
        torch.cuda.synchronize()
        ref, href = R.norm(d["x"], d["w"], res, gate, EPS)
        assert scale is None and (h is None) == (res is None)
        R.close(y, ref, ref.abs(), roundings(shape[-1]))
        if res is not None:
            assert torch.equal(h.cpu(), href.cpu())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,quant", [((3, 7), "row"), ((5, 128), "row"), ((2, 3, 128), "group"),
                                         ((4, 2048), "row"), ((4, 2048), "group"), ((3, 384), "group"),
                                         ((2, 1001), "row"), ((1, 40960), "group"), ((1, 40960), "row"),
                                         ((3, 200), "row"), ((2, 8192), "group"), ((33, 64), "row")])
def test_eight_bits(gdn, shape, quant, dtype):
    d = draw(shape, dtype, shape[-1] + 1)
    d["x"][0] = 0.0
    d["res"][0] = 0.0  # a row of zeros: the smallest scale, zeros
    D = shape[-1]
    group = D if quant == "row" else 128
    for res, gate in ((d["res"], None), (None, d["gate"])):
        y, scale, h = gdn.rms_norm_fwd(d["x"], d["w"], residual=res, gate=gate, eps=EPS, quant=quant)
        torch.cuda.synchronize()
        assert y.dtype == torch.float8_e4m3fn and scale.shape == shape[:-1] + (D // group,)
        ref, _ = R.norm(d["x"], d["w"], res, gate, EPS)
        parts = ref.reshape(shape[:-1] + (D // group, group))
        top = parts.abs().amax(-1).clamp_min(1e-30)
        R.close(scale, top / 448, top / 448, roundings(D) + 2)
        # the value stood for: half a step of e4m3 (2^-4 of the value, 2^-10 below 2^-6)
        value = y.float().cpu().double().reshape(parts.shape) * scale.cpu().double()[..., None]
        want = parts / (top / 448)[..., None]
        bound = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64))
        bound = (bound + want.abs() * (roundings(D) + 4) * R.U32) * (top / 448)[..., None] * 1.001
        assert ((value - parts).abs() <= bound).all()
        assert value.abs().amax() <= ref.abs().amax() * 1.001


def test_nan_and_infinity_stay_in_their_rows(gdn):
    for dtype, D in ((F32, 256), (BF16, 1024), (F32, 77)):
        d = draw((6, D), dtype, 3)
        d["x"][1, 5] = float("nan")
        d["x"][3, 6] = float("inf")
        for quant in (None, "row"):
            y, scale, h = gdn.rms_norm_fwd(d["x"], d["w"], residual=d["res"], quant=quant)
            y = y.float()
            assert torch.isfinite(y[[0, 2, 4, 5]]).all() and y[1].isnan().all() and y[3, 6].isnan()
            if quant:
                assert torch.isfinite(scale[[0, 2, 4, 5]]).all() and scale[[1, 3]].isnan().all()
        dx, dw, _ = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"])
        assert torch.isfinite(dx[[0, 2, 4, 5]].float()).all() and dx[1].isnan().all()


@pytest.mark.parametrize("dtype,D", [(F32, 256), (BF16, 1024), (F32, 131), (BF16, 384), (BF16, 40064)])
def test_an_infinite_value_in_8_bits(gdn, dtype, D):
    # no scale holds an infinity: the scale and the values of its row or group are NaN
    d = draw((5, D), dtype, 11)
    d["gate"][2, 3] = float("inf")
    for quant in ("row", "group") if D % 128 == 0 else ("row",):
        y, scale, _ = gdn.rms_norm_fwd(d["x"], d["w"], gate=d["gate"], quant=quant)
        n = D if quant == "row" else 128
        y = y.float()
        assert scale[2, 0].isnan() and y[2, :n].isnan().all()
        assert torch.isfinite(y[[0, 1, 3, 4]]).all() and torch.isfinite(scale[[0, 1, 3, 4]]).all()
        assert torch.isfinite(y[2, n:]).all() and torch.isfinite(scale[2, 1:]).all()


def test_rows_beyond_32_bit_offsets(gdn):
    # 2.2e9 elements, all zero but the last rows
    rows, D = 270_000, 8192
    x = torch.zeros(rows, D, dtype=BF16, device="cuda")
    dy = torch.zeros_like(x)
    d = draw((6, D), BF16, 12)
    x[-6:], dy[-6:] = d["x"], d["dy"]
    y, scale, _ = gdn.rms_norm_fwd(x, d["w"], quant="group")
    z, zs, _ = gdn.rms_norm_fwd(d["x"], d["w"], quant="group")
    assert torch.equal(y[-6:].float(), z.float()) and torch.equal(scale[-6:], zs)
    assert not (y[:-6].view(torch.uint8) & 0x7f).any()  # +0 or -0, as the weight
    del y, scale
    dx, dw, _ = gdn.rms_norm_bwd(dy, x, d["w"])
    ex, ew, _ = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"])
    assert torch.equal(dx[-6:], ex) and not dx[:-6].any()
    ref = R.norm_grads(d["dy"], d["x"], d["w"], None, None, EPS)
    R.close(dw, ref[1], ref[4], bwd_roundings(D, 6))


def test_gate_at_its_ends(gdn):
    d = draw((4, 128), F32, 4)
    d["gate"][0], d["gate"][1], d["gate"][2] = -200.0, 200.0, 0.0
    y, _, _ = gdn.rms_norm_fwd(d["x"], d["w"], gate=d["gate"])
    ref, _ = R.norm(d["x"], d["w"], None, d["gate"], EPS)
    R.close(y, ref, ref.abs() + 1e-30, roundings(128))
    dx, dw, dg = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=d["gate"])
    assert all(torch.isfinite(t).all() for t in (dx, dw, dg))


@pytest.mark.parametrize("dtype,D", [(F32, 128), (BF16, 2048), (F32, 77), (BF16, 40000)])
def test_in_place(gdn, dtype, D):
    # the residual stream updated in place, in either place, and y over x
    d = draw((5, D), dtype, 5)
    y, _, h = gdn.rms_norm_fwd(d["x"], d["w"], residual=d["res"])
    for at in ("res", "x"):
        e = {n: t.clone() for n, t in d.items()}
        y2, _, h2 = gdn.rms_norm_fwd(e["x"], e["w"], residual=e["res"], h_out=e[at])
        assert h2 is e[at] and torch.equal(h2, h) and torch.equal(y2, y)
    y3, _, _ = gdn.rms_norm_fwd(d["x"], d["w"])
    x = d["x"].clone()
    y4, _, _ = gdn.rms_norm_fwd(x, d["w"], out=x)
    assert y4 is x and torch.equal(x, y3)


def test_slices_and_float32_weights(gdn):
    for D, pad in ((128, 8), (100, 4), (64, 3)):
        d = draw((6, 3, D), BF16, D, param=F32)
        wide = lambda t: torch.cat([t.flatten(1), t.flatten(1)[:, :pad]], 1)[:, :3 * D].unflatten(1, (3, D))
        s = {n: wide(t) if t.dim() == 3 else t for n, t in d.items()}
        for kw in (dict(residual="res"), dict(gate="gate")):
            a = gdn.rms_norm_fwd(d["x"], d["w"], **{n: d[v] for n, v in kw.items()})
            b = gdn.rms_norm_fwd(s["x"], s["w"], **{n: s[v] for n, v in kw.items()})
            ref, _ = R.norm(d["x"], d["w"], d["res"] if "residual" in kw else None,
                            d["gate"] if "gate" in kw else None, EPS)
            R.close(a[0], ref, ref.abs(), roundings(D))
            R.close(b[0], ref, ref.abs(), roundings(D))
        ref = R.norm_grads(d["dy"], d["x"], d["w"], d["gate"], d["dres"], EPS)
        for e in (d, s):
            dx, dw, dg = gdn.rms_norm_bwd(e["dy"], e["x"], e["w"], gate=e["gate"], d_res=e["dres"])
            R.close(dx, ref[0], ref[3], bwd_roundings(D, 18))
            R.close(dw, ref[1], ref[4], bwd_roundings(D, 18))
            R.close(dg, ref[2], ref[5], bwd_roundings(D, 18))


def bwd_roundings(D, rows):
    # two sums over a row and their products; dw: a block's rows in a chain (148 blocks at
    # least), its row groups (64 at most) in a chain, then 888 blocks at most, 128 ways
    return max(32, D / 256) + 64 + rows / 148 + 64 + 24


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (70, 7), (3, 32), (4, 3, 64), (900, 16), (2, 2, 5, 128),
                                   (6, 200), (1300, 512), (3, 640), (2, 1001), (5, 1024), (700, 2048),
                                   (2, 2056), (3, 8192), (1, 12290), (2, 16384), (1, 40000)])
def test_gradients(gdn, shape, dtype):
    d = draw(shape, dtype, shape[-1] + 2)
    rows = d["x"].numel() // shape[-1]
    for gate, dres in ((None, None), (None, d["dres"]), (d["gate"], None), (d["gate"], d["dres"])):
        dx, dw, dg = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=gate, d_res=dres, eps=EPS)
        torch.cuda.synchronize()
        ref = R.norm_grads(d["dy"], d["x"], d["w"], gate, dres, EPS)
        c = bwd_roundings(shape[-1], rows)
        R.close(dx, ref[0], ref[3], c)
        R.close(dw, ref[1], ref[4], c)
        assert (dg is None) == (gate is None)
        if gate is not None:
            R.close(dg, ref[2], ref[5] + 1e-30, c)
        again = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=gate, d_res=dres, eps=EPS)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip((dx, dw, dg), again))


def test_gradients_against_differences(gdn):
    d = draw((6, 40), F32, 7)
    dx, dw, dg = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=d["gate"])
    g = torch.Generator().manual_seed(6)
    to = {n: torch.randn(d[n].shape, generator=g, dtype=torch.float64) for n in ("x", "w", "gate")}
    at = lambda n, s: d[n].cpu().double() + s * to[n]
    loss = lambda s: (R.norm(at("x", s), at("w", s), None, at("gate", s), EPS)[0]
                      * d["dy"].cpu().double()).sum()
    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    got = [(t.cpu().double() * to[n]) for t, n in ((dx, "x"), (dw, "w"), (dg, "gate"))]
    assert (slope - sum(t.sum() for t in got)).abs() <= 2e-5 * sum(t.abs().sum() for t in got)


def test_no_rows_and_graphs(gdn):
    d = draw((0, 64), BF16, 8)
    y, _, _ = gdn.rms_norm_fwd(d["x"], d["w"])
    dx, dw, _ = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"])
    assert y.shape == dx.shape == (0, 64) and (dw == 0).all()
    # forward and backward captured, then replayed on other values
    d, e = draw((40, 2048), BF16, 9), draw((40, 2048), BF16, 10)
    s = {n: t.clone() for n, t in d.items()}

    def both():
        y, _, h = gdn.rms_norm_fwd(s["x"], s["w"], residual=s["res"])
        return (y, h) + gdn.rms_norm_bwd(s["dy"], h, s["w"], d_res=s["dres"])[:2]

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for n in s:
        s[n].copy_(e[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, both()))


def test_a_given_workspace(gdn):
    # the same bits, nothing behind its size written; one that is too small is not used
    d = draw((300, 3, 96), BF16, 13)
    a = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=d["gate"])
    need = gdn.rms_norm_bwd_workspace_size(300, 3, 96)
    for size in (need, 16):
        ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
        b = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=d["gate"], workspace=ws[:size])
        assert all(torch.equal(s, t) for s, t in zip(a, b)) and (ws[size:] == 7).all()


# 4736 rows and more take other splits of a row over threads than few rows do
@pytest.mark.parametrize("shape,dtype", [((4736, 1032), BF16), ((4800, 2048), BF16), ((4737, 2056), BF16),
                                         ((4736, 4096), BF16), ((4736, 516), F32), ((4741, 1024), F32),
                                         ((4736, 2048), F32)])
def test_forward_of_many_rows(gdn, shape, dtype):
    d = draw(shape, dtype, shape[-1])
    D = shape[-1]
    for res, gate in ((None, None), (d["res"], None), (None, d["gate"])):
        ref, href = R.norm(d["x"], d["w"], res, gate, EPS)
        y, _, h = gdn.rms_norm_fwd(d["x"], d["w"], residual=res, gate=gate, eps=EPS)
        R.close(y, ref, ref.abs(), roundings(D))
        assert res is None or torch.equal(h.cpu(), href.cpu())
        for quant in ("row", "group") if D % 128 == 0 else ("row",):
            y, scale, h = gdn.rms_norm_fwd(d["x"], d["w"], residual=res, gate=gate, eps=EPS, quant=quant)
            assert res is None or torch.equal(h.cpu(), href.cpu())
            group = D if quant == "row" else 128
            parts = ref.unflatten(-1, (-1, group))
            top = parts.abs().amax(-1)
            R.close(scale, top / 448, top / 448, roundings(D) + 2)
            # as in test_eight_bits
            value = y.float().cpu().double().unflatten(-1, (-1, group)) * scale.cpu().double()[..., None]
            want = parts / (top / 448)[..., None]
            bound = (want.abs() * 2.0 ** -4).clamp_min(2.0 ** -10)
            bound = (bound + want.abs() * (roundings(D) + 4) * R.U32) * (top / 448)[..., None] * 1.001
            assert ((value - parts).abs() <= bound).all()


# rows for two rounds and more of the blocks that fit at once, with an uneven last one: the
# next row's loads, the sums' two places and the row groups of a block are used again
@pytest.mark.parametrize("rows,D,dtype", [
    (60000, 32, BF16), (30001, 64, BF16), (15003, 128, BF16), (8005, 256, BF16), (5007, 512, BF16),
    (1609, 1024, BF16), (1613, 2048, BF16), (700, 4096, BF16), (331, 8192, BF16), (311, 16384, BF16),
    (1901, 1001, BF16), (60000, 16, F32), (30001, 32, F32), (15003, 64, F32), (8005, 128, F32),
    (5007, 200, F32), (1609, 512, F32), (1613, 1000, F32), (700, 2048, F32), (331, 4096, F32),
    (311, 8192, F32), (1901, 77, F32)])
def test_gradients_of_many_rows(gdn, rows, D, dtype):
    d = draw((rows, D), dtype, D + 3)
    for gate, dres in ((None, d["dres"]), (d["gate"], None)):
        dx, dw, dg = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=gate, d_res=dres, eps=EPS)
        ref = R.norm_grads(d["dy"], d["x"], d["w"], gate, dres, EPS)
        c = bwd_roundings(D, rows)
        R.close(dx, ref[0], ref[3], c)
        R.close(dw, ref[1], ref[4], c)
        if gate is not None:
            R.close(dg, ref[2], ref[5] + 1e-30, c)
        again = gdn.rms_norm_bwd(d["dy"], d["x"], d["w"], gate=gate, d_res=dres, eps=EPS)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip((dx, dw, dg), again))
