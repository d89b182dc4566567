"""The short causal convolution and its gradients against float64."""
import pytest
import torch

import layer_ref as R
from test_decode_runs_gpu import offsets

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_130_b200 import binding
    return binding


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda") if x is not None else None


def draw(total, C, W, n_slots, dtype, seed, bias=True, param=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    p = param or dtype
    return dict(x=rnd(total, C).to(dtype).cuda(), w=(0.5 * rnd(C, W)).to(p).cuda(),
                b=rnd(C).to(p).cuda() if bias else None,
                states=rnd(n_slots, W - 1, C).to(dtype).cuda(), dy=rnd(total, C).to(dtype).cuda())


# a sum of W products and the bias, the exponential, the division and two products; the
# fast exponential and division add a few units more at |z| up to 20
FWD = 48


def check_fwd(gdn, d, cu, slots, silu=True, splits=None, pool=True, out=None):
    states = d["states"].clone() if pool else None
    C = d["x"].shape[1]
    if out is None:
        out = tuple(torch.full((d["x"].shape[0], c), 7.0, dtype=d["x"].dtype, device="cuda")
                    for c in (splits or [C]))
    y = gdn.short_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=dev(cu), states=states,
                           slots=dev(slots), silu=silu, splits=splits,
                           out=out if splits else out[0])
    torch.cuda.synchronize()
    y = torch.cat(y, 1) if splits else y
    ref, S, scale, covered = R.conv(d["x"], d["w"], d["b"], cu, d["states"] if pool else None, slots,
                                    silu)
    R.close(y[covered.cuda()], ref[covered], scale[covered], FWD)
    assert (y[~covered.cuda()] == 7).all()
    if pool:
        assert torch.equal(states.double().cpu(), S) or \
            ((states.double().cpu() == S) | (S.isnan() & states.cpu().isnan())).all()
    return y, states


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 8, 37, 96, 1032])
def test_forward_sizes(gdn, C, W, dtype):
    lens = [1, 2, 3, 4, 5, 40, 0, 17]
    d = draw(sum(lens), C, W, 9, dtype, C + W)
    check_fwd(gdn, d, offsets(lens), [4, 0, 8, 1, 2, 7, 5, 3])
    check_fwd(gdn, d, offsets(lens), None, silu=False, pool=False)


@pytest.mark.parametrize("lens", [[1], [1] * 70, [16, 16, 16], [15, 1, 16, 17, 14, 2, 2, 100],
                                  [3] * 40, [0, 0, 31, 0, 33, 0], [1000, 7], [2] * 900])
def test_tile_edges(gdn, lens):
    # sequences that begin and end at every place of a tile; the held inputs of a sequence
    # whose first tokens lie in two tiles.  2048 channels: both tile heights run
    d = draw(sum(lens), 2048, 4, len(lens), BF16, len(lens), bias=False)
    slots = torch.randperm(len(lens), generator=torch.Generator().manual_seed(3)).tolist()
    check_fwd(gdn, d, offsets(lens), slots)
    check_fwd(gdn, dict(d, b=None), offsets(lens), None, pool=False)


def test_one_token_each_without_offsets(gdn):
    d = draw(33, 384, 4, 40, BF16, 1)
    check_fwd(gdn, d, None, list(range(7, 40)))
    check_fwd(gdn, d, None, None)


def test_parts_and_slices(gdn):
    lens, C = [5, 9, 1], 96
    for dtype, splits in [(BF16, [32, 32, 32]), (F32, [40, 56]), (BF16, [30, 33, 33]), (F32, [96])]:
        d = draw(15, C, 4, 3, dtype, 2)
        a, sa = check_fwd(gdn, d, offsets(lens), [2, 0, 1], splits=splits)
        wide = torch.zeros(15, C + 48, dtype=dtype, device="cuda")
        wide[:, 16:16 + C] = d["x"]
        b, sb = check_fwd(gdn, dict(d, x=wide[:, 16:16 + C]), offsets(lens), [2, 0, 1])
        assert torch.equal(a, b) and torch.equal(sa, sb)
        # the parts as column slices of one array
        y = torch.full((15, C), 7.0, dtype=dtype, device="cuda")
        at = offsets(splits)
        if all(v * y.element_size() % 16 == 0 for v in at):
            check_fwd(gdn, d, offsets(lens), [2, 0, 1], splits=splits,
                      out=tuple(y[:, m:n] for m, n in zip(at[:-1], at[1:])))
            assert torch.equal(y, a)


def test_padding_rows_behind_and_a_slot_twice(gdn):
    lens = [3, 2, 1, 9, 4, 2]
    d = draw(sum(lens) + 5, 64, 4, 5, F32, 4)
    cu = offsets(lens)
    d["x"][cu[1]:cu[3]] = float("nan")
    d["x"][cu[6]:] = float("inf")
    d["states"][3] = float("nan")
    y, S = check_fwd(gdn, d, cu, [4, -1, 5, 2, 4, 0])
    assert (y[cu[1]:cu[3]] == 0).all() and (y[cu[4]:cu[5]] == 0).all()


@pytest.mark.parametrize("kind", ["tokens", "ragged", "long", "one slot"])
def test_many_sequences_slots_again(gdn, kind):
    # slots named again inside a tile, tiles apart, by sequences with and without tokens
    g = torch.Generator().manual_seed(12)
    n, C = 2500, 1024
    lens = [1] * n
    if kind == "ragged":
        lens = torch.randint(0, 6, (n,), generator=g).tolist()
    if kind == "long":
        n, lens = 9, [700, 0, 3, 700, 1, 1, 2, 900, 300]
    slots = torch.randint(-1, n // 2, (n,), generator=g)
    slots[slots % 7 == 3] += n  # some out of the pool
    if kind == "one slot":
        slots[:] = 5
    if kind == "long":
        slots = torch.tensor([3, 2, 2, 3, -1, 1, 2, 2, 0])
    d = draw(sum(lens), C, 4, n // 2, BF16, 12, bias=False)
    check_fwd(gdn, d, offsets(lens) if kind != "tokens" else None, slots.tolist())


def test_prompt_then_tokens(gdn):
    # a prompt, then its continuation one token at a time, is the whole sequence at once
    for dtype in (F32, BF16):
        d = draw(12, 40, 4, 1, dtype, 5)
        d["states"].zero_()
        S = d["states"].clone()
        whole = gdn.short_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=dev([0, 12]))
        parts = [gdn.short_conv_fwd(d["x"][:7], d["w"], d["b"], cu_seqlens=dev([0, 7]), states=S)]
        parts += [gdn.short_conv_fwd(d["x"][t:t + 1], d["w"], d["b"], states=S) for t in range(7, 12)]
        assert torch.equal(torch.cat(parts), whole)


def test_infinities_stay_in_their_window(gdn):
    d = draw(20, 16, 4, 2, F32, 6)
    d["x"][9] = float("inf")
    d["w"].abs_()
    y = gdn.short_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=dev([0, 8, 10, 20]))
    assert torch.isfinite(y[:9]).all() and torch.isfinite(y[10:]).all()


def test_offsets_that_are_none(gdn):
    d = draw(40, 32, 4, 4, F32, 7)
    S = d["states"].clone()
    for cu in ([0, 50, 20], [-4, 10, 10], [7, 3, 90], [0, -1, 40]):
        gdn.short_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=dev(cu), states=S)
        gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu))
    torch.cuda.synchronize()


def test_graph_replay_with_other_offsets(gdn):
    d = draw(64, 256, 4, 6, BF16, 8)
    cu, slots, S = dev([0, 20, 40, 64]), dev([0, 1, 2]), d["states"].clone()
    y = torch.zeros_like(d["x"])
    run = lambda: gdn.short_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=cu, states=S, slots=slots,
                                     out=y)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for c, s in [([0, 1, 17, 64], [5, 3, 0]), ([0, 16, 16, 60], [1, 2, 4])]:
        cu.copy_(dev(c))
        slots.copy_(dev(s))
        S.copy_(d["states"])
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        ref, want, scale, covered = R.conv(d["x"], d["w"], d["b"], c, d["states"], s, True)
        R.close(y[covered.cuda()], ref[covered], scale[covered], FWD)
        assert (y[~covered.cuda()] == 7).all() and torch.equal(S.double().cpu(), want)


# dz is a product of four with two fast functions behind a sum of W; dw adds a tile's
# tokens in a chain, then the tiles
def bwd_roundings(total):
    return 64 + min(total, 160) + total / 64


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("C,W,lens", [(1, 2, [1]), (37, 3, [1, 2, 3, 4, 5, 0, 17]),
                                      (96, 4, [127, 1, 128, 129, 2, 2, 2]), (24, 4, [300]),
                                      (1032, 4, [9, 31]), (8, 2, [1] * 140)])
def test_gradients(gdn, C, W, lens, silu, dtype):
    d = draw(sum(lens) + 3, C, W, 1, dtype, C + W, bias=C != 24)
    cu = offsets(lens)
    d["x"][cu[-1]:] = float("nan")  # rows of no sequence
    d["dy"][cu[-1]:] = float("nan")
    dx, dw, db = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu), silu=silu)
    torch.cuda.synchronize()
    rx, rw, rb, sx, sw, sb = R.conv_grads(d["dy"], d["x"], d["w"], d["b"], cu, silu)
    c = bwd_roundings(sum(lens))
    R.close(dx, rx, sx, c)
    R.close(dw, rw, sw, c)
    assert (db is None) == (d["b"] is None)
    if db is not None:
        R.close(db, rb, sb, c)
    again = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu), silu=silu)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip((dx, dw, db), again))


def test_gradients_in_parts_without_offsets_and_float32_weights(gdn):
    d = draw(50, 96, 4, 1, BF16, 9, param=F32)
    for cu in ([0, 50], None):
        a = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu))
        parts = tuple(p.contiguous() for p in d["dy"].split([32, 16, 48], 1))
        b = gdn.short_conv_bwd(parts, d["x"], d["w"], d["b"], cu_seqlens=dev(cu))
        assert all(torch.equal(s, t) for s, t in zip(a, b))
        ref = R.conv_grads(d["dy"], d["x"], d["w"], d["b"], cu, True)
        for got, want, scale in zip(a, ref[:3], ref[3:]):
            R.close(got, want, scale, bwd_roundings(50))


def test_gradients_against_differences(gdn):
    # the float64 forward's central difference along a random direction
    d = draw(23, 5, 4, 1, F32, 10)
    cu = [0, 6, 23]
    dx, dw, db = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu))
    g = torch.Generator().manual_seed(5)
    to = {n: torch.randn(d[n].shape, generator=g, dtype=torch.float64) for n in ("x", "w", "b")}
    loss = lambda s: (R.conv(d["x"].cpu().double() + s * to["x"], d["w"].cpu().double() + s * to["w"],
                             d["b"].cpu().double() + s * to["b"], cu, None, None, True)[0]
                      * d["dy"].cpu().double()).sum()
    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    mine = sum((got.cpu().double() * to[n]).sum() for got, n in ((dx, "x"), (dw, "w"), (db, "b")))
    size = sum((got.cpu().double() * to[n]).abs().sum() for got, n in ((dx, "x"), (dw, "w"), (db, "b")))
    assert (slope - mine).abs() <= 1e-5 * size  # differences: 1e-10 + 1e-11; float32: 90 u32


def test_tokens_beyond_32_bit_offsets(gdn):
    # 2.2e9 elements, all zero but the last tokens, which are two sequences
    total, C, n = 270_000, 8192, 40
    d = draw(n, C, 4, 2, BF16, 13)
    x = torch.zeros(total, C, dtype=BF16, device="cuda")
    dy = torch.zeros_like(x)
    x[-n:], dy[-n:] = d["x"], d["dy"]
    cu, some = dev([0, total - n, total - 7, total]), [0, n - 7, n]
    S, T = d["states"][[0, 0, 1]].clone(), d["states"].clone()
    y = gdn.short_conv_fwd(x, d["w"], cu_seqlens=cu, states=S)
    z = gdn.short_conv_fwd(d["x"], d["w"], cu_seqlens=dev(some), states=T)
    assert torch.equal(y[-n:], z) and torch.equal(S[1:], T) and not S[0].any()
    del y
    dx, dw, _ = gdn.short_conv_bwd(dy, x, d["w"], cu_seqlens=cu)
    assert not dx[:-n].any()
    rx, rw, _, sx, sw, _ = R.conv_grads(d["dy"], d["x"], d["w"], None, some, True)
    R.close(dx[-n:], rx, sx, bwd_roundings(n))
    R.close(dw, rw, sw, bwd_roundings(n))


def test_no_tokens(gdn):
    d = draw(0, 16, 4, 1, F32, 11)
    for cu in ([0], [0, 0], None):
        assert gdn.short_conv_fwd(d["x"], d["w"], d["b"], cu_seqlens=dev(cu)).shape == (0, 16)
        dx, dw, db = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu))
        assert dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    d = draw(4, 16, 4, 1, F32, 11)  # tokens, but no sequence
    dx, dw, db = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev([0]))
    assert (dx == 0).all() and (dw == 0).all() and (db == 0).all()


def test_a_given_workspace(gdn):
    # the same bits, nothing behind its size written; one that is too small is not used
    d = draw(700, 96, 4, 1, BF16, 22)
    cu = dev([0, 300, 700])
    a = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=cu)
    need = gdn.short_conv_bwd_workspace_size(700, 96, 4)
    for size in (need, 16):
        ws = torch.full((need + 64,), 7, dtype=torch.uint8, device="cuda")
        b = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=cu, workspace=ws[:size])
        assert all(torch.equal(s, t) for s, t in zip(a, b)) and (ws[size:] == 7).all()


@pytest.mark.parametrize("tokens", [12, 5000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_offsets_outside_the_tokens(gdn, tokens, dtype):
    # a sequence that begins before the tokens and one that ends behind them are left out, and
    # the slots that they name are free for the others
    lens = [3] * ((tokens - 5) // 3)
    cu = [-3, 2] + [2 + a for a in offsets(lens)[1:]] + [tokens + 4]
    n = len(cu) - 1
    slots = [1, 1] + list(range(2, n - 1)) + [0]
    d = draw(tokens, 64, 4, n, dtype, 23)
    y, S = check_fwd(gdn, d, cu, slots)
    assert (y[:2] == 7).all() and (y[2:5] != 0).any() and not torch.equal(S[1], d["states"][1])
    d = dict(d, b=None)
    got = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], cu_seqlens=dev(cu))
    ref = R.conv_grads(d["dy"], d["x"], d["w"], None, cu, True)
    R.close(got[0], ref[0], ref[3], bwd_roundings(tokens))
    R.close(got[1], ref[1], ref[4], bwd_roundings(tokens))
    assert (got[0][:2] == 0).all()


# ---- the kernel over tiles of tokens, which calls of few blocks do not reach

def mixed(total, seed):
    """Lengths that begin and end sequences at every place of a tile and reach over tiles."""
    g = torch.Generator().manual_seed(seed)
    kinds = [0, 1, 1, 2, 2, 3, 4, 5, 7, 8, 9, 17, 40, 300]
    lens = []
    while sum(lens) < total:
        lens.append(min(kinds[int(torch.randint(len(kinds), (1,), generator=g))], total - sum(lens)))
    return lens


def tiled(C, total, vec):
    """Whether a forward of these sizes goes by tiles (more blocks than a batch of few tokens has)."""
    return -(-C // (128 * vec)) * total > 148 * 32


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,total", [(36, 4999), (1032, 5003), (37, 5001), (1029, 4801)])
def test_tiles(gdn, C, total, W, dtype):
    assert tiled(C, total, 4)
    lens = mixed(total, C + W)
    n = len(lens)
    g = torch.Generator().manual_seed(W)
    slots = torch.randperm(n, generator=g).tolist()
    for i in range(0, n, 11):      # rows of padding, slots behind the pool, slots again
        slots[i] = [-1, n, slots[i // 2]][i // 11 % 3]
    d = draw(total, C, W, n, dtype, C + W)
    cu = offsets(lens)
    check_fwd(gdn, d, cu, slots)
    check_fwd(gdn, dict(d, b=None), cu, None, silu=False)
    check_fwd(gdn, d, cu, None, silu=False, pool=False)
    splits = [C // 3, C // 3, C - 2 * (C // 3)]
    check_fwd(gdn, d, cu, slots, splits=splits)
    check_fwd(gdn, dict(d, b=None), cu, None, splits=[C - 8, 8], pool=False)


def test_high_tiles(gdn):
    # tiles of more tokens than a block has threads, sequences around their edges
    C, total = 6144, 12000
    lens = mixed(total, 5)
    d = draw(total, C, 4, len(lens), BF16, 21, bias=False)
    slots = torch.randperm(len(lens), generator=torch.Generator().manual_seed(3)).tolist()
    check_fwd(gdn, d, offsets(lens), slots)


@pytest.mark.parametrize("lens", [[15, 1, 16, 17, 14, 2, 2, 4750], [7] * 700, [8] * 620, [3] * 1600, [4800, 7]])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tile_edges_of_many_tokens(gdn, lens, dtype):
    assert tiled(64, sum(lens), 4)
    d = draw(sum(lens), 64, 4, len(lens), dtype, len(lens), bias=False)
    slots = torch.randperm(len(lens), generator=torch.Generator().manual_seed(3)).tolist()
    check_fwd(gdn, d, offsets(lens), slots)


@pytest.mark.parametrize("dtype,C,W", [(F32, 1032, 4), (BF16, 1032, 4), (F32, 37, 3), (BF16, 1029, 2), (BF16, 36, 4)])
def test_gradients_of_many_tokens(gdn, dtype, C, W):
    total = 5003
    lens = mixed(total, W)
    d = draw(total, C, W, 1, dtype, C + W)
    cu = offsets(lens)
    for silu in (True, False):
        got = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu), silu=silu)
        ref = R.conv_grads(d["dy"], d["x"], d["w"], d["b"], cu, silu)
        for a, want, scale in zip(got, ref[:3], ref[3:]):
            R.close(a, want, scale, bwd_roundings(total))
        again = gdn.short_conv_bwd(d["dy"], d["x"], d["w"], d["b"], cu_seqlens=dev(cu), silu=silu)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
