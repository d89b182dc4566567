"""Runs of tokens over a pool of states (decode_runs) against the token recurrence in
float64, at the sizes and batches where the kernel can go wrong."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_130_b200 import binding
    return binding


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def draw(total, Hk, Hv, Dk, Dv, n_slots, dtype, seed, behind=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    rows = total + behind
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    d = dict(q=unit(rnd(rows, Hk, Dk)).to(dtype), k=unit(rnd(rows, Hk, Dk)).to(dtype),
             v=rnd(rows, Hv, Dv).to(dtype), la=-torch.nn.functional.softplus(rnd(rows, Hv)),
             be=torch.sigmoid(rnd(rows, Hv)), states=0.3 * rnd(n_slots, Hv, Dv, Dk))
    return {n: t.cuda() for n, t in d.items()}


def roundings(tokens, Dk):
    # a token: two dot products of Dk terms (4 or 8 per lane, then 5 levels), the product
    # sums of up to 8 tokens, the rank-one update, the gates' and the norms' functions
    return tokens * (Dk / 16 + 48)


def check(gdn, d, cu, slots, dtype, update=True, **kw):
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda") if x is not None else None
    out = torch.full(d["v"].shape, 7.0, dtype=dtype, device="cuda")
    states = d["states"].clone()
    o = gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], states, slots=dev(slots),
                        cu_seqlens=dev(cu), out=out, update=update, **kw)
    torch.cuda.synchronize()
    assert o is out
    ref = R.runs(d["q"], d["k"], d["v"], d["la"], d["be"], d["states"], slots, cu,
                 torch.full(d["v"].shape, 7.0), update, kw.get("l2norm_qk", False),
                 kw.get("gate_logits", False))
    longest = max([b - a for _, a, b in R.spans(cu, d["v"].shape[0])], default=1)
    c = roundings(longest, d["k"].shape[2])
    R.close(o, ref[0], ref[2], c)
    R.close(states, ref[1], ref[3], c)
    return o, states


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 16, 16), (2, 4, 128, 128), (3, 3, 72, 40),
                                         (1, 4, 64, 200), (2, 2, 256, 512), (1, 2, 20, 7),
                                         (2, 2, 7, 3), (1, 1, 1, 1), (1, 3, 130, 65),
                                         (2, 2, 33, 130), (1, 1, 255, 66)])
def test_sizes(gdn, Hk, Hv, Dk, Dv, dtype):
    lens = [1, 8, 3, 9, 2]
    d = draw(sum(lens), Hk, Hv, Dk, Dv, 7, dtype, Dk + Dv)
    check(gdn, d, offsets(lens), [6, 0, 3, 1, 5], dtype)


@pytest.mark.parametrize("lens", [[1], [0], [0, 1, 0], [7, 8, 9, 16, 17], [1] * 40, [100, 1, 33]])
@pytest.mark.parametrize("update", [True, False])
def test_lengths(gdn, lens, update):
    d = draw(sum(lens), 2, 4, 64, 72, len(lens), F32, len(lens))
    check(gdn, d, offsets(lens), list(range(len(lens)))[::-1], F32, update)


def test_one_token_each_without_offsets(gdn):
    d = draw(9, 2, 2, 128, 128, 9, BF16, 3)
    o, S = check(gdn, d, None, None, BF16)
    # the same as the dense decode step, whose sums run in another order
    S2 = d["states"].clone()
    o2 = gdn.decode_step(d["q"], d["k"], d["v"], d["la"], d["be"], S2)
    assert (S - S2).abs().max() <= 64 * R.U32 * S2.abs().max() * 4
    assert (o.float() - o2.float()).abs().max() <= 2 * R.U[BF16] * o2.float().abs().max()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_raw_inputs(gdn, dtype):
    lens = [5, 1, 12]
    d = draw(sum(lens), 2, 4, 96, 48, 3, dtype, 5)
    g = torch.Generator().manual_seed(8)
    for n in ("q", "k"):
        d[n] = (3 * torch.randn(d[n].shape, generator=g)).to(dtype).cuda()
    d["la"] = torch.randn(d["la"].shape, generator=g).cuda()
    d["be"] = torch.randn(d["be"].shape, generator=g).cuda()
    check(gdn, d, offsets(lens), [2, 0, 1], dtype, l2norm_qk=True, gate_logits=True)


# the kernels: runs of several tokens in float32 (at a vector and an odd width) and in bf16
# on the tensor cores, and batches of single tokens (token by token)
KERNELS = [(F32, 32, 24, [3, 2, 1, 9]), (F32, 37, 24, [3, 2, 1, 9]), (BF16, 128, 40, [3, 2, 1, 9]),
           (BF16, 64, 136, [8, 2, 1, 17]), (F32, 128, 24, [1, 1, 1, 1]), (BF16, 72, 24, [2, 1, 1, 1]),
           (BF16, 72, 24, [1, 1, 1, 1])]


@pytest.mark.parametrize("dtype,Dk,Dv,lens", KERNELS)
def test_padding_rows_and_rows_behind(gdn, dtype, Dk, Dv, lens):
    # rows of padding (a slot below 0 or behind the pool), rows behind the last sequence and
    # unused slots may hold anything and stay out of the results
    d = draw(sum(lens), 1, 2, Dk, Dv, 6, dtype, 11, behind=4)
    cu = offsets(lens)
    for n in ("q", "k", "v", "la", "be"):
        d[n][cu[1]:cu[3]] = float("nan")
        d[n][cu[4]:] = float("inf")
    d["states"][4] = float("nan")
    o, S = check(gdn, d, cu, [5, -1, 6, 2], dtype)
    assert (o[cu[1]:cu[3]] == 0).all() and (o[cu[4]:] == 7).all()
    assert S[4].isnan().all() and torch.equal(S[0], d["states"][0])


@pytest.mark.parametrize("dtype,Dk,Dv,lens", [(F32, 48, 40, [0, 2, 3, 2, 9]), (BF16, 128, 40, [0, 2, 3, 2, 9]),
                                              (BF16, 48, 40, [0, 1, 2, 1, 1])])
def test_a_slot_named_twice(gdn, dtype, Dk, Dv, lens):
    # the first sequence with tokens has it; read-only runs share it
    d = draw(sum(lens), 1, 2, Dk, Dv, 4, dtype, 12)
    o, _ = check(gdn, d, offsets(lens), [1, 3, 1, 1, 3], dtype)
    assert (o[sum(lens[:3]):] == 0).all()
    o, _ = check(gdn, d, offsets(lens), [1, 3, 1, 1, 3], dtype, update=False)
    assert (o[sum(lens[:3]):] != 0).any()


def test_many_sequences_one_slot_twice(gdn):
    # the scan for an earlier owner covers more sequences than a block has threads
    N = 700
    d = draw(N, 1, 1, 16, 16, N, F32, 13)
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(1)).tolist()
    slots[650] = slots[3]
    check(gdn, d, None, slots, F32)


@pytest.mark.parametrize("dtype,Dk", [(F32, 64), (BF16, 64), (BF16, 128), (BF16, 40)])
def test_gates_at_their_ends(gdn, dtype, Dk):
    # a decay of exactly 0 (log alpha = -inf) in a run, none at all, writes of 0 and 1
    lens = [9, 4]
    d = draw(sum(lens), 1, 2, Dk, 32, 2, dtype, 14)
    d["la"][2] = d["la"][7] = float("-inf")
    d["la"][5], d["la"][10] = 0.0, -1e30
    d["be"][3], d["be"][4] = 0.0, 1.0
    check(gdn, d, offsets(lens), None, dtype)


@pytest.mark.parametrize("dtype,Dk", [(F32, 64), (BF16, 128), (F32, 30), (BF16, 64)])
def test_a_later_token_leaves_the_earlier_ones_alone(gdn, dtype, Dk):
    # NaN in the fourth token's k and the sixth's v: the outputs before them are what they
    # were, bit for bit, those behind are NaN
    d = draw(16, 1, 1, Dk, 32, 2, dtype, 21)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    run = lambda: gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], d["states"].clone(),
                                  cu_seqlens=dev([0, 8, 16]))
    a = run()
    d["k"][3] = float("nan")
    d["v"][8 + 5] = float("nan")
    b = run()
    assert torch.equal(a[:3], b[:3]) and b[3:8].isnan().all()
    assert torch.equal(a[8:13], b[8:13]) and b[13:].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_equal_keys_without_decay(gdn, dtype):
    # the same unit key eight times, written with strength 1: each write replaces the last,
    # and the system that joins the tokens is as far from the identity as it gets
    d = draw(8, 1, 1, 128, 64, 1, dtype, 22)
    d["k"][:] = 0.0
    d["k"][:, :, :16] = 0.25  # |k| = 1, exact in bf16
    d["la"].zero_()
    d["be"].fill_(1.0)
    _, S = check(gdn, d, [0, 8], None, dtype)
    # S k is the last v
    got = (S[0, 0].double() @ d["k"][7, 0].double()).cpu()
    assert (got - d["v"][7, 0].double().cpu()).abs().max() <= 64 * R.U32 * (8 * d["v"].abs().max() + 4).item()


@pytest.mark.parametrize("dtype,Dk,Dv", [(BF16, 128, 128), (BF16, 64, 96), (F32, 128, 64), (F32, 256, 20)])
def test_states_of_all_magnitudes(gdn, dtype, Dk, Dv):
    # rows of the state from 1e-18 to 1e18: nothing is lost beside larger numbers
    d = draw(12, 1, 1, Dk, Dv, 2, dtype, 23)
    d["states"] *= 10.0 ** torch.linspace(-18, 18, Dv, device="cuda")[:, None]
    d["v"] *= 0
    check(gdn, d, [0, 4, 12], None, dtype)


def test_read_only_then_commit(gdn):
    # a draft's outputs without moving the states, then its accepted half moves them
    lens = [8, 8, 8]
    d = draw(24, 2, 4, 128, 128, 3, BF16, 15)
    cu, dev = offsets(lens), lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    S = d["states"].clone()
    o = gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], S, cu_seqlens=dev(cu), update=False)
    assert torch.equal(S, d["states"])
    take = torch.cat([torch.arange(a, a + 4) for a in cu[:-1]]).cuda()
    part = {n: d[n][take].contiguous() for n in ("q", "k", "v", "la", "be")}
    none = gdn.decode_runs(None, part["k"], part["v"], part["la"], part["be"], S,
                           cu_seqlens=dev([0, 4, 8, 12]), want_output=False)
    assert none is None
    S2 = d["states"].clone()
    o2 = gdn.decode_runs(part["q"], part["k"], part["v"], part["la"], part["be"], S2,
                         cu_seqlens=dev([0, 4, 8, 12]))
    assert torch.equal(S, S2)
    # the tokens' outputs do not depend on those behind them, up to the sums' order
    R.close(o2, o[take].double(), o.float().abs().max().item(), 2 ** 16)


def test_slices_of_a_projection(gdn):
    lens = [4, 1, 9]
    for dtype, Hk, Hv, Dk, Dv in [(BF16, 2, 4, 128, 64), (F32, 1, 2, 12, 20), (BF16, 1, 1, 24, 8)]:
        d = draw(14, Hk, Hv, Dk, Dv, 3, dtype, 16)
        wide = torch.cat([d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1)], 1)
        gates = torch.cat([d["la"], d["be"]], 1)
        s = dict(d, q=wide[:, :Hk * Dk].unflatten(1, (Hk, Dk)),
                 k=wide[:, Hk * Dk:2 * Hk * Dk].unflatten(1, (Hk, Dk)),
                 v=wide[:, 2 * Hk * Dk:].unflatten(1, (Hv, Dv)), la=gates[:, :Hv], be=gates[:, Hv:])
        a = check(gdn, s, offsets(lens), [1, 2, 0], dtype)
        b = check(gdn, d, offsets(lens), [1, 2, 0], dtype)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_that_are_none(gdn):
    # negative, decreasing and too far: these sequences are left out, the others run
    d = draw(8, 1, 2, 16, 16, 6, F32, 17)
    cu = [-3, 2, 5, 4, 8, 99]  # valid: 2..5 and 4..8 (sharing row 4, so read only)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    S = d["states"].clone()
    out = torch.full(d["v"].shape, 7.0, device="cuda")
    gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], S, cu_seqlens=dev(cu), out=out,
                    update=False)
    torch.cuda.synchronize()
    ref = R.runs(d["q"], d["k"], d["v"], d["la"], d["be"], d["states"], None, cu,
                 torch.full(d["v"].shape, 7.0), False)
    keep = [0, 1, 2, 3, 5, 6, 7]
    R.close(out[keep], ref[0][keep], ref[2][keep], roundings(4, 16))


def test_graph_replay_with_other_offsets_and_slots(gdn):
    d = draw(12, 2, 4, 128, 64, 6, BF16, 18)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu, slots = dev([0, 4, 8, 12]), dev([0, 1, 2])
    S, out = d["states"].clone(), torch.zeros_like(d["v"])
    run = lambda: gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], S, slots=slots,
                                  cu_seqlens=cu, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for c, s in [([0, 1, 9, 12], [5, 3, 0]), ([0, 5, 5, 7], [1, 2, -1])]:
        cu.copy_(dev(c))
        slots.copy_(dev(s))
        S.copy_(d["states"])
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        ref = R.runs(d["q"], d["k"], d["v"], d["la"], d["be"], d["states"], s, c,
                     torch.full(d["v"].shape, 7.0))
        R.close(out, ref[0], ref[2], roundings(8, 128))
        R.close(S, ref[1], ref[3], roundings(8, 128))


def test_equal_calls_give_equal_bits_on_any_stream(gdn):
    lens = [3, 8, 1, 20]
    d = draw(sum(lens), 2, 4, 128, 128, 4, F32, 19)
    a = check(gdn, d, offsets(lens), [3, 1, 0, 2], F32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        b = check(gdn, d, offsets(lens), [3, 1, 0, 2], F32)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_pool_beyond_32_bit_offsets(gdn):
    # 140,000 slots of 16,384 floats: element offsets above 2^31
    slots, D = 140_000, 128
    states = torch.empty(slots, 1, D, D, device="cuda")
    d = draw(6, 1, 1, D, D, 1, F32, 20)
    use = [139_999, 131_072, 70_000]
    first = 0.3 * torch.randn(3, 1, D, D, generator=torch.Generator().manual_seed(2))
    states[use] = first.cuda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    o = gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], states, slots=dev(use),
                        cu_seqlens=dev([0, 1, 3, 6]))
    ref = R.runs(d["q"], d["k"], d["v"], d["la"], d["be"], first, [0, 1, 2], [0, 1, 3, 6],
                 torch.zeros(6, 1, D))
    R.close(o, ref[0], ref[2], roundings(3, D))
    R.close(states[use], ref[1], ref[3], roundings(3, D))


@pytest.mark.parametrize("dtype,Dk,behind", [(F32, 32, 0), (F32, 32, 8), (BF16, 64, 0), (BF16, 64, 8), (BF16, 40, 8)])
def test_sequences_left_out_keep_no_slot(gdn, dtype, Dk, behind):
    # offsets before the first token, behind the last, decreasing: such a sequence does not hold
    # the slot that it names (token by token, up to 8 at once, on the tensor cores)
    d = draw(12, 1, 2, Dk, 24, 5, dtype, 25, behind=behind)
    cu = [-3, 2, 5, 99, 8, 12]  # 2..5 and 8..12 run
    o, S = check(gdn, d, cu, [0, 0, 1, 3, 1], dtype)
    assert (o[2:5] != 0).any() and (o[8:12] != 0).any() and (o[5:8] == 7).all()
    assert not torch.equal(S[0], d["states"][0]) and not torch.equal(S[1], d["states"][1])


# ---- blocks that take several tiles of a head's rows: 296 (sequence, head) pairs and more

def many(lens, Hv, Dk, Dv, dtype, seed):
    n = len(lens)
    assert n * Hv >= 296
    d = draw(sum(lens), Hv // 2, Hv, Dk, Dv, n + 2, dtype, seed)
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(seed)).tolist()[:n]
    for i in range(0, n, 9):  # rows of padding, slots behind the pool, slots again
        slots[i] = [-1, n + 2, slots[i // 2]][i // 9 % 3]
    return d, offsets(lens), slots


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Dk,Dv", [(128, 72), (16, 300), (256, 33), (96, 70), (33, 140)])
def test_row_tiles_of_single_tokens(gdn, Dk, Dv, dtype):
    lens = [1] * 74
    lens[3] = lens[40] = 2  # a run of more than one token among them
    d, cu, slots = many(lens, 4, Dk, Dv, dtype, Dk + Dv)
    check(gdn, d, cu, slots, dtype)
    check(gdn, d, cu, None, dtype, update=False)


@pytest.mark.parametrize("dtype,Dk,Dv", [(F32, 128, 72), (F32, 16, 300), (F32, 256, 36), (F32, 37, 140),
                                         (BF16, 72, 72), (BF16, 256, 36), (BF16, 128, 136), (BF16, 64, 144)])
def test_row_tiles_of_runs(gdn, dtype, Dk, Dv):
    lens = [2] * 74
    lens[5], lens[6], lens[7], lens[50] = 9, 1, 17, 8
    d, cu, slots = many(lens, 4, Dk, Dv, dtype, Dk + Dv)
    check(gdn, d, cu, slots, dtype)
    check(gdn, d, cu, None, dtype, update=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Dk,Dv", [(33, 40), (130, 65), (200, 24), (255, 7), (256, 256), (1, 1)])
def test_single_tokens_of_any_width(gdn, Dk, Dv, dtype):
    d = draw(9, 1, 2, Dk, Dv, 7, dtype, Dk, behind=2)
    check(gdn, d, [0, 1, 2, 2, 3, 5, 6, 7, 8, 9], [6, 0, 1, -1, 3, 4, 5, 2, 9], dtype)
    check(gdn, d, [0, 1, 2, 2, 3, 5, 6, 7, 8, 9], [6, 0, 1, 3, 3, 4, 5, 2, 2], dtype, update=False)


@pytest.mark.parametrize("dtype,Dk", [(F32, 64), (BF16, 128), (BF16, 64), (F32, 30)])
def test_an_infinite_query_stays_with_its_token(gdn, dtype, Dk):
    # its own outputs are infinite or NaN, all others and the states bit for bit what they were
    d = draw(16, 1, 1, Dk, 32, 2, dtype, 24)
    run = lambda S: gdn.decode_runs(d["q"], d["k"], d["v"], d["la"], d["be"], S,
                                    cu_seqlens=torch.tensor([0, 8, 16], dtype=torch.int32, device="cuda"))
    S, S2 = d["states"].clone(), d["states"].clone()
    a = run(S)
    d["q"][3, 0, 5] = float("inf")
    b = run(S2)
    assert torch.equal(S, S2) and not torch.isfinite(b[3]).any()
    rest = [t for t in range(16) if t != 3]
    assert torch.equal(a[rest], b[rest])
