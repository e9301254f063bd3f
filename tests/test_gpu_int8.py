"""GPU parity of the int8 experts with the oracle, and what must not change a bit.

Bit for bit: the activation codes and scales, the packed weights, the FC2 rows
from the GPU's own codes (the integer sums are exact and the two scale products
have one order), whole forwards whose SwiGLU rows hold no rounding, and any
forward across capacities, tile designs, streams and replays.  Elsewhere the
SwiGLU's exponential may move a bf16 rounding of the FC2 input: a SwiGLU value
then differs by at most one bf16 step (2^-7 of it), so a dequantized code by at
most 127 2^-7 + 1 + 2^-8 < 2.01 steps of its row, and the forward stays within
the framework's tolerance.
"""
import numpy as np
import pytest
import torch

import oracle
from workloads import WORKLOADS, Workload
from gpu_common import Case, assert_close, live_tensor, sentinel_out, to_dev_bits, SENTINEL_BITS

pytestmark = pytest.mark.gpu

CASES = {
    "tiny": Workload("tiny", 64, 64, 128, 256, 8, 2, "int8"),
    "one_token": Workload("one_token", 1, 3, 96, 64, 4, 3, "int8"),
    "smallest": Workload("smallest", 5, 5, 32, 32, 1, 1, "int8"),
    "odd": Workload("odd", 77, 80, 96, 160, 5, 3, "int8"),
    # capacity above 1024: the 256-row and the 64-row launches
    "odd_big": Workload("odd_big", 1500, 1600, 544, 288, 6, 2, "int8", bias=True),
    "k_below_256": Workload("k_below_256", 1200, 1200, 192, 224, 3, 2, "int8"),
    "one_expert": Workload("one_expert", 1100, 1100, 256, 288, 1, 1, "int8"),
    "decode_T64": Workload("decode_T64", 64, 64, 2048, 1024, 64, 6, "int8"),
    "bounded_T40": Workload("bounded_T40", 40, 2048, 2688, 1856, 16, 6, "int8"),
    "top16": Workload("top16", 33, 40, 64, 96, 1024, 16, "int8"),
    "rows_above_8192": Workload("rows_above_8192", 3, 3, 8224, 32, 2, 1, "int8"),
}
_cases = {}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import swiglu_expert_mlp_amd  # noqa: F401  (raises if the library is missing)


def get_case(name):
    if name not in _cases:
        _cases[name] = Case(CASES[name], seed=13, outliers=True)
    return _cases[name]


def new_moe(c):
    from swiglu_expert_mlp_amd import MoE
    moe = MoE(c.w.E, c.w.H, c.w.F, c.w.k, "int8")
    moe.load_weights(*c.weights_dev())
    return moe


def forward(c, moe=None, **kw):
    w = c.w
    moe = moe or new_moe(c)
    x, ids, probs = c.dev()
    ws = moe.new_workspace(w.T_cap)
    ws.fill_(0xA5)
    out = sentinel_out(w.T_cap, w.H)
    moe.forward(x, ids, probs, live_tensor(w.T), out=out, ws=ws, **kw)
    assert moe.check(ws) == 0
    return moe, ws, out.cpu().numpy()


def rows_of(moe, ws, w):
    idx = moe.get_indices(ws, w.T_cap)
    return idx, moe.get_rows(ws, w.T_cap, idx["n_rows"], idx["T"])


@pytest.mark.parametrize("name", list(CASES))
def test_activation_codes_and_weights_bitwise(name):
    c = get_case(name)
    w = c.w
    moe, ws, _ = forward(c)
    _, rows = rows_of(moe, ws, w)
    q, s = oracle.int8_quantize(oracle.bf16_value(c.inp["x_bits"][: w.T]))
    assert np.array_equal(rows["x_scales"], s)
    assert np.array_equal(rows["x_codes"], q)
    ref = oracle.pack(w.E, w.H, w.F, c.inp["w1_bits"], c.inp["w2_bits"], "int8")
    off = moe.kbuf.cpu().numpy()
    assert np.array_equal(off, ref) or _same_but_padding(off, ref, w)


def _same_but_padding(a, b, w):
    """The 256-byte padding after the scale sections is not written."""
    up = lambda v: (v + 255) // 256 * 256
    pitch = lambda K: (K + 63) // 64 * 64 if K < 256 else (K + 127) // 128 * 128
    at = 0
    for n in (w.E * 2 * w.F * pitch(w.H), w.E * w.H * pitch(w.F), 4 * w.E * 2 * w.F, 4 * w.E * w.H):
        if not np.array_equal(a[at: at + n], b[at: at + n]):
            return False
        at += up(n)
    return at == a.size


@pytest.mark.parametrize("name", list(CASES))
def test_fc2_rows_bitwise_from_own_codes(name):
    """(float)(integer sum) * weight scale * row scale, in fp32 and that order."""
    c = get_case(name)
    w = c.w
    moe, ws, _ = forward(c)
    idx, rows = rows_of(moe, ws, w)
    q2, s2 = oracle.int8_quantize(oracle.bf16_value(c.inp["w2_bits"]).reshape(-1, w.F))
    q2, s2 = q2.reshape(w.E, w.H, w.F), s2.reshape(w.E, w.H)
    for e in range(w.E):
        a, b = idx["offsets"][e], idx["offsets"][e + 1]
        if a == b:
            continue
        acc = rows["fc1_codes"][a:b].astype(np.float64) @ q2[e].astype(np.float64).T    # exact
        ref = acc.astype(np.float32) * s2[e][None, :] * rows["fc1_scales"][a:b, None]
        assert np.array_equal(rows["fc2_rows"][a:b], ref), e


@pytest.mark.parametrize("name", ["tiny", "one_token", "smallest", "odd", "odd_big", "k_below_256", "one_expert",
                                  "top16", "rows_above_8192"])
def test_forward_against_the_oracle(name):
    c = get_case(name)
    w = c.w
    moe, ws, out = forward(c)
    ref, err, extras = c.oracle_model().forward(c.inp["x_bits"], c.ids, c.probs, w.T, want_rows=True)
    assert err == 0
    _, rows = rows_of(moe, ws, w)
    n = rows["fc1_codes"].shape[0]
    got = rows["fc1_codes"] * rows["fc1_scales"][:, None]
    step = np.abs(extras["H"][:n]).max(axis=1, keepdims=True) / 127
    assert np.all(np.abs(got - extras["H"][:n]) <= 2.01 * step + 1e-30)
    assert_close(out[: w.T], ref[: w.T], name)
    assert np.all(out[w.T:].view(np.uint32) == SENTINEL_BITS), "rows past live were written"


@pytest.mark.parametrize("name", ["decode_T64", "bounded_T40"])
def test_forward_tokens_against_the_oracle(name):
    c = get_case(name)
    w = c.w
    _, _, out = forward(c)
    tokens = np.arange(0, w.T, max(1, w.T // 4))
    ref = c.oracle_model().forward_tokens(c.inp["x_bits"], c.ids, c.probs, tokens)
    assert_close(out[tokens], ref, name)


@pytest.mark.parametrize("T,cap", [(50, 50), (1300, 1300)])
def test_exact_experts_bitwise(T, cap):
    """x holds integers with 32 in coordinate 0, which every gate picks (g = 32 and
    silu(32) = 32); an up row picks one other coordinate: the SwiGLU row 32 x_j is a
    bf16 value, so every stage equals the oracle bit for bit, with given codes and
    scales (powers of two in FC1, any in FC2)."""
    from swiglu_expert_mlp_amd import MoE
    E, H, F, k = 4, 288, 160, 2
    rng = np.random.default_rng(T)
    x = rng.integers(-126, 127, (T, H)).astype(np.float32)
    x[:, 0], x[:, 1] = 32, 127                       # row scale 1
    w1 = np.zeros((E, 2 * F, H), np.int8)
    w1[:, :F, 0] = 2
    s1 = np.full((E, 2 * F), 0.5, np.float32)
    for e in range(E):
        w1[e, F + np.arange(F), rng.integers(1, H, F)] = rng.choice([-2, 2], F)
    w2 = rng.integers(-128, 128, (E, H, F)).astype(np.int8)
    s2 = rng.uniform(1e-4, 1e-2, (E, H)).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    probs = rng.uniform(0.1, 0.9, (T, k)).astype(np.float32)
    bits = oracle.bf16_bits(x)
    ref, err, _ = oracle.Model.quantized(E, H, F, k, w1, s1, w2, s2).forward(bits, ids, probs, T)
    assert err == 0
    moe = MoE(E, H, F, k, "int8")
    dev = lambda a: torch.from_numpy(a).cuda()
    moe.load_quantized(dev(w1), dev(s1), dev(w2), dev(s2))
    out = moe.forward(to_dev_bits(bits), dev(ids), dev(probs), live_tensor(T))
    assert np.array_equal(out.cpu().numpy(), ref)


def test_load_quantized_equals_load_weights():
    c = get_case("odd_big")
    w = c.w
    moe, _, a = forward(c)
    q1, s1 = oracle.int8_quantize(oracle.bf16_value(c.inp["w1_bits"]).reshape(-1, w.H))
    q2, s2 = oracle.int8_quantize(oracle.bf16_value(c.inp["w2_bits"]).reshape(-1, w.F))
    dev = lambda v, *shape: torch.from_numpy(v.reshape(shape)).cuda()
    # the refit: the same handle, weights of other sizes of value first
    moe.load_quantized(dev(q1 * 0, w.E, 2 * w.F, w.H), dev(s1, w.E, 2 * w.F), dev(q2, w.E, w.H, w.F),
                       dev(s2, w.E, w.H))
    _, _, z = forward(c, moe)
    assert not z[: w.T].any()
    moe.load_quantized(dev(q1, w.E, 2 * w.F, w.H), dev(s1, w.E, 2 * w.F), dev(q2, w.E, w.H, w.F),
                       dev(s2, w.E, w.H), kbuf=moe.kbuf)
    _, _, b = forward(c, moe)
    assert np.array_equal(a.view(np.uint32), b.view(np.uint32))


@pytest.mark.parametrize("name", ["odd_big", "k_below_256", "one_expert"])
def test_tile_designs_and_capacities_agree_bitwise(name):
    """A token's bits in a launch of 40 tokens (64-row tiles only) and in the whole one."""
    c = get_case(name)
    w = c.w
    moe, _, out = forward(c)
    x, ids, probs = c.dev()
    small = moe.forward(x[:40].contiguous(), ids[:40].contiguous(), probs[:40].contiguous(), live_tensor(40))
    assert np.array_equal(small.cpu().numpy(), out[:40])
    large = moe.forward(x, ids, probs, live_tensor(700))
    assert np.array_equal(large.cpu().numpy()[:700], out[:700])


@pytest.mark.parametrize("name", ["tiny", "odd_big"])
def test_combines_and_probabilities_in_fc1(name):
    c = get_case(name)
    w = c.w
    moe, ws, f32 = forward(c)
    idx, rows = rows_of(moe, ws, w)
    x, ids, probs = c.dev()
    live = live_tensor(w.T)
    b16 = moe.forward(x, ids, probs, live, combine="bf16")[: w.T]
    assert torch.equal(b16, torch.from_numpy(f32[: w.T]).cuda().to(torch.bfloat16))
    per_route = moe.forward(x, ids, None, live, combine="rows").cpu().numpy()[: w.T]
    assert np.array_equal(per_route, oracle.finalize_rows(rows["fc2_rows"], idx["dst"], w.H))
    # probabilities of one: the weighted rows are the rows
    ones = torch.ones_like(probs)
    a = moe.forward(x, ids, ones, live, topk_in_fc1=True)[: w.T]
    assert torch.equal(a, moe.forward(x, ids, ones, live)[: w.T])
    got = moe.forward(x, ids, probs, live, topk_in_fc1=True).cpu().numpy()
    ref, _, _ = c.oracle_model().forward(c.inp["x_bits"], c.ids, c.probs, w.T, topk_in_fc1=True)
    assert_close(got[: w.T], ref[: w.T], name)


def test_rows_of_zeros_tiny_and_non_finite_values():
    """A token of zeros gives +0; tokens near the ends of bf16's range keep their codes; a
    token with an infinity or a NaN gives NaN and touches no other token."""
    c = get_case("tiny")
    w = c.w
    bits = c.inp["x_bits"].copy()
    bits[1] = 0
    bits[2] = np.where(bits[2] & 0x8000, 0x8001, 1)            # subnormals
    bits[3] = (bits[3] & 0x807F) | 0x0080                       # just above 2^-126
    bits[4] = (bits[4] & 0x807F) | 0x7F00                       # near 2^127
    bits[5, 7] = 0x7F80
    bits[6, 9] = 0xFF80
    bits[7, 11] = 0x7FC0
    bits[8, 0] = 0xFFFF
    moe, _, clean = forward(c)
    _, ids, probs = c.dev()
    ws = moe.new_workspace(w.T_cap)
    out = moe.forward(to_dev_bits(bits), ids, probs, live_tensor(w.T), ws=ws).cpu().numpy()
    _, rows = rows_of(moe, ws, w)
    q, s = oracle.int8_quantize(oracle.bf16_value(bits[: w.T]))
    assert np.array_equal(rows["x_codes"], q)
    assert np.array_equal(rows["x_scales"].view(np.uint32)[:5], s.view(np.uint32)[:5])
    assert np.array_equal(out[1], np.zeros(w.H, np.float32))
    assert np.all(np.isnan(out[5:9])) and np.all(np.isnan(rows["x_scales"][5:9]))
    keep = np.r_[0, 9: w.T]
    assert np.array_equal(out[keep], clean[keep])


def test_dropped_routes_and_live_counts():
    from swiglu_expert_mlp_amd import DEVERR_BAD_EXPERT_ID, DEVERR_DUP_EXPERT_ID, DEVERR_LIVE_ABOVE_CAP
    c = get_case("odd")
    w = c.w
    moe, _, full = forward(c)
    x, ids, probs = c.dev()
    ids = ids.clone()
    ids[0, 1] = w.E + 4
    ids[1, 2] = ids[1, 1]
    ids[2] = -1                                                 # nothing left for token 2
    ws = moe.new_workspace(w.T_cap)
    out = moe.forward(x, ids, probs, live_tensor(w.T), ws=ws)
    assert moe.check(ws) == DEVERR_BAD_EXPERT_ID | DEVERR_DUP_EXPERT_ID
    ref, _, _ = c.oracle_model().forward(c.inp["x_bits"], ids.cpu().numpy(), c.probs, w.T)
    assert_close(out.cpu().numpy()[: w.T], ref[: w.T])
    assert not out[2].any()
    for live, bits in ((0, 0), (-3, 8), (w.T_cap + 5, DEVERR_LIVE_ABOVE_CAP | DEVERR_BAD_EXPERT_ID)):
        o = sentinel_out(w.T_cap, w.H)
        moe.forward(x, torch.from_numpy(c.ids).cuda(), probs, live_tensor(live), out=o, ws=ws)
        assert moe.check(ws) & bits == bits
        if live <= 0:
            assert np.all(o.cpu().numpy().view(np.uint32) == SENTINEL_BITS)
        else:
            assert np.array_equal(o.cpu().numpy()[: w.T], full[: w.T])


@pytest.mark.parametrize("name", ["tiny", "odd_big"])
def test_graph_replays_and_streams_bitwise(name):
    """A captured forward, replayed with eager work between, on new inputs each time."""
    c = get_case(name)
    w = c.w
    moe, _, _ = forward(c)
    x, ids, probs = c.dev()
    live = live_tensor(w.T)
    ws, ws2 = moe.new_workspace(w.T_cap), moe.new_workspace(w.T_cap)
    out = torch.zeros(w.T_cap, w.H, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.forward(x, ids, probs, live, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.forward(x, ids, probs, live, out=out, ws=ws)
    for n in range(4):
        x.copy_(torch.roll(x[: w.T], 1, 0) if w.T == w.T_cap else torch.cat([torch.roll(x[: w.T], 1, 0), x[w.T:]]))
        live.fill_(w.T - n)
        graph.replay()
        eager = moe.forward(x, ids, probs, live, ws=ws2)
        torch.cuda.synchronize()
        assert torch.equal(out[: w.T - n], eager[: w.T - n]), n


def _skewed(w, n_small=100, seed=7):
    """Routes: the first tokens to the upper half of the experts (about 50 rows each:
    64-row tiles), the rest to the lower half (256-row tiles)."""
    rng = np.random.default_rng(seed)
    half = w.E // 2
    ids = np.full((w.T_cap, w.k), -1, np.int32)
    for t in range(w.T):
        pool = np.arange(half, w.E) if t < n_small else np.arange(half)
        ids[t] = np.sort(rng.choice(pool, size=w.k, replace=False))
    probs = rng.uniform(0.1, 0.9, (w.T_cap, w.k)).astype(np.float32)
    return torch.from_numpy(ids).cuda(), torch.from_numpy(probs).cuda()


SPLIT = {
    # both stages have a 256-row and a 64-row launch: the 64-row chain is forked
    "both_split": Workload("both_split", 1400, 1500, 256, 288, 8, 2, "int8"),
    # one stage alone has two launches (the other's K is under 256): serial
    "fc1_split": Workload("fc1_split", 1400, 1500, 256, 96, 8, 2, "int8"),
    "fc2_split": Workload("fc2_split", 1400, 1500, 64, 256, 8, 2, "int8"),
}


@pytest.mark.parametrize("name", list(SPLIT))
def test_forked_chain_equals_the_serial_order(name):
    """Stage events keep the stages serial; the two orders give the same bits."""
    w = SPLIT[name]
    c = Case(w, seed=18)
    moe = new_moe(c)
    ids, probs = _skewed(w)
    x, live = c.dev()[0], live_tensor(w.T)
    ws = moe.new_workspace(w.T_cap)
    ws.fill_(0x5A)
    forked = moe.forward(x, ids, probs, live, out=sentinel_out(w.T_cap, w.H), ws=ws)
    counts = moe.get_indices(ws, w.T_cap)["counts"]
    assert counts[: w.E // 2].min() > 128 and 0 < counts[w.E // 2:].max() <= 128
    events = [torch.cuda.Event(enable_timing=True) for _ in range(6)]     # (the caller's: kept until the end)
    moe.set_stage_events(events)
    serial = moe.forward(x, ids, probs, live, out=sentinel_out(w.T_cap, w.H), ws=moe.new_workspace(w.T_cap))
    moe.set_stage_events(None)
    assert np.array_equal(forked.cpu().numpy().view(np.uint32), serial.cpu().numpy().view(np.uint32))
    ref, _, _ = c.oracle_model().forward(c.inp["x_bits"], ids.cpu().numpy(), probs.cpu().numpy(), w.T)
    assert_close(forked.cpu().numpy()[: w.T], ref[: w.T], name)


@pytest.mark.parametrize("F", [256, 1024, 2048, 4096, 8192, 8224])
def test_swiglu_rows_of_every_width(F):
    """Each width class of the SwiGLU rows' quantization, by all rows (serial) and by the
    tiles of each chain (forked), against the oracle's rows."""
    w = Workload(f"width_{F}", 1300, 1310, 256, F, 4, 1, "int8")
    c = Case(w, seed=19)
    moe = new_moe(c)
    ids, probs = _skewed(w)
    x, live = c.dev()[0], live_tensor(w.T)
    ref, err, extras = c.oracle_model().forward(c.inp["x_bits"], ids.cpu().numpy(), probs.cpu().numpy(), w.T,
                                                want_rows=True)
    assert err == 0
    events = [torch.cuda.Event(enable_timing=True) for _ in range(6)]
    seen = []
    for ev in (None, events):
        moe.set_stage_events(ev)
        ws = moe.new_workspace(w.T_cap)
        ws.fill_(0x5A)
        out = moe.forward(x, ids, probs, live, out=sentinel_out(w.T_cap, w.H), ws=ws).cpu().numpy()
        assert moe.check(ws) == 0
        _, rows = rows_of(moe, ws, w)
        codes, scales = rows["fc1_codes"], rows["fc1_scales"]
        n = codes.shape[0]
        assert n == w.T and np.all(np.abs(codes.astype(np.int32)).max(axis=1) == 127)
        step = np.abs(extras["H"][:n]).max(axis=1, keepdims=True) / 127
        assert np.all(np.abs(codes * scales[:, None] - extras["H"][:n]) <= 2.01 * step + 1e-30)
        assert_close(out[: w.T], ref[: w.T], w.name)
        seen.append((codes, scales, out.view(np.uint32)))
    moe.set_stage_events(None)
    assert all(np.array_equal(a, b) for a, b in zip(*seen))


def test_two_caller_streams_share_one_handle():
    """Forwards on two streams at once (one handle and so one side stream, two workspaces)."""
    w = SPLIT["both_split"]
    c = Case(w, seed=19)
    moe = new_moe(c)
    ids, probs = _skewed(w)
    live = live_tensor(w.T)
    xs = [c.dev()[0]]
    xs.append(torch.flip(xs[0][: w.T], dims=[0]).contiguous())
    xs[1] = torch.cat([xs[1], xs[0][w.T:]])
    refs = [moe.forward(x, ids, probs, live, out=sentinel_out(w.T_cap, w.H)) for x in xs]
    outs = [[sentinel_out(w.T_cap, w.H) for _ in range(4)] for _ in xs]
    wss = [moe.new_workspace(w.T_cap) for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for n in range(4):
        for i, s in enumerate(streams):
            moe.forward(xs[i], ids, probs, live, out=outs[i][n], ws=wss[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert np.array_equal(o.cpu().numpy().view(np.uint32), refs[i].cpu().numpy().view(np.uint32))


def test_forked_chain_captured_and_replayed():
    w = SPLIT["both_split"]
    c = Case(w, seed=20)
    moe = new_moe(c)
    ids, probs = _skewed(w)
    x, live = c.dev()[0], live_tensor(w.T)
    ws, ws2 = moe.new_workspace(w.T_cap), moe.new_workspace(w.T_cap)
    out = sentinel_out(w.T_cap, w.H)
    moe.forward(x, ids, probs, live, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.forward(x, ids, probs, live, out=out, ws=ws)
    for n in range(4):
        x[: w.T] = torch.roll(x[: w.T], 3, 0)
        live.fill_(w.T - 11 * n)
        graph.replay()
        eager = moe.forward(x, ids, probs, live, ws=ws2)
        torch.cuda.synchronize()
        assert torch.equal(out[: w.T - 11 * n], eager[: w.T - 11 * n]), n


def test_refused_options():
    c = get_case("tiny")
    moe = new_moe(c)
    x, ids, probs = c.dev()
    live = live_tensor(c.w.T)
    for kw in (dict(fused_ffn=True), dict(fused_finalize=True), dict(combine="rows", topk_in_fc1=True)):
        with pytest.raises(ValueError):
            moe.forward(x, ids, probs, live, **kw)
    with pytest.raises(TypeError):
        moe.forward(x.half(), ids, probs, live)
    noalloc = moe.forward_noalloc(x, ids, probs, live)
    assert torch.equal(noalloc, moe.forward(x, ids, probs, live))


@pytest.mark.parametrize("workload", ["bf16_16k", "logprob"])
def test_full_size_tokens(workload):
    """Sampled tokens of the full-size launches against the oracle's per-token loop, and
    the FC2 rows of one expert bit for bit."""
    from dataclasses import replace
    w = replace(WORKLOADS[workload], precision="int8")
    c = Case(w, seed=11, outliers=True)
    moe, ws, out = forward(c)
    tokens = np.linspace(0, w.T - 1, 6).astype(np.int64)
    m = oracle.Model(w.E, w.H, w.F, w.k, c.inp["w1_bits"], c.inp["w2_bits"], "int8")
    assert_close(out[tokens], m.forward_tokens(c.inp["x_bits"], c.ids, c.probs, tokens), workload)
    again = moe.forward(*c.dev(), live_tensor(w.T), ws=ws)
    assert np.array_equal(again.cpu().numpy(), out)
