"""GPU tests of the router's training operators against fp64 references: moe_balance,
moe_route_backward, moe_probs_backward, and a training step that runs them together
with the router and the experts.  Tolerances are counts of fp32 roundings
(router_train_ref.py)."""
import numpy as np
import pytest
import torch

from gpu_common import Case, live_tensor, to_dev_bits
from router_train_ref import EPS, balance_bounds, balance_ref, route_backward_ref, selected_probs
from workloads import Workload

pytestmark = pytest.mark.gpu

NAN = float("nan")
SENTINEL = 12345.678


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import swiglu_expert_mlp_amd  # noqa: F401  (raises if the library is missing)


def moe_of(E, k, H=32, F=32, precision="bf16"):
    from swiglu_expert_mlp_amd import MoE
    return MoE(E, H, F, k, precision)


def make(T, cap, E, k, seed=0, spread=1.0, mask=None):
    """Logits, ids (ascending), probabilities and their gradients, mask; rows past T are
    NaN, ids there out of range, the mask there set."""
    rng = np.random.default_rng(seed + 7 * T + E)
    z = np.full((cap, E), NAN, np.float32)
    z[:T] = rng.standard_normal((T, E)) * spread + rng.standard_normal(E)
    ids = np.full((cap, k), 0x7FC00000, np.int32)
    ids[:T] = np.sort(np.argsort(-z[:T], axis=1, kind="stable")[:, :k], axis=1)
    q = np.full((cap, k), NAN, np.float32)
    q[:T] = selected_probs(z[:T].astype(np.float64), ids[:T])
    d = np.full((cap, k), NAN, np.float32)
    d[:T] = rng.standard_normal((T, k))
    m = None
    if mask is not None:
        m = np.ones(cap, bool)
        m[:T] = rng.random(T) < mask
    return z, ids, q, d, m


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_balance(moe, z, ids, T, m, ws=None):
    ws = moe.new_balance_workspace(z.shape[0]) if ws is None else ws
    ws.fill_(0xA5)
    losses = torch.full((2,), SENTINEL, device="cuda")
    counts = torch.full((moe.E + 1,), -7, dtype=torch.int32, device="cuda")
    sums = torch.full((moe.E,), SENTINEL, device="cuda")
    moe.balance(dev(z), dev(ids), live_tensor(T), mask=dev(m), losses=losses, counts=counts, prob_sums=sums, ws=ws)
    return losses.cpu().numpy(), counts.cpu().numpy(), sums.cpu().numpy()


def in_order(T, E):
    """fp32 additions in a row of the balance sums: a lane's tokens, a wave's, 16 waves, a
    sixteenth of at most 512 partials, 16 again."""
    per = 64 if E <= 256 else 16
    blocks = 1 if T <= 4 * per else min(-(-T // per), 512)
    return -(-T // (blocks * per)) + 2 + 16 + 32 + 16 + 260 // 4


SIZES = [
    # T, cap, E, k
    (1, 1, 1, 1), (1, 4, 64, 6), (3, 3, 5, 5), (256, 256, 64, 6), (257, 300, 64, 6), (64, 64, 257, 16),
    (65, 70, 1024, 16), (1000, 1001, 63, 7), (777, 777, 130, 8), (2000, 2048, 128, 8), (500, 500, 512, 3),
    (300, 300, 1000, 10), (130, 130, 1023, 9), (4099, 4100, 256, 4), (40000, 40000, 8, 2), (30011, 30020, 6, 1),
]


@pytest.mark.parametrize("mask", [None, 0.7])
@pytest.mark.parametrize("T,cap,E,k", SIZES)
def test_balance(T, cap, E, k, mask):
    z, ids, _, _, m = make(T, cap, E, k, mask=mask)
    keep = np.ones(T, bool) if m is None else m[:T]
    losses, counts, sums = run_balance(moe_of(E, k), z, ids, T, m)
    rl, rc, rs = balance_ref(z[:T], ids[:T], keep)
    bl, bs = balance_bounds(z[:T], ids[:T], keep, in_order(cap, E))
    assert np.array_equal(counts, rc)
    assert np.all(np.abs(sums - rs) <= bs), np.max(np.abs(sums - rs) / bs)
    assert np.all(np.abs(losses - rl) <= bl), (losses, rl, bl)


@pytest.mark.parametrize("which", ["both", "probs", "losses"])
@pytest.mark.parametrize("mask", [None, 0.7])
@pytest.mark.parametrize("T,cap,E,k", SIZES)
def test_route_backward(T, cap, E, k, mask, which):
    z, ids, q, d, m = make(T, cap, E, k, mask=mask)
    keep = np.ones(T, bool) if m is None else m[:T]
    g = (0.5, 0.25)
    _, counts, _ = balance_ref(z[:T], ids[:T], keep)
    counts = counts.astype(np.int32)
    with_p, with_l = which != "losses", which != "probs"
    out = torch.full((cap, E), SENTINEL, device="cuda")
    moe_of(E, k).route_backward(
        dev(z), dev(ids) if with_p else None, live_tensor(T), d_logits=out, mask=dev(m),
        **(dict(probs=dev(q), d_probs=dev(d)) if with_p else {}),
        **(dict(counts=dev(counts), d_losses=torch.tensor(g, device="cuda")) if with_l else {}))
    out = out.cpu().numpy()
    ref, off = route_backward_ref(z[:T], ids[:T], keep, q[:T] if with_p else None, d[:T] if with_p else None,
                                  counts.astype(np.float64) if with_l else None, g)
    bad = np.abs(out[:T] - ref) > off
    assert not bad.any(), (np.argwhere(bad)[:4], np.max(np.abs(out[:T] - ref) / off))
    assert np.all(out[T:] == np.float32(SENTINEL)), "rows past live were written"


@pytest.mark.parametrize("E", [64, 128, 256, 512, 1024])
def test_logits_past_the_infinity_cache(E):
    """256 MiB of logits and more are read and written non-temporally: the sums against fp64
    on the GPU, sampled rows of the gradient against the reference."""
    k, T = 2, (1 << 26) // E + 5
    g = torch.Generator("cuda").manual_seed(E)
    z = torch.randn(T, E, generator=g, device="cuda")
    ids = z.topk(k, dim=1).indices.sort(dim=1).values.to(torch.int32)
    q = torch.softmax(z.gather(1, ids.long()), 1)
    d = torch.randn(T, k, generator=g, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") < 0.75
    moe, live = moe_of(E, k), live_tensor(T)
    losses, counts, sums = moe.balance(z, ids, live, mask=mask)
    n = int(mask.sum())
    ref, zl = torch.zeros(E, dtype=torch.float64, device="cuda"), 0.0
    for c in range(0, T, 1 << 16):
        zz = z[c: c + (1 << 16)][mask[c: c + (1 << 16)]].double()
        lse = torch.logsumexp(zz, 1)
        ref += torch.exp(zz - lse[:, None]).sum(0)
        zl += float(lse.square().sum())
    hits = torch.bincount(ids[mask].reshape(-1).long(), minlength=E)
    assert torch.equal(counts, torch.cat([hits, hits.new_tensor([n])]).to(torch.int32))
    # (2 |z - m| + 26) roundings a probability, |z - m| < 12, and those of the sum
    tol = (2 * 12 + 26 + in_order(T, E)) * EPS
    assert torch.all((sums.double() - ref).abs() <= tol * ref)
    bal = float((hits * ref).sum()) * E / (k * n * n)
    assert abs(float(losses[0]) - bal) <= (tol + (E / 64 + 40) * EPS) * bal
    # lse lies in [0, 13]: 2 (3 * 7 + 22 + |lse|) roundings of it, relative to its mean square
    assert abs(float(losses[1]) - zl / n) <= (2 * 60 * EPS * 13 / (zl / n) ** 0.5 + in_order(T, E) * EPS) * zl / n
    dz = moe.route_backward(z, ids, live, probs=q, d_probs=d, counts=counts,
                            d_losses=torch.tensor([0.5, 0.25], device="cuda"), mask=mask)
    rows = np.unique(np.r_[0:40, np.random.default_rng(E).integers(0, T, 100), T - 40: T])
    at = torch.from_numpy(rows).cuda()
    host = lambda t: t[at].cpu().numpy()
    ref, off = route_backward_ref(host(z), host(ids), host(mask), host(q), host(d),
                                  counts.cpu().numpy().astype(np.float64), (0.5, 0.25))
    assert np.all(np.abs(host(dz) - ref) <= off)


def test_kernel_gradient_against_differences():
    """The kernel's gradient against central differences of the losses in fp64."""
    T, E, k = 4, 6, 2
    z, ids, q, d, _ = make(T, T, E, k, seed=5)
    keep = np.ones(T, bool)
    gb, gz = 0.7, 0.3
    _, counts, _ = balance_ref(z, ids, keep)
    got = moe_of(E, k).route_backward(dev(z), dev(ids), live_tensor(T), probs=dev(q), d_probs=dev(d),
                                      counts=dev(counts.astype(np.int32)),
                                      d_losses=torch.tensor([gb, gz], device="cuda")).cpu().numpy()

    def value(zz):
        losses, _, _ = balance_ref(zz, ids, keep)
        return gb * losses[0] + gz * losses[1] + (d * selected_probs(zz, ids)).sum()

    z64 = z.astype(np.float64)
    for t in range(T):
        for e in range(E):
            up, dn = z64.copy(), z64.copy()
            up[t, e] += 1e-5
            dn[t, e] -= 1e-5
            # values of order one: some tens of fp32 roundings and 1e-9 of the difference
            assert abs((value(up) - value(dn)) / 2e-5 - got[t, e]) < 100 * EPS


def test_rows_that_leave_nothing():
    """Masked experts (-inf, the type's lowest value), whole rows of them, and NaN or
    infinities in tokens that do not count."""
    E, k, T = 8, 2, 6
    z, ids, q, d, _ = make(T, T, E, k)
    z[0, 3:] = -np.inf
    z[1] = -np.inf
    z[2, 1:] = np.finfo(np.float32).min
    z[3] = NAN
    z[4] = np.inf
    m = np.array([1, 1, 1, 0, 0, 1], bool)
    losses, counts, sums = run_balance(moe_of(E, k), z, ids, T, m)
    rz = z.astype(np.float64)
    rz[3:5] = 0
    rl, rc, rs = balance_ref(rz, ids, m)
    bl, bs = balance_bounds(rz, ids, m, in_order(T, E))
    assert np.array_equal(counts, rc) and np.all(np.abs(sums - rs) <= bs) and np.all(np.abs(losses - rl) <= bl)
    out = moe_of(E, k).route_backward(dev(z), None, live_tensor(T), mask=dev(m), counts=dev(rc.astype(np.int32)),
                                      d_losses=torch.tensor([0.5, 0.5], device="cuda")).cpu().numpy()
    ref, off = route_backward_ref(rz, ids, m, None, None, rc.astype(np.float64), (0.5, 0.5))
    assert np.all(np.abs(out - ref) <= off)
    assert not out[1].any() and not out[3:5].any() and not out[0, 3:].any()
    # a counted NaN is not hidden
    losses, _, sums = run_balance(moe_of(E, k), z, ids, T, None)
    assert np.isnan(losses).all() and np.isnan(sums).all()


@pytest.mark.parametrize("T,cap", [(0, 5), (0, 2000), (-4, 300)])
def test_no_tokens(T, cap):
    E, k = 70, 4
    z = np.full((cap, E), NAN, np.float32)
    ids = np.zeros((cap, k), np.int32)
    losses, counts, sums = run_balance(moe_of(E, k), z, ids, T, None)
    assert not losses.any() and not counts.any() and not sums.any()
    out = torch.full((cap, E), SENTINEL, device="cuda")
    f = torch.zeros(cap, k, device="cuda")
    moe_of(E, k).route_backward(dev(z), dev(ids), live_tensor(T), probs=f, d_probs=f, counts=dev(counts),
                                d_losses=torch.ones(2, device="cuda"), d_logits=out)
    assert torch.all(out == SENTINEL)
    # every token masked: no counted token, no division by zero
    z, ids, q, d, _ = make(9, 9, E, k)
    m = np.zeros(9, bool)
    losses, counts, sums = run_balance(moe_of(E, k), z, ids, 9, m)
    assert not losses.any() and not counts.any() and not sums.any()
    out = moe_of(E, k).route_backward(dev(z), None, live_tensor(9), mask=dev(m), counts=dev(counts),
                                      d_losses=torch.ones(2, device="cuda"))
    assert not out.any()


def test_live_count_above_the_capacity_is_clamped():
    z, ids, q, d, _ = make(50, 50, 12, 3)
    a = run_balance(moe_of(12, 3), z, ids, 50, None)
    b = run_balance(moe_of(12, 3), z, ids, 4000, None)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    g = [moe_of(12, 3).route_backward(dev(z), dev(ids), live_tensor(n), probs=dev(q), d_probs=dev(d)) for n in (50, 99)]
    assert torch.equal(*g)


@pytest.mark.parametrize("E", [20, 300])
def test_invalid_and_repeated_ids(E):
    """Ids outside [0, E) are in no count; a dropped route has no gradient and is in no sum."""
    k, T = 5, 40
    z, ids, q, d, _ = make(T, T, E, k)
    ids[0, 1], ids[1, 0], ids[2, 4] = E, -1, 2 ** 31 - 1
    ids[3, 2] = ids[3, 4]
    ids[4] = 7
    ids[5] = [9, 3, 9, 3, 3]
    ids[6] = -1
    _, counts, _ = run_balance(moe_of(E, k), z, ids, T, None)
    assert np.array_equal(counts, balance_ref(z, ids, np.ones(T, bool))[1])
    out = moe_of(E, k).route_backward(dev(z), dev(ids), live_tensor(T), probs=dev(q), d_probs=dev(d)).cpu().numpy()
    ref, off = route_backward_ref(z, ids, np.ones(T, bool), q, d, None, None)
    assert np.all(np.abs(out - ref) <= off)
    assert not out[6].any()


def test_balanced_loads_give_an_exact_zero():
    """Every expert with the same count: the balance loss has no gradient, to the bit."""
    E, k, T = 16, 2, 64
    z, _, _, _, _ = make(T, T, E, k)
    counts = np.append(np.full(E, T * k // E), T).astype(np.int32)
    out = moe_of(E, k).route_backward(dev(z), None, live_tensor(T), counts=dev(counts),
                                      d_losses=torch.tensor([1.0, 0.0], device="cuda"))
    assert not out.any()


def test_large_counts():
    """Counts summed over many batches: c E passes 32 bits."""
    E, k, T = 1024, 2, 8
    z, ids, _, _, _ = make(T, T, E, k)
    rng = np.random.default_rng(0)
    counts = np.append(rng.integers(0, 1 << 27, E), 1 << 30).astype(np.int32)
    out = moe_of(E, k).route_backward(dev(z), None, live_tensor(T), counts=dev(counts),
                                      d_losses=torch.tensor([1.0, 0.5], device="cuda")).cpu().numpy()
    ref, off = route_backward_ref(z, ids, np.ones(T, bool), None, None, counts.astype(np.float64), (1.0, 0.5))
    assert np.all(np.abs(out - ref) <= off)


def test_rows_do_not_depend_on_the_batch_and_repeats_agree():
    E, k, T = 128, 8, 3000
    z, ids, q, d, _ = make(T, T, E, k)
    moe = moe_of(E, k)
    _, counts, _ = balance_ref(z, ids, np.ones(T, bool))
    kw = dict(counts=dev(counts.astype(np.int32)), d_losses=torch.tensor([0.5, 0.1], device="cuda"))
    whole = moe.route_backward(dev(z), dev(ids), live_tensor(T), probs=dev(q), d_probs=dev(d), **kw)
    part = moe.route_backward(dev(z[1000:1037]), dev(ids[1000:1037]), live_tensor(37), probs=dev(q[1000:1037]),
                              d_probs=dev(d[1000:1037]), **kw)
    assert torch.equal(whole[1000:1037], part)
    a = run_balance(moe, z, ids, T, None)
    for _ in range(3):
        assert all(np.array_equal(x, y) for x, y in zip(a, run_balance(moe, z, ids, T, None)))


def test_two_streams_at_once():
    """Two calls in flight, each with its own workspace, outputs and stream."""
    cases, streams = [make(5000 + 13 * i, 5100, 256, 4, seed=i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    moe = moe_of(256, 4)
    alone = [run_balance(moe, c[0], c[1], 5000 + 13 * i, None) for i, c in enumerate(cases)]
    held = [(dev(c[0]), dev(c[1]), live_tensor(5000 + 13 * i), moe.new_balance_workspace(5100)) for i, c in enumerate(cases)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            z, ids, live, ws = held[i]
            with torch.cuda.stream(s):
                got[i].append(moe.balance(z, ids, live, ws=ws))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(g, alone[i]))


# ------------------------------------------------------------- probabilities of the combine

PROBS_CASES = {
    "tiny": Workload("tiny", 64, 64, 128, 256, 8, 2, "bf16"),
    "one": Workload("one", 1, 1, 32, 32, 1, 1, "bf16"),
    "decode": Workload("decode", 96, 100, 2048, 64, 32, 6, "int8"),
    "many": Workload("many", 3000, 3100, 96, 32, 20, 5, "bf16"),
    "odd_mxfp8": Workload("odd_mxfp8", 77, 80, 96, 160, 5, 3, "mxfp8"),
    "top16": Workload("top16", 40, 40, 544, 32, 64, 16, "int8"),
}
_cases = {}


def probs_case(name):
    if name not in _cases:
        c = Case(PROBS_CASES[name], seed=3)
        moe = moe_of(c.w.E, c.w.k, c.w.H, c.w.F, c.w.precision)
        moe.load_weights(*c.weights_dev())
        _cases[name] = (c, moe)
    return _cases[name]


def probs_ref(moe, ws, w, ids, d_out):
    """d_probs in listed order from the GPU's own rows, in fp64, and its bound."""
    idx = moe.get_indices(ws, w.T_cap)
    rows = moe.get_rows(ws, w.T_cap, idx["n_rows"], idx["T"])["fc2_rows"].astype(np.float64)
    T = idx["T"]
    ref, off = np.zeros((T, w.k)), np.zeros((T, w.k))
    for t in range(T):
        order = np.argsort(ids[t], kind="stable")
        for c, j in enumerate(order):
            r = idx["dst"][t, c]
            if r >= 0:
                prod = d_out[t].astype(np.float64) * rows[r]
                ref[t, j], off[t, j] = prod.sum(), np.abs(prod).sum()
    # a lane adds at most H / 64 products, then 6 lane steps and 8 waves
    return ref, off * (w.H / 64 + 16) * EPS + 1e-37


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", list(PROBS_CASES))
def test_probs_backward(name, grad):
    c, moe = probs_case(name)
    w = c.w
    x, ids, probs = c.dev()
    rng = np.random.default_rng(1)
    # listed in another order than the canonical one
    perm = np.stack([rng.permutation(w.k) for _ in range(w.T_cap)])
    ids = torch.from_numpy(np.take_along_axis(c.ids, perm, axis=1)).cuda()
    probs = torch.from_numpy(np.take_along_axis(c.probs, perm, axis=1)).cuda()
    ws = moe.new_workspace(w.T_cap)
    for combine in ("fp32", "bf16", "rows"):
        moe.forward(x, ids, probs, live_tensor(w.T), ws=ws, combine=combine)
        d_out = torch.full((w.T_cap, w.H), NAN, device="cuda", dtype=grad)
        d_out[: w.T] = torch.from_numpy(rng.standard_normal((w.T, w.H)).astype(np.float32)).cuda().to(grad)
        got = torch.full((w.T_cap, w.k), SENTINEL, device="cuda")
        moe.probs_backward(d_out, ids, ws, d_probs=got)
        assert moe.check(ws) == 0
        ref, off = probs_ref(moe, ws, w, ids.cpu().numpy(), d_out.float().cpu().numpy())
        got = got.cpu().numpy()
        assert np.all(np.abs(got[: w.T] - ref) <= off), combine
        assert np.all(got[w.T:] == np.float32(SENTINEL)), "rows past live were written"


def test_probs_backward_is_the_combine_gradient():
    """<d_out, out> is linear in the probabilities: its differences are the gradient."""
    c, moe = probs_case("tiny")
    w = c.w
    x, ids, probs = c.dev()
    live, ws = live_tensor(w.T), moe.new_workspace(w.T_cap)
    d_out = torch.randn(w.T_cap, w.H, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    value = lambda p: (moe.forward(x, ids, p, live).double() * d_out.double()).sum(1)
    moe.forward(x, ids, probs, live, ws=ws)
    got = moe.probs_backward(d_out, ids, ws).double()
    for j in range(w.k):
        up = probs.clone()
        up[:, j] += 1.0
        step = (up[:, j] - probs[:, j]).double()
        diff = (value(up) - value(probs)) / step
        # each out element is off by k + 1 roundings of its terms, the gradient by H / 64 + 16
        size = (moe.forward(x, ids, up, live).abs().double() * d_out.abs().double()).sum(1) * 4
        rows = moe.forward(x, ids, None, live, combine="rows").double().abs()[:, j]
        size = size + (rows * d_out.abs().double()).sum(1)
        assert torch.all((diff - got[:, j]).abs() <= size * (w.H / 64 + 20) * EPS)


def test_probs_backward_of_dropped_routes():
    c, moe = probs_case("odd_mxfp8")
    w = c.w
    x, ids, probs = c.dev()
    ids = ids.clone()
    ids[0, 1], ids[1, 2], ids[2] = w.E, ids[1, 0], -1
    ws = moe.new_workspace(w.T_cap)
    moe.forward(x, ids, probs, live_tensor(w.T), ws=ws)
    d_out = torch.randn(w.T_cap, w.H, device="cuda")
    got = moe.probs_backward(d_out, ids, ws).cpu().numpy()
    ref, off = probs_ref(moe, ws, w, ids.cpu().numpy(), d_out.cpu().numpy())
    assert np.all(np.abs(got[: w.T] - ref) <= off)
    assert got[0, 1] == 0 and got[1, 2] == 0 and not got[2].any()


def test_workspaces_without_the_rows_are_flagged():
    """No forward yet, another capacity, another shape, rows weighted inside FC1: nothing is
    read or written, and moe_check says so."""
    from swiglu_expert_mlp_amd import DEVERR_NO_ROWS, DEVERR_WEIGHTED_ROWS
    c, moe = probs_case("tiny")
    w = c.w
    x, ids, probs = c.dev()
    live = live_tensor(w.T)
    d_out = torch.randn(w.T_cap, w.H, device="cuda")
    got = torch.full((w.T_cap, w.k), SENTINEL, device="cuda")

    def flagged(ws, bit, n=w.T_cap):
        moe.probs_backward(d_out[:n], ids[:n], ws, d_probs=got[:n])
        assert moe.check(ws) == bit
        assert torch.all(got == SENTINEL)

    ws = moe.new_workspace(w.T_cap)
    for fill in (0, 0xA5, 0xFF):
        ws.fill_(fill)
        ws[:4] = 0                               # the error word of a workspace no call has run on
        flagged(ws, DEVERR_NO_ROWS)
    moe.forward(x, ids, probs, live, ws=ws)
    flagged(ws, DEVERR_NO_ROWS, w.T_cap - 8)
    other = moe_of(w.E, w.k, w.H, w.F, "int8")
    other.load_weights(*c.weights_dev())
    big = other.new_workspace(w.T_cap)
    other.forward(x, ids, probs, live, ws=big)
    flagged(big, DEVERR_NO_ROWS)
    moe.forward(x, ids, probs, live, ws=ws, topk_in_fc1=True)
    flagged(ws, DEVERR_WEIGHTED_ROWS)
    moe.forward(x, ids, probs, live, ws=ws)
    moe.probs_backward(d_out, ids, ws, d_probs=got)
    assert moe.check(ws) == 0 and not torch.any(got[: w.T] == SENTINEL)


def test_balance_in_a_forward_workspace_is_flagged():
    """A buffer that held a forward and then balance's partials holds no rows: the
    probabilities' gradient says so instead of reading the partials as indices."""
    from swiglu_expert_mlp_amd import DEVERR_NO_ROWS
    T, E, k, H = 1200, 64, 6, 64
    moe = moe_of(E, k, H, 32)
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=g)
    moe.load_weights(draw(E, 64, H).bfloat16(), draw(E, H, 32).bfloat16())
    z, live = draw(T, E), live_tensor(T)
    ws = moe.new_workspace(T)
    ids, probs = moe.route(z, live, ws=ws)
    moe.forward(draw(T, H).bfloat16(), ids, probs, live, ws=ws)
    assert moe.check(ws) == 0
    moe.balance(z, ids, live, ws=ws)
    got = torch.full((T, k), SENTINEL, device="cuda")
    moe.probs_backward(draw(T, H), ids, ws, d_probs=got)
    assert moe.check(ws) == DEVERR_NO_ROWS
    assert torch.all(got == SENTINEL)


def test_probs_backward_after_the_single_launch_modes():
    c, moe = probs_case("tiny")
    w = c.w
    x, ids, probs = c.dev()
    live, d_out = live_tensor(w.T), torch.randn(w.T_cap, w.H, device="cuda")
    got = []
    for kw in ({}, dict(fused_ffn=True), dict(fused_finalize=True)):
        ws = moe.new_workspace(w.T_cap)
        moe.forward(x, ids, probs, live, ws=ws, **kw)
        got.append(moe.probs_backward(d_out, ids, ws))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ------------------------------------------------------------- a training step

class Step:
    """Router -> experts -> losses -> gradients of the probabilities and of the logits."""

    def __init__(self, name="decode", seed=0):
        self.c, self.moe = probs_case(name)
        w, moe = self.c.w, self.moe
        self.x, _, _ = self.c.dev()
        self.logits = torch.from_numpy(self.c.inp["logits"]).cuda()
        self.live = live_tensor(w.T)
        self.mask = torch.rand(w.T_cap, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) < 0.8
        self.d_out = torch.randn(w.T_cap, w.H, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + 1))
        self.d_losses = torch.tensor([0.01, 0.001], device="cuda")
        self.ws, self.bws = moe.new_workspace(w.T_cap), moe.new_balance_workspace(w.T_cap)
        self.out = torch.zeros(w.T_cap, w.H, device="cuda")
        self.ids = torch.zeros(w.T_cap, w.k, dtype=torch.int32, device="cuda")
        self.probs, self.d_probs = (torch.zeros(w.T_cap, w.k, device="cuda") for _ in range(2))
        self.d_logits = torch.zeros(w.T_cap, w.E, device="cuda")
        self.losses, self.sums = torch.zeros(2, device="cuda"), torch.zeros(w.E, device="cuda")
        self.counts = torch.zeros(w.E + 1, dtype=torch.int32, device="cuda")

    def __call__(self):
        moe = self.moe
        moe.route(self.logits, self.live, ids=self.ids, probs=self.probs, ws=self.ws)
        moe.forward(self.x, self.ids, self.probs, self.live, out=self.out, ws=self.ws)
        moe.balance(self.logits, self.ids, self.live, mask=self.mask, losses=self.losses, counts=self.counts,
                    prob_sums=self.sums, ws=self.bws)
        moe.probs_backward(self.d_out, self.ids, self.ws, d_probs=self.d_probs)
        moe.route_backward(self.logits, self.ids, self.live, probs=self.probs, d_probs=self.d_probs,
                           counts=self.counts, d_losses=self.d_losses, mask=self.mask, d_logits=self.d_logits)

    def results(self):
        T = self.c.w.T
        return [self.out[:T], self.d_probs[:T], self.d_logits[:T], self.losses, self.counts, self.sums]


@pytest.mark.parametrize("name", ["decode", "many"])
def test_training_step_against_fp64_autograd(name):
    """The gradient of <d_out, out> + 0.01 balance + 0.001 z with respect to the logits, the
    experts' rows being constants, against torch's autograd in fp64 on the CPU."""
    s = Step(name)
    s()
    w, moe = s.c.w, s.moe
    assert moe.check(s.ws) == 0
    T = w.T
    idx = moe.get_indices(s.ws, w.T_cap)
    rows = moe.get_rows(s.ws, w.T_cap, idx["n_rows"], T)["fc2_rows"]
    o = torch.from_numpy(rows[idx["dst"]]).double()                      # [T, k, H]
    z = s.logits[:T].cpu().double().requires_grad_()
    ids, keep = s.ids[:T].cpu().long(), s.mask[:T].cpu()
    q = torch.softmax(z.gather(1, ids), dim=1)
    p, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
    n = int(keep.sum())
    counts = torch.bincount(ids[keep].reshape(-1), minlength=w.E).double()
    balance = w.E / (w.k * n * n) * (counts * p[keep].sum(0)).sum()
    z_loss = lse[keep].square().sum() / n
    d_out = s.d_out[:T].cpu().double()
    ((o * q[:, :, None]).sum(1) * d_out).sum().add(0.01 * balance + 0.001 * z_loss).backward()
    dp, q64 = (o * d_out[:, None]).sum(2).numpy(), q.detach().numpy()
    ref, off = route_backward_ref(z.detach().numpy(), ids.numpy(), keep.numpy(), q64, dp,
                                  np.append(counts.numpy(), n), (0.01, 0.001))
    assert np.allclose(ref, z.grad.numpy(), rtol=0, atol=1e-9 * np.abs(ref).max())
    # besides the kernel's own roundings: those of d_probs (H / 64 + 16 of its terms) and of the
    # router's probabilities (2e-6 of them), each through q (d - <q, d>)
    mag = (o * d_out[:, None]).abs().sum(2).numpy() * (w.H / 64 + 16) * EPS + 4 * 2e-6 * np.abs(dp)
    extra = q64 * (mag + (q64 * mag).sum(1, keepdims=True) + 2 * 2e-6 * np.abs(q64 * dp).sum(1, keepdims=True))
    np.put_along_axis(off, ids.numpy(), np.take_along_axis(off, ids.numpy(), 1) + extra, 1)
    got = s.d_logits[:T].cpu().numpy()
    assert np.all(np.abs(got - z.grad.numpy()) <= off), np.max(np.abs(got - z.grad.numpy()) / off)
    assert abs(float(s.losses[0]) - float(balance.detach())) <= 2e-5 * float(balance.detach())
    assert abs(float(s.losses[1]) - float(z_loss.detach())) <= 2e-5 * float(z_loss.detach())


def test_training_step_captured_and_replayed():
    """The whole step in one graph, replayed on new inputs with eager work between."""
    s, e = Step("decode"), Step("decode")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    for n in range(4):
        T = s.c.w.T - n
        s.live.fill_(T)
        s.logits[:T].copy_(torch.roll(s.logits[:T], 1, 0) * 1.1)
        s.d_out.mul_(-0.5)
        graph.replay()
        for a in ("logits", "d_out", "live"):
            getattr(e, a).copy_(getattr(s, a))
        e()
        torch.cuda.synchronize()
        for a, b in zip(s.results(), e.results()):
            m = min(T, a.shape[0]) if a.dim() == 2 else a.shape[0]
            assert torch.equal(a[:m], b[:m]), n


# ------------------------------------------------------------- far offsets

def test_logit_offsets_past_32_bits():
    """2.15e9 logits: the last rows' gradients, and sums that hold every row."""
    E, k, T = 1024, 2, 2_100_007
    z = torch.empty(T, E, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    at = torch.arange(T, device="cuda", dtype=torch.int32)
    ids = torch.stack([at % (E - 1), torch.full_like(at, E - 1)], 1).contiguous()
    q = torch.full((T, k), 0.5, device="cuda")
    d = torch.stack([at % 7, at % 5], 1).float()
    moe, live = moe_of(E, k), live_tensor(T)
    losses, counts, sums = moe.balance(z, ids, live)
    hits = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts, torch.cat([hits, hits.new_tensor([T])]).to(torch.int32))
    total = float(sums.double().sum())               # every row's probabilities sum to 1
    assert abs(total - T) <= T * (2 * 12 + 26 + in_order(T, E)) * EPS
    dz = moe.route_backward(z, ids, live, probs=q, d_probs=d, counts=counts,
                            d_losses=torch.tensor([0.5, 0.25], device="cuda"))
    sel = torch.cat([torch.arange(0, 20), torch.arange(T // 2, T // 2 + 20), torch.arange(T - 40, T)]).cuda()
    host = lambda t: t[sel].cpu().numpy()
    ref, off = route_backward_ref(host(z), host(ids), np.ones(len(sel), bool), host(q), host(d),
                                  counts.cpu().numpy().astype(np.float64), (0.5, 0.25))
    assert np.all(np.abs(host(dz) - ref) <= off)


def test_row_offsets_past_32_bits():
    """1.06 million tokens of 2048 int8 codes (past 2^31) and as many fp32 rows: sampled far
    tokens against a small launch, and the probabilities' gradient <d_out, out> (one route a
    token, probability 1)."""
    E, H, F, T = 4, 2048, 64, 1_060_003
    g = torch.Generator("cuda").manual_seed(3)
    moe = moe_of(E, 1, H, F, "int8")
    moe.load_weights((torch.randn(E, 2 * F, H, generator=g, device="cuda") * 0.02).bfloat16(),
                     (torch.randn(E, H, F, generator=g, device="cuda") * 0.1).bfloat16())
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % E)[:, None].contiguous()
    probs = torch.ones(T, 1, device="cuda")
    ws = moe.new_workspace(T)
    out = moe.forward(x, ids, probs, live_tensor(T), ws=ws)
    sel = torch.cat([torch.arange(0, 50), torch.arange(T - 150, T)]).cuda()
    small = moe.forward(x[sel].contiguous(), ids[sel].contiguous(), probs[sel].contiguous(), live_tensor(len(sel)))
    assert torch.equal(out[sel], small)
    d_out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    got = moe.probs_backward(d_out, ids, ws)
    assert moe.check(ws) == 0
    prod = d_out[sel].double() * out[sel].double()
    assert torch.all((got[sel, 0].double() - prod.sum(1)).abs() <= prod.abs().sum(1) * (H / 64 + 16) * EPS)


def test_side_stream_calls_keep_what_they_allocate():
    """Calls on another stream that allocate their outputs and workspaces."""
    moe = moe_of(256, 4)
    z, ids, q, d, _ = (dev(a) for a in make(6000, 6000, 256, 4))
    live = live_tensor(6000)
    ref = moe.balance(z, ids, live)
    grad = moe.route_backward(z, ids, live, probs=q, d_probs=d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        got.append((moe.balance(z, ids, live, stream=side), moe.route_backward(z, ids, live, probs=q, d_probs=d,
                                                                               stream=side)))
        torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")   # takes what was freed
    torch.cuda.synchronize()
    for b, g in got:
        assert all(torch.equal(u, v) for u, v in zip(b, ref)) and torch.equal(g, grad)


def test_python_refusals():
    moe = moe_of(8, 2)
    z, ids = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    live, f = live_tensor(4), torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError):
        moe.route_backward(z, ids, live)
    with pytest.raises(ValueError):
        moe.route_backward(z, ids, live, d_probs=f)
    with pytest.raises(ValueError):
        moe.route_backward(z, ids, live, probs=f, d_probs=f, d_logits=z)
    with pytest.raises(TypeError):
        moe.balance(z.half(), ids, live)
    with pytest.raises(TypeError):
        moe.balance(z, ids.long(), live)
    with pytest.raises(ValueError):
        moe.balance(z, ids, live, mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        moe.balance(z, ids, live, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        moe.balance(z.t().contiguous().t(), ids, live)
    with pytest.raises(TypeError):
        moe.probs_backward(torch.zeros(4, 32, device="cuda").half(), ids, moe.new_workspace(4))
