"""The experts' training operators on the GPU: the forward that keeps its gate and up in 8
bits, the backward pass, tokens sorted by expert and back, and their gradients."""
import pytest
import torch

from experts_train_ref import B, S, backward_ref, forward64, join, kept_values, row_of_ref, routes, split

pytestmark = pytest.mark.gpu
NAN = float("nan")

# T, cap, E, H, F, k, skew: one token; odd counts; a sum over 32 only, over odd multiples of
# 32 (half a stage); partial column tiles; experts of one row, of 64, of more than 128 and of
# several 256-row tiles; one expert; top-16; capacities with unused rows
SHAPES = [
    (1, 1, 2, 32, 32, 1, 0), (1, 3, 8, 64, 64, 2, 0), (7, 7, 3, 96, 32, 2, 0), (64, 64, 8, 128, 256, 2, 0),
    (33, 40, 4, 160, 96, 3, 0), (130, 131, 2, 64, 320, 1, 0), (257, 300, 1, 288, 64, 1, 0),
    (300, 300, 16, 96, 160, 16, 0), (520, 600, 3, 192, 288, 2, 1), (700, 701, 40, 256, 544, 4, 1),
    (1100, 1100, 5, 544, 128, 2, 1), (1300, 1400, 24, 320, 192, 6, 1), (90, 90, 100, 64, 96, 3, 0),
]


def _make(T, cap, E, H, F, k, skew, seed=0, std=0.08):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")     # noqa: E731
    z = rn(T, E) + (2 * rn(E) if skew else 0)
    ids = z.topk(k, dim=1).indices.to(torch.int32)                 # any order
    probs = torch.softmax(rn(T, k), dim=1)
    pad = lambda v, fill: torch.cat([v, torch.full((cap - T,) + v.shape[1:], fill, dtype=v.dtype, device="cuda")])  # noqa: E731
    return dict(x=pad(rn(T, H).bfloat16(), NAN), d_out=pad(rn(T, H).bfloat16(), NAN), ids=pad(ids, 1 << 30),
                probs=pad(probs, NAN), w1=(rn(E, 2 * F, H) * std).bfloat16(), w2=(rn(E, H, F) * std).bfloat16(),
                live=torch.tensor([T], dtype=torch.int32, device="cuda"))


def _moe(c, k, precision="bf16"):
    from swiglu_expert_mlp_amd import MoE
    E, H, F = c["w2"].shape
    m = MoE(E, H, F, k, precision)
    m.load_weights(c["w1"], c["w2"])
    return m


def _within(got, ref, bound, what):
    got = got.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(((got - ref).abs() / bound).nan_to_num(9e9).max()))


def _garbage(n):
    return torch.full((max(1, (n + 3) // 4),), 0x7FC00001, dtype=torch.int32, device="cuda").view(torch.uint8)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_checkpoint(shape):
    """out has the forward's bits; every kept value is within half a scale (and the sum's
    error) of the exact gate or up, and the scale is the smallest whose 127-fold reaches."""
    T, cap, E, H, F, k, skew = shape
    c = _make(*shape)
    m = _moe(c, k)
    codes, scales = m.new_checkpoint(cap)
    codes.fill_(99)
    scales.fill_(77)
    for combine in ("fp32", "bf16", "rows"):
        want = m.forward(c["x"], c["ids"], c["probs"], c["live"], combine=combine)
        got, _, _ = m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"], codes=codes, scales=scales,
                                         combine=combine)
        assert torch.equal(got[:T].view(torch.uint8), want[:T].view(torch.uint8))
    rows, off = routes(c["ids"][:T].tolist(), E, T)
    n = off[-1]
    assert (codes[n:] == 99).all() and (scales[n:] == 77).all()
    kept = kept_values(codes[:n], scales[:n])
    step = torch.exp2(scales[:n].double() - 127.0).repeat_interleave(32, dim=1)
    tok = torch.tensor([r[0] for r in rows], device="cuda")
    for e in range(E):
        r = slice(off[e], off[e + 1])
        xe, w = c["x"][tok[r]].double(), c["w1"][e].double()
        gu, mag = xe @ w.t(), xe.abs() @ w.abs().t()
        want = join(gu[:, :F], gu[:, F:])
        err = join(mag[:, :F], mag[:, F:]) * (H + 4) * S
        _within(kept[r], want, step[r] * 0.5 + err, "kept")
        amax = want.abs().view(-1, F // 16, 32).max(dim=2).values
        slack = err.view(-1, F // 16, 32).max(dim=2).values
        one = step[r].view(-1, F // 16, 32)[:, :, 0]
        assert (amax <= 127 * one + slack).all() and (amax >= 63.5 * one - slack).all()


def test_kept_codes_exact():
    """Gate and up that are exact in fp32: codes, ties and scale bytes bit for bit, blocks of
    zeros, of a single huge value and of values that are no numbers."""
    E, H, F, T = 1, 64, 64, 6
    w1 = torch.zeros((E, 2 * F, H))
    w1[0, :, 0] = torch.arange(2 * F) - 63.0            # integers, gate -63 .. 0, up 1 .. 64
    w1[0, :, 1] = (torch.arange(2 * F) % 7) * 0.125 - 0.375
    w1[0, :, 2] = (torch.arange(2 * F) == 5).float() * 2.0 ** 100
    w1[0, :, 3] = 1.0
    x = torch.zeros((T, H))
    x[0, 0], x[1, 0], x[2, 1], x[4, 2], x[5, 3] = 1.0, 2.0, 1.0, 1.0, 2.0 ** -120
    x[1, 3] = 0.5                                        # 2 (i - 63) + 1/2
    bf = lambda v: v.bfloat16().cuda()                   # noqa: E731
    w1b, w2b = bf(w1), bf(torch.zeros((E, H, F)))
    c = dict(w1=w1b, w2=w2b)
    m = _moe(c, 1)
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ones = torch.ones((T, 1), device="cuda")
    live = torch.tensor([T], dtype=torch.int32, device="cuda")
    _, codes, scales = m.forward_checkpoint(bf(x), ids, ones, live)
    gu = x.bfloat16().double() @ w1.bfloat16()[0].double().t()
    want = join(gu[:, :F], gu[:, F:]).view(T, F // 16, 32)
    for t in range(T):
        for b in range(F // 16):
            v = want[t, b]
            amax = float(v.abs().max())
            e = -126
            while amax > 127.0 * 2.0 ** e:
                e += 1
            assert int(scales[t, b]) == e + 127, (t, b)
            assert codes[t, 32 * b: 32 * b + 32].tolist() == torch.round(v / 2.0 ** e).int().tolist(), (t, b)
    # an infinite and a NaN product: that block alone is lost
    xb = bf(x)
    xb[3, 2] = float("inf")
    xb[2, 1] = NAN
    _, codes2, scales2 = m.forward_checkpoint(xb, ids, ones, live)
    assert (scales2[2:4] == 255).all() and (codes2[2:4] == 0).all()       # 0 times inf is NaN in every column
    keep = [0, 1, 4, 5]
    assert torch.equal(codes2[keep], codes[keep]) and torch.equal(scales2[keep], scales[keep])


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, wide):
    """Every gradient within its bound of fp64; rows past the live tokens untouched, nothing
    read there (NaN), the workspace's contents without effect; repeated bit for bit."""
    T, cap, E, H, F, k, skew = shape
    c = _make(*shape, seed=3)
    m = _moe(c, k)
    _, codes, scales = m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"])
    d_out = c["d_out"].float() if wide else c["d_out"]       # (bf16 values: the same operand)
    ws = _garbage(m.new_backward_workspace(cap).numel())
    d_x = torch.full((cap, H), 7.0, dtype=torch.bfloat16, device="cuda")
    d_p = torch.full((cap, k), 7.0, device="cuda")
    got = m.backward(d_out, c["x"], c["ids"], c["probs"], c["live"], codes, scales, d_x=d_x, d_probs=d_p, ws=ws,
                     grad_dtype="fp32" if wide else "bf16")
    assert m.check(ws) == 0
    ref = backward_ref(c["d_out"], c["x"], c["ids"][:T], c["probs"], T, codes, scales, c["w1"], c["w2"], wide)
    for name, v in zip(("d_x", "d_w1", "d_w2", "d_probs"), got):
        v = v[:T] if name in ("d_x", "d_probs") else v
        _within(v, *ref[name], name)
    assert (d_x[T:] == 7.0).all() and (d_p[T:] == 7.0).all()
    again = m.backward(d_out, c["x"], c["ids"], c["probs"], c["live"], codes, scales,
                       grad_dtype="fp32" if wide else "bf16")
    for a, b in zip(got, again):
        n = T if a.shape[0] == cap and a.dim() == 2 else a.shape[0]
        assert torch.equal(a[:n], b[:n])


def test_backward_matches_differences():
    """Where gate and up are integers (kept exactly), the gradients are those of the layer in
    fp64: central differences in every direction tried."""
    E, H, F, T, k = 3, 32, 32, 4, 2
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-1, 2, (T, H), generator=g).double()
    w1 = torch.zeros((E, 2 * F, H), dtype=torch.float64)
    w1.scatter_(2, torch.randint(0, H, (E, 2 * F, 3), generator=g), 1.0)
    w2 = torch.randint(-2, 3, (E, H, F), generator=g).double() / 4
    ids = torch.tensor([[0, 2], [1, 0], [2, 1], [0, 1]], dtype=torch.int32)
    probs = torch.tensor([[0.25, 0.75], [0.5, 0.5], [0.125, 0.875], [1.0, 0.0]], dtype=torch.float64)
    d_out = torch.randint(-3, 4, (T, H), generator=g).double()
    c = dict(w1=w1.bfloat16().cuda(), w2=w2.bfloat16().cuda())
    m = _moe(c, k)
    args = (x.bfloat16().cuda(), ids.cuda(), probs.float().cuda(), torch.tensor([T], dtype=torch.int32, device="cuda"))
    _, codes, scales = m.forward_checkpoint(*args)
    got = dict(zip(("x", "w1", "w2", "probs"), m.backward(d_out.bfloat16().cuda(), *args, codes, scales, grad_dtype="fp32")))
    bounds = backward_ref(d_out.cuda(), args[0], args[1], args[2], T, codes, scales, c["w1"], c["w2"], True)
    loss = lambda **kw: float((d_out * forward64(*[kw.get(n, v) for n, v in  # noqa: E731
                                                   (("x", x), ("ids", ids), ("probs", probs), ("w1", w1), ("w2", w2))])).sum())
    for name, base in (("x", x), ("w1", w1), ("w2", w2), ("probs", probs)):
        for s in range(3):
            v = torch.randn(base.shape, generator=g, dtype=torch.float64)
            h = 1e-5
            want = (loss(**{name: base + h * v}) - loss(**{name: base - h * v})) / (2 * h)
            grad = got[name].double().cpu()
            # the gradients' own bounds; differences are off by h^2 of third derivatives
            # (values up to 10^3) and 1e-16 / h of the loss
            tol = float((bounds["d_" + name][1].cpu() * v.abs()).sum()) + 1e-5
            assert abs(float((grad * v).sum()) - want) <= tol, (name, s)


def test_backward_dropped_routes_and_empty_experts():
    """Invalid and repeated ids have no row (gradient 0, the rest as without them); experts
    without rows have gradients of exactly 0; no live token at all."""
    T, E, H, F, k = 70, 12, 64, 96, 3
    c = _make(T, T, E, H, F, k, 0, seed=8)
    ids = c["ids"] % 5                                   # experts 5 .. 11 stay empty, repeats appear
    ids[3] = torch.tensor([-1, E, 2], dtype=torch.int32)
    ids[4] = torch.tensor([1 << 30, -7, -7], dtype=torch.int32)
    ids[5] = 4
    m = _moe(c, k)
    _, codes, scales = m.forward_checkpoint(c["x"], ids, c["probs"], c["live"])
    ws = m.new_backward_workspace(T)
    d1, d2 = torch.full_like(c["w1"], NAN), torch.full_like(c["w2"], NAN)
    got = m.backward(c["d_out"], c["x"], ids, c["probs"], c["live"], codes, scales, d_w1=d1, d_w2=d2, ws=ws)
    assert m.check(ws) == 3
    ref = backward_ref(c["d_out"], c["x"], ids, c["probs"], T, codes, scales, c["w1"], c["w2"], False)
    for name, v in zip(("d_x", "d_w1", "d_w2", "d_probs"), got):
        _within(v, *ref[name], name)
    assert (d1[5:] == 0).all() and (d2[5:] == 0).all()
    assert (got[0][4] == 0).all() and (got[3][4] == 0).all() and (got[3][5, 1:] == 0).all()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    d1.fill_(NAN)
    d_x = torch.full_like(c["x"], 3.0)
    m.backward(c["d_out"], c["x"], ids, c["probs"], none, codes, scales, d_x=d_x, d_w1=d1, d_w2=d2, ws=ws)
    assert (d1 == 0).all() and (d2 == 0).all() and (d_x == 3.0).all() and m.check(ws) == 0


def test_backward_no_number_stays_with_its_token():
    """A NaN in one token's d_out, an infinity in another's x: other tokens' d_x and d_probs
    and other experts' gradients keep their bits."""
    T, E, H, F, k = 300, 6, 96, 64, 2
    c = _make(T, T, E, H, F, k, 0, seed=9)
    m = _moe(c, k)
    _, codes, scales = m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"])
    args = (c["ids"], c["probs"], c["live"], codes, scales)
    clean = m.backward(c["d_out"], c["x"], *args)
    d, x = c["d_out"].clone(), c["x"].clone()
    d[17, 5], x[101, 7] = NAN, float("inf")
    got = m.backward(d, x, *args)
    keep = [t for t in range(T) if t != 17]
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[3][keep], clean[3][keep])
    assert got[0][17].isnan().all()
    for e in range(E):
        touched = {int(v) for v in c["ids"][17]}, {int(v) for v in c["ids"][101]}
        if e not in touched[0]:
            assert torch.equal(got[2][e], clean[2][e])
        if e not in touched[0] and e not in touched[1]:
            assert torch.equal(got[1][e], clean[1][e])
        if e in touched[1] and e not in touched[0]:
            others = [h for h in range(H) if h != 7]
            assert torch.equal(got[1][e][:, others], clean[1][e][:, others])
            assert not got[1][e][:, 7].isfinite().any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_dispatch_and_combine(shape, dtype):
    """The permutation and the copied rows exactly; sums and gradients within their roundings;
    rows and tokens past the live ones untouched."""
    T, cap, E, H, F, k, skew = shape
    c = _make(*shape, seed=4)
    from swiglu_expert_mlp_amd import MoE
    m = MoE(E, H, F, k)
    ids = c["ids"].clone()
    if T > 6:
        ids[2, 0] = -1
        if k > 1:
            ids[6, 1] = ids[6, 0]
    x = c["x"].to(dtype)
    R = cap * k
    rows = torch.full((R, H), 5.0, dtype=dtype, device="cuda")
    row_of = torch.full((cap, k), -9, dtype=torch.int32, device="cuda")
    ws = _garbage(m.new_dispatch_workspace(cap).numel())
    rows, row_of, offsets = m.dispatch(x, ids, c["live"], rows=rows, row_of=row_of, ws=ws)
    want_of, off = row_of_ref(ids[:T].cpu(), E, T)
    n = off[-1]
    assert m.check(ws) == (0 if T <= 6 else (1 if k == 1 else 3))
    assert offsets.tolist() == off and torch.equal(row_of[:T].cpu(), want_of) and (row_of[T:] == -9).all()
    where = want_of.cuda().long()
    for j in range(k):
        ok = where[:, j] >= 0
        assert torch.equal(rows[where[ok, j]], x[:T][ok])
    assert (rows[n:] == 5.0).all()
    # back, from rows of any values; rows past the last one are NaN
    g = torch.Generator(device="cuda").manual_seed(6)
    y = torch.full((R, H), NAN, dtype=dtype, device="cuda")
    y[:n] = torch.randn((n, H), generator=g, device="cuda").to(dtype)
    y64, p64 = y.double(), c["probs"].double()
    eps = B if dtype == torch.bfloat16 else S
    ok = (where >= 0).double()
    r64 = torch.where(ok[..., None] > 0, y64[where.clamp(min=0)], torch.zeros((), dtype=torch.float64, device="cuda"))
    for probs in (c["probs"], None):
        w = (p64[:T] if probs is not None else torch.ones_like(ok))[..., None]
        want, mag = (r64 * w).sum(dim=1), (r64 * w).abs().sum(dim=1)
        for out_dtype in (torch.float32, torch.bfloat16):
            oe = B if out_dtype == torch.bfloat16 else S
            out = torch.full((cap, H), 8.0, dtype=out_dtype, device="cuda")
            if probs is not None:
                m.combine(y, row_of, probs, c["live"], out=out)
            else:
                m.dispatch_backward(y, row_of, c["live"], d_x=out)
            _within(out[:T], want, mag * (k + 1) * S + want.abs() * oe + 1e-37, "combine")
            assert (out[T:] == 8.0).all()
    for out_dtype in (torch.float32, torch.bfloat16):
        d_out = c["d_out"].to(out_dtype)
        d_rows = torch.full((R, H), 5.0, dtype=dtype, device="cuda")
        d_p = torch.full((cap, k), 6.0, device="cuda")
        m.combine_backward(d_out, y, row_of, c["probs"], c["live"], d_rows=d_rows, d_probs=d_p)
        d64 = d_out[:T].double()
        for j in range(k):
            o = where[:, j] >= 0
            want = p64[:T][o, j, None] * d64[o]
            _within(d_rows[where[o, j]], want, want.abs() * (eps + S) + 1e-37, "d_rows")
            assert (d_p[:T][~o, j] == 0).all()
        _within(d_p[:T], (r64 * d64[:, None]).sum(dim=2), (r64 * d64[:, None]).abs().sum(dim=2) * (H + 2) * S + 1e-37, "d_probs")
        assert (d_rows[n:] == 5.0).all() and (d_p[T:] == 6.0).all()
        alone, nothing = m.combine_backward(d_out, None, row_of, c["probs"], c["live"],
                                            d_rows=torch.full_like(d_rows, 5.0))
        assert nothing is None and torch.equal(alone, d_rows)


def test_combine_rows_outside_and_infinities():
    """A row index outside the rows adds nothing and reads nothing; the sum's order is the
    rows', not the routes'; an infinity stays in its token."""
    from swiglu_expert_mlp_amd import MoE
    m = MoE(4, 32, 32, 3)
    rows = torch.randn((6, 32), device="cuda")
    rows[4, 3] = float("inf")
    big = 2.0 ** 25
    rows[0], rows[1], rows[2] = big, 1.0, -big
    live = torch.tensor([2], dtype=torch.int32, device="cuda")
    row_of = torch.tensor([[2, 0, 1], [6, -1, 4]], dtype=torch.int32, device="cuda")
    ones = torch.ones((2, 3), device="cuda")
    out = m.combine(rows, row_of, ones, live)
    assert (out[0] == 0.0).all()                        # ((2^25 + 1) - 2^25) in fp32
    assert torch.equal(out[1], rows[4])
    d_rows, d_p = m.combine_backward(out[:2].clone().fill_(1.0), rows, row_of, ones, live,
                                     d_rows=torch.zeros_like(rows))
    assert d_p[1, 0] == 0 and d_p[1, 1] == 0 and d_p[1, 2].isinf() and (d_rows[[3, 5]] == 0).all()


def test_a_workspace_of_another_call_holds_no_forward():
    """Indices and rows are read from a forward's workspace only, and so is the gradient of the
    combine's probabilities; a forward on the same memory makes them readable again."""
    T, E, H, F, k = 40, 8, 64, 96, 2
    for T in (40, 300):                                  # dispatch in one launch and in three
        c = _make(T, T, E, H, F, k, 0, seed=31)
        m = _moe(c, k)
        ws = _garbage(max(m.new_workspace(T).numel(), m.new_backward_workspace(T).numel()))
        out, codes, scales = m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"], ws=ws)
        want = m.get_indices(ws, T)
        d = m.probs_backward(c["d_out"], c["ids"], ws)
        for other in (lambda: m.dispatch(c["x"], c["ids"], c["live"], ws=ws),
                      lambda: m.backward(c["d_out"], c["x"], c["ids"], c["probs"], c["live"], codes, scales, ws=ws)):
            other()
            assert m.check(ws) == 0
            with pytest.raises(ValueError):
                m.get_indices(ws, T)
            with pytest.raises(ValueError):
                m.get_rows(ws, T, want["n_rows"], T)
            m.probs_backward(c["d_out"], c["ids"], ws)
            assert m.check(ws) == 32                     # no rows: not written
            m.forward(c["x"], c["ids"], c["probs"], c["live"], ws=ws)
            got = m.get_indices(ws, T)
            assert all((got[n] == want[n]).all() if hasattr(got[n], "all") else got[n] == want[n] for n in want)
            assert torch.equal(m.probs_backward(c["d_out"], c["ids"], ws), d)


def test_whole_step_together():
    """A training step with experts of the library and one with the caller's own experts
    between dispatch and combine agree with fp64 autograd of the layer."""
    T, E, H, F, k = 200, 8, 96, 64, 2
    c = _make(T, T, E, H, F, k, 0, seed=12, std=0.15)
    m = _moe(c, k)
    rows, row_of, offsets = m.dispatch(c["x"].float(), c["ids"], c["live"])
    off = offsets.tolist()
    leaf = {n: c[n].double().requires_grad_() for n in ("x", "w1", "w2", "probs")}
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(E):
            t = (c["ids"][:, j] == e).nonzero()[:, 0]
            gu = leaf["x"][t] @ leaf["w1"][e].t()
            y = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ leaf["w2"][e].t()
            out = out.index_add(0, t, leaf["probs"][t, j, None] * y)
    d_out = c["d_out"].float()
    out.backward(d_out.double())
    # the caller's own experts, fp32
    r = rows.clone().requires_grad_()
    w1, w2 = c["w1"].float().requires_grad_(), c["w2"].float().requires_grad_()
    parts = []
    for e in range(E):
        gu = r[off[e]:off[e + 1]] @ w1[e].t()
        parts.append((torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ w2[e].t())
    y = torch.cat(parts)
    got_out = m.combine(y.detach(), row_of, c["probs"], c["live"])
    d_rows, d_probs = m.combine_backward(d_out, y.detach(), row_of, c["probs"], c["live"])
    y.backward(d_rows)
    d_x = m.dispatch_backward(r.grad, row_of, c["live"])
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())     # noqa: E731
    for a, b in ((got_out, out.detach()), (d_x, leaf["x"].grad), (d_probs, leaf["probs"].grad), (w1.grad, leaf["w1"].grad),
                 (w2.grad, leaf["w2"].grad)):
        # fp32 sums of at most 2 F + H terms of random sign: well inside their linear bound
        assert rel(a, b) <= (2 * F + H) * S
    # the library's experts: kept values are off by at most 1/127 of their block's largest,
    # which is under 4.5 of their standard deviations here, so by a mean of
    # 4.5 / 127 / sqrt(12) of it or less; each gradient depends on gate and up with a
    # relative slope of at most 3 in the mean; and four roundings to bf16
    tol = 3 * 4.5 / 127 / 12 ** 0.5 + 4 * B
    out2, codes, scales = m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"])
    g = m.backward(d_out, c["x"], c["ids"], c["probs"], c["live"], codes, scales)
    assert rel(out2, out.detach()) <= 2 * B
    for a, b in zip(g, (leaf["x"].grad, leaf["w1"].grad, leaf["w2"].grad, leaf["probs"].grad)):
        assert rel(a, b) <= tol


def test_captured_replayed_and_on_streams():
    """A step captured into a graph and replayed between eager work on other inputs, a call on
    another stream and two streams at once: the bits of the plain call."""
    shape = (900, 1500, 16, 128, 192, 3, 1)
    T, cap, E, H, F, k, _ = shape
    a, b = _make(*shape, seed=21), _make(*shape, seed=22)
    m = _moe(a, k)

    def step(c, ws, bws, dws, stream=None):
        out, codes, scales = m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"], ws=ws, stream=stream)
        grads = m.backward(c["d_out"], c["x"], c["ids"], c["probs"], c["live"], codes, scales, ws=bws, stream=stream)
        rows, row_of, _ = m.dispatch(c["x"], c["ids"], c["live"], ws=dws, stream=stream)
        back = m.combine_backward(c["d_out"], rows, row_of, c["probs"], c["live"], stream=stream)
        y = m.combine(rows, row_of, c["probs"], c["live"], stream=stream)
        n = int(T * k)
        return [v[:T] for v in (out, grads[0], grads[3], y, back[1])] + [grads[1], grads[2], rows[:n], back[0][:n], codes[:n]]

    spaces = lambda: (m.new_workspace(cap), m.new_backward_workspace(cap), m.new_dispatch_workspace(cap))  # noqa: E731
    want = {id(c): [v.clone() for v in step(c, *spaces())] for c in (a, b)}
    same = lambda got, c: all(torch.equal(x, y) for x, y in zip(got, want[id(c)]))     # noqa: E731
    ws = spaces()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = step(a, *ws)
    for i in range(4):
        for v in held:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, a), i
        assert same(step(b, *ws), b)                    # eager work in the same workspaces
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    r1 = step(a, *spaces(), stream=s1)
    r2 = step(b, *spaces(), stream=s2)
    torch.cuda.synchronize()
    assert same(r1, a) and same(r2, b)
    with torch.cuda.stream(s2):                         # the current stream, nothing given
        r3 = step(a, *spaces())
    torch.cuda.synchronize()
    assert same(r3, a)


def test_both_tile_designs_on_one_stream_and_beside_each_other():
    """Enough rows per expert that the 64-row tiles stay on the call's stream: the bits of the
    same tokens at a capacity whose mean puts them beside the 256-row ones, and the bounds."""
    T, E, H, F, k = 1300, 4, 96, 160, 2
    c = _make(T, T, E, H, F, k, 0, seed=41)
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(T, 1)
    ids[::13, 0], ids[5::17, 1] = 2, 3                       # experts 2 and 3 keep at most 128 rows
    m = _moe(c, k)
    _, codes, scales = m.forward_checkpoint(c["x"], ids, c["probs"], c["live"])
    ref = backward_ref(c["d_out"], c["x"], ids, c["probs"], T, codes, scales, c["w1"], c["w2"], False)
    assert T * k >= 4 * 128 * E
    got = m.backward(c["d_out"], c["x"], ids, c["probs"], c["live"], codes, scales)
    for name, v in zip(("d_x", "d_w1", "d_w2", "d_probs"), got):
        _within(v, *ref[name], name)
    # the same experts among twice as many: the mean is under the threshold
    wide = dict(c, w1=torch.cat([c["w1"], c["w1"]]), w2=torch.cat([c["w2"], c["w2"]]))
    assert T * k < 4 * 128 * 2 * E
    m2 = _moe(wide, k)
    again = m2.backward(c["d_out"], c["x"], ids, c["probs"], c["live"], codes, scales)
    assert torch.equal(again[0], got[0]) and torch.equal(again[3], got[3])
    assert torch.equal(again[1][:E], got[1]) and torch.equal(again[2][:E], got[2]) and (again[1][E:] == 0).all()


def test_eager_backward_beside_a_capture():
    """A captured backward leaves the side stream in the capture until it ends: an eager one on
    another stream meanwhile stays out of the graph; replays beside eager calls, the same bits."""
    shape = (1400, 1500, 16, 96, 192, 2, 1)
    T, cap, E, H, F, k, _ = shape
    a, b = _make(*shape, seed=51), _make(*shape, seed=52)
    m = _moe(a, k)
    kept = {id(c): m.forward_checkpoint(c["x"], c["ids"], c["probs"], c["live"])[1:] for c in (a, b)}
    bf = torch.bfloat16

    def buffers():
        e = lambda s, t: torch.full(s, NAN, dtype=t, device="cuda")      # noqa: E731
        return dict(d_x=e((cap, H), bf), d_w1=e((E, 2 * F, H), bf), d_w2=e((E, H, F), bf), d_probs=e((cap, k), torch.float32),
                    ws=_garbage(m.new_backward_workspace(cap).numel()))

    def back(c, o, stream=None):
        return m.backward(c["d_out"], c["x"], c["ids"], c["probs"], c["live"], *kept[id(c)], stream=stream, **o)

    cut = lambda g: (g[0][:T].clone(), g[1].clone(), g[2].clone(), g[3][:T].clone())     # noqa: E731
    want = {id(c): cut(back(c, buffers())) for c in (a, b)}
    names = ("d_x", "d_w1", "d_w2", "d_probs")
    same = lambda o, c: all(torch.equal(x, y) for x, y in zip(cut([o[n] for n in names]), want[id(c)]))   # noqa: E731
    outs = [buffers() for _ in range(4)]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        back(a, outs[0])
        back(b, outs[1], other)                              # not captured
        back(b, outs[2])
        back(a, outs[3], other)                              # not captured
    torch.cuda.synchronize()
    assert same(outs[1], b) and same(outs[3], a)
    for n in range(3):
        for o in (outs[0], outs[2], outs[1]):
            for name in names:
                o[name].fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        back(b, outs[1], other)                              # beside the replay
        torch.cuda.synchronize()
        assert same(outs[0], a) and same(outs[2], b) and same(outs[1], b), n


@pytest.mark.parametrize("H,F", [(2080, 64), (64, 2080)])
def test_offsets_past_32_bits(H, F):
    """Buffers past 4 GiB (rows of H columns, then those of F): tokens at both ends and in the
    middle agree with a small call on them alone."""
    T, E, k = 530000, 8, 2
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    from swiglu_expert_mlp_amd import MoE
    g = torch.Generator(device="cuda").manual_seed(2)
    m = MoE(E, H, F, k)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 53000):
        x[i:i + 53000] = torch.randn((53000, H), generator=g, device="cuda").bfloat16()
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    probs = torch.rand((T, k), generator=g, device="cuda")
    live = torch.tensor([T], dtype=torch.int32, device="cuda")
    w1 = (torch.randn((E, 2 * F, H), generator=g, device="cuda") * 0.05).bfloat16()
    w2 = (torch.randn((E, H, F), generator=g, device="cuda") * 0.05).bfloat16()
    m.load_weights(w1, w2)
    pick = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    small = torch.tensor([5], dtype=torch.int32, device="cuda")
    rows, row_of, off = m.dispatch(x, ids, live)
    assert int(off[E]) == T * k and T * k * max(H, F) * 2 > 1 << 32
    assert torch.equal(rows[row_of[pick].long()], x[pick][:, None].expand(5, k, H))
    y = m.combine(rows, row_of, probs, live)
    srows, srow_of, _ = m.dispatch(x[pick], ids[pick], small)
    assert torch.equal(y[pick], m.combine(srows, srow_of, probs[pick], small))
    del y
    d_rows, d_p = m.combine_backward(x, rows, row_of, probs, live)
    sd, sp = m.combine_backward(x[pick], srows, srow_of, probs[pick], small)
    assert torch.equal(d_rows[row_of[pick].long()], sd[srow_of.long()]) and torch.equal(d_p[pick], sp)
    del d_rows, rows
    ws = m.new_workspace(T)
    out, codes, scales = m.forward_checkpoint(x, ids, probs, live, ws=ws, combine="bf16")
    del ws
    _, sc, ss = m.forward_checkpoint(x[pick], ids[pick], probs[pick], small, combine="bf16")
    at, sat = row_of[pick].long(), srow_of.long()
    assert torch.equal(codes[at], sc[sat]) and torch.equal(scales[at], ss[sat])
    grads = m.backward(x, x, ids, probs, live, codes, scales)
    sg = m.backward(x[pick], x[pick], ids[pick], probs[pick], small, sc, ss)
    assert torch.equal(grads[0][pick], sg[0]) and torch.equal(grads[3][pick], sg[3])
    for v in grads:
        assert v.isfinite().all()


@pytest.mark.parametrize("H,F", [(2080, 64), (64, 2080)])
def test_weights_gradients_past_32_bits(H, F):
    """The gradients of the weights over rows past 4 GiB are the sums of those over pieces of
    the tokens, which are smaller than 2 GiB."""
    T, E, k, piece = 530000, 8, 2, 53000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    from swiglu_expert_mlp_amd import MoE
    g = torch.Generator(device="cuda").manual_seed(4)
    m = MoE(E, H, F, k)
    m.load_weights((torch.randn((E, 2 * F, H), generator=g, device="cuda") * 0.05).bfloat16(),
                   (torch.randn((E, H, F), generator=g, device="cuda") * 0.05).bfloat16())
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, piece):
        x[i:i + piece] = torch.randn((piece, H), generator=g, device="cuda").bfloat16()
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    probs = torch.rand((T, k), generator=g, device="cuda")
    live = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")     # noqa: E731
    _, codes, scales = m.forward_checkpoint(x, ids, probs, live(T), combine="bf16")
    got = m.backward(x, x, ids, probs, live(T), codes, scales, grad_dtype="fp32")[1:3]
    del codes, scales
    n = live(piece)
    want = [torch.zeros(v.shape, dtype=torch.float64, device="cuda") for v in got]
    for i in range(0, T, piece):
        xs, it, pt = x[i:i + piece], ids[i:i + piece], probs[i:i + piece]
        _, sc, ss = m.forward_checkpoint(xs, it, pt, n, combine="bf16")
        for w, v in zip(want, m.backward(xs, xs, it, pt, n, sc, ss, grad_dtype="fp32")[1:3]):
            w += v
    for v, w in zip(got, want):
        # fp32 sums of about T k / E terms of random sign, of the same products: well inside
        # their linear bound
        assert float((v.double() - w).norm() / w.norm()) <= 2 * T * k / E * S
