"""The experts' backward pass where its sums, types and values are at their ends."""
import pytest
import torch

from experts_train_ref import backward_ref
from test_gpu_experts_train import _make, _moe, _within
from test_gpu_experts_train import test_forward_checkpoint as check_forward_checkpoint

pytestmark = pytest.mark.gpu
NAMES = ("d_x", "d_w1", "d_w2", "d_probs")


@pytest.mark.parametrize("T", [90, 1100], ids=["64-row tiles", "256-row tiles"])
@pytest.mark.parametrize("H", [96, 128])
def test_an_infinite_weight(H, T):
    """An infinity in W2 makes the sums it is part of infinite, not NaN (a hidden size that is an
    odd multiple of 32 ends half a stage early), and leaves the other expert's gradients alone."""
    E, F, k = 2, 64, 1
    c = _make(T, T, E, H, F, k, 0, seed=61)
    m = _moe(c, k)
    args = (c["x"], c["ids"], c["probs"], c["live"])
    _, codes, scales = m.forward_checkpoint(*args)
    clean = m.backward(c["d_out"], *args, codes, scales)
    c["w2"][0, H - 1, 5] = float("inf")
    m.load_weights(c["w1"], c["w2"])
    got = m.backward(c["d_out"], *args, codes, scales)
    ref = backward_ref(c["d_out"], c["x"], c["ids"], c["probs"], T, codes, scales, c["w1"], c["w2"], False)
    mine, other = (c["ids"][:, 0] == 0), (c["ids"][:, 0] == 1)
    want = ref["d_probs"][0]
    assert want[mine].isinf().float().mean() > 0.9           # (a kept value of 0 makes it NaN)
    assert torch.equal(got[3].double()[mine].nan_to_num(7.0), want[mine].nan_to_num(7.0))
    # up's gradient, the second half of d_w1's operand: row 5 of both halves is lost, no other
    lost = torch.zeros(2 * F, dtype=torch.bool, device="cuda")
    lost[[5, F + 5]] = True
    assert not got[1][0][lost].isfinite().any()
    assert torch.equal(got[1][0][~lost], clean[1][0][~lost])
    assert torch.equal(got[0][other], clean[0][other]) and torch.equal(got[3][other], clean[3][other])
    assert torch.equal(got[1][1], clean[1][1]) and torch.equal(got[2], clean[2])


@pytest.mark.parametrize("T,cap", [(90, 90), (1100, 1200)], ids=["64-row tiles", "256-row tiles"])
def test_fp32_d_out_is_rounded_first(T, cap):
    """d_out in fp32, with values that are no bf16 ones (ties, infinities and the largest numbers
    among them): the bits of the same call on its bf16 rounding."""
    E, H, F, k = 6, 160, 96, 2
    c = _make(T, cap, E, H, F, k, 1, seed=62)
    m = _moe(c, k)
    args = (c["x"], c["ids"], c["probs"], c["live"])
    _, codes, scales = m.forward_checkpoint(*args)
    g = torch.Generator(device="cuda").manual_seed(63)
    d = torch.full((cap, H), float("nan"), device="cuda")
    d[:T] = torch.randn((T, H), generator=g, device="cuda")
    # halfway between neighbours: 1 + 2^-8 to 1, 1 + 3 2^-8 to 1 + 2^-6
    d[3, :4] = torch.tensor([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -8, 2.0 ** -130], device="cuda")
    d[5, 7], d[6, 8], d[7, 9] = float("inf"), 3.4e38, float("nan")
    assert (d[:T].bfloat16().float() != d[:T]).float().mean() > 0.9
    got = m.backward(d, *args, codes, scales)
    want = m.backward(d.bfloat16(), *args, codes, scales)
    for a, b in zip(got, want):
        n = T if a.shape[0] == cap and a.dim() == 2 else a.shape[0]
        bits = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(a[:n].contiguous().view(bits), b[:n].contiguous().view(bits))


# the largest |gate|: the sigmoid is within (|g| + 6) S of its value; past |g| = 87 it, or its
# distance from 1, is below the smallest normal number and may be 0: off by 2^-126 at most, in
# an output by 1e-25 at most (raw < 500, gate and up < 512, sums of at most 1100 terms below 10^6)
@pytest.mark.parametrize("top,slack", [(64, 0.0), (512, 1e-25)])
@pytest.mark.parametrize("T", [90, 1100], ids=["64-row tiles", "256-row tiles"])
def test_large_gates(T, top, slack, monkeypatch):
    import experts_train_ref as ref_module
    E, H, F, k = 4, 128, 96, 2
    c = _make(T, T, E, H, F, k, 1, seed=64)
    m = _moe(c, k)
    g = torch.Generator(device="cuda").manual_seed(65)
    codes = torch.randint(-127, 128, (T * k, 2 * F), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.empty((T * k, F // 16), dtype=torch.uint8, device="cuda")
    hi = 120 + top.bit_length()                  # 127 2^(hi - 127) < top
    scales[:, 0::2] = torch.randint(hi - 3, hi + 1, (T * k, F // 32), generator=g, device="cuda").to(torch.uint8)
    scales[:, 1::2] = torch.randint(118, 123, (T * k, F // 32), generator=g, device="cuda").to(torch.uint8)
    got = m.backward(c["d_out"], c["x"], c["ids"], c["probs"], c["live"], codes, scales, grad_dtype="fp32")
    monkeypatch.setattr(ref_module, "SIG", (top + 6) * ref_module.S)
    ref = backward_ref(c["d_out"], c["x"], c["ids"], c["probs"], T, codes, scales, c["w1"], c["w2"], True)
    for name, v in zip(NAMES, got):
        value, bound = ref[name]
        _within(v, value, bound + slack, name)


def test_error_against_the_layer_itself():
    """Gradients from kept values against those of the layer in fp64.  A kept value is off by
    step / sqrt(12) in the mean; over blocks of 32 normal values (largest magnitude squared 4.9
    variances in the mean, steps from 1 to 2 times largest / 127, evenly in their logarithm) by
    0.0074 of the deviation.  Every gradient is a product with one or two of up, silu(gate) and
    its slope, whose relative errors in the mean are that of the kept value or less (deviation
    about 1): sqrt(2) 0.0074 = 0.0105, and two roundings to bf16, 0.0024: 0.0108; allowed half
    as much again."""
    T, E, H, F, k = 600, 4, 256, 128, 2
    c = _make(T, T, E, H, F, k, 0, seed=66, std=0.06)
    m = _moe(c, k)
    leaf = {n: c[n].double().requires_grad_() for n in ("x", "w1", "w2", "probs")}
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(E):
            t = (c["ids"][:, j] == e).nonzero()[:, 0]
            gu = leaf["x"][t] @ leaf["w1"][e].t()
            y = (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]) @ leaf["w2"][e].t()
            out = out.index_add(0, t, leaf["probs"][t, j, None] * y)
    out.backward(c["d_out"].double())
    args = (c["x"], c["ids"], c["probs"], c["live"])
    ws = m.new_workspace(T)
    _, codes, scales = m.forward_checkpoint(*args, ws=ws)
    got = m.backward(c["d_out"], *args, codes, scales)
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())     # noqa: E731
    off = {n: rel(v, leaf[n[2:]].grad) for n, v in zip(NAMES, got)}
    assert max(off.values()) <= 1.5 * 0.0108, off
    # the combine's gradient on the forward's own rows: their bf16 operand's rounding alone, 2^-8
    # of h in each term of the sum
    assert rel(m.probs_backward(c["d_out"], c["ids"], ws), leaf["probs"].grad) <= 2.0 ** -8


@pytest.mark.parametrize("H,F", [(2080, 64), (64, 2080)])
def test_weights_gradients_past_32_bits_by_expert(H, F):
    """Rows past 4 GiB against the sum over pieces below 2 GiB, each expert by itself.  d_out is
    independent of x, so the terms have random signs: one lost row of the n = 132,500 of an expert
    is about 1 / sqrt(n) = 2.7e-3 of its gradient's norm.  An fp32 sum of n terms is off by S sqrt(n)
    in the mean where its roundings are independent, by n S over the 16 terms of an instruction at
    most were they all one way; both sides of the comparison: 16 sqrt(n) S + n / 8 S = 1.3e-3."""
    from swiglu_expert_mlp_amd import MoE
    T, E, k, piece = 530000, 8, 2, 53000
    S = 2.0 ** -24
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device="cuda").manual_seed(67)
    m = MoE(E, H, F, k)
    m.load_weights((torch.randn((E, 2 * F, H), generator=g, device="cuda") * 0.05).bfloat16(),
                   (torch.randn((E, H, F), generator=g, device="cuda") * 0.05).bfloat16())
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    d = torch.empty_like(x)
    for i in range(0, T, piece):
        for v in (x, d):
            v[i:i + piece] = torch.randn((piece, H), generator=g, device="cuda").bfloat16()
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    probs = 0.5 + torch.rand((T, k), generator=g, device="cuda")
    live = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")     # noqa: E731
    _, codes, scales = m.forward_checkpoint(x, ids, probs, live(T), combine="bf16")
    args = (d, x, ids, probs, live(T), codes, scales)
    got = m.backward(*args, grad_dtype="fp32")[1:3]
    for a, b in zip(m.backward(*args, grad_dtype="bf16")[1:3], got):
        assert torch.equal(a, b.bfloat16())              # the same sums, rounded once
    del codes, scales, args

    def pieces(last):
        want = [torch.zeros(v.shape, dtype=torch.float64, device="cuda") for v in got]
        for i in range(0, T, piece):
            n = live(last if i + piece == T else piece)
            xs, it, pt = x[i:i + piece], ids[i:i + piece], probs[i:i + piece]
            _, sc, ss = m.forward_checkpoint(xs, it, pt, n, combine="bf16")
            for w, v in zip(want, m.backward(d[i:i + piece], xs, it, pt, n, sc, ss, grad_dtype="fp32")[1:3]):
                w += v
        return want

    def off(want):
        return [(v.double() - w).flatten(1).norm(dim=1) / w.flatten(1).norm(dim=1) for v, w in zip(got, want)]

    rows = T * k / E
    tol = 16 * rows ** 0.5 * S + rows / 8 * S
    for o in off(pieces(piece)):
        assert o.max() <= tol, o
    for o in off(pieces(piece - 32)):                     # an oracle without the last 32 tokens is told apart
        assert o.min() > tol, o


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [70, 1100], ids=["64-row tiles", "256-row tiles"])
def test_an_expert_whose_weights_pass_32_bits(T, wide):
    """An expert's W1 of more than 2 GiB: the kept values and every gradient within the bounds of
    fp64, where a 32-bit offset into the weights would have wrapped."""
    E, H, F, k = 2, 32768, 16416, 1
    assert 4 * F * H >= 1 << 31
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    check_forward_checkpoint((T, T, E, H, F, k, 0))
    torch.cuda.empty_cache()
    c = _make(T, T, E, H, F, k, 0, seed=68, std=0.01)
    m = _moe(c, k)
    args = (c["x"], c["ids"], c["probs"], c["live"])
    _, codes, scales = m.forward_checkpoint(*args)
    got = m.backward(c["d_out"], *args, codes, scales, grad_dtype="fp32" if wide else "bf16")
    ref = backward_ref(c["d_out"], c["x"], c["ids"], c["probs"], T, codes, scales, c["w1"], c["w2"], wide)
    for name, v in zip(NAMES, got):
        value, bound = ref.pop(name)
        for e in range(E) if value.dim() == 3 else (slice(None),):
            _within(v[e], value[e], bound[e], name)
        del value, bound
