"""GPU tests of the router's training calls and of the forward they read from, at the edges
of their contract: rows that are not numbers, workspaces without a forward, calls on other
streams, an eager call beside a capture."""
import numpy as np
import pytest
import torch

from gpu_common import live_tensor
from router_train_ref import balance_bounds, balance_ref
from test_gpu_router_train import NAN, dev, in_order, make, moe_of, run_balance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import swiglu_expert_mlp_amd  # noqa: F401  (raises if the library is missing)


# ------------------------------------------------------------- rows that are not numbers

def _nan_and_low(row):
    row[:] = -np.inf
    row[len(row) // 2] = NAN


BAD_ROWS = {
    "all_nan": lambda row: row.fill(NAN),
    "nan_and_low": _nan_and_low,
    "one_nan": lambda row: row.__setitem__(len(row) - 1, NAN),
    "one_inf": lambda row: row.__setitem__(0, np.inf),
}


# one launch (at most four turns of a workgroup) and two; lanes past E and none
@pytest.mark.parametrize("T", [6, 1100])
@pytest.mark.parametrize("E", [8, 60, 64, 130, 256, 1000])
@pytest.mark.parametrize("bad", list(BAD_ROWS))
def test_one_bad_row_reaches_both_losses_and_its_gradient(bad, E, T):
    """A single counted row with a NaN or +inf logit makes prob_sums and both losses NaN, and
    its own gradient; left out by the mask it changes nothing."""
    k, at = 2, T // 2
    z, ids, _, _, _ = make(T, T, E, k)
    BAD_ROWS[bad](z[at])
    moe = moe_of(E, k)
    losses, counts, sums = run_balance(moe, z, ids, T, None)
    assert np.array_equal(counts, balance_ref(np.where(np.isfinite(z), z, 0), ids, np.ones(T, bool))[1])
    assert np.isnan(losses[0]) and np.isnan(losses[1]), losses
    assert np.isnan(sums).all()
    g = dict(counts=dev(counts), d_losses=torch.tensor([0.5, 0.25], device="cuda"))
    grad = moe.route_backward(dev(z), None, live_tensor(T), **g).cpu().numpy()
    others = np.arange(T) != at
    assert np.isnan(grad[at]).all() and np.isfinite(grad[others]).all()
    # the same row, not counted
    losses, counts, sums = run_balance(moe, z, ids, T, others)
    ref = np.where(others[:, None], z, 0)
    rl, rc, rs = balance_ref(ref, ids, others)
    bl, bs = balance_bounds(ref, ids, others, in_order(T, E))
    assert np.array_equal(counts, rc) and np.all(np.abs(sums - rs) <= bs) and np.all(np.abs(losses - rl) <= bl)
    grad = moe.route_backward(dev(z), None, live_tensor(T), mask=dev(others), **g).cpu().numpy()
    assert not grad[at].any() and np.isfinite(grad).all()


# ------------------------------------------------------------- calls on another stream

def _pending_writes(sizes):
    """Blocks of these sizes, freed on the current stream behind some milliseconds of its work
    that ends by overwriting them."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    busy = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    for _ in range(40):
        busy.fill_(1.0)
    for b in blocks:
        b.fill_(0xFF)


def _nbytes(*tensors):
    return [t.numel() * t.element_size() for t in tensors]


@pytest.mark.parametrize("T", [200, 6000])
def test_training_calls_on_a_stream_do_not_write_where_work_is_pending(T):
    """What a call on another stream makes for itself is not memory that the current stream
    has freed with writes to it still to come."""
    E, k, H = 256, 4, 64
    moe = moe_of(E, k, H)
    z, ids, q, d, _ = (dev(a) for a in make(T, T, E, k))
    g = torch.Generator(device="cuda").manual_seed(T)
    moe.load_weights(torch.randn(E, 64, H, device="cuda", generator=g).bfloat16(),
                     torch.randn(E, H, 32, device="cuda", generator=g).bfloat16())
    x, d_out = torch.randn(T, H, device="cuda", generator=g).bfloat16(), torch.randn(T, H, device="cuda", generator=g)
    live, ws = live_tensor(T), moe.new_workspace(T)
    moe.forward(x, ids, q, live, ws=ws)
    calls = {
        "balance": lambda **kw: moe.balance(z, ids, live, **kw),
        "route_backward": lambda **kw: (moe.route_backward(z, ids, live, probs=q, d_probs=d, **kw),),
        "probs_backward": lambda **kw: (moe.probs_backward(d_out, ids, ws, **kw),),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        ref = [r.cpu() for r in call()]
        torch.cuda.synchronize()
        _pending_writes(_nbytes(*ref, moe.new_balance_workspace(T)))
        got = call(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b.cpu()) for a, b in zip(ref, got)), name


def test_a_returned_tensor_is_kept_for_the_current_stream():
    """A result of a call on another stream, read by pending work of the current one when it
    is dropped, is not handed to the next call on that stream."""
    E, k, T = 256, 4, 6000
    moe = moe_of(E, k)
    z, ids, q, d, _ = (dev(a) for a in make(T, T, E, k))
    live, side = live_tensor(T), torch.cuda.Stream()
    ref, other = moe.route_backward(z, ids, live, probs=q, d_probs=d), q * 2
    busy = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    grad = moe.route_backward(z, ids, live, probs=q, d_probs=d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(40):
        busy.fill_(1.0)
    copy = grad.clone()
    del grad
    for _ in range(3):
        moe.route_backward(z, ids, live, probs=other, d_probs=d, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, ref)


# ------------------------------------------------------------- weights and forwards on another stream

def _int8_layer(E=6, k=2, H=128, F=96, T=900, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=g)
    w1 = (draw(E, 2 * F, H) * 20).round().clamp(-127, 127).to(torch.int8)
    w2 = (draw(E, H, F) * 20).round().clamp(-127, 127).to(torch.int8)
    codes = (w1, torch.full((E, 2 * F), 0.01, device="cuda"), w2, torch.full((E, H), 0.01, device="cuda"))
    z = draw(T, E)
    return moe_of(E, k, H, F, "int8"), codes, draw(T, H).bfloat16(), z, live_tensor(T)


def test_loads_and_forwards_on_a_stream_do_not_write_where_work_is_pending():
    """As the training calls: the packed weights, the router's results, the forward's output
    and its workspace."""
    moe, codes, x, z, live = _int8_layer()
    T = x.shape[0]
    moe.load_quantized(*codes)
    ids, probs = moe.route(z, live)
    out = moe.forward(x, ids, probs, live)
    ref = [t.cpu() for t in (moe.kbuf, ids, probs, out)]
    side = torch.cuda.Stream()
    calls = {
        "load": lambda: (moe.load_quantized(*codes, stream=side),),
        "route": lambda: moe.route(z, live, stream=side),
        "forward": lambda: (moe.forward(x, ids, probs, live, stream=side),),
        "forward_noalloc": lambda: (moe.forward_noalloc(x[:300], ids[:300], probs[:300], live, stream=side),),
    }
    want = {"load": ref[:1], "route": ref[1:3], "forward": ref[3:], "forward_noalloc": [ref[3][:300]]}
    for name, call in calls.items():
        torch.cuda.synchronize()
        _pending_writes(_nbytes(*want[name], moe.new_workspace(T)))
        got = call()
        torch.cuda.synchronize()
        if name == "load":        # (the padding of the sections is not written)
            got = (moe.forward(x, ids, probs, live),)
            assert torch.equal(got[0].cpu(), ref[3])
        else:
            assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want[name])), name


@pytest.mark.parametrize("bound", [False, True])
@pytest.mark.parametrize("load", ["load_weights", "load_quantized"])
def test_a_refit_keeps_the_old_weights_for_forwards_in_flight(load, bound):
    """A forward waits on its stream for earlier work; the refit drops the weights that it will
    read and the next allocations of the same size are overwritten at once."""
    moe, codes, x, z, live = _int8_layer(seed=2)
    w = codes if load == "load_quantized" else tuple(
        (codes[i].float() * codes[i + 1][..., None]).bfloat16() for i in (0, 2))
    ids, probs = moe.route(z, live)
    ws, out = moe.new_workspace(x.shape[0]), torch.zeros(x.shape[0], moe.H, device="cuda")
    getattr(moe, load)(*w)
    moe.forward(x, ids, probs, live, out=out, ws=ws)
    ref = out.clone()
    side = torch.cuda.Stream()
    call = moe.bind_forward(x, ids, probs, live, out, ws, stream=side)
    getattr(moe, load)(*w)                      # weights newer than the binding
    out.zero_()
    busy = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(40):
            busy.fill_(1.0)
    if bound:
        call()
    else:
        moe.forward(x, ids, probs, live, out=out, ws=ws, stream=side)
    getattr(moe, load)(*w)                      # drops them
    junk = [torch.full((moe.weight_bytes,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and len(junk) == 3


def test_bound_calls_keep_their_handle():
    """A bound call outlives the name of its layer: the handle it passes is not freed."""
    import gc
    import weakref
    moe, codes, x, z, live = _int8_layer(T=40)
    moe.load_quantized(*codes)
    ids, probs = moe.route(z, live)
    ws, out = moe.new_workspace(40), torch.zeros(40, moe.H, device="cuda")
    ref = moe.forward(x, ids, probs, live)
    calls = [moe.bind_route(z, live, ids, probs, ws), moe.bind_forward(x, ids, probs, live, out, ws)]
    seen = weakref.ref(moe)
    del moe
    gc.collect()
    assert seen() is not None
    for call in calls:
        call()
    assert torch.equal(out, ref)
    del call, calls
    gc.collect()
    assert seen() is None


# ------------------------------------------------------------- error bits without a forward

def _probs_setup():
    moe, codes, x, z, live = _int8_layer(T=40)
    moe.load_quantized(*codes)
    d_out = torch.randn(40, moe.H, device="cuda")
    got = torch.full((40, moe.topk), 12345.0, device="cuda")
    return moe, x, z, live, d_out, got


@pytest.mark.parametrize("fill", [0, 0x5A, 0xA5, 0xFF])
def test_a_workspace_of_any_contents_gives_the_one_bit(fill):
    """No call has run on the workspace: its error word is not one to add to."""
    from swiglu_expert_mlp_amd import DEVERR_NO_ROWS
    moe, x, z, live, d_out, got = _probs_setup()
    ids = torch.zeros(40, moe.topk, dtype=torch.int32, device="cuda")
    ws = moe.new_workspace(40)
    ws.fill_(fill)
    for _ in range(2):
        moe.probs_backward(d_out, ids, ws, d_probs=got)
        moe.probs_backward(d_out, ids, ws, d_probs=got)
        assert moe.check(ws) == DEVERR_NO_ROWS
        assert moe.check(ws) == 0
    assert torch.all(got == 12345.0)


def test_bits_of_earlier_calls_stay_beside_it():
    from swiglu_expert_mlp_amd import (DEVERR_BAD_EXPERT_ID, DEVERR_LIVE_ABOVE_CAP, DEVERR_NO_ROWS,
                                       DEVERR_WEIGHTED_ROWS)
    moe, x, z, live, d_out, got = _probs_setup()
    ws = moe.new_workspace(40)
    ws.fill_(0x5A)
    ids, probs = moe.route(z, live_tensor(50), ws=ws)            # a router alone: no rows
    moe.probs_backward(d_out, ids, ws, d_probs=got)
    assert moe.check(ws) == DEVERR_LIVE_ABOVE_CAP | DEVERR_NO_ROWS
    bad = ids.clone()
    bad[3, 0] = -1
    moe.forward(x, bad, probs, live_tensor(40), ws=ws)
    moe.probs_backward(d_out[:30], bad[:30].contiguous(), ws, d_probs=got[:30])      # another capacity
    assert moe.check(ws) == DEVERR_BAD_EXPERT_ID | DEVERR_NO_ROWS
    moe.forward(x, bad, probs, live_tensor(40), ws=ws, topk_in_fc1=True)
    moe.probs_backward(d_out, bad, ws, d_probs=got)
    assert moe.check(ws) == DEVERR_BAD_EXPERT_ID | DEVERR_WEIGHTED_ROWS
    assert torch.all(got == 12345.0)
    # balance's partials in the workspace: its word is known, and holds nothing
    big, T = moe_of(64, 2), 1200
    ws = big.new_workspace(T)
    ws.fill_(0x5A)
    zz = torch.randn(T, 64, device="cuda")
    ids = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    big.balance(zz, ids, live_tensor(T), ws=ws)
    assert big.check(ws) == 0


def test_check_names_every_bit():
    """moe_last_error has a text for each bit of the word."""
    import swiglu_expert_mlp_amd as m
    moe, ws = moe_of(4, 2), moe_of(4, 2).new_workspace(8)
    bits = {getattr(m, n) for n in m.__all__ if n.startswith("DEVERR_")}
    seen = set()
    for b in sorted(bits):
        ws[:4] = torch.tensor([b], dtype=torch.int32, device="cuda").view(torch.uint8)
        assert moe.check(ws) == b and moe.check(ws) == 0
        ws[:4] = torch.tensor([b], dtype=torch.int32, device="cuda").view(torch.uint8)
        moe.check(ws)
        text = m.lib().moe_last_error().decode().split(":", 2)[2].strip()
        assert text and text not in seen, (b, text)
        seen.add(text)
