"""Router training operators on the CPU: the boundary's refusals and sizes, and the
formulas of the GPU tests' reference against differences (no compute calls)."""
import ctypes

import numpy as np
import pytest

from router_train_ref import balance_ref, route_backward_ref, selected_probs

P = ctypes.c_void_p
FAKE, ODD = P(1 << 20), P((1 << 20) + 4)


@pytest.fixture(scope="module")
def L():
    import swiglu_expert_mlp_amd as m
    return m.lib()


@pytest.fixture()
def handle(L):
    h = ctypes.c_void_p()
    assert L.moe_create(8, 128, 256, 2, 0, ctypes.byref(h)) == 0
    yield h
    L.moe_destroy(h)


def test_error_bits_match_the_header(L):
    import os
    import re
    import swiglu_expert_mlp_amd as m
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe.h")).read()
    bits = {n: int(v) for n, v in re.findall(r"#define\s+MOE_(DEVERR_[A-Z_]+)\s+(\d+)u", text)}
    assert bits["DEVERR_NO_ROWS"] == m.DEVERR_NO_ROWS == 32
    assert bits["DEVERR_WEIGHTED_ROWS"] == m.DEVERR_WEIGHTED_ROWS == 64
    assert len(set(bits.values())) == len(bits)


def test_balance_workspace_sizes(L, handle):
    sizes = [L.moe_balance_workspace_bytes(handle, T) for T in (0, 1, 256, 1000, 65536, 1 << 26)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 and s > 0 for s in sizes)
    assert L.moe_balance_workspace_bytes(None, 64) == 0 and L.moe_balance_workspace_bytes(handle, -1) == 0


def test_balance_refusals(L, handle):
    need = L.moe_balance_workspace_bytes(handle, 64)

    def call(logits=FAKE, ids=FAKE, T=64, live=FAKE, mask=None, losses=FAKE, counts=FAKE, sums=FAKE, ws=FAKE,
             n=need, h=handle):
        return L.moe_balance(h, logits, ids, T, live, mask, losses, counts, sums, ws, n, None)

    assert call(h=None) == -1 and call(T=-1) == -1 and call(T=(1 << 26) + 1) == -1
    assert call(n=need - 1) == -1 and b"ws_bytes" in L.moe_last_error()
    for name in ("logits", "ids", "losses", "counts", "sums", "ws"):
        assert call(**{name: None}) == -1 and b"NULL" in L.moe_last_error(), name
        assert call(**{name: ODD}) == -1 and b"aligned" in L.moe_last_error(), name
    assert call(live=None) == -1 and call(mask=ODD) == -1


def test_route_backward_refusals(L, handle):
    def call(logits=FAKE, ids=FAKE, probs=FAKE, d_probs=FAKE, T=64, live=FAKE, mask=None, counts=FAKE, d_losses=FAKE,
             d_logits=P(1 << 24), h=handle):
        return L.moe_route_backward(h, logits, ids, probs, d_probs, T, live, mask, counts, d_losses, d_logits, None)

    assert call(h=None) == -1 and call(T=-1) == -1 and call(T=(1 << 26) + 1) == -1
    for name in ("logits", "live", "d_logits", "ids", "probs", "d_probs", "counts", "d_losses"):
        assert call(**{name: None}) == -1, name
    for name in ("logits", "ids", "probs", "d_probs", "mask", "counts", "d_losses", "d_logits"):
        assert call(**{name: ODD}) == -1 and b"aligned" in L.moe_last_error(), name
    assert call(probs=None, d_probs=None, counts=None, d_losses=None) == -1
    assert call(d_logits=FAKE) == -1 and b"must not be" in L.moe_last_error()


def test_probs_backward_refusals(L, handle):
    need = L.moe_workspace_bytes(handle, 64)

    def call(d_out=FAKE, combine=0, ids=FAKE, T=64, d_probs=FAKE, ws=FAKE, n=need, h=handle):
        return L.moe_probs_backward(h, d_out, combine, ids, T, d_probs, ws, n, None)

    assert call(h=None) == -1 and call(T=-1) == -1 and call(T=(1 << 26) + 1) == -1
    for c in (2, 3, -1, 0x100, 0x200):
        assert call(combine=c) == -1 and b"combine" in L.moe_last_error()
    assert call(n=need - 1) == -1
    for name in ("d_out", "ids", "d_probs", "ws"):
        assert call(**{name: None}) == -1 and call(**{name: ODD}) == -1, name


@pytest.mark.parametrize("T,E,k,masked", [(7, 5, 2, False), (6, 4, 4, True), (3, 9, 1, False), (1, 1, 1, False)])
def test_reference_gradient_against_differences(T, E, k, masked):
    """The formula of the gradient against central differences of
    gb balance + gz z + <d_probs, q> in fp64 (step 1e-5: curvature below 1e-9)."""
    rng = np.random.default_rng(T * E)
    z = rng.standard_normal((T, E))
    ids = np.sort(np.stack([rng.permutation(E)[:k] for _ in range(T)]), axis=1)
    keep = rng.random(T) < 0.6 if masked else np.ones(T, bool)
    d = rng.standard_normal((T, k))
    gb, gz = 0.7, 0.3

    def value(zz):
        losses, counts, _ = balance_ref(zz, ids, keep)
        return gb * losses[0] + gz * losses[1] + (d * selected_probs(zz, ids)).sum()

    _, counts, _ = balance_ref(z, ids, keep)
    grad, _ = route_backward_ref(z, ids, keep, selected_probs(z, ids), d, counts, (gb, gz))
    for t in range(T):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += 1e-5
            dn[t, e] -= 1e-5
            assert abs((value(up) - value(dn)) / 2e-5 - grad[t, e]) < 1e-8


def test_tensors_of_another_device_are_refused(monkeypatch):
    import torch
    import swiglu_expert_mlp_amd as m

    class Fake:
        device = torch.device("cuda:1")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        m._on_current(None, (None, Fake()))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    m._on_current(None, (None, Fake()))


def test_streams_of_another_device_are_refused(monkeypatch):
    import torch
    import swiglu_expert_mlp_amd as m

    class Stream:
        device = torch.device("cuda:1")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="stream"):
        m._on_current(Stream(), ())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    m._on_current(Stream(), ())


@pytest.mark.parametrize("call", ["load_weights", "load_quantized", "route", "forward", "forward_noalloc",
                                  "bind_forward", "bind_route"])
def test_every_call_refuses_tensors_of_another_device(call, monkeypatch):
    """The kernels run on the current device: another one's memory would be read from there."""
    import torch
    import swiglu_expert_mlp_amd as m

    class Fake:
        device = torch.device("cuda:1")
        shape = (4, 8)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    moe = m.MoE(8, 32, 32, 2, "int8")
    n = {"load_weights": 2, "load_quantized": 4, "route": 2, "forward": 4, "forward_noalloc": 4, "bind_forward": 6,
         "bind_route": 5}[call]
    with pytest.raises(ValueError, match="current device"):
        getattr(moe, call)(*[Fake()] * n)


@pytest.mark.parametrize("name,size", [("logits", 64 * 8 * 4), ("ids", 64 * 2 * 4), ("probs", 64 * 2 * 4),
                                       ("d_probs", 64 * 2 * 4), ("live", 4), ("mask", 64), ("counts", 9 * 4),
                                       ("d_losses", 8)])
def test_route_backward_refuses_outputs_inside_an_input(L, handle, name, size):
    """Partly over an input's last bytes, and an input inside the output's rows."""
    rows, out = 64 * 8 * 4, 1 << 26

    def call(p):
        where = dict(logits=1 << 20, ids=2 << 20, probs=3 << 20, d_probs=4 << 20, live=5 << 20, mask=6 << 20,
                      counts=7 << 20, d_losses=8 << 20)
        where[name] = p
        a = {n: P(v) for n, v in where.items()}
        return L.moe_route_backward(handle, a["logits"], a["ids"], a["probs"], a["d_probs"], 64, a["live"], a["mask"],
                                    a["counts"], a["d_losses"], P(out), None)

    for p in (out - (size - 1) // 16 * 16, out, out + rows - 16):
        assert call(p) == -1 and b"must not be" in L.moe_last_error(), p
