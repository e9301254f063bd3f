"""Which workspaces moe_get_indices and moe_get_rows read: a forward's of the handle's shape,
precision and capacity.  One that another call wrote over since is refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E, H, F, K = 8, 64, 96, 2


def _case(T, seed=1):
    from swiglu_expert_mlp_amd import MoE
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")     # noqa: E731
    m = MoE(E, H, F, K)
    m.load_weights((rn(E, 2 * F, H) * 0.1).bfloat16(), (rn(E, H, F) * 0.1).bfloat16())
    c = dict(x=rn(T, H).bfloat16(), d_out=rn(T, H).bfloat16(), logits=rn(T, E),
             ids=rn(T, E).topk(K, dim=1).indices.to(torch.int32), probs=torch.softmax(rn(T, K), dim=1),
             live=torch.tensor([T], dtype=torch.int32, device="cuda"))
    n = max(m.new_workspace(T).numel(), m.new_backward_workspace(T).numel(), m.new_balance_workspace(T).numel())
    return m, c, torch.empty(n, dtype=torch.uint8, device="cuda")


def _read(m, ws, T):
    idx = m.get_indices(ws, T)
    return idx, m.get_rows(ws, T, idx["n_rows"], idx["T"])


def _same(a, b):
    return all((a[n] == b[n]).all() if hasattr(a[n], "all") else a[n] == b[n] for n in a)


def _refused(m, ws, T, rows):
    with pytest.raises(ValueError, match="moe_get_indices"):
        m.get_indices(ws, T)
    with pytest.raises(ValueError, match="moe_get_rows"):
        m.get_rows(ws, T, rows, T)


@pytest.mark.parametrize("before", ["forward", "dispatch", "backward"])
def test_a_balance_loss_over_a_forward(before):
    """The balance loss of many tokens writes its partial sums where a forward's indices are."""
    T = 4000
    m, c, ws = _case(T)
    args = (c["x"], c["ids"], c["probs"], c["live"])
    _, codes, scales = m.forward_checkpoint(*args, ws=ws)
    want = _read(m, ws, T)
    if before == "dispatch":
        m.dispatch(c["x"], c["ids"], c["live"], ws=ws)
    elif before == "backward":
        m.backward(c["d_out"], *args, codes, scales, ws=ws)
    m.balance(c["logits"], c["ids"], c["live"], ws=ws)
    _refused(m, ws, T, want[0]["n_rows"])
    m.forward(*args, ws=ws)
    got = _read(m, ws, T)
    assert _same(got[0], want[0]) and _same(got[1], want[1])


def test_calls_that_leave_a_forward_readable():
    """A balance loss that one workgroup takes writes nothing there, a route its error bits."""
    T = 16
    m, c, ws = _case(T)
    m.forward(c["x"], c["ids"], c["probs"], c["live"], ws=ws)
    want = _read(m, ws, T)
    m.balance(c["logits"], c["ids"], c["live"], ws=ws)
    m.route(c["logits"], c["live"], ws=ws)
    m.probs_backward(c["d_out"], c["ids"], ws)
    got = _read(m, ws, T)
    assert _same(got[0], want[0]) and _same(got[1], want[1])


def test_what_holds_no_forward_of_the_handle():
    """Memory that no forward has used (its counts are anything), a route alone, another
    capacity, another handle's shape."""
    from swiglu_expert_mlp_amd import MoE
    T = 300
    m, c, ws = _case(T)
    ws.fill_(0x7F)
    _refused(m, ws, T, 1)
    m.route(c["logits"], c["live"], ws=ws)
    _refused(m, ws, T, 1)
    m.forward(c["x"], c["ids"], c["probs"], c["live"], ws=ws)
    n = m.get_indices(ws, T)["n_rows"]
    for cap in (0, T - 1, T + 1, 2 * T, -1):
        with pytest.raises(ValueError):
            m.get_indices(ws, cap)
    other = MoE(E, H, F, K + 1)
    _refused(other, ws, T, n)
    assert m.get_indices(ws, T)["n_rows"] == n
