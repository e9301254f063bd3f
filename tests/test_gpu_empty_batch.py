"""Calls on a batch without tokens (empty tensors, whose address is null): every output that
has a size is written, nothing is refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E, H, F, K = 6, 96, 64, 2
NAN = float("nan")


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _moe():
    from swiglu_expert_mlp_amd import MoE
    m = MoE(E, H, F, K)
    g = torch.Generator(device="cuda").manual_seed(1)
    m.load_weights(torch.randn((E, 2 * F, H), generator=g, device="cuda").bfloat16(),
                   torch.randn((E, H, F), generator=g, device="cuda").bfloat16())
    return m


@pytest.mark.parametrize("live_count", [0, 3], ids=["none", "more than the capacity"])
@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
def test_experts(wide, live_count):
    m = _moe()
    live = torch.tensor([live_count], dtype=torch.int32, device="cuda")
    bf = torch.bfloat16
    x, ids, probs = _empty(0, H, dtype=bf), _empty(0, K, dtype=torch.int32), _empty(0, K)
    out, codes, scales = m.forward_checkpoint(x, ids, probs, live)
    assert out.shape == (0, H) and codes.shape == (0, 2 * F) and scales.shape == (0, F // 16)
    gt = torch.float32 if wide else bf
    d1, d2 = torch.full((E, 2 * F, H), NAN, dtype=gt, device="cuda"), torch.full((E, H, F), NAN, dtype=gt, device="cuda")
    ws = torch.full((m.new_backward_workspace(0).numel(),), 0x7F, dtype=torch.uint8, device="cuda")
    d_x, _, _, d_p = m.backward(_empty(0, H, dtype=gt), x, ids, probs, live, codes, scales, d_w1=d1, d_w2=d2, ws=ws)
    assert d_x.shape == (0, H) and d_p.shape == (0, K)
    assert (d1 == 0).all() and (d2 == 0).all()
    assert m.check(ws) == (4 if live_count else 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_dispatch_and_combine(dtype):
    m = _moe()
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, ids, probs = _empty(0, H, dtype=dtype), _empty(0, K, dtype=torch.int32), _empty(0, K)
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((m.new_dispatch_workspace(0).numel(),), 0x7F, dtype=torch.uint8, device="cuda")
    rows, row_of, _ = m.dispatch(x, ids, live, offsets=offsets, ws=ws)
    assert rows.shape == (0, H) and row_of.shape == (0, K) and (offsets == 0).all() and m.check(ws) == 0
    assert m.combine(rows, row_of, probs, live).shape == (0, H)
    assert m.dispatch_backward(rows, row_of, live).shape == (0, H)
    d_rows, d_p = m.combine_backward(x, rows, row_of, probs, live)
    assert d_rows.shape == (0, H) and d_p.shape == (0, K)
    assert m.combine_backward(x, None, row_of, probs, live)[0].shape == (0, H)


@pytest.mark.parametrize("precision", ["bf16", "mxfp8", "mxfp4", "int8"])
def test_forward_and_router(precision):
    from swiglu_expert_mlp_amd import MoE
    m = MoE(E, 128, 128, K, precision)
    g = torch.Generator(device="cuda").manual_seed(2)
    m.load_weights(torch.randn((E, 256, 128), generator=g, device="cuda").bfloat16(),
                   torch.randn((E, 128, 128), generator=g, device="cuda").bfloat16())
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((m.new_workspace(0).numel(),), 0x7F, dtype=torch.uint8, device="cuda")
    logits = _empty(0, E)
    ids, probs = m.route(logits, live, ws=ws)
    assert ids.shape == (0, K) and probs.shape == (0, K) and m.check(ws) == 0
    x = _empty(0, 128, dtype=torch.bfloat16)
    options = [dict(combine="fp32"), dict(combine="bf16"), dict(combine="rows"), dict(topk_in_fc1=True)]
    if precision == "bf16":
        options += [dict(fused_ffn=True), dict(fused_finalize=True)]
    for o in options:
        ws.fill_(0x7F)
        assert m.forward(x, ids, probs, live, ws=ws, **o).shape[0] == 0
        idx = m.get_indices(ws, 0)
        assert m.check(ws) == 0 and idx["T"] == 0 and idx["n_rows"] == 0 and (idx["offsets"] == 0).all()
        assert m.forward_noalloc(x, ids, probs, live, **o).shape[0] == 0
    assert m.probs_backward(_empty(0, 128), ids, ws).shape == (0, K)
    losses, counts, prob_sums = m.balance(logits, ids, live)
    assert (losses == 0).all() and (counts == 0).all() and (prob_sums == 0).all()
    d = m.route_backward(logits, ids, live, probs=probs, d_probs=probs, counts=counts, d_losses=losses)
    assert d.shape == (0, E)
    assert m.route_backward(logits, ids, live, counts=counts, d_losses=losses).shape == (0, E)
    assert m.route_backward(logits, ids, live, probs=probs, d_probs=probs).shape == (0, E)
