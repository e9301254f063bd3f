"""The experts' backward pass where its sums, types and values are at their ends."""
import pytest
import torch

from experts_train_ref import backward_ref
from test_gpu_experts_train import _make, _moe, _within

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
