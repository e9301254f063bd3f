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
