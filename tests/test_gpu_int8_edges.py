"""GPU parity of the int8 experts on both sides of the padded length (256 codes) from which
a stage has 256-row tiles: FC1, FC2, both or neither on them above a 1024-token capacity."""
import numpy as np
import pytest
import torch

import oracle
from gpu_common import Case, assert_close, live_tensor, SENTINEL_BITS
from test_gpu_int8 import _skewed, forward, new_moe, rows_of
from workloads import Workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import swiglu_expert_mlp_amd  # noqa: F401  (raises if the library is missing)


PITCH = {32: 64, 160: 192, 192: 192, 224: 256, 256: 256}


@pytest.mark.parametrize("H,F", [(192, 160), (32, 192), (192, 224), (224, 160), (224, 224), (256, 192), (160, 256)])
def test_stages_around_the_shortest_256_row_product(H, F):
    """Against the oracle, FC2 rows bit for bit from their own codes, and the bits of a small
    launch (64-row tiles alone), with experts of both sizes."""
    w = Workload(f"h{H}_f{F}", 1200, 1210, H, F, 6, 2, "int8")
    c = Case(w, seed=29)
    moe = new_moe(c)
    ids, probs = _skewed(w)
    c.ids, c.probs = ids.cpu().numpy(), probs.cpu().numpy()
    _, ws, out = forward(c, moe)
    idx, rows = rows_of(moe, ws, w)
    counts = idx["counts"]
    assert counts[: w.E // 2].min() > 128 and 0 < counts[w.E // 2:].max() <= 128
    q2, s2 = oracle.int8_quantize(oracle.bf16_value(c.inp["w2_bits"]).reshape(-1, F))
    q2, s2 = q2.reshape(w.E, H, F), s2.reshape(w.E, H)
    for e in range(w.E):
        a, b = idx["offsets"][e], idx["offsets"][e + 1]
        acc = rows["fc1_codes"][a:b].astype(np.float64) @ q2[e].astype(np.float64).T     # exact
        ref = acc.astype(np.float32) * s2[e][None, :] * rows["fc1_scales"][a:b, None]
        assert np.array_equal(rows["fc2_rows"][a:b], ref), e
    ref, err, _ = c.oracle_model().forward(c.inp["x_bits"], c.ids, c.probs, w.T)
    assert err == 0
    assert_close(out[: w.T], ref[: w.T], w.name)
    assert np.all(out[w.T:].view(np.uint32) == SENTINEL_BITS), "rows past live were written"
    x, at = c.dev()[0], slice(60, 160)           # tokens of both kinds of experts
    small = moe.forward(x[at].contiguous(), ids[at].contiguous(), probs[at].contiguous(), live_tensor(100))
    assert np.array_equal(small.cpu().numpy(), out[at])


@pytest.mark.parametrize("K", sorted(PITCH))
def test_padded_lengths(K):
    """The pitch that the tests' shapes stand for, read from the packed buffer's size."""
    up = lambda v: (v + 255) // 256 * 256
    from swiglu_expert_mlp_amd import MoE
    E, N = 3, 64
    moe = MoE(E, K, N // 2, 1, "int8")
    size = up(E * N * PITCH[K]) + up(E * K * 64) + up(4 * E * N) + up(4 * E * K)
    assert moe.weight_bytes == size
