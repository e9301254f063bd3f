"""The workspaces of dispatch and of the experts' backward pass hold the permutation and what
their own kernels use, nothing of the single-launch forwards."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    import swiglu_expert_mlp_amd as m
    return m.lib()


def _sizes(L, E, H, F, k, T):
    h = P()
    assert L.moe_create(E, H, F, k, 0, ctypes.byref(h)) == 0
    out = L.moe_dispatch_workspace_bytes(h, T), L.moe_backward_workspace_bytes(h, T), L.moe_workspace_bytes(h, T)
    L.moe_destroy(h)
    return out


@pytest.mark.parametrize("T", [1, 256, 4096, 100001])
@pytest.mark.parametrize("E,k", [(8, 2), (128, 8), (1024, 16)])
def test_dispatch_workspace_is_the_permutation(L, T, E, k):
    R, chunks = T * k, (T + 255) // 256
    # header; counts, offsets and each chunk's; ranks, ids, probabilities and rows of the routes
    # both ways; a table entry per 64-row and per 256-row tile; each of the twelve rounded up to 256
    need = 256 + 4 * E + 4 * (E + 1) + 4 * E * chunks + 4 * chunks + 5 * 4 * R
    need += 8 * (E + (R + 63) // 64 + 1) + 8 * (E + (R + 255) // 256 + 1)
    sizes = [_sizes(L, E, H, 64, k, T)[0] for H in (32, 2048, 65536)]
    assert len(set(sizes)) == 1 and need <= sizes[0] <= need + 12 * 256


def test_backward_workspace_grows_by_its_rows_alone(L):
    E, F, k, T = 8, 64, 2, 4096
    R = T * k
    a, b = (_sizes(L, E, H, F, k, T)[1] for H in (1024, 2048))
    assert b - a == 2 * R * 1024 + R * 64 + 2 * T * 1024      # rows of x's gradient, their scales, d_out
