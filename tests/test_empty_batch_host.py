"""Host checks with a capacity of no tokens: only tensors without a size may be NULL.  (Every
call here ends before anything is launched.)"""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    import swiglu_expert_mlp_amd as m
    return m.lib()


def _refused(L, st, word):
    assert st == -1 and word in L.moe_last_error().decode(), (st, L.moe_last_error())


def test_what_may_be_null(L):
    h = P()
    assert L.moe_create(8, 128, 256, 2, 0, ctypes.byref(h)) == 0
    a = [P((i + 1) << 30) for i in range(3)]
    _refused(L, L.moe_dispatch(h, None, 1, None, 0, a[0], None, None, a[1], a[2], 64, None), "ws_bytes")
    for i in range(3):
        b = a[:i] + [None] + a[i + 1:]
        _refused(L, L.moe_dispatch(h, None, 1, None, 0, b[0], None, None, b[1], b[2], 64, None), "NULL")
    _refused(L, L.moe_dispatch(h, None, 1, P(8), 0, a[0], None, None, a[1], a[2], 64, None), "aligned")
    _refused(L, L.moe_dispatch(h, None, 1, None, 1, a[0], None, None, a[1], a[2], 64, None), "NULL")
    _refused(L, L.moe_combine_rows(h, None, 0, None, None, 0, None, None, 0, None), "NULL")
    _refused(L, L.moe_combine_backward(h, None, 0, None, 0, None, None, 0, None, None, None, None), "NULL")
    _refused(L, L.moe_route(h, None, 0, a[0], None, None, a[1], 8, None), "too small")
    _refused(L, L.moe_balance(h, None, None, 0, a[0], None, a[0], a[1], a[2], a[0], 64, None), "ws_bytes")
    _refused(L, L.moe_balance(h, None, None, 0, a[0], None, None, a[1], a[2], a[0], 64, None), "NULL")
    _refused(L, L.moe_probs_backward(h, None, 0, None, 0, None, a[0], 64, None), "ws_bytes")
    _refused(L, L.moe_route_backward(h, None, None, None, None, 0, a[0], None, a[1], None, None, None), "counts")
    fc = L.moe_forward_checkpoint(h, None, None, None, 0, a[0], 0, None, None, None, a[1], 64, None)
    assert fc == -3                                       # no weights: past the pointers
    L.moe_destroy(h)
