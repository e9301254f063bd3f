"""Host-side checks of the experts' training calls: no GPU, nothing is launched."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import swiglu_expert_mlp_amd as m
    return m.lib()


def _create(L, E=8, H=128, F=256, k=2, p=0):
    h = P()
    assert L.moe_create(E, H, F, k, p, ctypes.byref(h)) == 0
    return h


def _at(i):
    """Distinct fake addresses, 1 GiB apart."""
    return P((i + 1) << 30)


def _refused(L, st, *words):
    msg = L.moe_last_error().decode()
    assert st == -1 and all(w in msg for w in words), (st, msg)


def test_workspace_sizes(L):
    h = _create(L)
    for fn in (L.moe_backward_workspace_bytes, L.moe_dispatch_workspace_bytes):
        assert fn(None, 64) == 0 and fn(h, -1) == 0
        sizes = [fn(h, T) for T in (0, 1, 64, 1000, 65536)]
        assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    T, k, H, F = 1000, 2, 128, 256
    rows = T * k
    assert L.moe_backward_workspace_bytes(h, T) >= L.moe_dispatch_workspace_bytes(h, T) + rows * (6 * F + 2 * H)
    L.moe_destroy(h)


def _dispatch(L, h, T=64, a=None, type=1, n=BIG):
    a = [_at(i) for i in range(7)] if a is None else a
    return L.moe_dispatch(h, a[0], type, a[1], T, a[2], a[3], a[4], a[5], a[6], n, None)


def test_dispatch_refusals(L):
    h = _create(L)
    _refused(L, _dispatch(L, None), "handle")
    _refused(L, _dispatch(L, h, T=-1), "T_cap")
    _refused(L, _dispatch(L, h, T=(1 << 26) + 1), "T_cap")
    _refused(L, _dispatch(L, h, type=2), "type")
    _refused(L, _dispatch(L, h, n=64), "ws_bytes")
    for i in range(7):
        a = [_at(j) for j in range(7)]
        a[i] = None
        _refused(L, _dispatch(L, h, a=a), "NULL")
        a[i] = P((i + 1 << 30) + 4)
        _refused(L, _dispatch(L, h, a=a), "aligned")
    for i, j in ((3, 0), (4, 1), (5, 2), (6, 0)):        # outputs in an input's memory
        a = [_at(n) for n in range(7)]
        a[i] = a[j]
        _refused(L, _dispatch(L, h, a=a), "input's memory")
    a = [_at(n) for n in range(7)]
    a[4] = P(a[3].value + 256)
    _refused(L, _dispatch(L, h, a=a), "share")
    L.moe_destroy(h)


def test_combine_refusals(L):
    h = _create(L)
    a = [_at(i) for i in range(5)]

    def call(a, h=h, T=64, t=0, o=0):
        return L.moe_combine_rows(h, a[0], t, a[1], a[2], T, a[3], a[4], o, None)
    _refused(L, call(a, h=None), "handle")
    _refused(L, call(a, T=-5), "T_cap")
    _refused(L, call(a, t=3), "type")
    _refused(L, call(a, o=-1), "type")
    for i in (0, 1, 3, 4):
        _refused(L, call(a[:i] + [None] + a[i + 1:]), "NULL")
    _refused(L, call(a[:2] + [P(8)] + a[3:]), "aligned")
    _refused(L, call(a[:4] + [P(a[0].value + 128)]), "input's memory")

    b = [_at(i) for i in range(7)]

    def back(b, h=h, T=64, t=0, o=0):
        return L.moe_combine_backward(h, b[0], o, b[1], t, b[2], b[3], T, b[4], b[5], b[6], None)
    _refused(L, back(b, h=None), "handle")
    _refused(L, back(b, t=9), "type")
    _refused(L, back(b[:1] + [None] + b[2:]), "d_probs needs rows")
    _refused(L, back(b[:6] + [None]), "d_probs needs rows")
    for i in (0, 2, 3, 4, 5):
        _refused(L, back(b[:i] + [None] + b[i + 1:]), "NULL")
    _refused(L, back(b[:5] + [b[1], b[6]]), "input's memory")
    _refused(L, back(b[:6] + [b[5]]), "share")
    L.moe_destroy(h)


def test_backward_refusals(L):
    a = [_at(i) for i in range(12)]

    def call(h, a=a, T=64, dt=1, wt=1, n=BIG):
        return L.moe_backward(h, a[0], dt, a[1], a[2], a[3], T, a[4], a[5], a[6], a[7], a[8], a[9], wt, a[10], a[11], n,
                              None)
    _refused(L, call(None), "handle")
    for p in (1, 2, 4):
        h = _create(L, p=p)
        _refused(L, call(h), "bf16")
        fc = L.moe_forward_checkpoint(h, a[0], a[1], a[2], 64, a[3], 0, a[4], a[5], a[6], a[7], BIG, None)
        _refused(L, fc, "bf16")
        L.moe_destroy(h)
    for H, F in ((32, (1 << 20) + 32), ((1 << 20) + 32, 32)):
        h = _create(L, 1, H, F, 1)
        assert call(h) == -2 and b"above" in L.moe_last_error()
        L.moe_destroy(h)
    h = _create(L)
    assert call(h) == -3 and b"load" in L.moe_last_error()

    def fc(combine=0, codes=a[5], scales=a[6]):
        return L.moe_forward_checkpoint(h, a[0], a[1], a[2], 64, a[3], combine, a[4], codes, scales, a[7], BIG, None)
    for combine in (3, 0x100, 0x200, 0x401, -1):
        _refused(L, fc(combine), "combine")
    _refused(L, fc(codes=None), "NULL")
    _refused(L, fc(scales=P(24)), "aligned")
    _refused(L, fc(scales=a[4]), "input's memory")
    _refused(L, fc(scales=a[5]), "share")
    assert fc() == -3
    L.moe_destroy(h)


def test_binding_refusals():
    from swiglu_expert_mlp_amd import MoE
    m = MoE(4, 32, 32, 2)
    codes, scales = m.new_checkpoint(8, device="cpu")
    assert codes.shape == (16, 64) and codes.dtype == torch.int8
    assert scales.shape == (16, 2) and scales.dtype == torch.uint8
    with pytest.raises(ValueError):
        m.combine(None, None, None, None)
    with pytest.raises(ValueError):
        m.bind_combine(None, None, None, None, None)
    with pytest.raises(ValueError):
        m.backward(None, None, None, None, None, None, None, grad_dtype="fp16")
    with pytest.raises(ValueError):
        m.combine(None, None, torch.zeros(1), None, combine="rows")
