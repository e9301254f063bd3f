"""int8 experts on the CPU: the oracle's quantizer, layer and packed layout against
independent formulations, and the boundary's refusals (no compute calls)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle
from workloads import Workload, make_inputs

INT8 = 4


@pytest.fixture(scope="module")
def L():
    import swiglu_expert_mlp_amd as m
    return m.lib()


def _handle(L, E, H, F, k, p=INT8):
    h = ctypes.c_void_p()
    return L.moe_create(E, H, F, k, p, ctypes.byref(h)), h


def test_codes_are_the_rational_formula():
    """sign(v) floor(127 |v| / amax + 1/2) in exact rationals, ties among them."""
    rng = np.random.default_rng(3)
    v = oracle.bf16_value(oracle.bf16_bits(rng.standard_normal((40, 96)).astype(np.float32)))
    v[0, :4] = [127.0, 63.5, -63.5, 0.5]           # ties of a row whose amax is 127
    v[0, 4:] = 0.0
    v[1, :3] = [3.0, 1.5, -1.5]                    # 63.5 again, amax 3
    v[1, 3:] = 0.0
    v[2] = 0.0
    v[3] = oracle.bf16_value(np.uint16(1))         # the smallest bf16 subnormal
    q, s = oracle.int8_quantize(v)
    assert list(q[0, :4]) == [127, 64, -64, 1] and list(q[1, :3]) == [127, 64, -64]
    assert s[2] == 0 and not q[2].any() and np.all(q[3] == 127)
    for r in range(40):
        amax = Fraction(float(np.abs(v[r]).max()))
        assert s[r] == np.float32(np.abs(v[r]).max()) / np.float32(127)
        for c in range(96):
            if amax:
                e = (abs(Fraction(float(v[r, c]))) * 127 / amax + Fraction(1, 2)).__floor__()
                assert q[r, c] == (-e if v[r, c] < 0 else e), (r, c)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_row_with_a_non_finite_value_has_scale_nan(bad):
    v = np.ones((2, 32), np.float32)
    v[1, 5] = bad
    q, s = oracle.int8_quantize(v)
    assert s[0] == np.float32(1) / np.float32(127) and np.isnan(s[1]) and not q[1].any()


def test_layer_against_integer_numpy():
    """The oracle's forward against int64 products and fp64 scaling."""
    w = Workload("t", 20, 20, 96, 64, 5, 3, "int8")
    inp = make_inputs(w, seed=5)
    ids, probs, _ = oracle.route(inp["logits"], w.T, w.k)
    m = oracle.Model(w.E, w.H, w.F, w.k, inp["w1_bits"], inp["w2_bits"], "int8")
    out, err, _ = m.forward(inp["x_bits"], ids, probs, w.T)
    assert err == 0
    xq, sx = oracle.int8_quantize(oracle.bf16_value(inp["x_bits"]))
    q1, s1 = oracle.int8_quantize(oracle.bf16_value(inp["w1_bits"]).reshape(-1, w.H))
    q2, s2 = oracle.int8_quantize(oracle.bf16_value(inp["w2_bits"]).reshape(-1, w.F))
    q1, s1 = q1.reshape(w.E, 2 * w.F, w.H).astype(np.int64), s1.reshape(w.E, 2 * w.F).astype(np.float64)
    q2, s2 = q2.reshape(w.E, w.H, w.F).astype(np.int64), s2.reshape(w.E, w.H).astype(np.float64)
    ref = np.zeros((w.T, w.H))
    for t in range(w.T):
        for j in range(w.k):
            e = ids[t, j]
            gu = (q1[e] @ xq[t].astype(np.int64)) * s1[e] * sx[t]
            h = gu[: w.F] / (1 + np.exp(-gu[: w.F])) * gu[w.F:]
            hq, sh = oracle.int8_quantize(oracle.bf16_value(oracle.bf16_bits(h.astype(np.float32)))[None])
            ref[t] += probs[t, j] * (q2[e] @ hq[0].astype(np.int64)) * s2[e] * float(sh[0])
    # fp32 scaling and SwiGLU (a few 2^-24 each) may move a bf16 rounding of h in a
    # few of the 64 x 60 elements, by one code (1 / 127 of a row's largest) each
    assert np.linalg.norm(out - ref) <= 2e-3 * np.linalg.norm(ref)
    tok = m.forward_tokens(inp["x_bits"], ids, probs, np.arange(w.T))
    assert np.array_equal(tok, out)
    mq = oracle.Model.quantized(w.E, w.H, w.F, w.k, q1, s1, q2, s2)
    assert np.array_equal(mq.forward(inp["x_bits"], ids, probs, w.T)[0], out)


@pytest.mark.parametrize("E,H,F", [(2, 96, 160), (1, 32, 64), (3, 544, 288), (2, 128, 256)])
def test_packed_layout_inverted_by_reshapes(E, H, F):
    rng = np.random.default_rng(H + F)
    w1 = oracle.bf16_bits(rng.standard_normal((E, 2 * F, H)).astype(np.float32))
    w2 = oracle.bf16_bits(rng.standard_normal((E, H, F)).astype(np.float32))
    buf = oracle.pack(E, H, F, w1, w2, "int8")
    up = lambda v: (v + 255) // 256 * 256
    pitch = lambda K: (K + 63) // 64 * 64 if K < 256 else (K + 127) // 128 * 128
    at = 0
    for N, K, w, fc1 in ((2 * F, H, w1, True), (H, F, w2, False)):
        q, _ = oracle.int8_quantize(oracle.bf16_value(w).reshape(E * N, K))
        q = q.reshape(E, N, K)
        if fc1:
            q = q.reshape(E, 2, F // 32, 32, K).transpose(0, 2, 1, 3, 4).reshape(E, N, K)
        Kp = pitch(K)
        got = buf[at: at + E * N * Kp].view(np.int8).reshape(E, N * Kp)
        rows = []
        for g0 in range(0, N // 16, 32):           # 512-row groups, the last one narrower
            width = min(32, N // 16 - g0)
            part = got[:, g0 * 16 * Kp: (g0 + width) * 16 * Kp]
            part = part.reshape(E, Kp // 64, width, 4, 16, 16).transpose(0, 2, 4, 1, 3, 5)
            rows.append(part.reshape(E, width * 16, Kp))
        got = np.concatenate(rows, axis=1)
        assert np.array_equal(got[:, :, :K], q) and not got[:, :, K:].any()
        at += up(E * N * Kp)
    for N, K, w, fc1 in ((2 * F, H, w1, True), (H, F, w2, False)):
        _, s = oracle.int8_quantize(oracle.bf16_value(w).reshape(E * N, K))
        s = s.reshape(E, N)
        if fc1:
            s = s.reshape(E, 2, F // 32, 32).transpose(0, 2, 1, 3).reshape(E, N)
        assert np.array_equal(buf[at: at + 4 * E * N].view(np.float32).reshape(E, N), s)
        at += up(4 * E * N)
    assert at == buf.size


def test_create_and_sizes(L):
    import swiglu_expert_mlp_amd as m
    st, h = _handle(L, 8, 128, 288, 2)
    assert st == 0 and L.moe_weight_bytes(h) == oracle.pack_bytes(8, 128, 288, "int8")
    sizes = [L.moe_workspace_bytes(h, T) for T in (0, 1, 64, 1000)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    L.moe_destroy(h)
    assert m.MoE(8, 128, 256, 2, "int8").precision == "int8"
    # an int32 sum holds K products of 128 x 128 for K below 131072
    for H, F in ((131072, 32), (32, 131072)):
        assert _handle(L, 1, H, F, 1)[0] == -2 and b"int8" in L.moe_last_error()
    st, h = _handle(L, 1, 131072 - 32, 32, 1)
    assert st == 0
    L.moe_destroy(h)


def test_refusals(L):
    P = ctypes.c_void_p
    fake = P(1 << 20)
    st, h = _handle(L, 8, 128, 256, 2, 0)
    assert L.moe_load_quantized(h, fake, fake, fake, fake, fake, 1 << 30, None) == -1
    assert b"not int8" in L.moe_last_error()
    L.moe_destroy(h)
    st, h = _handle(L, 8, 128, 256, 2)
    need = L.moe_weight_bytes(h)
    good = [fake] * 5
    for i in range(5):
        for p in (None, P((1 << 20) + 4)):
            args = good[:i] + [p] + good[i + 1:]
            assert L.moe_load_quantized(h, *args, need, None) == -1, (i, p)
    assert L.moe_load_quantized(h, *good, need - 1, None) == -1 and b"kbuf_bytes" in L.moe_last_error()
    assert L.moe_load_quantized(None, *good, need, None) == -1
    assert L.moe_forward(h, fake, fake, fake, 64, fake, fake, fake, 1 << 30, None) == -3
    L.moe_destroy(h)
