"""Timed cases of the experts' training and of tokens sorted by expert and back.

Operators (each in a plain form, and as the library's own call):

  forward_checkpoint  the routed SwiGLU MoE forward that also keeps every row's gate and
                      up values in 8 bits (a power-of-two scale per 32 values)
  backward            the gradients of x, of both weights and of the probabilities, from
                      those kept values
  dispatch            tokens copied to rows sorted by expert, and the gradient of that
  combine             rows summed back into tokens with the probabilities applied, and
                      the gradients of the rows and of the probabilities
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a small layer, as in a unit test: launch latency counts
        dict(name="train_forward_tiny", op="forward_checkpoint", T=64, cap=64, H=128, F=256, E=8, k=2, skew=False),
        # a training micro-batch whose experts are loaded unevenly
        dict(name="train_forward_4k", op="forward_checkpoint", T=4096, cap=4096, H=2048, F=1024, E=128, k=8, skew=True),
        # the backward pass of the small layer
        dict(name="backward_tiny", op="backward", T=64, cap=64, H=128, F=256, E=8, k=2, skew=False),
        # a short micro-batch in a buffer for more tokens: the weights and their gradients stream from memory
        dict(name="backward_1k", op="backward", T=1000, cap=1024, H=2048, F=1024, E=64, k=6, skew=False),
        # the backward pass of the uneven micro-batch
        dict(name="backward_4k", op="backward", T=4096, cap=4096, H=2048, F=1024, E=128, k=8, skew=True),
        # 16K tokens: bound by the matrix products
        dict(name="backward_16k", op="backward", T=16384, cap=16384, H=2048, F=1024, E=128, k=8, skew=False),
        # a serving batch sorted for experts of the caller's own
        dict(name="dispatch_256", op="dispatch", back=False, T=256, cap=256, H=2048, E=64, k=6, dtype="bf16"),
        # a training batch sorted for them
        dict(name="dispatch_16k", op="dispatch", back=False, T=16384, cap=16384, H=2048, E=128, k=8, dtype="bf16"),
        # the gradient of an odd number of tokens, in fp32
        dict(name="dispatch_backward_4k", op="dispatch", back=True, T=4099, cap=4100, H=2688, E=128, k=6, dtype="fp32"),
        # a serving batch's rows summed back
        dict(name="combine_256", op="combine", back=False, T=256, cap=256, H=2048, E=64, k=6, dtype="bf16"),
        # a training batch's rows in fp32
        dict(name="combine_16k", op="combine", back=False, T=16384, cap=16384, H=2048, E=128, k=8, dtype="fp32"),
        # and the gradients of a training batch's bf16 rows and probabilities
        dict(name="combine_backward_16k", op="combine", back=True, T=16384, cap=16384, H=2048, E=128, k=8, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward_checkpoint", "backward", "backward", "dispatch", "combine"])
    H = 32 * _log_int(rng, 2, 84)
    E = _log_int(rng, 2, 128)
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, 16384)
    if op in ("dispatch", "combine"):
        T = max(1, min(T, (1 << 28) // (H * k)))
        return dict(op=op, back=rng.random() < 0.5, T=T, cap=T + rng.choice([0, 0, 1, 37]), H=H, E=E, k=k,
                    dtype=rng.choice(["bf16", "fp32"]))
    F = 32 * _log_int(rng, 2, 64)
    T = max(1, min(T, int(1.6e12 / (6.0 * H * F * k))))
    cap = T if rng.random() < 0.7 else min(16384, T + _log_int(rng, 1, 2048))
    return dict(op=op, T=T, cap=cap, H=H, F=F, E=E, k=k, skew=rng.random() < 0.5)


def work(case):
    T, k, E, H = case["T"], case["k"], case["E"], case["H"]
    R = T * k
    if case["op"] in ("forward_checkpoint", "backward"):
        F = case["F"]
        touched = E * (1.0 - (1.0 - k / E) ** T)      # experts with a route, were all equally likely
        kept = R * (2.0 * F + F / 16.0)
        if case["op"] == "forward_checkpoint":
            return {"bytes": touched * 6.0 * H * F + T * (4.0 * H + 8 * k) + kept, "flops": 6.0 * H * F * R}
        return {"bytes": (touched + E) * 6.0 * H * F + T * (6.0 * H + 12 * k) + kept, "flops": 12.0 * H * F * R}
    size = 2.0 if case["dtype"] == "bf16" else 4.0
    if case["op"] == "dispatch":
        extra = 4.0 * R if case["back"] else 8.0 * R + 4.0 * E
        return {"bytes": (T + R) * H * size + extra, "flops": 1.0 * R * H if case["back"] else 0.0}
    if case["back"]:
        return {"bytes": (T + 2 * R) * H * size + 12.0 * R, "flops": 3.0 * R * H}
    return {"bytes": (T + R) * H * size + 8.0 * R, "flops": 2.0 * R * H}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _route(g, T, E, k, skew):
    """Top-k experts in ascending order and their renormalized probabilities."""
    z = _randn(g, T, E)
    if skew:
        z = z + _randn(g, E)
    ids = z.topk(k, dim=1).indices.sort(dim=1).values
    return ids.to(torch.int32), torch.softmax(z.gather(1, ids), dim=1)


def _buffer(v, cap, fill):
    """`v` in the first rows of a buffer of `cap` rows, the others filled."""
    b = torch.full((cap,) + tuple(v.shape[1:]), fill, dtype=v.dtype, device=DEV)
    b[: v.shape[0]] = v
    return b


def _weights(g, E, N, K, std):
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e] = (_randn(g, N, K) * std).to(torch.bfloat16)
    return w


def _kept(v):
    """int8 codes [.., C] and scale bytes [.., C / 32] of the rows of v: a scale 2^(byte - 127) per
    32 columns, the smallest whose 127-fold reaches every magnitude."""
    b = v.reshape(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(dim=2))           # amax = m 2^e, 1/2 <= m < 1
    e = (e - 7 + (m > 127.0 / 128.0).to(torch.int32)).clamp(-127, 127)
    codes = torch.round(torch.ldexp(b, -e[..., None]))
    return codes.reshape(v.shape).to(torch.int8), (e + 127).to(torch.uint8)


def _row_order(ids, E):
    """Routes (t k + j) in the order of their rows: by expert, then by token."""
    return torch.argsort(ids.reshape(-1).long(), stable=True)


def _interleave(gate, up):
    """Columns of gate and up in blocks of 32 by turns."""
    n, F = gate.shape
    return torch.stack([gate.reshape(n, F // 32, 32), up.reshape(n, F // 32, 32)], dim=2).reshape(n, 2 * F)


def _inputs(case, seed):
    """The case's inputs, the same whatever computes them."""
    g = _gen(seed)
    T, cap, E, k, H = case["T"], case["cap"], case["E"], case["k"], case["H"]
    s = dict(case)
    ids, probs = _route(g, T, E, k, case.get("skew", False))
    s["ids"], s["probs"] = _buffer(ids, cap, -1), _buffer(probs, cap, float("nan"))
    if case["op"] in ("forward_checkpoint", "backward"):
        F = case["F"]
        x = _randn(g, T, H)
        x[torch.rand(T, generator=g, device=DEV) < 0.05] *= 3.0        # louder tokens
        x = x.to(torch.bfloat16)
        s["x"] = _buffer(x, cap, float("nan"))
        s["w1"], s["w2"] = _weights(g, E, 2 * F, H, 0.02), _weights(g, E, H, F, 0.02)
        if case["op"] == "backward":
            s["d_out"] = _buffer((_randn(g, T, H) / T).to(torch.bfloat16), cap, float("nan"))
            # what a forward keeps: rows by expert, the blocks of gate and up by turns
            s["codes"] = torch.zeros((cap * k, 2 * F), dtype=torch.int8, device=DEV)
            s["scales"] = torch.zeros((cap * k, F // 16), dtype=torch.uint8, device=DEV)
            order = _row_order(ids, E)
            ends = torch.bincount(ids.reshape(-1).long(), minlength=E).cumsum(0).tolist()
            for e in range(E):
                r0, r1 = (ends[e - 1] if e else 0), ends[e]
                if r1 > r0:
                    gu = (x[order[r0:r1] // k] @ s["w1"][e].t()).float()
                    s["codes"][r0:r1], s["scales"][r0:r1] = _kept(_interleave(gu[:, :F], gu[:, F:]))
        return s
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    row_of = torch.empty(T * k, dtype=torch.int32, device=DEV)
    row_of[_row_order(ids, E)] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    s["row_of"] = _buffer(row_of.view(T, k), cap, -1)
    if case["op"] == "dispatch" and not case["back"]:
        s["x"] = _buffer(_randn(g, T, H).to(dt), cap, float("nan"))
        return s
    s["rows"] = _buffer(_randn(g, T * k, H).to(dt), cap * k, float("nan"))
    if case["op"] == "combine" and case["back"]:
        s["d_out"] = _buffer(_randn(g, T, H).to(dt), cap, float("nan"))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from swiglu_expert_mlp_amd import MoE

    cap, E, k, H = case["cap"], case["E"], case["k"], case["H"]
    live = torch.tensor([case["T"]], dtype=torch.int32, device=DEV)
    s["live"] = live
    moe = MoE(E, H, case.get("F", 32), k)
    s["moe"] = moe
    if case["op"] in ("forward_checkpoint", "backward"):
        moe.load_weights(s["w1"], s["w2"])
        if case["op"] == "forward_checkpoint":
            s["out"] = torch.empty((cap, H), dtype=torch.bfloat16, device=DEV)
            s["codes"], s["scales"] = moe.new_checkpoint(cap)
            s["call"] = moe.bind_forward_checkpoint(s["x"], s["ids"], s["probs"], live, s["out"], s["codes"],
                                                    s["scales"], moe.new_workspace(cap), combine="bf16")
        else:
            s["d_x"], s["d_probs"] = torch.empty_like(s["x"]), torch.empty((cap, k), device=DEV)
            s["d_w1"], s["d_w2"] = torch.empty_like(s["w1"]), torch.empty_like(s["w2"])
            s["call"] = moe.bind_backward(s["d_out"], s["x"], s["ids"], s["probs"], live, s["codes"], s["scales"],
                                          s["d_x"], s["d_w1"], s["d_w2"], s["d_probs"],
                                          moe.new_backward_workspace(cap))
    elif case["op"] == "dispatch":
        if case["back"]:
            s["d_x"] = torch.empty((cap, H), dtype=s["rows"].dtype, device=DEV)
            s["call"] = moe.bind_dispatch_backward(s["rows"], s["row_of"], live, s["d_x"])
        else:
            s["rows"] = torch.empty((cap * k, H), dtype=s["x"].dtype, device=DEV)
            s["to"] = torch.empty((cap, k), dtype=torch.int32, device=DEV)
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
            s["call"] = moe.bind_dispatch(s["x"], s["ids"], live, s["rows"], s["to"], s["offsets"],
                                          moe.new_dispatch_workspace(cap))
    elif case["back"]:
        s["d_rows"], s["d_probs"] = torch.empty_like(s["rows"]), torch.empty((cap, k), device=DEV)
        s["call"] = moe.bind_combine_backward(s["d_out"], s["rows"], s["row_of"], s["probs"], live, s["d_rows"],
                                              s["d_probs"])
    else:
        s["out"] = torch.empty((cap, H), dtype=s["rows"].dtype, device=DEV)
        s["call"] = moe.bind_combine(s["rows"], s["row_of"], s["probs"], live, s["out"])
    return s


# ------------------------------------------------------------------ plain forms

def _values(codes, scales, dtype):
    """The numbers that kept codes stand for (7 bits and a power of two: exact in bf16)."""
    n, C = codes.shape
    step = (scales.to(torch.int16) << 7).view(torch.bfloat16)           # 2^(byte - 127), 0 for byte 0
    return (codes.view(n, C // 32, 32) * step[:, :, None].to(dtype)).view(n, C)


def _slots(s):
    """Every route's place in [E, M] (its expert, its rank there), the routes' order by rows, and M."""
    E, k, T = s["E"], s["k"], s["T"]
    ids = s["ids"][:T].long().reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    order = torch.argsort(ids, stable=True)
    M = int(counts.max())
    slot = torch.empty_like(ids)
    slot[order] = ids[order] * M + torch.arange(T * k, device=DEV) - (torch.cumsum(counts, 0) - counts)[ids[order]]
    return slot, order, M


def _padded(v, slot, E, M):
    b = torch.zeros((E * M, v.shape[1]), device=DEV)
    b[slot] = v
    return b.view(E, M, v.shape[1])


def _plain_forward(s):
    T, H, F, E, k = s["T"], s["H"], s["F"], s["E"], s["k"]
    slot, order, M = _slots(s)
    tok = torch.arange(T * k, device=DEV) // k
    a = _padded(s["x"][:T].float()[tok], slot, E, M)
    gu = torch.bmm(a, s["w1"].float().transpose(1, 2).contiguous())
    gate, up = gu[..., :F], gu[..., F:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    o = torch.bmm(h, s["w2"].float().transpose(1, 2).contiguous())
    out = (o.view(E * M, H)[slot].view(T, k, H) * s["probs"][:T, :, None]).sum(dim=1).to(torch.bfloat16)
    rows = gu.view(E * M, 2 * F)[slot[order]]
    codes, scales = _kept(_interleave(rows[:, :F], rows[:, F:]))
    return {"out": out, "kept": _values(codes, scales, torch.bfloat16)}


def _plain_backward(s):
    T, H, F, E, k = s["T"], s["H"], s["F"], s["E"], s["k"]
    slot, order, M = _slots(s)
    tok = torch.arange(T * k, device=DEV) // k
    w1, w2 = s["w1"].float(), s["w2"].float()
    kept = _values(s["codes"][: T * k], s["scales"][: T * k], torch.float32).view(T * k, F // 32, 2, 32)
    gate = _padded(kept[:, :, 0].reshape(T * k, F), slot[order], E, M)
    up = _padded(kept[:, :, 1].reshape(T * k, F), slot[order], E, M)
    x = _padded(s["x"][:T].float()[tok], slot, E, M)
    d = _padded(s["d_out"][:T].float()[tok], slot, E, M)
    p = _padded(s["probs"][:T].reshape(-1, 1), slot, E, M)
    dh = torch.bmm(d, w2)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    h = gate * sig * up
    d_probs = (dh * h).sum(dim=2).view(-1)[slot].view(T, k)
    dh = dh * p
    dgu = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig], dim=2)
    dx = torch.bmm(dgu, w1).view(E * M, H)[slot].view(T, k, H).sum(dim=1)
    d_w1 = torch.bmm(dgu.transpose(1, 2).contiguous(), x)
    d_w2 = torch.bmm((d * p).transpose(1, 2).contiguous(), h)
    return {"d_x": dx.to(torch.bfloat16), "d_w1": d_w1.to(torch.bfloat16), "d_w2": d_w2.to(torch.bfloat16),
            "d_probs": d_probs}


def _plain_dispatch(s):
    T, E, k = s["T"], s["E"], s["k"]
    if s["back"]:
        return s["rows"][s["row_of"][:T].long()].float().sum(dim=1).to(s["rows"].dtype)
    ids = s["ids"][:T].long().reshape(-1)
    order = torch.argsort(ids, stable=True)
    row_of = torch.empty(T * k, dtype=torch.int32, device=DEV)
    row_of[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(ids, minlength=E).cumsum(0)
    return {"rows": s["x"][order // k], "row_of": row_of.view(T, k), "offsets": offsets}


def _plain_combine(s):
    T, k = s["T"], s["k"]
    p, row_of = s["probs"][:T, :, None], s["row_of"][:T].long()
    rows = s["rows"][row_of].float()
    if not s["back"]:
        return (rows * p).sum(dim=1).to(s["rows"].dtype)
    d = s["d_out"][:T].float()[:, None, :]
    d_rows = torch.empty_like(s["rows"][: T * k])
    d_rows[row_of] = (p * d).to(d_rows.dtype)
    return {"d_rows": d_rows, "d_probs": (rows * d).sum(dim=2)}


def run(state):
    s = state
    T, k = s["T"], s["k"]
    if not own:
        plain = {"forward_checkpoint": _plain_forward, "backward": _plain_backward, "dispatch": _plain_dispatch,
                 "combine": _plain_combine}
        return plain[s["op"]](s)
    s["call"]()
    if s["op"] == "forward_checkpoint":
        return {"out": s["out"][:T], "kept": _values(s["codes"][: T * k], s["scales"][: T * k], torch.bfloat16)}
    if s["op"] == "backward":
        return {"d_x": s["d_x"][:T], "d_w1": s["d_w1"], "d_w2": s["d_w2"], "d_probs": s["d_probs"][:T]}
    if s["op"] == "dispatch":
        return s["d_x"][:T] if s["back"] else {"rows": s["rows"][: T * k], "row_of": s["to"][:T],
                                               "offsets": s["offsets"]}
    return {"d_rows": s["d_rows"][: T * k], "d_probs": s["d_probs"][:T]} if s["back"] else s["out"][:T]


# ------------------------------------------------------------------ 64 bits

def _kept64(v):
    """The values that the kept codes of the rows of v stand for."""
    b = v.view(v.shape[0], -1, 32)
    top = b.abs().max(dim=2, keepdim=True).values
    step = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 127.0)))
    return (torch.round(b / step) * step).view(v.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    T, E, k, H = case["T"], case["E"], case["k"], case["H"]
    ids, probs = s["ids"][:T].long(), s["probs"][:T].double()
    if case["op"] in ("forward_checkpoint", "backward"):
        F = case["F"]
        f64 = dict(dtype=torch.float64, device=DEV)
        x = s["x"][:T].double()
        back = case["op"] == "backward"
        if back:
            d_out = s["d_out"][:T].double()
            dx, d_probs = torch.zeros((T, H), **f64), torch.zeros((T, k), **f64)
            d_w1, d_w2 = torch.zeros((E, 2 * F, H), **f64), torch.zeros((E, H, F), **f64)
        else:
            out, kept = torch.zeros((T, H), **f64), torch.zeros((T * k, 2 * F), **f64)
        r0 = 0
        for e in range(E):
            t, j = (ids == e).nonzero(as_tuple=True)
            n = t.numel()
            if n == 0:
                continue
            w1, w2, p = s["w1"][e].double(), s["w2"][e].double(), probs[t, j][:, None]
            if not back:
                gu = x[t] @ w1.t()
                h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
                out.index_add_(0, t, p * (h @ w2.t()))
                kept[r0:r0 + n] = _kept64(_interleave(gu[:, :F], gu[:, F:]))
            else:
                scale = torch.exp2(s["scales"][r0:r0 + n].double() - 127.0)
                gu = (s["codes"][r0:r0 + n].double().view(n, -1, 32) * scale[..., None]).view(n, -1, 2, 32)
                gate, up = gu[:, :, 0].reshape(n, F), gu[:, :, 1].reshape(n, F)
                sig = torch.sigmoid(gate)
                raw = d_out[t] @ w2
                h = gate * sig * up
                d_probs[t, j] = (raw * h).sum(dim=1)
                dh = raw * p
                dgu = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], dim=1)
                dx.index_add_(0, t, dgu @ w1)
                d_w1[e] = dgu.t() @ x[t]
                d_w2[e] = (p * d_out[t]).t() @ h
            r0 += n
        if back:
            return {"d_x": dx, "d_w1": d_w1, "d_w2": d_w2, "d_probs": d_probs}
        return {"out": out, "kept": kept}
    row_of = s["row_of"][:T].long()
    if case["op"] == "dispatch":
        if not case["back"]:
            rows = torch.empty((T * k, H), dtype=torch.float64, device=DEV)
            for i in range(k):
                rows[row_of[:, i]] = s["x"][:T].double()
            ends = [int((ids < e).sum()) for e in range(E + 1)]
            return {"rows": rows, "row_of": row_of.to(torch.int32),
                    "offsets": torch.tensor(ends, dtype=torch.int32, device=DEV)}
        out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        for i in range(k):
            out += s["rows"][row_of[:, i]].double()
        return out
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    if not case["back"]:
        for i in range(k):
            out += probs[:, i, None] * s["rows"][row_of[:, i]].double()
        return out
    d = s["d_out"][:T].double()
    d_rows = torch.empty((T * k, H), dtype=torch.float64, device=DEV)
    d_probs = torch.empty((T, k), dtype=torch.float64, device=DEV)
    for i in range(k):
        d_rows[row_of[:, i]] = probs[:, i, None] * d
        d_probs[:, i] = (d * s["rows"][row_of[:, i]].double()).sum(dim=1)
    return {"d_rows": d_rows, "d_probs": d_probs}
