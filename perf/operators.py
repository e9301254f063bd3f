"""Timed cases of the 8-bit integer experts and of the router's training operators.

Operators (each in a plain form, and as the library's own call):

  int8_forward    the routed SwiGLU MoE forward with 8-bit integer weights (a scale
                  per output channel) and activations (a scale per token)
  balance         per-expert counts, the balance loss and the z loss of the router
  route_backward  the gradient of the logits from both losses and from the
                  gradients of the selected probabilities
  probs_backward  the gradient of the combine's probabilities from the expert rows
                  that the forward left in its workspace
"""
import math

import torch

own = False

DEV = "cuda"
BALANCE_WEIGHT, Z_WEIGHT = 1e-2, 1e-3


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a small layer, as in a unit test or a draft model: launch latency counts
        dict(name="int8_tiny", op="int8_forward", T=64, cap=64, H=128, F=256, E=8, k=2, skew=False),
        # a decode step of a serving batch: the weights stream from memory
        dict(name="int8_decode", op="int8_forward", T=256, cap=256, H=2048, F=1024, E=64, k=6, skew=False),
        # decode in a buffer sized for the largest batch, with the live count on the device
        dict(name="int8_bounded", op="int8_forward", T=512, cap=65536, H=2688, F=1856, E=128, k=6, skew=False),
        # a log-prob forward whose experts are loaded unevenly
        dict(name="int8_logprob", op="int8_forward", T=4096, cap=4096, H=2048, F=1024, E=128, k=8, skew=True),
        # prefill of 16K tokens: bound by the matrix products
        dict(name="int8_16k", op="int8_forward", T=16384, cap=16384, H=2048, F=1024, E=128, k=8, skew=False),
        # the losses of a small micro-batch
        dict(name="balance_256", op="balance", T=256, cap=256, E=64, k=6, mask=False),
        # a training batch with padding tokens inside it
        dict(name="balance_16k", op="balance", T=16384, cap=16384, E=128, k=8, mask=True),
        # a long batch over many small experts
        dict(name="balance_64k_wide", op="balance", T=65536, cap=65536, E=1024, k=16, mask=False),
        # the gradients of the same batches
        dict(name="route_backward_4k", op="route_backward", T=4096, cap=4096, E=128, k=8, mask=True),
        dict(name="route_backward_64k_wide", op="route_backward", T=65536, cap=65536, E=1024, k=16, mask=False),
        # the probabilities' gradient of a micro-batch, the output's gradient in bf16
        dict(name="probs_backward_256", op="probs_backward", T=256, cap=256, H=2048, E=64, k=6, grad="bf16"),
        # and of a 16K-token batch in fp32
        dict(name="probs_backward_16k", op="probs_backward", T=16384, cap=16384, H=2048, E=128, k=8, grad="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int8_forward", "int8_forward", "balance", "route_backward", "probs_backward"])
    if op == "int8_forward":
        H, F = 32 * _log_int(rng, 2, 84), 32 * _log_int(rng, 2, 64)
        E = _log_int(rng, 2, 128)
        k = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 16384)
        T = max(1, min(T, int(1.6e12 / (6.0 * H * F * k))))
        cap = T if rng.random() < 0.7 else min(16384, T + _log_int(rng, 1, 2048))
        return dict(op=op, T=T, cap=cap, H=H, F=F, E=E, k=k, skew=rng.random() < 0.5)
    if op == "probs_backward":
        H = 32 * _log_int(rng, 2, 84)
        E = _log_int(rng, 2, 128)
        k = rng.randint(1, min(16, E))
        T = max(1, min(_log_int(rng, 1, 16384), (1 << 28) // (H * k)))
        return dict(op=op, T=T, cap=T + rng.choice([0, 0, 1, 37]), H=H, E=E, k=k, grad=rng.choice(["bf16", "fp32"]))
    E = _log_int(rng, 2, 1024)
    k = rng.randint(1, min(16, E))
    T = _log_int(rng, 1, 65536)
    return dict(op=op, T=T, cap=T + rng.choice([0, 0, 1, 37]), E=E, k=k, mask=rng.random() < 0.5)


def work(case):
    T, k, E = case["T"], case["k"], case["E"]
    if case["op"] == "int8_forward":
        H, F = case["H"], case["F"]
        touched = E * (1.0 - (1.0 - k / E) ** T)      # experts with a route, were all equally likely
        return {"bytes": touched * (3.0 * H * F + 4 * (2 * F + H)) + T * (2.0 * H + 2.0 * H + 8 * k),
                "flops": 6.0 * H * F * T * k}
    if case["op"] == "balance":
        return {"bytes": T * (4.0 * E + 4 * k) + 8.0 * E, "flops": 5.0 * T * E}
    if case["op"] == "route_backward":
        return {"bytes": T * (8.0 * E + 12 * k) + 4.0 * E, "flops": 9.0 * T * E}
    H = case["H"]
    return {"bytes": T * (4.0 * H * k + H * (2 if case["grad"] == "bf16" else 4) + 8 * k), "flops": 2.0 * T * k * H}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _logits(g, T, E, skew):
    z = _randn(g, T, E)
    return z + _randn(g, E) if skew else z


def _route(z, k):
    """Top-k experts in ascending order and their renormalized probabilities."""
    ids = z.topk(k, dim=1).indices.sort(dim=1).values
    return ids.to(torch.int32), torch.softmax(z.gather(1, ids), dim=1)


def _buffer(v, cap, fill):
    """`v` in the first rows of a buffer of `cap` rows, the others filled."""
    b = torch.full((cap,) + tuple(v.shape[1:]), fill, dtype=v.dtype, device=DEV)
    b[: v.shape[0]] = v
    return b


def _channel_codes(g, E, N, K, std):
    """Weights of a quantized checkpoint: int8 codes [E, N, K] and a scale per row."""
    codes = torch.empty((E, N, K), dtype=torch.int8, device=DEV)
    scales = torch.empty((E, N), dtype=torch.float32, device=DEV)
    for e in range(E):
        w = _randn(g, N, K) * std
        amax = w.abs().amax(dim=1)
        codes[e] = torch.round(w * (127.0 / amax)[:, None]).to(torch.int8)
        scales[e] = amax / 127.0
    return codes, scales


def _exact_experts(g, T, H, E):
    """Inputs and weights of experts whose SwiGLU rows hold no rounding: coordinate 0 of x
    is 32, which every gate picks (silu(32) = 32 in fp32), and every up row picks one
    other coordinate.  Gives x, W1, W2 (bf16) and the coordinates [E, 32]."""
    x = _randn(g, T, H)
    x[:, 0] = 32.0
    pick = torch.randint(1, H, (E, 32), generator=g, device=DEV)
    w1 = torch.zeros((E, 64, H), dtype=torch.bfloat16, device=DEV)
    w1[:, :32, 0] = 1.0
    w1[:, 32:].scatter_(2, pick[:, :, None], 1.0)
    w2 = (_randn(g, E, H, 32) * (0.7 / 181.0)).to(torch.bfloat16)
    return x.to(torch.bfloat16), w1, w2, pick


def _live(T):
    return torch.tensor([T], dtype=torch.int32, device=DEV)


def _inputs(case, seed):
    """The case's inputs, the same whatever computes them."""
    g = _gen(seed)
    T, cap, E, k = case["T"], case["cap"], case["E"], case["k"]
    s = dict(case)
    if case["op"] == "int8_forward":
        H, F = case["H"], case["F"]
        x = _randn(g, T, H)
        x[torch.rand(T, generator=g, device=DEV) < 0.05] *= 30.0       # outlier tokens
        s["x"] = _buffer(x.to(torch.bfloat16), cap, float("nan"))
        ids, probs = _route(_logits(g, T, E, case["skew"]), k)
        s["ids"], s["probs"] = _buffer(ids, cap, -1), _buffer(probs, cap, float("nan"))
        s["w1"], s["s1"] = _channel_codes(g, E, 2 * F, H, 0.02)
        s["w2"], s["s2"] = _channel_codes(g, E, H, F, 0.02)
        return s
    if case["op"] == "probs_backward":
        H = case["H"]
        x, s["w1"], s["w2"], s["pick"] = _exact_experts(g, T, H, E)
        s["x"] = _buffer(x, cap, float("nan"))
        ids, probs = _route(_logits(g, T, E, False), k)
        s["ids"], s["probs"] = _buffer(ids, cap, -1), _buffer(probs, cap, float("nan"))
        d_out = _randn(g, T, H).to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
        s["d_out"] = _buffer(d_out, cap, float("nan"))
        return s
    z = _logits(g, T, E, True)
    ids, probs = _route(z, k)
    s["logits"], s["ids"] = _buffer(z, cap, float("nan")), _buffer(ids, cap, -1)
    s["probs"] = _buffer(probs, cap, float("nan"))
    s["mask"] = None
    if case["mask"]:                                                   # False: a padding token
        s["mask"] = _buffer(torch.rand(T, generator=g, device=DEV) >= 0.25, cap, False)
    if case["op"] == "route_backward":
        s["d_probs"] = _buffer(_randn(g, T, k) / T, cap, float("nan"))
        s["d_losses"] = torch.tensor([BALANCE_WEIGHT, Z_WEIGHT], device=DEV)
        counted = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"][:T]
        c = torch.bincount(ids[counted].reshape(-1).long(), minlength=E)
        s["counts"] = torch.cat([c, counted.sum().reshape(1)]).to(torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    T, cap, E, k = case["T"], case["cap"], case["E"], case["k"]
    if own:
        from swiglu_expert_mlp_amd import MoE

        live = _live(T)
        s["live"] = live
        if case["op"] == "int8_forward":
            moe = MoE(E, case["H"], case["F"], k, "int8")
            moe.load_quantized(s["w1"], s["s1"], s["w2"], s["s2"])
            s["out"] = torch.empty((cap, case["H"]), dtype=torch.bfloat16, device=DEV)
            s["call"] = moe.bind_forward(s["x"], s["ids"], s["probs"], live, s["out"], moe.new_workspace(cap),
                                         combine="bf16")
        elif case["op"] == "balance":
            moe = MoE(E, 32, 32, k)
            s["losses"] = torch.empty(2, device=DEV)
            s["counts"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
            s["prob_sums"] = torch.empty(E, device=DEV)
            s["call"] = moe.bind_balance(s["logits"], s["ids"], live, s["losses"], s["counts"], s["prob_sums"],
                                         moe.new_balance_workspace(cap), mask=s["mask"])
        elif case["op"] == "route_backward":
            moe = MoE(E, 32, 32, k)
            s["d_logits"] = torch.empty((cap, E), device=DEV)
            s["call"] = moe.bind_route_backward(s["logits"], s["ids"], live, s["d_logits"], probs=s["probs"],
                                                d_probs=s["d_probs"], counts=s["counts"], d_losses=s["d_losses"],
                                                mask=s["mask"])
        else:
            moe = MoE(E, case["H"], 32, k)
            moe.load_weights(s["w1"], s["w2"])
            ws = moe.new_workspace(cap)
            moe.forward(s["x"], s["ids"], s["probs"], live, ws=ws)      # leaves its expert rows in ws
            s["d_probs"] = torch.empty((cap, k), device=DEV)
            s["call"] = moe.bind_probs_backward(s["d_out"], s["ids"], s["d_probs"], ws)
        s["moe"] = moe
    elif case["op"] == "probs_backward":
        rows = torch.empty((T, k, case["H"]), device=DEV)
        for e in range(E):
            t, j = (s["ids"][:T] == e).nonzero(as_tuple=True)
            rows[t, j] = (32.0 * s["x"][t].float()[:, s["pick"][e]]) @ s["w2"][e].float().t().contiguous()
        s["rows"] = rows
    return s


# ------------------------------------------------------------------ plain forms

def _row_codes(v):
    """Codes and scales of the rows of v: round half away from zero of 127 v / amax."""
    amax = v.abs().amax(dim=-1, keepdim=True)
    q = torch.floor(v.abs() * 127.0 / amax.clamp_min(1e-30) + 0.5) * torch.sign(v)
    return q, amax / 127.0


def _plain_int8(s):
    T, H, F, E, k = s["T"], s["H"], s["F"], s["E"], s["k"]
    x, ids, probs = s["x"][:T].float(), s["ids"][:T].long().reshape(-1), s["probs"][:T]
    xq, sx = _row_codes(x)
    counts = torch.bincount(ids, minlength=E)
    order = torch.argsort(ids, stable=True)
    M = int(counts.max())
    # every route's place in [E, M]: its expert, and its rank among the expert's routes
    slot = torch.empty_like(ids)
    slot[order] = ids[order] * M + torch.arange(T * k, device=DEV) - (torch.cumsum(counts, 0) - counts)[ids[order]]
    tok = torch.arange(T * k, device=DEV) // k
    a = torch.zeros((E * M, H), device=DEV)
    a[slot] = xq[tok]
    sa = torch.zeros((E * M, 1), device=DEV)
    sa[slot] = sx[tok]
    g = torch.bmm(a.view(E, M, H), s["w1"].float().transpose(1, 2).contiguous())
    g = g * sa.view(E, M, 1) * s["s1"][:, None, :]
    gate, up = g[..., :F], g[..., F:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16).float()     # the operator's FC2 input is bf16
    hq, sh = _row_codes(h)
    o = torch.bmm(hq, s["w2"].float().transpose(1, 2).contiguous()) * sh * s["s2"][:, None, :]
    return (o.view(E * M, H)[slot].view(T, k, H) * probs[:, :, None]).sum(dim=1).to(torch.bfloat16)


def _plain_balance(s):
    T, E, k = s["T"], s["E"], s["k"]
    z, ids = s["logits"][:T], s["ids"][:T].long()
    m = torch.ones(T, device=DEV) if s["mask"] is None else s["mask"][:T].float()
    top = z.amax(dim=1, keepdim=True)
    w = torch.exp(z - top)
    total = w.sum(dim=1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    prob_sums = (w / total * m[:, None]).sum(dim=0)
    counts = torch.zeros(E, device=DEV, dtype=torch.int32)
    counts.index_add_(0, ids.reshape(-1), m.to(torch.int32)[:, None].expand(T, k).reshape(-1))
    n = m.to(torch.int32).sum(dtype=torch.int32)
    nf = n.clamp_min(1).float()
    balance = E / k * (counts / nf * prob_sums / nf).sum()
    z_loss = (lse * lse * m).sum() / nf
    return {"losses": torch.stack([balance, z_loss]), "counts": torch.cat([counts, n.reshape(1)]),
            "prob_sums": prob_sums}


def _plain_route_backward(s):
    T, E, k = s["T"], s["E"], s["k"]
    z, ids, q, d = s["logits"][:T], s["ids"][:T].long(), s["probs"][:T], s["d_probs"][:T]
    m = torch.ones(T, device=DEV) if s["mask"] is None else s["mask"][:T].float()
    top = z.amax(dim=1, keepdim=True)
    w = torch.exp(z - top)
    total = w.sum(dim=1, keepdim=True)
    p, lse = w / total, top + torch.log(total)
    n = s["counts"][E].clamp_min(1).float()
    c = s["d_losses"][0] * (E / k) * s["counts"][:E] / n / n
    grad = p * (c - (p * c).sum(dim=1, keepdim=True) + s["d_losses"][1] * 2.0 * lse / n) * m[:, None]
    grad.scatter_add_(1, ids, q * (d - (q * d).sum(dim=1, keepdim=True)))
    return grad


def _plain_probs_backward(s):
    T = s["T"]
    return (s["rows"] * s["d_out"][:T].float()[:, None, :]).sum(dim=2)


def run(state):
    s = state
    T = s["T"]
    if own:
        s["call"]()
        if s["op"] == "int8_forward":
            return s["out"][:T]
        if s["op"] == "balance":
            return {"losses": s["losses"], "counts": s["counts"], "prob_sums": s["prob_sums"]}
        return s["d_logits"][:T] if s["op"] == "route_backward" else s["d_probs"][:T]
    plain = {"int8_forward": _plain_int8, "balance": _plain_balance, "route_backward": _plain_route_backward,
             "probs_backward": _plain_probs_backward}
    return plain[s["op"]](s)


# ------------------------------------------------------------------ 64 bits

def _codes64(v):
    amax = v.abs().max(dim=1).values
    ratio = 127.0 * v.abs() / torch.where(amax > 0, amax, torch.ones_like(amax))[:, None]
    return torch.copysign((ratio + 0.5).floor(), v), amax / 127.0


def exact(case, seed):
    s = _inputs(case, seed)
    T, E, k = case["T"], case["E"], case["k"]
    ids = s["ids"][:T].long()
    if case["op"] == "int8_forward":
        F = case["F"]
        xq, sx = _codes64(s["x"][:T].double())
        out = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV)
        for e in range(E):
            t, j = (ids == e).nonzero(as_tuple=True)
            if t.numel() == 0:
                continue
            gu = (xq[t] @ s["w1"][e].double().t()) * sx[t, None] * s["s1"][e].double()
            h = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
            hq, sh = _codes64(h.to(torch.bfloat16).double())
            row = (hq @ s["w2"][e].double().t()) * sh[:, None] * s["s2"][e].double()
            out.index_add_(0, t, row * s["probs"][t, j].double()[:, None])
        return out
    if case["op"] == "probs_backward":
        out = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        for e in range(E):
            t, j = (ids == e).nonzero(as_tuple=True)
            h = 32.0 * s["x"][t].double()[:, s["pick"][e]]
            out[t, j] = (s["d_out"][t].double() @ s["w2"][e].double() * h).sum(dim=1)
        return out
    z = s["logits"][:T].double()
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"][:T]
    lse = torch.logsumexp(z, dim=1)
    p = torch.exp(z - lse[:, None])
    if case["op"] == "balance":
        n = int(keep.sum())
        hits = torch.nn.functional.one_hot(ids[keep].reshape(-1), E).sum(dim=0) if n else ids.new_zeros(E)
        sums = p[keep].sum(dim=0)
        losses = torch.stack([(hits.double() * sums).sum() * E / (k * max(n, 1) ** 2),
                              lse[keep].square().sum() / max(n, 1)])
        return {"losses": losses, "counts": torch.cat([hits, hits.new_tensor([n])]).to(torch.int32),
                "prob_sums": sums}
    n = max(int(s["counts"][E]), 1)
    gb, gz = (float(v) for v in s["d_losses"].double())
    share = s["counts"][:E].double() * (gb * E / (k * n * n))
    inner = share[None, :] - (p @ share)[:, None] + gz * 2.0 * lse[:, None] / n
    grad = torch.where(keep[:, None], p * inner, torch.zeros_like(p))
    q, d = s["probs"][:T].double(), s["d_probs"][:T].double()
    back = q * (d - (q * d).sum(dim=1, keepdim=True))
    for i in range(k):
        grad[torch.arange(T, device=DEV), ids[:, i]] += back[:, i]
    return grad
