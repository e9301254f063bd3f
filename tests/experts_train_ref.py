"""fp64 references of the experts' training operators (torch, no code of the library),
with elementwise bounds on what their fp32 sums and bf16 roundings may be off by.

A rounding to bf16 is off by at most B = 2^-8 of the value, one to fp32 by S = 2^-24; a sum
of n products in fp32 by n S of the sum of the magnitudes.  The sigmoid is within
(|g| + 6) S of its value (the exponent's product is off by |g| S, the exponential, the sum
and the reciprocal by units in the last place): 2^-20 for the |g| <= 10 that the tests have.
"""
import torch

B, S, SIG = 2.0 ** -8, 2.0 ** -24, 2.0 ** -20


def routes(ids, E, T):
    """Grouped rows of the live tokens: (token, place) per row, and the offsets [E + 1];
    a route whose id is outside [0, E) or repeats an earlier one of its token has none."""
    seen, per = set(), [[] for _ in range(E)]
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if 0 <= e < E and (t, e) not in seen:
                seen.add((t, e))
                per[e].append((t, j))
    off = [0]
    for p in per:
        off.append(off[-1] + len(p))
    return [r for p in per for r in p], off


def row_of_ref(ids, E, T):
    rows, off = routes(ids.tolist(), E, T)
    out = torch.full((T, ids.shape[1]), -1, dtype=torch.int32)
    for r, (t, j) in enumerate(rows):
        out[t, j] = r
    return out, off


def kept_values(codes, scales):
    """fp64 values of codes [n, 2F] with scale bytes [n, F / 16]."""
    n, C = codes.shape
    step = torch.exp2(scales.double() - 127.0)
    step = torch.where(scales == 255, torch.full_like(step, float("nan")), step)
    return (codes.double().view(n, C // 32, 32) * step[..., None]).view(n, C)


def split(v):
    """gate, up of the interleaved columns"""
    n, C = v.shape
    b = v.view(n, C // 64, 2, 32)
    return b[:, :, 0].reshape(n, C // 2), b[:, :, 1].reshape(n, C // 2)


def join(gate, up):
    n, F = gate.shape
    return torch.stack([gate.view(n, F // 32, 32), up.view(n, F // 32, 32)], dim=2).reshape(n, 2 * F)


def backward_ref(d_out, x, ids, probs, T, codes, scales, w1, w2, wide):
    """Gradients {name: (value, bound)} in fp64.  wide: the weights' gradients are fp32."""
    E, _, H = w1.shape
    F, k = w2.shape[2], ids.shape[1]
    dev = x.device
    rows, off = routes(ids.tolist(), E, T)
    f64 = dict(dtype=torch.float64, device=dev)
    dx, bx = torch.zeros((T, H), **f64), torch.zeros((T, H), **f64)
    mag_x = torch.zeros((T, H), **f64)
    dp, bp = torch.zeros((T, k), **f64), torch.zeros((T, k), **f64)
    dw1, b1 = torch.zeros((E, 2 * F, H), **f64), torch.zeros((E, 2 * F, H), **f64)
    dw2, b2 = torch.zeros((E, H, F), **f64), torch.zeros((E, H, F), **f64)
    kept = kept_values(codes[: off[-1]], scales[: off[-1]])
    out_eps = S if wide else B
    for e in range(E):
        n = off[e + 1] - off[e]
        if n == 0:
            continue
        t = torch.tensor([r[0] for r in rows[off[e]: off[e + 1]]], device=dev)
        j = torch.tensor([r[1] for r in rows[off[e]: off[e + 1]]], device=dev)
        g, u = split(kept[off[e]: off[e + 1]])
        p = probs[t, j].double()[:, None]
        d, v1, v2 = d_out[t].double(), w1[e].double(), w2[e].double()
        raw = d @ v2
        raw_off = (H + 4) * S * (d.abs() @ v2.abs())
        s = torch.sigmoid(g)
        silu, h = g * s, g * s * u
        dsilu = s + silu * (1 - s)
        dsilu_off = SIG * (s + silu.abs() * (2 - s)) * 2
        dp[t, j] = (raw * h).sum(dim=1)
        bp[t, j] = (raw_off * h.abs() + raw.abs() * h.abs() * (2 * SIG + (F + 8) * S)).sum(dim=1)
        dg, du = p * raw * u * dsilu, p * raw * silu
        og = p * u.abs() * (raw_off * dsilu.abs() + raw.abs() * dsilu_off) + dg.abs() * (B + 4 * S)
        ou = p * silu.abs() * (raw_off + raw.abs() * SIG) + du.abs() * (B + 4 * S)
        hp = p * h
        oh = hp.abs() * (B + 2 * SIG)
        dgu, ogu = torch.cat([dg, du], dim=1), torch.cat([og, ou], dim=1)
        row = dgu @ v1
        # a route's row: its operand's rounding, the sum's, and that of 16-bit integers whose
        # scale 16 columns share: half of one, 2^-15 of the largest of the 16
        row_off = (ogu + (2 * F + 4) * S * (dgu.abs() + ogu)) @ v1.abs()
        top = (row.abs() + row_off).view(n, H // 16, 16).max(dim=2, keepdim=True).values
        row_off = row_off + (2.0 ** -15 * top).expand(n, H // 16, 16).reshape(n, H)
        dx.index_add_(0, t, row)
        bx.index_add_(0, t, row_off)
        mag_x.index_add_(0, t, row.abs() + row_off)
        xt = x[t].double()
        dw1[e] = dgu.t() @ xt
        b1[e] = (ogu + (n + 4) * S * (dgu.abs() + ogu)).t() @ xt.abs()
        dw2[e] = d.t() @ hp
        b2[e] = d.abs().t() @ (oh + (n + 4) * S * (hp.abs() + oh))
    bx = bx + (k + 2) * S * mag_x
    tiny = 1e-36                                   # below the smallest normal numbers
    fin = lambda v, b, eps: (v, b * (1 + eps) + v.abs() * eps + tiny)   # noqa: E731
    return {"d_x": fin(dx, bx, B), "d_w1": fin(dw1, b1, out_eps), "d_w2": fin(dw2, b2, out_eps), "d_probs": fin(dp, bp, S)}


def forward64(x, ids, probs, w1, w2):
    """The layer in fp64, without roundings: out [T, H]."""
    T, (E, H, F) = x.shape[0], w2.shape
    out = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j, e in enumerate(ids[t].tolist()):
            gu = w1[e] @ x[t]
            out[t] += probs[t, j] * (w2[e] @ (gu[:F] * torch.sigmoid(gu[:F]) * gu[F:]))
    return out
