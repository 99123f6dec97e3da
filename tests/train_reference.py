"""The norms around a block, the router's losses and the gradient norm in 64 bits from their formulas, with bounds of what
rounding may do.

As in block_reference: a rounding moves a value by at most half a step r (fp32: E32), and the bounds carry these through each
operator to first order.  A sum over a row runs over at most 64 terms in a thread and 10 in the tree above: 80 roundings with
the division by the row's length.
"""
import torch

from block_reference import D, E32, half_step

ROW = 80 * E32


def norm(v, e_v, kind, eps):
    """(v^, its error, rstd, rstd's relative error) of the rows v known to e_v."""
    if kind == "none":
        return v, e_v, torch.ones_like(v[:, :1]), torch.zeros_like(v[:, :1])
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    rstd = ((v - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    n = (v - mean) * rstd
    e_mean = (ROW * v.abs() + e_v).mean(1, keepdim=True) if kind == "layer" else 0.0
    # d rstd / rstd = -mean(n dv) rstd: the rows' own errors, and the sum's, the division's and the root's roundings
    e_r = ROW + 8 * E32 + rstd * (n.abs() * (e_v + e_mean)).mean(1, keepdim=True)
    e_n = rstd * (e_v + e_mean + 2 * E32 * (v.abs() + mean.abs())) + n.abs() * e_r
    return n, e_n, rstd, e_r


def norm_back(a, e_a, n, e_n, rstd, e_r, kind):
    """The gradient of v from that of v^."""
    if kind == "none":
        return a, e_a
    mn = (a * n).mean(1, keepdim=True)
    e_mn = (ROW * (a * n).abs() + a.abs() * e_n + n.abs() * e_a).mean(1, keepdim=True)
    core, e = a - n * mn, e_a + e_n * mn.abs() + n.abs() * e_mn + 4 * E32 * (a.abs() + (n * mn).abs())
    if kind == "layer":
        ma = a.mean(1, keepdim=True)
        core, e = core - ma, e + (ROW * a.abs() + e_a).mean(1, keepdim=True) + 4 * E32 * ma.abs()
    return rstd * core, rstd * e + (rstd * core).abs() * (e_r + 2 * E32)


def residual_norm(x, h, w, post, pre, rho, eps, row_gate=None, ds=None, dn=None):
    """{name: (value, bound)} of s, n (and dx, dh and the gradients of the parameters in w and of row_gate).  w: by name."""
    r = half_step(x.dtype)
    T, d = x.shape
    x, h = x.to(D), h.to(D)
    pr = {k: half_step(t.dtype) for k, t in w.items()}
    w = {k: t.to(D) for k, t in w.items()}
    one, zero = torch.ones(d, dtype=D, device=x.device), torch.zeros(d, dtype=D, device=x.device)
    w1, b1, g = w.get("post_weight", one), w.get("post_bias", zero), w.get("gate", one)
    w2, b2 = w.get("pre_weight", one), w.get("pre_bias", zero)
    c = torch.ones(T, 1, dtype=D, device=x.device) if row_gate is None else row_gate.to(D)[:, None]
    n1, e_n1, r1, e_r1 = norm(h, torch.zeros_like(h), post, eps)
    z, parts = n1 * w1 + b1, (n1 * w1).abs() + b1.abs()
    e_z = e_n1 * w1.abs() + 2 * E32 * parts
    s = rho * x + c * g * z
    # products with gate and c, in whichever order, and the sum
    e_s = (c * g).abs() * (e_z + 4 * E32 * parts) + 2 * E32 * ((rho * x).abs() + s.abs())
    out = {"s": (s, e_s + r * s.abs())}
    n2, e_n2, r2, e_r2 = norm(s, e_s, pre, eps)
    if pre != "none":
        n = n2 * w2 + b2
        out["n"] = (n, e_n2 * w2.abs() + 2 * E32 * (n2 * w2).abs() + E32 * b2.abs() + r * n.abs())
    if ds is None and dn is None:
        return out
    k = (T + 12) * E32  # at most T additions, in whichever groups
    total, e_t = (torch.zeros_like(x) if ds is None else ds.to(D)), torch.zeros_like(x)

    def param(name, value, bound):
        if name in w:
            out[name] = (value, bound + pr[name] * value.abs())

    if pre != "none":
        dn = dn.to(D)
        a = dn * w2
        back, e_b = norm_back(a, E32 * a.abs(), n2, e_n2, r2, e_r2, pre)
        total, e_t = total + back, e_b
        param("pre_weight", (dn * n2).sum(0), (k * (dn * n2).abs() + dn.abs() * e_n2).sum(0))
        param("pre_bias", dn.sum(0), k * dn.abs().sum(0))
    e_t = e_t + E32 * total.abs()
    out["dx"] = (rho * total, abs(rho) * (e_t + E32 * total.abs()) + r * (rho * total).abs())
    a = c * g * w1 * total
    e_a = (c * g * w1).abs() * (e_t + 4 * E32 * total.abs())
    dh, e_h = norm_back(a, e_a, n1, e_n1, r1, e_r1, post)
    out["dh"] = (dh, e_h + r * dh.abs())
    u1, u0 = (c * total * n1).sum(0), (c * total).sum(0)
    e_u1 = (k * (c * total * n1).abs() + c.abs() * (e_t * n1.abs() + total.abs() * e_n1)).sum(0)
    e_u0 = (k * (c * total).abs() + c.abs() * e_t).sum(0)
    param("post_weight", g * u1, g.abs() * (e_u1 + 2 * E32 * u1.abs()))
    param("post_bias", g * u0, g.abs() * (e_u0 + 2 * E32 * u0.abs()))
    param("gate", w1 * u1 + b1 * u0, w1.abs() * (e_u1 + 2 * E32 * u1.abs()) + b1.abs() * (e_u0 + 2 * E32 * u0.abs()))
    if row_gate is not None:
        each = total * g * z
        # z with the gate in whichever order: 4 roundings of its parts
        e = e_t * (g * z).abs() + (total * g).abs() * (e_z + 4 * E32 * parts) + (ROW + E32) * each.abs()
        out["row_gate"] = (each.sum(1), e.sum(1) + E32 * each.sum(1).abs())
    return out


def rows_of(spans, T, sequences):
    """[(first, last)] of the sequences."""
    if spans is None:
        return [(s * (T // sequences), (s + 1) * (T // sequences)) for s in range(sequences)]
    out = []
    for first, last in spans.tolist():
        first = min(max(first, 0), T)
        out.append((first, min(max(last, first), T)))
    return out


def router_loss(logits, idx, sequences, balance, z, spans=None, d_weights=None, d_loss=1.0, dtype=torch.float32):
    """{name: (value, bound)} of losses {loss, B, Z} and dlogits, and the counts.  All logits but those of -inf are finite."""
    T, G = logits.shape
    l, idx = logits.to(D), idx.long()
    gone = torch.isinf(l).all(1)
    top = l.amax(1, keepdim=True).nan_to_num(neginf=0.0)
    e = torch.exp(l - top)
    den = e.sum(1, keepdim=True)
    p = torch.where(gone[:, None], 0.0, e / den)
    # exp(x) as 2^(x log2 e): x is a rounded difference, its product is rounded, log2 e in fp32 is off by 0.22 E32 of it, together
    # 2.25 E32 |x| of the result; the power itself within 2 steps of 2 E32 each; sums of at most 16 + 6 terms
    rel = torch.where(torch.isinf(l), 0.0, E32 * (2.25 * (l - top).abs() + 6))
    rel_den = (p * rel).sum(1, keepdim=True) + 24 * E32
    rel_p = rel + rel_den + 2 * E32
    lse = torch.where(gone[:, None], 0.0, top + torch.log(den))
    e_lse = rel_den + 4 * E32 * (top.abs() + lse.abs() + torch.log(den).nan_to_num(neginf=0.0).abs())
    spans = rows_of(spans, T, sequences)
    live = [(a, b) for a, b in spans if b > a]
    N, S = max(1, sum(b - a for a, b in live)), max(1, len(live))
    counts = torch.zeros(len(spans), G, dtype=torch.int32, device=l.device)
    grad, e_grad = torch.zeros_like(l), torch.zeros_like(l)
    B = e_B = Z = e_Z = torch.zeros((), dtype=D, device=l.device)
    for q, (a, b) in enumerate(spans):
        if b <= a:
            continue
        i = idx[a:b]
        good = (i >= 0) & (i < G)
        counts[q] = torch.bincount(i[good], minlength=G).to(torch.int32)
        f = counts[q].to(D) * (G / max(1, int(counts[q].sum())))
        P, rp = p[a:b], rel_p[a:b]
        B, e_B = B + (P @ f).sum() / (b - a) / S, e_B + ((P * (rp + 30 * E32)) @ f).sum() / (b - a) / S
        Z, e_Z = Z + lse[a:b].square().sum() / N, e_Z + (2 * lse[a:b].abs() * e_lse[a:b]).sum() / N
        share = d_loss * balance / (S * (b - a))
        v = (share * f).expand_as(P).clone()
        e_v = 8 * E32 * v.abs()
        if d_weights is not None:
            dw = torch.where(good, d_weights[a:b].to(D), 0.0)
            v.scatter_add_(1, i.clamp(0, G - 1), dw)
            many = e_v + 0.0
            many.scatter_add_(1, i.clamp(0, G - 1), idx.shape[1] * E32 * dw.abs())  # sums of slots with one expert
            e_v = many + E32 * v.abs()
        cz = d_loss * z * 2 / N
        dot, e_dot = (P * v).sum(1, keepdim=True), (P * (v.abs() * (rp + 24 * E32) + e_v)).sum(1, keepdim=True)
        inner = v - dot + cz * lse[a:b]
        e_in = e_v + e_dot + abs(cz) * e_lse[a:b] + 6 * E32 * (v.abs() + dot.abs() + (cz * lse[a:b]).abs())
        grad[a:b] = P * inner
        e_grad[a:b] = P * (e_in + inner.abs() * (rp + 2 * E32))
    losses = torch.stack([balance * B + z * Z, B, Z])
    e_losses = torch.stack([abs(balance) * e_B + abs(z) * e_Z, e_B, e_Z]) + 2 * E32 * losses.abs()
    return counts, {"losses": (losses, e_losses), "dlogits": (grad, e_grad + half_step(dtype) * grad.abs())}


def grad_norm(grads, max_norm, factor):
    """(norm, scale) of the gradients, each rounded once from 64 bits."""
    norm = factor * torch.stack([g.to(D).square().sum() for g in grads]).sum().sqrt() if grads else torch.zeros((), dtype=D)
    return norm, factor * (torch.ones_like(norm) if max_norm == float("inf") else (max_norm / (norm + 1e-6)).clamp(max=1.0))
