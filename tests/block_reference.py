"""Layer norm, the shared expert's block and AdamW in 64 bits from their formulas, with bounds of what rounding may do.

A rounding to a type moves a value by at most half a step, r = finfo.eps / 2 of it (bf16 2^-8, fp32 2^-24).  A sum of K
fp32 products is off by at most (K + 2) 2^-24 of the sum of their magnitudes.  The bounds carry these through each operator to
first order; SECOND covers the products of two errors, which are smaller than a hundredth of the first order here.
"""
import torch

D = torch.float64
E32 = 2.0 ** -24
SECOND = 1.01


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, bound, what):
    got = got.to(D)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - SECOND * bound - 1e-30
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError("%s: %d of %d out of bounds, worst at %d: %r for %r, bound %r" % (
            what, int((over > 0).sum()), over.numel(), i, got.reshape(-1)[i].item(), ref.reshape(-1)[i].item(),
            bound.expand_as(ref).reshape(-1)[i].item()))


def layer_norm(x, w, b, eps, dy=None, residual=None):
    """{name: (value, bound)} of y (and dx, dweight, dbias)."""
    r, pr = half_step(x.dtype), half_step(w.dtype)
    x, w, b = x.to(D), w.to(D), b.to(D)
    T, d = x.shape
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    n = (x - mean) * rstd
    # a sum of d terms runs over at most 64 terms in a thread and 10 in the tree above: 80 roundings with the division;
    # the mean is off by that share of mean |x|, n by that (and as much again through rstd, relative), and some steps
    e_mean = 80 * E32 * x.abs().mean(1, keepdim=True)
    e_n = e_mean * rstd + n.abs() * (80 * E32 + 8 * E32) + 2 * E32 * (x.abs() + mean.abs()) * rstd
    y = n * w + b
    out = {"y": (y, e_n * w.abs() + 2 * E32 * (n * w).abs() + E32 * b.abs() + r * y.abs())}
    if dy is None:
        return out
    dy = dy.to(D)
    a = dy * w
    ma, mn = a.mean(1, keepdim=True), (a * n).mean(1, keepdim=True)
    dx = rstd * (a - ma - n * mn)
    e_ma = 80 * E32 * a.abs().mean(1, keepdim=True)
    e_mn = 80 * E32 * (a * n).abs().mean(1, keepdim=True) + (a.abs() * e_n).mean(1, keepdim=True)
    e = rstd * (4 * E32 * a.abs() + e_ma + e_n * mn.abs() + n.abs() * e_mn + 4 * E32 * (ma.abs() + (n * mn).abs()))
    e = e + 90 * E32 * dx.abs()
    if residual is not None:
        dx = dx + residual.to(D)
        e = e + E32 * dx.abs()
    out["dx"] = (dx, e + r * dx.abs())
    k = T + 2  # at most T additions, in whichever groups
    dw, db = (dy * n).sum(0), dy.sum(0)
    out["dweight"] = (dw, (dy.abs() * e_n).sum(0) + k * E32 * (dy * n).abs().sum(0) + pr * dw.abs())
    out["dbias"] = (db, k * E32 * dy.abs().sum(0) + pr * db.abs())
    return out


def shared_ffn(x, w_gate_up, w_down, residual=None, dy=None):
    """{name: (value, bound)}: y (with the residual unless dy is given), and with dy: dx (with it), dw_gate_up, dw_down."""
    r = half_step(x.dtype)
    f = w_down.shape[1]
    T, d = x.shape
    x, wd = x.to(D), w_down.to(D)
    W = w_gate_up.to(D)
    gu, e_gu = x @ W.T, (d + 2) * E32 * (x.abs() @ W.abs().T)
    g, u = gu[:, :f], gu[:, f:]
    sig = torch.sigmoid(g)
    s, ds = g * sig, sig * (1 + g * (1 - sig))
    # |silu'| <= 1.1, |silu''| <= 0.5; exp of an argument off by 2^-24 of it, a reciprocal and four products: 2^-20 in all
    # for |g| up to 16 or so, which sigmoid's own slope damps
    h = s * u
    e_s = 1.1 * e_gu[:, :f] + 2.0 ** -20 * s.abs()
    e_h = e_s * u.abs() + s.abs() * e_gu[:, f:] + (r + 2 * E32) * h.abs()
    y = h @ wd.T
    e_y = e_h @ wd.abs().T + (f + 2) * E32 * (h.abs() @ wd.abs().T)
    out = {}
    if dy is None and residual is not None:
        y = y + residual.to(D)
        e_y = e_y + E32 * y.abs()
    out["y"] = (y, e_y + r * y.abs())
    if dy is None:
        return out
    dy = dy.to(D)
    dh, e_dh = dy @ wd, (d + 2) * E32 * (dy.abs() @ wd.abs())
    e_g, e_u = e_gu[:, :f], e_gu[:, f:]  # kept in fp32
    du, dg = dh * s, dh * u * ds
    e_du = e_dh * s.abs() + dh.abs() * 1.1 * e_g + (2.0 ** -20 + r) * du.abs()
    e_dg = e_dh * (u * ds).abs() + (dh * ds).abs() * e_u + (dh * u).abs() * (0.5 * e_g + 2.0 ** -20) + r * dg.abs()
    dgu, e_dgu = torch.cat([dg, du], 1), torch.cat([e_dg, e_du], 1)
    dx = dgu @ W
    e_dx = e_dgu @ W.abs() + (2 * f + 2) * E32 * (dgu.abs() @ W.abs())
    if residual is not None:
        dx = dx + residual.to(D)
        e_dx = e_dx + E32 * dx.abs()
    out["dx"] = (dx, e_dx + r * dx.abs())
    dw = dgu.T @ x
    out["dw_gate_up"] = (dw, e_dgu.T @ x.abs() + (T + 2) * E32 * (dgu.abs().T @ x.abs()) + r * dw.abs())
    dw = dy.T @ h
    out["dw_down"] = (dw, dy.abs().T @ e_h + (T + 2) * E32 * (dy.abs().T @ h.abs()) + r * dw.abs())
    return out


BLOCK = 32


def power(n):
    """2^n in 64 bits, exactly (a power function need not be exact)."""
    return (n.long() + 1023 << 52).view(D)


def m_values(codes, scale):
    n = codes.numel()
    s = power(scale.long() - 127).repeat_interleave(BLOCK)[:n]
    return codes.view(torch.float8_e4m3fn).to(D) * s


def root_values(codes, scale):
    n, c = codes.numel(), codes.long()
    v = (1 + (c % 16).to(D) / 16) * power(c // 16 - 15)
    v = torch.where(c == 0, 0.0, torch.where(c == 255, float("nan"), v))
    return v * power(scale.long() - 127).repeat_interleave(BLOCK)[:n]


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, scale=1.0):
    """(value, bound) of p (before its rounding to its type), m and v from fp64 inputs."""
    g = g * scale
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    e_m = 4 * E32 * ((beta1 * m).abs() + ((1 - beta1) * g).abs())
    e_v = 6 * E32 * v1
    c1, c2 = 1 - beta1 ** step, 1 - beta2 ** step
    den = (v1 / c2).sqrt() + eps
    up = lr / c1 * m1 / den
    p1 = p - lr * decay * p - up
    # the update: m's error, the root's and the reciprocal's (1 ulp = 2 E32 each), half of v's, seven roundings
    e_p = lr / c1 * e_m / den + (2 + 2 + 3 + 7) * E32 * up.abs() + 4 * E32 * (lr * decay * p).abs() + 2 * E32 * (p.abs() + p1.abs())
    return (p1, e_p), (m1, e_m), (v1, e_v)
