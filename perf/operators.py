"""The operators around the routed experts of a mixture-of-experts block, as cases to measure: layer norm (forward and
backward), the shared expert's gated feed-forward block (forward and backward), and AdamW over many tensors at once.

Where ``own`` is false, ``run`` computes an operator from elementary torch operations in 32 bits, rounded once at the
end; where it is true, it calls the framework.  ``exact`` gives the same results in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32  # elements that share a scale of the 8-bit optimizer states
BETA1, BETA2, EPS, NORM_EPS = 0.9, 0.95, 1e-8, 1e-5
LR, DECAY, STEP = 2e-5, 0.1, 1000  # a fine-tuning run's rate, in the middle of it


# ---- cases -------------------------------------------------------------------------------------------------------

def norm(rows, d, dtype, train, residual=False, params="f32", pad=0, **kw):
    """pad: elements between the rows of x (a slice of a wider buffer)."""
    return dict(op="norm", rows=rows, d=d, dtype=dtype, train=train, residual=residual, params=params, pad=pad, **kw)


def ffn(tokens, d, f, dtype, train, residual=False, **kw):
    return dict(op="ffn", tokens=tokens, d=d, f=f, dtype=dtype, train=train, residual=residual, **kw)


def adamw(experts, d, f, small, bits, params, grads, **kw):
    """The weights of `experts` local experts, a router's and a norm's, and `small` tensors of odd sizes.  params: "master"
    (fp32, with the bf16 copy that the layer reads), "f32" or "bf16"."""
    return dict(op="adamw", experts=experts, d=d, f=f, small=small, bits=bits, params=params, grads=grads, **kw)


def listed():
    return [
        # one new token's row before the router: latency alone
        norm(1, 7168, "bf16", False, name="norm, one token"),
        # the pre-norm of a training step on the DeepSeek-V3-shaped rank's 8 x 2048 tokens, with the residual's gradient
        norm(16384, 7168, "bf16", True, residual=True, name="norm, training"),
        # single precision, a width that no vector load divides, rows of a wider buffer
        norm(1021, 1407, "f32", True, pad=9, name="norm, odd width, f32"),
        # decoding one token: the weights stream past once
        ffn(1, 7168, 2048, "bf16", False, name="ffn, one token"),
        # a decode batch through Mixtral-shaped weights, added to the routed experts' output
        ffn(24, 4096, 14336, "bf16", False, residual=True, name="ffn, decode batch"),
        # an odd prompt through the skewed workload's widths
        ffn(777, 2048, 1408, "bf16", False, residual=True, name="ffn, prompt"),
        # a training step of one rank with few tokens
        ffn(2048, 2048, 1408, "bf16", True, name="ffn, training, small"),
        # a training step on the DeepSeek-V3-shaped rank's 8 x 2048 tokens
        ffn(16384, 7168, 2048, "bf16", True, residual=True, name="ffn, training"),
        # single precision and sizes that nothing divides
        ffn(301, 333, 517, "f32", True, residual=True, name="ffn, odd sizes, f32"),
        # a tiny layer and a tail of odd tensors: latency alone
        adamw(1, 64, 128, 40, 32, "f32", "f32", name="adamw, small tensors"),
        # the skewed workload's 16 local experts: fp32 master weights and gradients, and the bf16 copy
        adamw(16, 2048, 1408, 4, 32, "master", "f32", name="adamw, 32-bit states"),
        # the same with the states in 8 bits
        adamw(16, 2048, 1408, 4, 8, "master", "f32", name="adamw, 8-bit states"),
    ]


def between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def width(rng, lo, hi):
    """A width: mostly whole 64s, some whole 8s, some that nothing divides."""
    step = rng.choice([64, 64, 64, 8, 1])
    return max(lo, between(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["norm", "ffn", "ffn", "adamw"])
    if op == "norm":
        d = width(rng, 64, 16384)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = between(rng, 1, max(1, min(65536, 16384 * 7168 // d // (1 if dtype == "bf16" else 2))))
        return norm(rows, d, dtype, rng.random() < 0.6, rng.random() < 0.5, rng.choice(["f32", dtype]),
                    rng.choice([0, 0, 64, 3]))
    if op == "ffn":
        d, f = width(rng, 64, 7168), width(rng, 64, 14336)
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        train = rng.random() < 0.5
        most = 16384 * 7168 * 2048 // (d * f) // (1 if dtype == "bf16" else 16)
        return ffn(between(rng, 1, max(1, min(16384, most))), d, f, dtype, train, rng.random() < 0.5)
    d, f = width(rng, 64, 4096), width(rng, 64, 4096)
    experts = between(rng, 1, max(1, min(32, 16 * 2048 * 1408 // (d * f))))
    return adamw(experts, d, f, rng.randint(0, 64), rng.choice([8, 32]), rng.choice(["master", "f32", "bf16"]),
                 rng.choice(["f32", "bf16"]))


def work(case):
    c = case
    if c["op"] == "norm":
        s = 2 if c["dtype"] == "bf16" else 4
        ps = 2 if c["params"] == "bf16" else 4
        n = c["rows"] * c["d"]
        nbytes = 2 * n * s + 2 * c["d"] * ps + 8 * c["rows"]
        if c["train"]:
            nbytes += (3 + c["residual"]) * n * s + 3 * c["d"] * ps
        return {"bytes": nbytes, "flops": n * (22 if c["train"] else 8)}
    if c["op"] == "ffn":
        s = 2 if c["dtype"] == "bf16" else 4
        td, df = c["tokens"] * c["d"], c["d"] * c["f"]
        nbytes = (2 + c["residual"]) * td * s + 3 * df * s
        if c["train"]:
            nbytes += 2 * td * s + 3 * df * s  # dy, dx, the weights' gradients
        return {"bytes": nbytes, "flops": (18 if c["train"] else 6) * c["tokens"] * df}
    n = sum(k for k, _ in sizes(c))
    p = {"master": 10, "f32": 8, "bf16": 4}[c["params"]]
    g = 4 if c["grads"] == "f32" else 2
    # 8-bit states: codes and scales read and written, and their values given back
    states = 16 if c["bits"] == 32 else 4 + 4 / BLOCK + 4
    return {"bytes": n * (p + g + states), "flops": n * 16}


# ---- inputs ------------------------------------------------------------------------------------------------------

def sizes(c):
    """(elements, whether weight decay acts on it) of each tensor: matrices decay, vectors do not."""
    e, d, f = c["experts"], c["d"], c["f"]
    got = [(e * 2 * f * d, True), (e * d * f, True), (4 * e * d, True), (d, False), (d, False)]
    return got + [(1 + (k * k * 37) % 2999, False) for k in range(c["small"])]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    if c["op"] == "norm":
        T, d, dt, pt = c["rows"], c["d"], DTYPES[c["dtype"]], DTYPES[c["params"]]
        # a residual stream: every channel with its own offset and size, some far larger than the others
        x = randn(T, d) * torch.exp(0.5 * randn(d)) + 0.3 * randn(d)
        x[:, :: 97] *= 20.0
        wide = torch.zeros(T, d + c["pad"], device="cuda", dtype=dt)
        wide[:, :d] = x
        s = {"case": c, "x": wide[:, :d], "w": (1 + 0.2 * randn(d)).to(pt), "b": (0.1 * randn(d)).to(pt)}
        if c["train"]:
            s["dy"] = randn(T, d).to(dt)
            s["residual"] = randn(T, d).to(dt) if c["residual"] else None
        if own:
            from expert_output_overlap_amd.runtime import LayerNorm

            s["op"] = LayerNorm(T, d, dtype=c["dtype"], param_dtype=c["params"], eps=NORM_EPS, train=c["train"])
        return s
    if c["op"] == "ffn":
        T, d, f, dt = c["tokens"], c["d"], c["f"], DTYPES[c["dtype"]]
        s = {"case": c, "x": randn(T, d).to(dt), "w_gate_up": (randn(2 * f, d) / math.sqrt(d)).to(dt),
             "w_down": (randn(d, f) / math.sqrt(d)).to(dt), "residual": randn(T, d).to(dt) if c["residual"] else None}
        if c["train"]:
            s["dy"] = randn(T, d).to(dt)
        if own:
            from expert_output_overlap_amd.runtime import SharedFFN

            s["op"] = SharedFFN(T, d, f, dtype=c["dtype"], train=c["train"])
        return s
    # flat buffers, as a trainer holds them: matrices in one, vectors in the other, each tensor at a multiple of 32
    # elements, zeros between them
    s = {"case": c, "groups": [], "clip": 0.3 + 0.7 * torch.rand(1, generator=gen, device="cuda")}  # clip: of the norm
    scale = 1.0 / math.sqrt(c["d"])
    for decayed in (True, False):
        spans, n = [], 0
        for k, w in sizes(c):
            if w == decayed:
                spans.append((n, k))
                n += -(-k // BLOCK) * BLOCK
        used = torch.zeros(n, device="cuda")
        for at, k in spans:
            used[at: at + k] = 1
        p = (scale * randn(n) if decayed else 1 + 0.1 * randn(n)) * used
        size = 1e-3 * torch.exp(randn(n // BLOCK)).repeat_interleave(BLOCK) * used  # gradients of very different sizes
        g = randn(n) * size
        m = 0.3 * randn(n) * size
        v = (size * (0.5 + torch.rand(n, generator=gen, device="cuda"))) ** 2
        q = {"spans": spans, "decay": DECAY if decayed else 0.0, "g": g.to(DTYPES[c["grads"]]),
             "p": p.to(torch.bfloat16 if c["params"] == "bf16" else torch.float32),
             "copy": p.to(torch.bfloat16) if c["params"] == "master" else None}
        if c["bits"] == 32:
            q["m"], q["v"] = m, v
        else:
            q["m"], q["m_scale"] = pack_m(m)
            q["v"], q["v_scale"] = pack_root(torch.sqrt(v))
            q["m_values"], q["root_values"] = (torch.empty(n, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        s["groups"].append(q)
    if own:
        from expert_output_overlap_amd.runtime import AdamW

        tensors = []
        for q in s["groups"]:
            for at, k in q["spans"]:
                t = {name: q[name][at: at + k] for name in ("p", "g", "m", "v")}
                if q["copy"] is not None:
                    t["copy"] = q["copy"][at: at + k]
                if c["bits"] == 8:
                    b = slice(at // BLOCK, at // BLOCK + -(-k // BLOCK))
                    t["m_scale"], t["v_scale"] = q["m_scale"][b], q["v_scale"][b]
                    t["m_values"], t["root_values"] = (q[name][at: at + k] for name in ("m_values", "root_values"))
                t["weight_decay"] = q["decay"]
                tensors.append(t)
        s["op"] = AdamW(tensors, betas=(BETA1, BETA2), eps=EPS)
        for q in s["groups"]:  # the gaps between the tensors hold no values
            if c["bits"] == 8:
                q["m_values"].zero_()
                q["root_values"].zero_()
    return s


# ---- the operators -----------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return run_norm(state) if op == "norm" else run_ffn(state) if op == "ffn" else run_adamw(state)


def run_norm(s):
    x, w, b = s["x"], s["w"], s["b"]
    if own:
        op = s["op"]
        y = op.forward(x, w, b)
        if not s["case"]["train"]:
            return y
        dx = op.backward(s["dy"], x, w, residual=s["residual"])
        return y, dx, op.dweight, op.dbias
    dt, pt, xf, wf = x.dtype, w.dtype, x.float(), w.float()
    mean = xf.mean(1, keepdim=True)
    xc = xf - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + NORM_EPS)
    xh = xc * rstd
    y = (xh * wf + b.float()).to(dt)
    if not s["case"]["train"]:
        return y
    dy = s["dy"].float()
    a = dy * wf
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return y, dx.to(dt), (dy * xh).sum(0).to(pt), dy.sum(0).to(pt)


def run_ffn(s):
    x, wgu, wd, res = s["x"], s["w_gate_up"], s["w_down"], s["residual"]
    train = s["case"]["train"]
    if own:
        op = s["op"]
        if not train:
            return op.forward(x, wgu, wd, residual=res)
        y = op.forward(x, wgu, wd)
        dx = op.backward(s["dy"], x, wgu, wd, residual=res)
        return y, dx, op.dw_gate_up, op.dw_down
    dt, f = x.dtype, wd.shape[1]
    xf, wguf, wdf = x.float(), wgu.float(), wd.float()
    gu = xf @ wguf.T
    g, u = gu[:, :f], gu[:, f:]
    sig = torch.sigmoid(g)
    h = g * sig * u
    y = h @ wdf.T
    if not train:
        return (y if res is None else y + res.float()).to(dt)
    dy = s["dy"].float()
    dh = dy @ wdf
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1)
    dx = dgu @ wguf
    if res is not None:
        dx = dx + res.float()
    return y.to(dt), dx.to(dt), (dgu.T @ xf).to(dt), (dy.T @ h).to(dt)


def run_adamw(s):
    if own:
        s["op"].step(STEP, lr=LR, grad_scale=s["clip"])
        if s["case"]["bits"] == 8:
            s["op"].read_states()
    else:
        adamw_plain(s["groups"][0], s["clip"])
        adamw_plain(s["groups"][1], s["clip"])
    return [given(s["groups"][0]), given(s["groups"][1])]


def given(q):
    """What the step leaves: the parameters, their copy, and the states (in 8 bits: their values, which bf16 holds exactly:
    4 and 5 significant bits times a power of two)."""
    got = {"p": q["p"], "m": q.get("m_values", q["m"]), "v": q.get("root_values", q["v"])}
    return got if q["copy"] is None else {**got, "copy": q["copy"]}


def adamw_plain(q, clip):
    p, g, small = q["p"].float(), q["g"].float() * clip, "m_scale" in q
    m = unpack_m(q["m"], q["m_scale"]) if small else q["m"]
    v = unpack_root(q["v"], q["v_scale"]).square() if small else q["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = torch.sqrt(v)
    update = m / (root * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS)
    p = p * (1 - LR * q["decay"]) - update * (LR / (1 - BETA1 ** STEP))
    q["p"].copy_(p)
    if q["copy"] is not None:
        q["copy"].copy_(p)
    if small:
        codes, scale = pack_m(m)
        q["m"].copy_(codes)
        q["m_scale"].copy_(scale)
        codes, scale = pack_root(root)
        q["v"].copy_(codes)
        q["v_scale"].copy_(scale)
        q["m_values"].copy_(unpack_m(q["m"], q["m_scale"]))
        q["root_values"].copy_(unpack_root(q["v"], q["v_scale"]))
    else:
        q["m"].copy_(m)
        q["v"].copy_(v)


# The 8-bit states.  m: e4m3 codes times 2^(b - 127), with b (one byte for 32 elements) the smallest exponent at which
# the block's largest |m| is at most 448.  The second moment's root: an unsigned float with 4 exponent and 4 mantissa
# bits, times 2^(b - 127): code 16 e + k stands for (1 + k / 16) 2^(e - 15), 0 for 0, 255 for no finite value, and
# a positive value is never below code 1, so no step divides by a root that rounding made zero; b is the smallest
# exponent at which the block's largest root is at most 1.875.

def power(n):
    """2^n as fp32, exactly, for -127 < n < 128."""
    return (n.int() + 127 << 23).view(torch.float32)


def exponent(top, over, lead):
    """(Biased exponent of `top`) - lead, one more where its significand is over `over`, at least 1."""
    mant, e = torch.frexp(top)  # top = mant 2^e, mant in [0.5, 1)
    b = e + 126 - lead + (2 * mant > over).int()
    return torch.where(top > 0, b, 1).clamp_(min=1)


def pack_m(m):
    blocks = m.view(-1, BLOCK)
    b = exponent(blocks.abs().amax(1), 1.75, 8)
    codes = (blocks * power(127 - b)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(-1), b.to(torch.uint8)


def unpack_m(codes, b):
    return (codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * power(b.int() - 127)[:, None]).view(-1)


def pack_root(r):
    blocks = r.view(-1, BLOCK)
    b = exponent(blocks.amax(1), 1.875, 0).clamp_(min=16)
    mant, e = torch.frexp(blocks * power(127 - b)[:, None])
    code = (torch.round(mant * 32) - 16 + 16 * (e + 14)).clamp_(min=1).to(torch.uint8)  # round: ties to even
    return torch.where(blocks > 0, code, 0).view(-1), b.to(torch.uint8)


def unpack_root(codes, b):
    c = codes.int().view(-1, BLOCK)
    value = (1 + (c & 15).float() / 16) * power((c >> 4) - 15 + (b.int() - 127)[:, None])
    return torch.where(c > 0, value, 0.0).view(-1)


# ---- in 64 bits --------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        x, w, b = s["x"].to(D), s["w"].to(D), s["b"].to(D)
        d = x.shape[1]
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        inv = 1 / (var + NORM_EPS).sqrt()
        y = (x - mean) * inv * w + b
        if not case["train"]:
            return y
        dy = s["dy"].to(D)
        # the derivative through x, through the mean and through the variance
        dxh = dy * w
        dvar = (dxh * (x - mean)).sum(1, keepdim=True) * -0.5 * inv ** 3
        dmean = -inv * dxh.sum(1, keepdim=True)
        dx = dxh * inv + dvar * 2 * (x - mean) / d + dmean / d
        if s["residual"] is not None:
            dx += s["residual"].to(D)
        return y, dx, (dy * (x - mean) * inv).sum(0), dy.sum(0)
    if case["op"] == "ffn":
        x, wd = s["x"].to(D), s["w_down"].to(D)
        wg, wu = s["w_gate_up"].to(D).chunk(2)
        g, u = x.mm(wg.t()), x.mm(wu.t())
        e = torch.exp(-g)
        silu = g / (1 + e)
        h = silu * u
        y = h.mm(wd.t())
        if not case["train"]:
            return y if s["residual"] is None else y + s["residual"].to(D)
        dy = s["dy"].to(D)
        dh = dy.mm(wd)
        dg = dh * u * (1 + e + g * e) / (1 + e) ** 2
        du = dh * silu
        dx = dg.mm(wg) + du.mm(wu)
        if s["residual"] is not None:
            dx += s["residual"].to(D)
        return y, dx, torch.cat([dg.t().mm(x), du.t().mm(x)]), dy.t().mm(h)
    return [exact_adamw(q, s["clip"], case["bits"] == 8) for q in s["groups"]]


def exact_adamw(q, clip, small):
    D = torch.float64
    g, p = q["g"].to(D) * clip.to(D), q["p"].to(D)
    if small:
        scale_m, scale_v = ((2.0 ** (q[k].to(D) - 127)).repeat_interleave(BLOCK) for k in ("m_scale", "v_scale"))
        m = q["m"].view(torch.float8_e4m3fn).to(D) * scale_m
        c = q["v"].long()
        root = torch.where(c > 0, (16 + c % 16).to(D) * 2.0 ** ((c // 16).to(D) - 19), 0.0) * scale_v
        v = root * root
    else:
        m, v = q["m"].to(D), q["v"].to(D)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    m_hat, v_hat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    p = p - LR * q["decay"] * p - LR * m_hat / (v_hat.sqrt() + EPS)
    if small:
        m, v = on_grid(m, 8, 3, 448.0, -6), on_grid(v.sqrt(), 0, 4, 1.875, -15)
    got = {"p": p, "m": m, "v": v}
    return got if q["copy"] is None else {**got, "copy": p}


def on_grid(x, top, bits, most, low):
    """x on the grid of its block's 8-bit floats: `bits` mantissa bits, the block's scale the smallest power of two at which
    its largest magnitude is at most `most`, the lowest binade at 2^low (e4m3: steps stay the same below it; the
    root's format: a positive value is at least its code 1)."""
    blocks = x.view(-1, BLOCK)
    peak = blocks.abs().amax(1, keepdim=True)
    live = peak > 0
    scale = 2.0 ** torch.ceil(torch.log2(torch.where(live, peak, 1.0) / most))
    z = blocks / scale
    mag = z.abs().clamp(min=1e-300)
    step = 2.0 ** (torch.floor(torch.log2(mag)).clamp(min=low) - bits)
    z = torch.round(z / step) * step
    if top == 0:
        z = torch.where(blocks > 0, z.clamp(min=2.0 ** low * (1 + 2.0 ** -bits)), z)
    return torch.where(live, z * scale, 0.0).view(-1)
