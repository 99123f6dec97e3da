"""The operators that complete a mixture-of-experts block's training step, as cases to measure: the norms after and before a
block with its gate and the residual's scale (forward and backward), the router's balance loss with per-expert counts and
the gradient of the logits, and the global gradient norm over many tensors with clipping.

Where ``own`` is false, ``run`` computes an operator from elementary torch operations in 32 bits, rounded once at the
end; where it is true, it calls the framework.  ``exact`` gives the same results in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NORM_EPS, CLIP_EPS = 1e-5, 1e-6
ALIGN = 32  # elements at whose multiples a flat buffer's tensors start


# ---- cases -------------------------------------------------------------------------------------------------------

def join(rows, d, dtype, train, post="rms", pre="rms", bias=False, gate=True, row_gate=False, rho=1.0, params="f32", pad=0,
         **kw):
    """post, pre: the norm of the block's output and that in front of the next block ("none", "layer", "rms"); rho: the
    residual's scale; pad: elements between the rows of x (a slice of a wider buffer)."""
    return dict(op="join", rows=rows, d=d, dtype=dtype, train=train, post=post, pre=pre, bias=bias, gate=gate,
                row_gate=row_gate, rho=rho, params=params, pad=pad, **kw)


def router(tokens, experts, k, train, sequences=1, padded=False, z=1e-3, weights=True, dtype="f32", **kw):
    """padded: sequences of lengths of their own with rows of no sequence between them; weights: the routing weights'
    gradient reaches the logits too; dtype: of the logits' gradient."""
    return dict(op="router", tokens=tokens, experts=experts, k=k, train=train, sequences=sequences, padded=padded, z=z,
                weights=weights, dtype=dtype, **kw)


def clip(experts, d, f, small, grads, out, **kw):
    """The gradients of `experts` local experts' weights, a router's and a norm's, and `small` tensors of odd sizes.  out:
    None (the norm and the coefficient alone, for an optimizer that takes it) or the type of the clipped gradients."""
    return dict(op="clip", experts=experts, d=d, f=f, small=small, grads=grads, out=out, **kw)


def listed():
    return [
        # one new token between two blocks: latency alone
        join(1, 7168, "bf16", False, name="join, one token"),
        # a decode batch through Mixtral-shaped blocks, a gate per token, layer norms
        join(24, 4096, "bf16", False, "layer", "layer", True, row_gate=True, rho=0.5, name="join, decode batch"),
        # a training step on the DeepSeek-V3-shaped rank's 8 x 2048 tokens
        join(16384, 7168, "bf16", True, name="join, training"),
        # single precision, a width that no vector load divides, rows of a wider buffer, everything that the operator has
        join(1021, 1407, "f32", True, "layer", "layer", True, row_gate=True, rho=0.7, pad=9, name="join, odd width, f32"),
        # the tiny layer's router: latency alone
        router(64, 8, 2, True, name="router, tiny"),
        # the Mixtral-shaped rank's 4 x 1024 tokens, one balance for all of them
        router(4096, 8, 2, True, name="router, 8 experts"),
        # the skewed workload's 4 x 2048 tokens, packed from many short sequences
        router(8192, 64, 6, True, sequences=200, padded=True, name="router, short sequences"),
        # a training step on the DeepSeek-V3-shaped rank's 8 x 2048 tokens, a balance for each padded sequence
        router(16384, 256, 8, True, sequences=8, padded=True, z=0.0, dtype="bf16", name="router, training"),
        # a tiny layer and a tail of odd tensors: latency alone
        clip(1, 64, 128, 40, "f32", None, name="clip, small tensors"),
        # the skewed workload's 16 local experts: the norm of bf16 gradients, for the optimizer's coefficient
        clip(16, 2048, 1408, 4, "bf16", None, name="clip, norm"),
        # the same with fp32 accumulators, clipped into bf16 gradients
        clip(16, 2048, 1408, 4, "f32", "bf16", name="clip, into bf16"),
    ]


def between(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def width(rng, lo, hi):
    """A width: mostly whole 64s, some whole 8s, some that nothing divides."""
    step = rng.choice([64, 64, 64, 8, 1])
    return max(lo, between(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["join", "join", "router", "clip"])
    if op == "join":
        d = width(rng, 64, 16384)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = between(rng, 1, max(1, min(65536, 16384 * 7168 // d // (1 if dtype == "bf16" else 2))))
        return join(rows, d, dtype, rng.random() < 0.6, rng.choice(["none", "layer", "rms", "rms"]),
                    rng.choice(["none", "layer", "rms", "rms"]), rng.random() < 0.5, rng.random() < 0.7,
                    rng.random() < 0.4, rng.choice([1.0, 1.0, 0.7]), rng.choice(["f32", dtype]), rng.choice([0, 0, 64, 3]))
    if op == "router":
        experts = rng.choice([8, 64, 128, 256, between(rng, 2, 1024)])
        tokens = between(rng, 1, min(65536, 65536 * 64 // experts))
        sequences = rng.choice([1, 1, between(rng, 1, max(1, min(1000, tokens // 4)))])
        return router(tokens, experts, rng.randint(1, min(experts, 16)), rng.random() < 0.8, sequences, rng.random() < 0.5,
                      rng.choice([0.0, 1e-3]), rng.random() < 0.7, rng.choice(["f32", "bf16"]))
    d, f = width(rng, 64, 4096), width(rng, 64, 4096)
    experts = between(rng, 1, max(1, min(32, 16 * 2048 * 1408 // (d * f))))
    return clip(experts, d, f, rng.randint(0, 64), rng.choice(["f32", "bf16"]), rng.choice([None, "f32", "bf16"]))


def params_of(c):
    """The parameters that a join has, by name."""
    names = []
    for where in ("post", "pre"):
        if c[where] != "none":
            names += [where + "_weight"] + ([where + "_bias"] if c["bias"] and c[where] == "layer" else [])
    return names + (["gate"] if c["gate"] else [])


def work(case):
    c = case
    if c["op"] == "join":
        s = 2 if c["dtype"] == "bf16" else 4
        ps = 2 if c["params"] == "bf16" else 4
        n, np = c["rows"] * c["d"], len(params_of(c)) * c["d"] * ps
        nbytes = (3 + (c["pre"] != "none")) * n * s + np + 4 * c["rows"] * c["row_gate"]
        if c["train"]:
            nbytes += (3 + (c["pre"] != "none")) * n * s + np + 4 * c["rows"] * c["row_gate"]
        return {"bytes": nbytes, "flops": n * (60 if c["train"] else 18)}
    if c["op"] == "router":
        n, ids = c["tokens"] * c["experts"], c["tokens"] * c["k"]
        nbytes = 4 * n + 4 * ids + 4 * c["sequences"] * c["experts"] + 12
        if c["train"]:
            nbytes += (2 if c["dtype"] == "bf16" else 4) * n + 4 * ids * c["weights"]
        return {"bytes": nbytes, "flops": n * (25 if c["train"] else 10)}
    n = sum(sizes(c))
    nbytes = n * ((2 if c["grads"] == "bf16" else 4) + {None: 0, "bf16": 2, "f32": 4}[c["out"]]) + 8
    return {"bytes": nbytes, "flops": n * (3 if c["out"] else 2)}


# ---- inputs ------------------------------------------------------------------------------------------------------

def sizes(c):
    """Elements of each gradient."""
    e, d, f = c["experts"], c["d"], c["f"]
    return [e * 2 * f * d, e * d * f, 4 * e * d, d, d] + [1 + (k * k * 37) % 2999 for k in range(c["small"])]


def spans_of(c, gen):
    """[sequences, 2] first and last rows: equal parts of the tokens, the padded ones between a quarter and all of a part."""
    T, S = c["tokens"], c["sequences"]
    edge = torch.arange(S + 1, device="cuda") * T // S
    first, part = edge[:-1], edge[1:] - edge[:-1]
    share = 0.25 + 0.75 * torch.rand(S, generator=gen, device="cuda") if c["padded"] else torch.ones(S, device="cuda")
    return torch.stack([first, first + torch.ceil(part * share).long().clamp(max=T)], 1).to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    if c["op"] == "join":
        T, d, dt, pt = c["rows"], c["d"], DTYPES[c["dtype"]], DTYPES[c["params"]]
        # a residual stream: every channel with its own offset and size, some far larger than the others
        x = randn(T, d) * torch.exp(0.5 * randn(d)) + 0.3 * randn(d)
        x[:, :: 97] *= 20.0
        wide = torch.zeros(T, d + c["pad"], device="cuda", dtype=dt)
        wide[:, :d] = x
        h = randn(T, d) * torch.exp(0.3 * randn(d)) * torch.exp(0.5 * randn(T, 1))  # a block's output, rows of any size
        w = {}
        for name in params_of(c):
            w[name] = ((0.1 * randn(d)) if name.endswith("bias") else 0.5 + 0.2 * randn(d) if name == "gate" else
                       1 + 0.2 * randn(d)).to(pt)
        s = {"case": c, "x": wide[:, :d], "h": h.to(dt), "w": w,
             "row_gate": torch.sigmoid(randn(T)) if c["row_gate"] else None}
        if c["train"]:
            s["ds"], s["dn"] = randn(T, d).to(dt), randn(T, d).to(dt) if c["pre"] != "none" else None
        if own:
            from expert_output_overlap_amd.runtime import ResidualNorm

            s["op"] = ResidualNorm(T, d, dtype=c["dtype"], param_dtype=c["params"], post=c["post"], pre=c["pre"],
                                   residual_scale=c["rho"], eps=NORM_EPS, train=c["train"])
        return s
    if c["op"] == "router":
        T, G, k = c["tokens"], c["experts"], c["k"]
        logits = randn(T, G) + 0.7 * randn(G)  # experts of their own popularity
        s = {"case": c, "logits": logits, "topk_idx": torch.topk(logits, k, 1).indices.to(torch.int32),
             "spans": spans_of(c, gen), "d_weights": 1e-2 * randn(T, k) if c["train"] and c["weights"] else None}
        if own:
            from expert_output_overlap_amd.runtime import RouterLoss

            s["op"] = RouterLoss(T, G, k, sequences=c["sequences"], balance=0.01, z=c["z"], dtype=c["dtype"])
        return s
    # flat buffers, as a trainer holds its gradients: each tensor at a multiple of 32 elements, zeros between them
    spans, n = [], 0
    for k in sizes(c):
        spans.append((n, k))
        n += -(-k // ALIGN) * ALIGN
    g = torch.zeros(n, device="cuda")
    for at, k in spans:  # gradients of very different sizes
        g[at: at + k] = 1e-3 * randn(k) * torch.exp(randn(1))
    g = g.to(DTYPES[c["grads"]])
    s = {"case": c, "g": g, "out": torch.zeros(n, device="cuda", dtype=DTYPES[c["out"]]) if c["out"] else None,
         "max_norm": 1.0 if n > 1 << 22 else 0.05, "factor": 0.25}  # the mean of four accumulated batches
    if own:
        from expert_output_overlap_amd.runtime import GradNorm

        s["op"] = GradNorm([{"g": g[at: at + k], **({"out": s["out"][at: at + k]} if c["out"] else {})} for at, k in spans])
    return s


# ---- the operators -----------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return run_join(state) if op == "join" else run_router(state) if op == "router" else run_clip(state)


def normed(v, kind):
    """(n, rstd) of the rows of v."""
    if kind == "none":
        return v, torch.ones_like(v[:, :1])
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + NORM_EPS)
    return v * rstd, rstd


def normed_back(a, n, rstd, kind):
    """The gradient of a norm's input from that of n."""
    if kind == "none":
        return a
    out = a - n * (a * n).mean(1, keepdim=True)
    return rstd * (out - a.mean(1, keepdim=True) if kind == "layer" else out)


def run_join(s):
    c, x, h, w = s["case"], s["x"], s["h"], s["w"]
    if own:
        op = s["op"]
        out, n = op.forward(x, h, w, row_gate=s["row_gate"])
        if not c["train"]:
            return [t for t in (out, n) if t is not None]
        dx, dh = op.backward(s["ds"], s["dn"], x, h, w, row_gate=s["row_gate"])
        names = params_of(c) + (["row_gate"] if c["row_gate"] else [])
        return [t for t in (out, n) if t is not None] + [dx, dh] + [op.grads[name] for name in names]
    dt, pt, rho = x.dtype, DTYPES[c["params"]], c["rho"]
    p = {name: t.float() for name, t in w.items()}
    n1, r1 = normed(h.float(), c["post"])
    z = n1 * p["post_weight"] if "post_weight" in p else n1
    if "post_bias" in p:
        z = z + p["post_bias"]
    g = p["gate"] if "gate" in p else 1.0
    if c["row_gate"]:
        g = g * s["row_gate"][:, None]
    out = rho * x.float() + g * z
    got = [out.to(dt)]
    if c["pre"] != "none":
        n2, r2 = normed(out, c["pre"])
        n = n2 * p["pre_weight"]
        got.append((n + p["pre_bias"] if "pre_bias" in p else n).to(dt))
    if not c["train"]:
        return got
    D, grads = s["ds"].float(), {}
    if c["pre"] != "none":
        dn = s["dn"].float()
        grads["pre_weight"], grads["pre_bias"] = (dn * n2).sum(0), dn.sum(0)
        D = D + normed_back(dn * p["pre_weight"], n2, r2, c["pre"])
    dz = D * g
    grads["post_weight"], grads["post_bias"] = (dz * n1).sum(0), dz.sum(0)
    dgate = D * z
    if c["row_gate"]:
        grads["row_gate"] = (dgate * p["gate"] if "gate" in p else dgate).sum(1)
        dgate = dgate * s["row_gate"][:, None]
    grads["gate"] = dgate.sum(0)
    dh = normed_back(dz * p["post_weight"] if "post_weight" in p else dz, n1, r1, c["post"])
    got += [(rho * D).to(dt), dh.to(dt)] + [grads[name].to(pt) for name in params_of(c)]
    return got + ([grads["row_gate"]] if c["row_gate"] else [])


def run_router(s):
    c, logits, idx, spans, dw = s["case"], s["logits"], s["topk_idx"], s["spans"], s["d_weights"]
    if own:
        op = s["op"]
        losses = op.forward(logits, idx, spans=spans)
        if not c["train"]:
            return losses, op.counts
        return losses, op.counts, op.backward(logits, idx, d_weights=dw, spans=spans)
    T, G, S = c["tokens"], c["experts"], c["sequences"]
    rows = torch.arange(T, device=logits.device, dtype=torch.int32)
    seq = torch.searchsorted(spans[:, 0].contiguous(), rows, right=True) - 1  # the last that begins at or before the row
    live = (seq >= 0) & (rows < spans[seq.clamp(min=0), 1])
    seq = torch.where(live, seq, S)  # S: none
    counts = torch.zeros((S + 1) * G, device=logits.device, dtype=torch.int32)
    counts.index_add_(0, (seq[:, None] * G + idx).view(-1), torch.ones(idx.numel(), device=idx.device, dtype=torch.int32))
    counts = counts.view(S + 1, G)[:S]
    length = (spans[:, 1] - spans[:, 0]).float()
    share = 1.0 / (length.clamp(min=1) * (length > 0).sum())  # of a row in the mean over rows and sequences
    n_rows = length.sum().clamp(min=1)
    f = counts * (G / counts.sum(1, keepdim=True).clamp(min=1).float())
    f = torch.cat([f * share[:, None], torch.zeros(1, G, device=f.device)])[seq]
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    p, lse = e / total, top + torch.log(total)
    balance = (f * p).sum()
    z = (torch.where(live[:, None], lse, 0.0) ** 2).sum() / n_rows
    losses = torch.stack([0.01 * balance + c["z"] * z, balance, z])
    if not c["train"]:
        return losses, counts
    grad = 0.01 * f
    if dw is not None:
        grad = grad.scatter_add(1, idx.long(), dw)
    dl = p * (grad - (p * grad).sum(1, keepdim=True) + (2 * c["z"] / n_rows) * lse)
    return losses, counts, torch.where(live[:, None], dl, 0.0).to(DTYPES[c["dtype"]])


def run_clip(s):
    c, g = s["case"], s["g"]
    if own:
        op = s["op"]
        if c["out"] is None:
            return op.norm(s["max_norm"], factor=s["factor"]), op.scale
        return op.clip(s["max_norm"], factor=s["factor"]), op.scale, s["out"]
    gf = g.float()
    norm = s["factor"] * torch.sqrt((gf * gf).sum())
    scale = s["factor"] * (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    if c["out"] is None:
        return norm.view(1), scale.view(1)
    s["out"].copy_(gf * scale)
    return norm.view(1), scale.view(1), s["out"]


# ---- in 64 bits --------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"join": exact_join, "router": exact_router, "clip": exact_clip}[case["op"]](s)


def exact_join(s):
    """The gradients through each mean, variance and product by itself."""
    D = torch.float64
    c, x, h, d = s["case"], s["x"].to(D), s["h"].to(D), s["case"]["d"]
    w = {name: t.to(D) for name, t in s["w"].items()}
    one, rg = torch.ones(d, dtype=D, device=x.device), s["row_gate"]
    rg = torch.ones(len(x), 1, dtype=D, device=x.device) if rg is None else rg.to(D)[:, None]

    def norm(v, kind, where):
        if kind == "none":
            return v, None
        mu = v.mean(1, keepdim=True) if kind == "layer" else 0.0
        inv = 1 / (((v - mu) ** 2).sum(1, keepdim=True) / d + NORM_EPS).sqrt()
        return (v - mu) * inv * w.get(where + "_weight", one) + w.get(where + "_bias", 0.0), (mu, inv)

    def back(dy, v, st, kind, where):
        if kind == "none":
            return dy, {}
        mu, inv = st
        da = dy * w.get(where + "_weight", one)
        dvar = (da * (v - mu)).sum(1, keepdim=True) * -0.5 * inv ** 3
        dv = da * inv + dvar * 2 * (v - mu) / d
        if kind == "layer":
            dv = dv - inv * da.sum(1, keepdim=True) / d
        return dv, {where + "_weight": (dy * (v - mu) * inv).sum(0), where + "_bias": dy.sum(0)}

    z, st1 = norm(h, c["post"], "post")
    gate = w.get("gate", one)
    out = c["rho"] * x + rg * (gate * z)
    n, st2 = norm(out, c["pre"], "pre")
    got = [out] + ([n] if c["pre"] != "none" else [])
    if not c["train"]:
        return got
    total, grads = s["ds"].to(D), {}
    if c["pre"] != "none":
        dv, more = back(s["dn"].to(D), out, st2, c["pre"], "pre")
        total = total + dv
        grads.update(more)
    dh, more = back(total * rg * gate, h, st1, c["post"], "post")
    grads.update(more)
    grads["gate"] = (total * rg * z).sum(0)
    grads["row_gate"] = (total * gate * z).sum(1)
    names = params_of(c) + (["row_gate"] if c["row_gate"] else [])
    return got + [c["rho"] * total, dh] + [grads[name] for name in names]


def exact_router(s):
    """Sequence by sequence."""
    D = torch.float64
    c, G, idx = s["case"], s["case"]["experts"], s["topk_idx"].long()
    logits, spans = s["logits"].to(D), s["spans"].tolist()
    live = [(a, b) for a, b in spans if b > a]
    n_rows = max(1, sum(b - a for a, b in live))
    counts = torch.zeros(len(spans), G, dtype=torch.int32, device=idx.device)
    dl = torch.zeros_like(logits)
    balance = torch.zeros((), dtype=D, device=idx.device)
    z = balance.clone()
    logp = torch.log_softmax(logits, 1)
    lse = torch.logsumexp(logits, 1)
    prob = logp.exp()
    for q, (a, b) in enumerate(spans):
        if b <= a:
            continue
        c_q = torch.bincount(idx[a:b].reshape(-1), minlength=G)
        counts[q] = c_q.to(torch.int32)
        f = c_q.to(D) * G / c_q.sum()
        p = prob[a:b]
        balance += f @ p.mean(0) / len(live)
        z += (lse[a:b] ** 2).sum() / n_rows
        if c["train"]:
            e = 0.01 * f.expand_as(p) / ((b - a) * len(live))
            if s["d_weights"] is not None:
                e = e.clone().scatter_add_(1, idx[a:b], s["d_weights"][a:b].to(D))
            dl[a:b] = p * e - p * (p * e).sum(1, keepdim=True) + c["z"] / n_rows * 2 * lse[a:b, None] * p
    losses = torch.stack([0.01 * balance + c["z"] * z, balance, z])
    return (losses, counts, dl) if c["train"] else (losses, counts)


def exact_clip(s):
    g = s["g"].to(torch.float64)
    norm = torch.linalg.vector_norm(g) * s["factor"]
    scale = s["factor"] * min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))
    got = [norm.view(1), torch.full((1,), scale, dtype=torch.float64, device=g.device)]
    return tuple(got + [g * scale] if s["case"]["out"] else got)
