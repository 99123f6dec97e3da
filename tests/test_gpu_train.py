"""The operators that complete a block's training step on the GPU against 64-bit formulas, with bounds counted from their
roundings."""
import itertools

import numpy as np
import pytest
import torch

import train_reference as ref
from block_reference import D, E32, half_step, within

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
RHO = float(np.float32(0.7))


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def spread(t, pad):
    """t's rows as a slice of a wider tensor, whose other elements are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


# ---- the norms around a block ------------------------------------------------------------------------------------

def names_of(post, pre, gate=True):
    return [n for n in ("post_weight", "post_bias", "gate", "pre_weight", "pre_bias")
            if not (n.startswith("post") and post == "none" or n.startswith("pre") and pre == "none" or n == "gate" and not gate)]


def residual_case(rows, d, dtype, params, post="rms", pre="rms", rho=1.0, pad=0, seed=0, gate=True, row_gate=False, ds=True,
                  bias=True):
    rnd = gen(3100 + seed)
    dt, pt = DT[dtype], DT[params]
    x = (rnd(rows, d) * torch.exp(0.5 * rnd(d)) + 0.5 * rnd(d)).to(dt)
    x[:, :: 37] *= 16
    h = (rnd(rows, d) * torch.exp(0.3 * rnd(d)) * torch.exp(rnd(rows, 1)) + 0.5 * rnd(d)).to(dt)
    w = {n: (0.1 * rnd(d) if n.endswith("bias") else 1 + 0.2 * rnd(d)).to(pt) for n in names_of(post, pre, gate)
         if bias or not n.endswith("bias")}
    c = torch.sigmoid(rnd(rows)) if row_gate else None
    gs, gn = (rnd(rows, d).to(dt) if ds else None), (rnd(rows, d).to(dt) if pre != "none" else None)
    if pad:
        x, h = spread(x, pad), spread(h, pad + 1)
        gs, gn = (spread(t, 2 * pad) if t is not None else None for t in (gs, gn))
    return dict(x=x, h=h, w=w, row_gate=c, ds=gs, dn=gn), dict(post=post, pre=pre, residual_scale=rho)


def residual_run(t, kinds, op=None):
    from expert_output_overlap_amd.runtime import ResidualNorm

    rows, d = t["x"].shape
    names = {torch.bfloat16: "bf16", torch.float32: "f32"}
    pt = next(iter(t["w"].values())).dtype if t["w"] else torch.float32
    if op is None:
        op = ResidualNorm(rows, d, names[t["x"].dtype], names[pt], **kinds)
    s, n = op.forward(t["x"], t["h"], t["w"], row_gate=t["row_gate"])
    dx, dh = op.backward(t["ds"], t["dn"], t["x"], t["h"], t["w"], row_gate=t["row_gate"])
    got = {"s": s, "dx": dx, "dh": dh, **{k: op.grads[k] for k in t["w"]}}
    if n is not None:
        got["n"] = n
    if t["row_gate"] is not None:
        got["row_gate"] = op.grads["row_gate"][:rows]
    return op, got


def residual_want(t, kinds):
    return ref.residual_norm(t["x"], t["h"], t["w"], kinds["post"], kinds["pre"], kinds["residual_scale"], 1e-5, t["row_gate"],
                             t["ds"], t["dn"])


def residual_check(got, want, tag):
    assert set(got) == set(want), tag
    for k in want:
        within(got[k], *want[k], (tag, k))


SIZES = [(2, 64), (16, 100), (64, 120), (65, 120), (33, 200), (16, 400), (17, 400), (4, 1000), (5, 1000), (4, 4096), (3, 4097), (1, 64), (1, 7168), (3, 1), (5, 7), (17, 65), (300, 512), (70, 513), (33, 1024), (40, 1407), (64, 2048), (9, 2049),
         (700, 4096), (21, 7168), (2000, 5000), (13, 8192), (7, 8193), (6, 16383), (5, 16384), (9000, 96)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_residual_norm(rows, d, dtype, params):
    k = rows + d
    post, pre = ("rms", "layer")[k % 2], ("layer", "rms", "rms")[k % 3]
    t, kinds = residual_case(rows, d, dtype, params, post, pre, RHO if k % 2 else 1.0, pad=k % 3, row_gate=k % 2 == 0, seed=k)
    _, got = residual_run(t, kinds)
    residual_check(got, residual_want(t, kinds), (rows, d, dtype, params))


@pytest.mark.parametrize("post,pre", itertools.product(["none", "layer", "rms"], repeat=2))
@pytest.mark.parametrize("rows,d,dtype", [(37, 200, "bf16"), (50, 3000, "f32"), (300, 5000, "bf16")])
def test_residual_norm_kinds(post, pre, rows, d, dtype):
    for i, (gate, row_gate, ds, bias) in enumerate(itertools.product([True, False], repeat=4)):
        if pre == "none" and not ds:
            continue
        t, kinds = residual_case(rows, d, dtype, "f32", post, pre, RHO, gate=gate, row_gate=row_gate, ds=ds, bias=bias, seed=i)
        _, got = residual_run(t, kinds)
        residual_check(got, residual_want(t, kinds), (post, pre, gate, row_gate, ds, bias))


@pytest.mark.parametrize("rows,d", [(1100, 16384), (1031, 8200), (1500, 12001), (4100, 7168), (3001, 2100)])
@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_residual_norm_of_many_rows(rows, d, dtype, params):
    """Several rows for each group of threads, and the same again into the same buffers."""
    t, kinds = residual_case(rows, d, dtype, params, "layer", "layer", RHO, pad=1, row_gate=True)
    op, got = residual_run(t, kinds)
    residual_check(got, residual_want(t, kinds), (rows, d, dtype))
    first = {k: v.clone() for k, v in got.items()}
    for _ in range(2):
        _, again = residual_run(t, kinds, op)
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("d", [7, 64, 100, 127, 128, 129, 250, 500, 1000, 1023, 1500, 2900, 4096, 5003, 8190, 8192])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_norm_of_rows_for_every_wave(d, dtype):
    """Enough rows that the forward gives a wave, or a part of one, to each: every width class, whole chunks and not, with biases and
    without."""
    for bias in (False, True):
        t, kinds = residual_case(2100, d, dtype, "f32", "layer" if bias else "rms", "layer", RHO, pad=d % 2, bias=bias, seed=d)
        _, got = residual_run(t, kinds)
        residual_check(got, residual_want(t, kinds), (d, dtype, bias))


@pytest.mark.parametrize("rows,d", [(2500, 8192), (2048, 4100), (40, 16384)])
def test_residual_norm_captured_with_much_lds(rows, d):
    """Launches with more LDS than the default limit in a graph, replayed with new inputs between eager calls."""
    t, kinds = residual_case(rows, d, "bf16", "f32", "layer", "layer")
    op, _ = residual_run(t, kinds)
    other = residual_run(t, kinds)[0]
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        _, got = residual_run(t, kinds, op)
    rnd = gen(9)
    for _ in range(3):
        t["x"].copy_(rnd(rows, d))
        t["dn"].copy_(rnd(rows, d))
        torch.cuda.synchronize()
        graph.replay()
        _, want = residual_run(t, kinds, other)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_residual_norm_in_place():
    from expert_output_overlap_amd.runtime import ResidualNorm

    for rows, d in ((1, 7168), (150, 1536), (700, 7168), (2200, 100), (2200, 5001), (60, 16000)):
        t, kinds = residual_case(rows, d, "bf16", "f32", "rms", "layer")
        op, got = residual_run(t, kinds)
        keep = {k: v.clone() for k, v in got.items()}
        ds, dn = t["ds"].clone(), t["dn"].clone()
        op.backward(ds, dn, t["x"], t["h"], t["w"], dx=ds, dh=dn)
        assert torch.equal(ds, keep["dx"]) and torch.equal(dn, keep["dh"])
        ds, dn = t["ds"].clone(), t["dn"].clone()
        op.backward(ds, dn, t["x"], t["h"], t["w"], dx=dn, dh=ds)
        assert torch.equal(dn, keep["dx"]) and torch.equal(ds, keep["dh"])
        assert all(torch.equal(op.grads[k], keep[k]) for k in t["w"])
        serve = ResidualNorm(rows, d, **kinds, train=False)
        x, h = t["x"].clone(), t["h"].clone()
        serve.forward(x, h, t["w"], s=x, n=h)
        assert torch.equal(x, keep["s"]) and torch.equal(h, keep["n"])
        x, h = t["x"].clone(), t["h"].clone()
        serve.forward(x, h, t["w"], s=h, n=x)
        assert torch.equal(h, keep["s"]) and torch.equal(x, keep["n"])
        with pytest.raises(RuntimeError, match="train"):
            serve.backward(t["ds"], t["dn"], t["x"], t["h"], t["w"])


def test_residual_norm_leaves_what_is_not_its_own():
    """Fewer rows than the buffers hold, results as slices, and gradients of parameters that are not there."""
    from expert_output_overlap_amd.runtime import ResidualNorm

    for d in (96, 1000, 5000):
        t, kinds = residual_case(10, d, "bf16", "f32", "rms", "rms", bias=False, row_gate=True)
        op = ResidualNorm(64, d, **kinds)
        for q in (op.s, op.n, op.dx, op.dh, op.stats, *op.grads.values()):
            q.fill_(7.0)
        wide = torch.full((10, 4 * d + 5), 7.0, device="cuda", dtype=torch.bfloat16)
        at = [slice(1 + i * (d + 1), 1 + i * (d + 1) + d) for i in range(4)]
        op.forward(t["x"], t["h"], t["w"], row_gate=t["row_gate"], s=wide[:, at[0]], n=wide[:, at[1]])
        op.backward(t["ds"], t["dn"], t["x"], t["h"], t["w"], row_gate=t["row_gate"], dx=wide[:, at[2]], dh=wide[:, at[3]])
        got = dict(s=wide[:, at[0]], n=wide[:, at[1]], dx=wide[:, at[2]], dh=wide[:, at[3]], **{k: op.grads[k] for k in t["w"]},
                   row_gate=op.grads["row_gate"][:10])
        residual_check(got, residual_want(t, kinds), d)
        outside = torch.ones(4 * d + 5, dtype=torch.bool, device="cuda")
        for a in at:
            outside[a] = False
        assert (wide[:, outside] == 7).all()
        for q in (op.s, op.n, op.dx, op.dh, op.grads["post_bias"], op.grads["pre_bias"], op.stats[10:], op.grads["row_gate"][10:]):
            assert (q == 7).all()
        op.forward(t["x"], t["h"], t["w"])
        assert (op.s[10:] == 7).all() and (op.n[10:] == 7).all()


def test_residual_norm_of_nothing():
    from expert_output_overlap_amd.runtime import ResidualNorm

    op, none = ResidualNorm(8, 200, "f32", "bf16"), torch.empty(0, 200, device="cuda")
    w = {n: torch.ones(200, device="cuda", dtype=torch.bfloat16) for n in names_of("rms", "rms")}
    for g in op.grads.values():
        g.fill_(5.0)
    s, n = op.forward(none, none, w)
    assert s.shape == (0, 200) and n.shape == (0, 200)
    op.backward(none, none, none, none, w)
    assert all((op.grads[k] == 0).all() for k in w) and (op.grads["row_gate"] == 5).all()
    bare = ResidualNorm(8, 200, "f32", post="none", pre="none")
    assert bare.forward(none, none, {})[1] is None
    bare.backward(none, None, none, none, {})


def test_residual_norm_of_constant_and_bad_rows():
    """A row without variance, rows of zeros, and NaN and infinities, which stay in their rows."""
    t, kinds = residual_case(9, 768, "f32", "f32", "layer", "layer", row_gate=True)
    x, h = t["x"], t["h"]
    h[1] = 3.25
    x[2], h[2] = 0.0, 0.0
    x[3, 5], h[4, 700], x[5, 0], t["row_gate"][6] = float("nan"), float("inf"), -float("inf"), float("nan")
    _, got = residual_run(t, kinds)
    want = residual_want(t, kinds)
    good = [0, 1, 2, 7, 8]
    for k in ("s", "n", "dx", "dh", "row_gate"):
        within(got[k][good], want[k][0][good], want[k][1][good], k)
    for k in ("n", "dx", "dh"):
        for r in (3, 4, 5, 6):
            assert not torch.isfinite(got[k][r]).any(), (k, r)
    ones = {n: torch.ones(64, device="cuda") for n in ("post_weight", "pre_weight")}
    z = dict(x=torch.zeros(2, 64, device="cuda"), h=torch.zeros(2, 64, device="cuda"), w=ones, row_gate=None,
             ds=torch.ones(2, 64, device="cuda"), dn=torch.zeros(2, 64, device="cuda"))
    _, got = residual_run(z, dict(post="rms", pre="rms", residual_scale=1.0))
    assert (got["s"] == 0).all() and (got["n"] == 0).all() and (got["dx"] == 1).all()
    assert (got["dh"].double() - 1e-5 ** -0.5).abs().max() < 1e-3 * 1e-5 ** -0.5


# a group of 16 lanes, a wave of one and of sixteen chunks a lane, workgroups of every size, odd widths, rows in LDS in the backward
LEVEL_SIZES = [(2100, 96), (2100, 100), (2051, 1000), (2048, 7168), (20, 33), (30, 512), (30, 1407), (30, 4096), (30, 7168), (9, 8200),
               (6, 16384)]


@pytest.mark.parametrize("rows,d", LEVEL_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_of_equal_elements_is_its_bias(rows, d, dtype):
    """A row of equal elements v has v^ = 0, whatever v is: the row sum's rounding leaves the mean by at most ROW |v| off, the
    differences are exact and their mean corrects it to that share of itself, less than half a step of v.  So s, n and the weights'
    gradients, which are sums of v^, are what the biases alone make; the variance is off by at most 3 ROW (ROW v)^2, against eps."""
    rnd, dt, eps = gen(rows + d), DT[dtype], 1e-5
    v = torch.tensor([3.25, 1000.3, 30000.0, -700.7, 1e-3], device="cuda").repeat(rows)[:rows, None].expand(rows, d).to(dt)
    w = {"post_weight": 1 + 0.2 * rnd(d), "post_bias": 0.1 * rnd(d), "gate": 1 + 0.2 * rnd(d)}
    t = dict(x=rnd(rows, d).to(dt), h=v.contiguous(), w=w, row_gate=torch.sigmoid(rnd(rows)), ds=rnd(rows, d).to(dt), dn=None)
    _, got = residual_run(t, dict(post="layer", pre="none", residual_scale=RHO))
    W = {k: x.to(D) for k, x in w.items()}
    c, x, ds, r = t["row_gate"].to(D)[:, None], t["x"].to(D), t["ds"].to(D), half_step(dt)
    part = c * W["gate"] * W["post_bias"]
    s = RHO * x + part
    within(got["s"], s, 4 * E32 * part.abs() + 2 * E32 * ((RHO * x).abs() + s.abs()) + r * s.abs(), "s")
    assert (got["post_weight"] == 0).all()
    u0, e_u0 = (c * ds).sum(0), ((rows + 12) * E32 * (c * ds).abs()).sum(0)
    within(got["post_bias"], W["gate"] * u0, W["gate"].abs() * (e_u0 + 2 * E32 * u0.abs()), "post_bias")
    within(got["gate"], W["post_bias"] * u0, W["post_bias"].abs() * (e_u0 + 2 * E32 * u0.abs()), "gate")
    a = c * W["gate"] * W["post_weight"] * ds
    zero, e_r = torch.zeros_like(a), 1.5 * ref.ROW * (ref.ROW * v[:, :1].to(D)) ** 2 / eps + 8 * E32
    dh, e = ref.norm_back(a, 4 * E32 * a.abs(), zero, zero, torch.full_like(a[:, :1], eps ** -0.5), e_r, "layer")
    within(got["dh"], dh, e + r * dh.abs(), "dh")
    # in front of the next block: s = v up to a factor
    w = {"pre_weight": 1 + 0.2 * rnd(d), "pre_bias": 0.1 * rnd(d)}
    t = dict(x=v.contiguous(), h=torch.zeros_like(t["h"]), w=w, row_gate=None, ds=None, dn=t["ds"])
    _, got = residual_run(t, dict(post="none", pre="layer", residual_scale=RHO))
    assert torch.equal(got["n"], w["pre_bias"].to(dt).expand(rows, d)) and (got["pre_weight"] == 0).all()
    within(got["pre_bias"], ds.sum(0), ((rows + 12) * E32 * ds.abs()).sum(0), "pre_bias")


@pytest.mark.parametrize("rows,d", LEVEL_SIZES)
@pytest.mark.parametrize("dtype,level", [("bf16", 200.0), ("f32", 1000.0)])
def test_layer_norm_far_from_zero(rows, d, dtype, level):
    """Rows of level - 1 and level + 1 in equal numbers (and one of the level itself where d is odd): the row's sum, mean, differences and
    their squares are exact, so v^ = (v - mean) rstd is off by the roundings of rstd and of one product alone, 8 E32 of itself,
    and not by steps of the level."""
    rnd, dt = gen(rows + d), DT[dtype]
    e = torch.ones(rows, d, device="cuda")
    e[:, 1::2] = -1
    if d % 2:
        e[:, -1] = 0
    v, zero = (level + e).to(dt), torch.zeros(rows, d, device="cuda", dtype=dt)
    assert torch.equal(v.float(), level + e)
    rstd = torch.full((rows, 1), (d // 2 * 2 / d + 1e-5) ** -0.5, dtype=D, device="cuda")
    n, g, r, k = e.to(D) * rstd, rnd(rows, d).to(dt), half_step(dt), (rows + 12) * E32
    for post, pre in (("layer", "none"), ("none", "layer")):
        w = {"post_weight" if pre == "none" else "pre_weight": torch.ones(d, device="cuda")}
        t = dict(x=zero if pre == "none" else v, h=v if pre == "none" else zero, w=w, row_gate=None, ds=g if pre == "none" else None,
                 dn=None if pre == "none" else g)
        _, got = residual_run(t, dict(post=post, pre=pre, residual_scale=1.0))
        within(got["s" if pre == "none" else "n"], n, (8 * E32 + r) * n.abs(), (post, pre))
        a = g.to(D)
        back, e_b = ref.norm_back(a, 0 * a, n, 8 * E32 * n.abs(), rstd, torch.full_like(rstd, 8 * E32), "layer")
        within(got["dh" if pre == "none" else "dx"], back, e_b + (E32 + r) * back.abs(), (post, pre))
        within(got[next(iter(w))], (a * n).sum(0), ((k + 8 * E32) * (a * n).abs()).sum(0), (post, pre, "weight"))


@pytest.mark.parametrize("rows,d", [(40, 100), (7, 1000), (2100, 96), (5, 5000), (5, 9000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pre", ["none", "rms"])
def test_residual_norm_without_a_post_norm_keeps_bad_values_out_of_dh(rows, d, dtype, pre):
    """Without N1, dh = c gate D, whatever h is: an infinity or a NaN in it reaches its row's other gradients through a pre norm alone, and
    the gate's in its column.  Rows without one are as ever."""
    t, kinds = residual_case(rows, d, dtype, "f32", "none", pre, RHO, row_gate=True, bias=False, seed=d)
    bad = {0: (d - 1, float("inf")), 2: (0, float("nan")), 4: (d // 2, -float("inf"))}
    for row, (col, value) in bad.items():
        t["h"][row, col] = value
    _, got = residual_run(t, kinds)
    clean = {**t, "h": torch.where(torch.isfinite(t["h"]), t["h"], 1.0)}
    want = residual_want(clean, kinds)
    rest = [k for k in range(rows) if k not in bad]
    for k in ("s", "dx", "dh", "row_gate"):
        within(got[k][rest], want[k][0][rest], want[k][1][rest], k)
    for row, (col, _) in bad.items():
        assert not torch.isfinite(got["s"][row, col]) and not torch.isfinite(got["row_gate"][row])
        assert not torch.isfinite(got["gate"][col])
    cols = [k for k in range(d) if k not in [col for col, _ in bad.values()]]
    if pre == "none":
        for k in ("dx", "dh"):
            within(got[k], want[k][0], want[k][1], k)
        within(got["gate"][cols], want["gate"][0][cols], want["gate"][1][cols], "gate")
    else:
        assert not torch.isfinite(got["dh"][[0, 2, 4]]).any()


def test_residual_norm_gradients_against_differences():
    """A step e along a direction changes the loss by e times the gradient's product with it: central differences of the operator's own
    fp32 forward.  The loss is a sum of 2 x 6 x 40 products, each known to 40 E32 of its size or so (row sums of 40, some products);
    that over 2 e, and e^2 of third derivatives of the order of the gradient."""
    from expert_output_overlap_amd.runtime import ResidualNorm

    e = 2.0 ** -7
    for post, pre in (("layer", "rms"), ("rms", "layer"), ("none", "rms"), ("rms", "none")):
        t, kinds = residual_case(6, 40, "f32", "f32", post, pre, RHO, row_gate=True)
        t["x"].clamp_(-3, 3), t["h"].clamp_(-3, 3)
        op, got = residual_run(t, kinds)
        got = {k: v.clone() for k, v in got.items()}
        rnd = gen(8)
        fwd = ResidualNorm(6, 40, "f32", **kinds, train=False)

        def loss(x, h, w, c):
            s, n = fwd.forward(x, h, w, row_gate=c)
            parts = (s.double() * t["ds"].double())
            if n is not None:
                parts = torch.cat([parts, n.double() * t["dn"].double()])
            return parts.sum(), parts.abs().sum()

        for name in ("x", "h", *t["w"], "row_gate"):
            at = t["w"][name] if name in t["w"] else t[name]
            way = rnd(*at.shape).sign() * 0.1
            ends = []
            for sign in (1, -1):
                moved = at + sign * e * way
                u = {**t, "w": dict(t["w"])}
                (u["w"] if name in t["w"] else u)[name] = moved
                ends.append(loss(u["x"], u["h"], u["w"], u["row_gate"]))
            diff = (ends[0][0] - ends[1][0]) / (2 * e)
            grad = got[{"x": "dx", "h": "dh"}.get(name, name)].double()
            want = (grad * way.double()).sum()
            size = (grad * way.double()).abs().sum()
            bound = 40 * E32 * ends[0][1] / e + 0.05 * e * size + 100 * E32 * size
            assert (diff - want).abs() <= bound, (post, pre, name, diff, want, bound)


def test_residual_norm_refusals():
    from expert_output_overlap_amd.runtime import ResidualNorm

    t, kinds = residual_case(8, 64, "bf16", "f32")
    op = ResidualNorm(8, 64, **kinds)
    x, h, w = t["x"], t["h"], t["w"]
    for kw, words in ((dict(x=x.float()), "wanted"), (dict(h=h[:4]), "wanted"), (dict(x=x.T.contiguous().T), "side by side"),
                      (dict(x=x.cpu()), "wanted"), (dict(w={**w, "gate": w["gate"].bfloat16()}), "wanted"),
                      (dict(w={**w, "gate": w["gate"][:32]}), "wanted"), (dict(row_gate=torch.ones(7, device="cuda")), "wanted"),
                      (dict(x=torch.cat([x, x]), h=torch.cat([h, h])), "up to 8")):
        with pytest.raises(ValueError, match=words):
            op.forward(**{**dict(x=x, h=h, w=w), **kw})
    from expert_output_overlap_amd import binding as B
    with pytest.raises(B.MoeError, match="overlaps"):
        op.forward(x, h, w, s=x)
    op.forward(x, h, w)
    with pytest.raises(B.MoeError, match="only then"):
        op.backward(t["ds"], None, x, h, w)
    with pytest.raises(B.MoeError, match="overlaps"):
        op.backward(t["ds"], t["dn"], x, h, w, dx=x)
    with pytest.raises(KeyError):
        ResidualNorm(8, 64, post="batch")
    with pytest.raises(B.MoeError):
        ResidualNorm(8, 16385)


# ---- the router's losses -----------------------------------------------------------------------------------------

def spans_for(T, S, seed):
    """Ascending spans with gaps, some empty, some of one row."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, T + 1, (2 * S,), generator=g).sort().values.view(S, 2)
    if S > 2:
        cuts[S // 2] = cuts[S // 2][:1]
    return cuts.to(torch.int32).cuda()


def router_case(T, G, k, S, padded, seed=0, weights=True):
    rnd = gen(4100 + seed)
    logits = (rnd(T, G) + 0.7 * rnd(G)) * 2
    idx = torch.topk(logits, k, 1).indices.to(torch.int32)
    return logits, idx, spans_for(T, S, seed) if padded else None, 1e-2 * rnd(T, k) if weights else None


def router_check(T, G, k, S, padded, z, dtype="f32", weights=True, seed=0, d_loss=None, balance=0.01):
    from expert_output_overlap_amd.runtime import RouterLoss

    logits, idx, spans, dw = router_case(T, G, k, S, padded, seed, weights)
    op = RouterLoss(T, G, k, S, balance, z, dtype)
    d = None if d_loss is None else torch.full((1,), d_loss, device="cuda")
    losses = op.forward(logits, idx, spans)
    dl = op.backward(logits, idx, dw, d, spans)
    counts, want = ref.router_loss(logits, idx, S, float(np.float32(balance)), float(np.float32(z)), spans, dw,
                                   1.0 if d_loss is None else d_loss, DT[dtype])
    assert torch.equal(op.counts, counts)
    live = [(a, b) for a, b in ref.rows_of(spans, T, S) if b > a]
    assert op.means.tolist() == [len(live), sum(b - a for a, b in live)]
    within(losses, *want["losses"], "losses")
    within(dl, *want["dlogits"], "dlogits")
    return op, (logits, idx, spans, dw)


ROUTER_SIZES = [(1, 1, 1), (1, 8, 2), (3, 2, 1), (64, 8, 2), (100, 7, 7), (65, 16, 16), (257, 33, 3), (1000, 64, 6), (77, 100, 5),
                (4096, 8, 2), (513, 129, 8), (2050, 256, 8), (300, 257, 4), (129, 512, 10), (90, 700, 16), (64, 1024, 8),
                (5, 1023, 1), (20000, 4, 1), (9000, 60, 4)]


@pytest.mark.parametrize("T,G,k", ROUTER_SIZES)
def test_router_loss(T, G, k):
    n = T + G
    router_check(T, G, k, 1, False, 1e-3, "f32", seed=n)
    router_check(T, G, k, min(T, 5), True, 0.0 if n % 2 else 2e-2, "bf16", weights=n % 3 > 0, seed=n, d_loss=0.5)


@pytest.mark.parametrize("T,G,k,S,padded", [(64, 8, 2, 4, False), (64, 8, 2, 64, False), (1000, 16, 2, 250, True),
                                            (3000, 64, 6, 700, True), (3000, 64, 6, 5000, True), (40, 4, 2, 1, True),
                                            (16384, 32, 4, 8, True), (16000, 256, 8, 8, False)])
def test_router_sequences(T, G, k, S, padded):
    for seed in range(2):
        op, (logits, idx, spans, dw) = router_check(T, G, k, S, padded, 1e-3, seed=seed)
        losses, counts, dl = op.losses.clone(), op.counts.clone(), op.dlogits.clone()
        for _ in range(2):  # the same bits
            op.forward(logits, idx, spans)
            op.backward(logits, idx, dw, spans=spans)
            assert torch.equal(op.losses, losses) and torch.equal(op.counts, counts) and torch.equal(op.dlogits, dl)


def test_router_losses_of_nothing_and_of_padding():
    from expert_output_overlap_amd.runtime import RouterLoss

    op = RouterLoss(10, 8, 2, sequences=3, z=1.0)
    none, ids = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    for q in (op.counts, op.means, op.losses):
        q.fill_(9)
    op.forward(none, ids)
    assert (op.losses == 0).all() and (op.counts == 0).all() and op.means.tolist() == [0, 0]
    assert op.backward(none, ids).shape == (0, 8)
    # rows of no sequence: NaN logits, wild ids and gradients of their weights reach nothing
    rnd = gen(3)
    logits, dw = rnd(10, 8), rnd(10, 2)
    idx = torch.topk(logits, 2).indices.to(torch.int32)
    spans = torch.tensor([[2, 5], [5, 5], [7, 8]], dtype=torch.int32, device="cuda")
    bad = [0, 1, 5, 6, 8, 9]
    want = [op.forward(logits, idx, spans).clone(), op.counts.clone(), op.backward(logits, idx, dw, spans=spans).clone()]
    logits[bad], dw[bad], idx[bad] = float("nan"), float("inf"), 1 << 30
    got = [op.forward(logits, idx, spans), op.counts, op.backward(logits, idx, dw, spans=spans)]
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (got[2][bad] == 0).all()
    # nothing but padding
    empty = torch.tensor([[0, 0], [4, 4], [10, 10]], dtype=torch.int32, device="cuda")
    op.forward(logits, idx, empty)
    assert (op.losses == 0).all() and (op.counts == 0).all() and (op.backward(logits, idx, dw, spans=empty) == 0).all()
    # spans that leave the rows are cut
    out = torch.tensor([[-5, 1], [1, 1], [8, 90]], dtype=torch.int32, device="cuda")
    clean = rnd(10, 8)
    op.forward(clean, idx.clamp(max=7), out)
    assert op.means.tolist() == [2, 3] and op.counts.sum() == 6


def test_router_loss_leaves_the_rows_behind():
    from expert_output_overlap_amd.runtime import RouterLoss

    logits, idx, _, dw = router_case(7, 13, 3, 1, False)
    op = RouterLoss(20, 13, 3)
    op.dlogits.fill_(7.0)
    op.forward(logits, idx)
    op.backward(logits, idx, dw)
    assert (op.dlogits[7:] == 7).all() and not (op.dlogits[:7] == 7).any()


@pytest.mark.parametrize("G", [4, 37, 200, 1000])
def test_router_rows_that_are_not_finite(G):
    """-inf takes an expert away, all of them leave the row without a gradient; lowest values are ordinary numbers; NaN and +inf stay
    in their rows' gradients."""
    from expert_output_overlap_amd.runtime import RouterLoss

    T, k, low = 12, 2, torch.finfo(torch.float32).min
    logits, idx, _, dw = router_case(T, G, k, 1, False, seed=G)
    logits[0, 0] = logits[1, 1:] = -float("inf")
    logits[2] = -float("inf")
    logits[3, ::2] = low
    logits[4] = low
    idx = torch.topk(logits, k).indices.to(torch.int32)
    idx[2] = torch.tensor([0, 1])
    dw[3] *= 1e3
    op = RouterLoss(T, G, k, z=0.0)
    op.forward(logits, idx)
    dl = op.backward(logits, idx, dw)
    counts, want = ref.router_loss(logits, idx, 1, float(np.float32(0.01)), 0.0, None, dw)
    assert torch.equal(op.counts, counts) and (dl[2] == 0).all()
    within(op.losses[:2], want["losses"][0][:2], want["losses"][1][:2], "losses")  # Z's square of the lowest value is over fp32's range
    within(dl, *want["dlogits"], "dlogits")
    for value in (float("nan"), float("inf")):
        bad = logits.clone()
        bad[6, G - 1] = value
        op.forward(bad, idx)
        got = op.backward(bad, idx, dw)
        assert torch.isnan(op.losses).all() and torch.isnan(got[6]).all()
        rest = [t for t in range(T) if t != 6]
        assert torch.equal(got[rest], dl[rest])


def test_router_ids_that_repeat_or_are_none():
    """The same expert twice in a row's choices counts twice, and its slots' gradients add up; ids outside count nowhere."""
    from expert_output_overlap_amd.runtime import RouterLoss

    for G in (9, 64, 100, 256, 600, 1024):
        logits, idx, _, dw = router_case(50, G, 4, 1, False)
        idx[3] = 5
        idx[4, 1] = idx[4, 0]
        idx[5] = -1
        idx[6, 2], idx[7, 0] = G, -(1 << 31)
        op = RouterLoss(50, G, 4, z=1e-3)
        op.forward(logits, idx)
        first = op.backward(logits, idx, dw).clone()
        counts, want = ref.router_loss(logits, idx, 1, float(np.float32(0.01)), float(np.float32(1e-3)), None, dw)
        assert torch.equal(op.counts, counts) and counts.sum() == 50 * 4 - 6
        within(op.losses, *want["losses"], "losses")
        within(op.dlogits, *want["dlogits"], "dlogits")
        assert torch.equal(op.backward(logits, idx, dw), first)


def test_router_workspace_serves_other_calls():
    """Calls of fewer and more tokens in turn on one operator give what an operator of their own gives."""
    from expert_output_overlap_amd.runtime import RouterLoss

    for G, S in ((8, 1), (256, 3), (1000, 40), (16, 300)):
        op = RouterLoss(9000, G, 2, S, z=1e-3)
        for T in (9000, 10, 4500, 0, 9000, 700, 1, 9000):
            logits, idx, spans, _ = router_case(T, G, 2, S, True, seed=T) if T else router_case(1, G, 2, S, True)
            logits, idx = logits[:T], idx[:T]
            own = RouterLoss(max(T, 1), G, 2, S, z=1e-3)
            assert torch.equal(op.forward(logits, idx, spans), own.forward(logits, idx, spans)), (G, S, T)
            assert torch.equal(op.counts, own.counts) and torch.equal(op.means, own.means)


@pytest.mark.parametrize("G", [2, 16, 60, 100, 250, 500, 1000])
def test_router_experts_far_below_the_top(G):
    """A slot's gradient of an expert x below its row's top logit: the others are so far down that the sum of exp is 1 to the last bit, and
    the logit's gradient is p (1 - p) dw with p = exp(x), off by the exponential's two steps (2 E32 each) and three roundings: 8 E32 of
    itself, however far down."""
    from expert_output_overlap_amd.runtime import RouterLoss

    T = 57
    x = -(30.0 + torch.arange(T, device="cuda"))  # to exp(-86), above the smallest normal number
    logits = torch.full((T, G), -float("inf"), device="cuda")
    logits[:, 0] = 5.0
    at = 1 + torch.arange(T, device="cuda") * 7 % (G - 1)
    rows = torch.arange(T, device="cuda")
    logits[rows, at] = 5.0 + x
    idx, dw = at.int()[:, None].contiguous(), gen(G)(T, 1)
    op = RouterLoss(T, G, 1, balance=0.0, z=0.0)
    op.forward(logits, idx)
    got = op.backward(logits, idx, dw)
    p = torch.exp(x.to(D))
    want = p * (1 - p) * dw[:, 0].to(D)
    off = (got[rows, at].to(D) / want - 1).abs()
    assert off.max() <= 8 * E32, (int(off.argmax()), off.max().item() / E32)


@pytest.mark.parametrize("G", [66, 128, 256, 500, 1024])
def test_router_slots_of_one_expert_add_up(G):
    """All slots of a row at one expert, in pairs, and one twice among others: the gradients add up whichever lanes hold them."""
    from expert_output_overlap_amd.runtime import RouterLoss

    T, k = 203, 16
    logits, idx, _, dw = router_case(T, G, k, 1, False, seed=G)
    idx[0::5] = idx[0::5, :1]
    idx[1::5] = idx[1::5, :8].repeat(1, 2)
    idx[2::5] = idx[2::5, :8].repeat_interleave(2, 1)
    idx[3::5, 15] = idx[3::5, 0]
    op = RouterLoss(T, G, k, z=1e-3)
    op.forward(logits, idx)
    got = op.backward(logits, idx, dw)
    counts, want = ref.router_loss(logits, idx, 1, float(np.float32(0.01)), float(np.float32(1e-3)), None, dw)
    assert torch.equal(op.counts, counts)
    within(got, *want["dlogits"], "dlogits")


def test_router_gradient_against_differences():
    """Central differences of the operator's own losses (fp32, 3 roundings of its size, its rows' products within 60 E32), and e^2
    of third derivatives of the order of the gradient."""
    from expert_output_overlap_amd.runtime import RouterLoss

    T, G, k, e = 6, 10, 3, 2.0 ** -6
    logits, idx, _, _ = router_case(T, G, k, 1, False, weights=False)
    for balance, z in ((1.0, 0.0), (0.0, 1.0), (1.0, 0.5)):
        op = RouterLoss(T, G, k, 2, balance, z)
        size = op.forward(logits, idx)[0].item()
        grad = op.backward(logits, idx).double()
        way = gen(4)(T, G).sign()
        ends = [op.forward(logits + s * e * way, idx)[0].item() for s in (1, -1)]
        want = (grad * way.double()).sum().item()
        slack = 64 * E32 * abs(size) / e + 2 * e * e * (grad.abs().sum().item() + z)
        assert abs((ends[0] - ends[1]) / (2 * e) - want) <= slack, (balance, z)


def test_router_refusals():
    from expert_output_overlap_amd import binding as B
    from expert_output_overlap_amd.runtime import RouterLoss

    logits, idx, spans, dw = router_case(8, 16, 2, 4, True)
    op = RouterLoss(8, 16, 2, 4)
    for a, words in (((logits.double(), idx), "wanted"), ((logits, idx.long()), "wanted"), ((logits[:, :8], idx), "wanted"),
                     ((logits, idx[:4]), "wanted"), ((logits, idx, spans[:3]), "wanted"), ((logits, idx, spans.long()), "wanted"),
                     ((torch.cat([logits] * 2), torch.cat([idx] * 2)), "up to 8"), ((logits.T.contiguous().T, idx), "contiguous")):
        with pytest.raises(ValueError, match=words):
            op.forward(*a)
    op.forward(logits, idx, spans)
    for kw in (dict(d_weights=dw[:3]), dict(d_loss=torch.ones(2, device="cuda")), dict(dlogits=op.dlogits.bfloat16())):
        with pytest.raises(ValueError, match="wanted"):
            op.backward(logits, idx, spans=spans, **kw)
    with pytest.raises(B.MoeError, match="multiple"):
        op.forward(logits[:7], idx[:7])
    with pytest.raises(RuntimeError, match="train"):
        RouterLoss(8, 16, 2, train=False).backward(logits, idx)
    with pytest.raises(B.MoeError):
        RouterLoss(8, 1025, 2)


# ---- the gradient norm -------------------------------------------------------------------------------------------

def grads_of(sizes, dtype, seed=0, offset=0):
    """Gradients of very different sizes, each at `offset` elements into its buffer."""
    rnd = gen(5100 + seed)
    return [(rnd(n + offset) * 1e-3 * torch.exp(2 * rnd(1))).to(DT[dtype])[offset:] for n in sizes]


GRAD_SIZES = [[1], [7], [8192], [8193, 5], [1, 2, 3, 4, 5, 6, 7, 8, 9], [100000, 1, 65536, 70001], [3000001], [33] * 300, [0, 5, 0]]


@pytest.mark.parametrize("sizes", GRAD_SIZES, ids=lambda s: "%d-%d" % (len(s), sum(s)))
@pytest.mark.parametrize("dtype,out", [("f32", None), ("f32", "bf16"), ("f32", "f32"), ("bf16", None), ("bf16", "bf16"),
                                       ("bf16", "f32")])
def test_grad_norm(sizes, dtype, out):
    from expert_output_overlap_amd.runtime import GradNorm

    for offset in (0, 1, 3):
        g = grads_of(sizes, dtype, len(sizes), offset)
        outs = [torch.full((t.numel() + offset,), 7.0, device="cuda", dtype=DT[out])[offset:] for t in g] if out else None
        op = GradNorm([{"g": t, **({"out": outs[i]} if out else {})} for i, t in enumerate(g)])
        before = [t.clone() for t in g]
        free, _ = ref.grad_norm(before, 1.0, 1.0)
        for max_norm, factor in ((0.25 * free.item(), 0.5), (10 * free.item(), 1.0), (float("inf"), 0.125)):
            norm, scale = ref.grad_norm(before, max_norm, factor)
            for t, b in zip(g, before):
                t.copy_(b)
            total = op.norm(max_norm, factor)
            first = (total.clone(), op.scale.clone())
            assert all(torch.equal(t, b) for t, b in zip(g, before))
            # 64-bit sums, one rounding of each result
            within(total[0], norm, 1.001 * E32 * norm, "norm")
            within(op.scale[0], scale, 1.001 * E32 * scale, "scale")
            op.clip(max_norm, factor)
            assert torch.equal(op.total, first[0]) and torch.equal(op.scale, first[1])
            f = op.scale.item()
            for t, b, o in zip(g, before, outs or g):
                want = b.to(D) * f  # the operator's own scale, which is right to half a step
                r = half_step(o.dtype) + (E32 if o.dtype is torch.bfloat16 else 0)
                within(o, want, r * want.abs(), "out")
                assert o is t or torch.equal(t, b)


def test_grad_norm_of_nothing():
    from expert_output_overlap_amd.runtime import GradNorm

    for tensors in ([], [{"g": torch.empty(0, device="cuda")}]):
        op = GradNorm(tensors)
        op.clip(2.0, 0.5)
        assert op.total.item() == 0 and op.scale.item() == 0.5


def test_grad_norm_of_values_out_of_the_ordinary():
    """Squares beyond fp32's range on both sides, and values that are not finite."""
    from expert_output_overlap_amd.runtime import GradNorm

    for value in (1e30, 1e-30, 1e-42):
        g = torch.full((5000,), value, device="cuda")
        op = GradNorm([{"g": g}])
        norm, scale = ref.grad_norm([g], 1e-3, 1.0)
        op.norm(1e-3)
        within(op.total[0], norm, 1.001 * E32 * norm + 2.0 ** -149, "norm")
        within(op.scale[0], scale, 1.001 * E32 * scale, "scale")
    g = torch.ones(5000, device="cuda")
    op = GradNorm([{"g": g}, {"g": torch.ones(10, device="cuda", dtype=torch.bfloat16)}])
    g[4321] = float("inf")
    assert op.norm(1.0).item() == float("inf") and op.scale.item() == 0
    assert op.norm().item() == float("inf") and op.scale.item() == 1
    g[4321] = float("nan")
    assert np.isnan(op.norm(1.0).item()) and np.isnan(op.scale.item())
    op.clip(1.0)
    assert torch.isnan(g).all()


def test_grad_clip_takes_a_scale_of_one_in_place():
    from expert_output_overlap_amd.runtime import GradNorm

    g = grads_of([10000], "f32")[0]
    g[3], before = -0.0, None
    before, out = g.clone(), torch.empty_like(g)
    GradNorm([{"g": g}]).clip(1e9)
    assert torch.equal(g, before)
    GradNorm([{"g": g, "out": out}]).clip(1e9)
    assert torch.equal(out, before)


def test_grad_norm_refusals():
    from expert_output_overlap_amd import binding as B
    from expert_output_overlap_amd.runtime import GradNorm

    g = torch.ones(100, device="cuda")
    for bad in ({"g": g.half()}, {"g": g.view(10, 10).T}, {"g": g, "out": g[:50]}, {"g": g, "out": torch.ones(100)},
                {"g": g, "out": g.long()}):
        with pytest.raises(ValueError, match="wanted"):
            GradNorm([bad])
    for bad in ([{"g": g}, {"g": g}], [{"g": g[:60]}, {"g": g[59:]}], [{"g": g, "out": g}], [{"g": g[:50], "out": g[25:75]}]):
        with pytest.raises(B.MoeError, match="overlaps"):
            GradNorm(bad)
    op = GradNorm([{"g": g}])
    for kw in (dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(factor=0.0), dict(factor=float("inf"))):
        with pytest.raises(B.MoeError, match="max_norm"):
            op.norm(**kw)


# ---- streams and graphs ------------------------------------------------------------------------------------------

def everything(seed, T=150, d=520):
    """One set of the operators and their run on given inputs: {name: result}."""
    from expert_output_overlap_amd.runtime import GradNorm, ResidualNorm, RouterLoss

    t, kinds = residual_case(T, d, "bf16", "f32", "layer", "rms", row_gate=True, seed=seed)
    logits, idx, spans, dw = router_case(T, 24, 3, 6, True, seed=seed)
    norm, loss = ResidualNorm(T, d, **kinds), RouterLoss(T, 24, 3, 6, z=1e-3, dtype="bf16")
    clipped = {k: torch.empty_like(g) for k, g in norm.grads.items() if k in t["w"]}
    grads = GradNorm([{"g": norm.grads[k], "out": c} for k, c in clipped.items()] + [{"g": loss.dlogits}])

    def run(stream=None):
        s, n = norm.forward(t["x"], t["h"], t["w"], row_gate=t["row_gate"], stream=stream)
        losses = loss.forward(logits, idx, spans, stream=stream)
        dl = loss.backward(logits, idx, dw, spans=spans, stream=stream)
        dx, dh = norm.backward(t["ds"], t["dn"], t["x"], t["h"], t["w"], row_gate=t["row_gate"], stream=stream)
        grads.clip(0.5, 0.25, stream=stream)
        return dict(s=s, n=n, losses=losses, counts=loss.counts, dl=dl, dx=dx, dh=dh, total=grads.total, scale=grads.scale, **clipped)

    return run, t, logits


def test_training_operators_captured_and_replayed():
    """Captured into one graph; each replay after new inputs equals the eager calls, with eager work between."""
    everything(1)[0]()
    torch.cuda.synchronize()
    (eager, t, logits), (captured, t2, logits2) = everything(2), everything(2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = captured()
    rnd = gen(6)
    for _ in range(4):
        for a, b in ((t["x"], t2["x"]), (t["dn"], t2["dn"]), (logits, logits2)):
            a.copy_(rnd(*a.shape))
            b.copy_(a)
        torch.cuda.synchronize()
        graph.replay()
        want = eager()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(want[k], got[k]), k


def test_training_operators_on_two_streams():
    """Two sets at the same time give what each gives alone."""
    sets = []
    for seed, T, d in ((3, 150, 520), (4, 2000, 1000)):
        run = everything(seed, T, d)[0]
        want = {k: v.clone() for k, v in run().items()}
        sets.append((run, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        # the clipped router gradient is in place: made anew by each run before it is clipped
        got = [run(stream) for run, _, stream in sets]
        torch.cuda.synchronize()
        for g, (_, want, _) in zip(got, sets):
            for k in want:
                assert torch.equal(g[k], want[k]), k


# ---- all of them together ----------------------------------------------------------------------------------------

def test_two_blocks_together():
    """Two training steps of two MoE blocks: norm, router, routed experts, shared expert, the balance loss, the join with its post norm
    and gate that makes the next block's input, all of their backward, the clipped gradients' norm and AdamW with its coefficient, against
    float64 autograd.  A result has passed at most eight roundings to bf16 in a row in each block and two at the join, forward and
    backward, each 2^-8 at most and of random sign, some of them through a norm that keeps their share: 24 x 2^-8 of its norm."""
    from expert_output_overlap_amd import binding as B
    from expert_output_overlap_amd.runtime import AdamW, GradNorm, MoeBlock, MoePath

    R, T_o, G, k, d, f, fs, M = 2, 40, 4, 2, 128, 128, 192, 16
    T, rnd, rho = R * T_o, gen(21), 0.75
    balance, z = float(np.float32(0.05)), float(np.float32(0.01))
    joins = [dict(post="rms", pre="layer", residual_scale=rho), dict(post="layer", pre="none", residual_scale=1.0)]
    blocks, weights, routers = [], [], []
    for j in joins:
        blocks.append(MoeBlock(MoePath(R, T_o, G, G, k, d, f, M), fs, losses=dict(balance=balance, z=z), join=j))
        w = {"norm_weight": 1 + 0.1 * rnd(d), "norm_bias": 0.1 * rnd(d), "w_gate_up": (rnd(G, 2 * f, d) / d ** 0.5).bfloat16(),
             "w_down": (rnd(G, d, f) / d ** 0.5).bfloat16(), "shared_gate_up": (rnd(2 * fs, d) / d ** 0.5).bfloat16(),
             "shared_down": (rnd(d, fs) / d ** 0.5).bfloat16()}
        w.update({n: 1 + 0.1 * rnd(d) if not n.endswith("bias") else 0.1 * rnd(d) for n in names_of(j["post"], j["pre"])})
        weights.append(w)
        routers.append(rnd(G, d) / d ** 0.5)
    used = [[n for n in w if i == 0 or not n.startswith("norm_")] for i, w in enumerate(weights)]  # the second's input comes from the join
    grads = []
    for b, names in zip(blocks, used):
        have = {"norm_weight": b.norm_op.dweight, "norm_bias": b.norm_op.dbias, "w_gate_up": b.path.bwd_buffers()["dw_gate_up"],
                "w_down": b.path.bwd_buffers()["dw_down"], "shared_gate_up": b.shared.dw_gate_up, "shared_down": b.shared.dw_down,
                **b.join_op.grads}
        grads.append({n: have[n] for n in names})
        grads[-1]["router"] = torch.zeros(G, d, device="cuda")
    params = [{**{n: w[n] for n in names}, "router": r} for w, names, r in zip(weights, used, routers)]
    flat = [(i, n) for i, p in enumerate(params) for n in p]
    master = {(i, n): params[i][n].float().clone() for i, n in flat}
    opt = AdamW([{"p": master[i, n], "g": grads[i][n], **AdamW.states(master[i, n]),
                  **({"copy": params[i][n]} if params[i][n].dtype is torch.bfloat16 else {})} for i, n in flat])
    clip = GradNorm([{"g": grads[i][n]} for i, n in flat])
    for step in (1, 2):
        x, d_out = rnd(T, d).bfloat16(), rnd(T, d).bfloat16()
        leaf = {(i, n): params[i][n].to(D).requires_grad_() for i, n in flat}
        x0 = x.to(D).requires_grad_()
        # the framework
        n, stream, kept, total = blocks[0].norm(x, weights[0]), x, [], torch.zeros(1, device="cuda")
        for b, w, r in zip(blocks, weights, routers):
            b.n = n
            logits = n.float() @ r.T
            out = b.experts(logits, w).clone()
            total = total + b.router_loss(logits)[:1]
            kept.append((n, logits, stream, out))
            stream, n = b.join(stream, out, w)
        ds, dn = d_out, None
        for i in (1, 0):
            b, w, r, (n, logits, stream_in, out) = blocks[i], weights[i], routers[i], kept[i]
            ds, dh = b.join_backward(ds, dn, stream_in, out, w)
            b.n = n
            dn = b.experts_backward(dh, w)
            dl = b.router_backward(logits)
            grads[i]["router"].copy_(dl.T.contiguous() @ n.float())
            dn = (dn.float() + dl @ r).bfloat16()
        dx = blocks[0].norm_backward(dn, x, weights[0], residual=ds)
        # float64, the routing as it is

        def norm(v, kind, wt, bias):
            if kind == "layer":
                v = v - v.mean(1, keepdim=True)
            return v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt() * wt + (0 if bias is None else bias)

        def mlp(rows, gu, down):
            a = rows @ gu.T
            h = gu.shape[0] // 2
            return (torch.nn.functional.silu(a[:, :h]) * a[:, h:]) @ down.T

        n64, s64, loss64 = norm(x0, "layer", leaf[0, "norm_weight"], leaf[0, "norm_bias"]), x0, 0
        for i, (b, j) in enumerate(zip(blocks, joins)):
            l = n64 @ leaf[i, "router"].T
            p, idx = torch.softmax(l, 1), b.path.topk_idx.long()
            h64 = mlp(n64, leaf[i, "shared_gate_up"], leaf[i, "shared_down"])
            for e in range(G):
                we = (p.gather(1, idx) * (idx == e)).sum(1, keepdim=True)
                h64 = h64 + we * mlp(n64, leaf[i, "w_gate_up"][e], leaf[i, "w_down"][e])
            for q in range(R):
                rows = slice(q * T_o, (q + 1) * T_o)
                share = torch.bincount(idx[rows].reshape(-1), minlength=G).to(D) * G / (T_o * k)
                loss64 = loss64 + balance * (share * p[rows].mean(0)).sum() / R
            loss64 = loss64 + z * torch.logsumexp(l, 1).square().mean()
            get = lambda name: leaf.get((i, name))
            s64 = j["residual_scale"] * s64 + get("gate") * norm(h64, j["post"], get("post_weight"), get("post_bias"))
            n64 = norm(s64, j["pre"], get("pre_weight"), get("pre_bias")) if j["pre"] != "none" else None
        ((s64 * d_out.to(D)).sum() + loss64).backward()
        pairs = [("s", stream, s64.detach()), ("dx", dx, x0.grad), ("loss", total[0], loss64.detach())]
        pairs += [((i, n), grads[i][n].view(params[i][n].shape), leaf[i, n].grad) for i, n in flat]
        for name, got, want in pairs:
            assert (got.to(D) - want).norm() <= 24 * 2.0 ** -8 * want.norm(), (step, name)
        # clipped to half of its norm; the optimizer takes the coefficient
        want, _ = ref.grad_norm([grads[i][n] for i, n in flat], 1.0, 1.0)
        total_norm = clip.norm(0.5 * want.item())
        within(total_norm[0], want, 1.001 * E32 * want, "norm")
        before = {q: t.clone() for q, t in master.items()}
        moments = [(t["m"].to(D).clone(), t["v"].to(D).clone()) for t in opt.tensors]
        opt.step(step, 1e-3, grad_scale=clip.scale)
        for (i, n), t, (m, v) in zip(flat, opt.tensors, moments):
            g = grads[i][n].to(D).view(-1) * clip.scale.to(D)
            m, v = 0.9 * m + 0.1 * g, 0.95 * v + 0.05 * g * g
            move = 1e-3 * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.95 ** step)).sqrt() + 1e-8)
            p = before[i, n].to(D).view(-1)
            # m and v to a few roundings of their parts (m: of its terms' sizes), the update to ten, p to one
            e = 10 * E32 * move.abs() + 2e-3 * 8 * E32 + 2 * E32 * p.abs()
            assert ((master[i, n].to(D).view(-1) - (p - move)).abs() <= e).all(), (step, i, n)
            if params[i][n].dtype is torch.bfloat16:
                assert torch.equal(params[i][n], master[i, n].bfloat16())
            else:
                params[i][n].copy_(master[i, n])
    assert all(b.path.status() == B.MOE_OK for b in blocks)


def test_block_with_losses_and_a_join_for_serving():
    """Made without training: the same losses, counts and joined rows, and no gradients."""
    from expert_output_overlap_amd.runtime import MoeBlock, MoePath

    R, T_o, G, k, d, f, fs, M = 2, 40, 4, 2, 128, 128, 192, 16
    T, rnd = R * T_o, gen(23)
    w = {"norm_weight": 1 + 0.1 * rnd(d), "norm_bias": 0.1 * rnd(d), "w_gate_up": (rnd(G, 2 * f, d) / d ** 0.5).bfloat16(),
         "w_down": (rnd(G, d, f) / d ** 0.5).bfloat16(), "shared_gate_up": (rnd(2 * fs, d) / d ** 0.5).bfloat16(),
         "shared_down": (rnd(d, fs) / d ** 0.5).bfloat16(), "gate": rnd(d)}
    x, router, got = rnd(T, d).bfloat16(), rnd(G, d) / d ** 0.5, []
    for train in (True, False):
        b = MoeBlock(MoePath(R, T_o, G, G, k, d, f, M), fs, train=train, losses=dict(z=1e-3), join=dict(post="rms", pre="rms"))
        logits = b.norm(x, w).float() @ router.T
        out = b.experts(logits, w)
        got.append([t.clone() for t in (b.router_loss(logits), b.losses_op.counts, *b.join(x, out, w))])
    assert all(torch.equal(a, c) for a, c in zip(*got))
    for call in (lambda: b.router_backward(logits), lambda: b.join_backward(x, x, x, out, w)):
        with pytest.raises(RuntimeError, match="train"):
            call()


def test_block_without_losses_or_a_join_says_so():
    from expert_output_overlap_amd.runtime import MoeBlock, MoePath

    b = MoeBlock(MoePath(1, 16, 4, 4, 2, 128, 128, 16), 64)
    x = torch.zeros(16, 128, device="cuda", dtype=torch.bfloat16)
    for call, name in ((lambda: b.router_loss(x), "losses"), (lambda: b.router_backward(x), "losses"), (lambda: b.join(x, x, {}), "join"),
                       (lambda: b.join_backward(x, x, x, x, {}), "join")):
        with pytest.raises(RuntimeError, match="made without %s=" % name):
            call()
