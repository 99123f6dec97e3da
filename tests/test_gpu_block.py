"""The operators around the routed experts on the GPU against 64-bit formulas, with bounds counted from their roundings."""
import pytest
import torch

import block_reference as ref
from expert_output_overlap_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def spread(t, pad):
    """t's rows as a slice of a wider tensor, whose other elements are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def check(got, want, names, tag):
    for n in names:
        ref.within(got[n], *want[n], (tag, n))


# ---- layer norm --------------------------------------------------------------------------------------------------

def norm_case(rows, d, dtype, params, pad=0, seed=0, residual=True):
    from expert_output_overlap_amd.runtime import LayerNorm

    rnd = gen(1000 + seed)
    dt, pt = DT[dtype], DT[params]
    x = (rnd(rows, d) * torch.exp(0.5 * rnd(d)) + 3 * rnd(d)).to(dt)
    x[:, :: 37] *= 16
    w, b = (1 + 0.2 * rnd(d)).to(pt), (0.1 * rnd(d)).to(pt)
    dy, res = rnd(rows, d).to(dt), rnd(rows, d).to(dt) if residual else None
    if pad:
        x, dy = spread(x, pad), spread(dy, pad + 1)
    op = LayerNorm(rows, d, dtype, params)
    y = op.forward(x, w, b)
    dx = op.backward(dy, x, w, residual=res)
    got = {"y": y, "dx": dx, "dweight": op.dweight, "dbias": op.dbias}
    return op, (x, w, b, dy, res), got, ref.layer_norm(x, w, b, 1e-5, dy, res)


NORM_SIZES = [(1, 64), (1, 7168), (3, 1), (5, 7), (17, 65), (300, 512), (70, 513), (33, 1024), (40, 1407), (64, 2048),
              (9, 2049), (700, 4096), (21, 7168), (2000, 5000), (13, 8192), (7, 8193), (6, 16383), (5, 16384), (9000, 96)]


@pytest.mark.parametrize("rows,d", NORM_SIZES)
@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_norm(rows, d, dtype, params):
    _, _, got, want = norm_case(rows, d, dtype, params, pad=(rows + d) % 3)
    check(got, want, ("y", "dx", "dweight", "dbias"), (rows, d, dtype, params))


@pytest.mark.parametrize("rows,d", [(1100, 16384), (1031, 8200), (1500, 12001)])
@pytest.mark.parametrize("dtype,params", [("bf16", "f32"), ("f32", "f32")])
def test_norm_of_many_wide_rows(rows, d, dtype, params):
    """Rows of more than 8192 elements, several for each group of threads, and again into the same buffers."""
    op, (x, w, b, dy, res), got, want = norm_case(rows, d, dtype, params, pad=1, seed=3)
    check(got, want, ("y", "dx", "dweight", "dbias"), (rows, d, dtype, params))
    first = {k: v.clone() for k, v in got.items()}
    op.forward(x, w, b)
    op.backward(dy, x, w, residual=res)
    assert all(torch.equal(first[k], got[k]) for k in first)


def test_norm_is_the_same_each_time_and_in_place():
    op, (x, w, b, dy, res), got, _ = norm_case(1500, 1536, "bf16", "f32", residual=True)
    first = {k: v.clone() for k, v in got.items()}
    for _ in range(2):
        op.forward(x, w, b)
        op.backward(dy, x, w, residual=res)
        assert all(torch.equal(first[k], got[k]) for k in first)
    dy2, res2, x2 = dy.clone(), res.clone(), x.clone()
    op.backward(dy2, x, w, residual=res, dx=dy2)
    assert torch.equal(dy2, first["dx"])
    op.backward(dy, x, w, residual=res2, dx=res2)
    assert torch.equal(res2, first["dx"])
    assert torch.equal(op.forward(x2, w, b, y=x2), first["y"])


def test_norm_leaves_what_is_not_its_own():
    """Fewer rows than the buffers hold, results as slices: everything else stays."""
    from expert_output_overlap_amd.runtime import LayerNorm

    rnd = gen(3)
    op = LayerNorm(64, 96, "bf16", "f32")
    x, w = rnd(10, 96).bfloat16(), 1 + rnd(96)
    y = torch.full((10, 130), 7.0, device="cuda", dtype=torch.bfloat16)
    for t in (op.y, op.dx, op.mean, op.rstd):
        t.fill_(7.0)
    op.forward(x, w, None, y=y[:, 17:113])
    assert (y[:, :17] == 7).all() and (y[:, 113:] == 7).all() and (op.y == 7).all() and (op.mean[10:] == 7).all()
    op.backward(y[:, 17:113], x, w)
    assert (op.dx[10:] == 7).all() and not (op.dx[:10] == 7).all()
    want = ref.layer_norm(x, w, torch.zeros(96, device="cuda"), 1e-5)
    ref.within(y[:, 17:113], *want["y"], "y")


def test_norm_between_its_own_rows():
    """x, y, dy and dx as slices of one wide tensor."""
    from expert_output_overlap_amd.runtime import LayerNorm

    rnd = gen(5)
    op = LayerNorm(33, 96, "bf16", "f32")
    wide = torch.empty(33, 4 * 96 + 1, device="cuda", dtype=torch.bfloat16).copy_(rnd(33, 4 * 96 + 1))
    x, y, dy, dx = (wide[:, 96 * i: 96 * (i + 1)] for i in (1, 0, 3, 2))
    x0, dy0, w, b = x.clone(), dy.clone(), 1 + rnd(96), rnd(96)
    last = wide[:, -1].clone()
    op.forward(x, w, b, y=y)
    op.backward(dy, x, w, dx=dx)
    want = ref.layer_norm(x0, w, b, 1e-5, dy0)
    check({"y": y, "dx": dx, "dweight": op.dweight, "dbias": op.dbias}, want, ("y", "dx", "dweight", "dbias"), "slices")
    assert torch.equal(x, x0) and torch.equal(dy, dy0) and torch.equal(wide[:, -1], last)


def test_norm_of_nothing_and_without_parameters():
    from expert_output_overlap_amd.runtime import LayerNorm

    rnd = gen(4)
    op = LayerNorm(8, 200, "f32", "f32")
    none = torch.empty(0, 200, device="cuda")
    op.dweight.fill_(5.0)
    op.dbias.fill_(5.0)
    assert op.forward(none).shape == (0, 200)
    op.backward(none, none)
    assert (op.dweight == 0).all() and (op.dbias == 0).all()
    x, dy = rnd(8, 200), rnd(8, 200)
    one, zero = torch.ones(200, device="cuda"), torch.zeros(200, device="cuda")
    want = ref.layer_norm(x, one, zero, 1e-5, dy)
    got = {"y": op.forward(x), "dx": op.backward(dy, x), "dweight": op.dweight, "dbias": op.dbias}
    check(got, want, ("y", "dx", "dweight", "dbias"), "no parameters")


def test_norm_of_constant_and_bad_rows():
    """A row without variance gives its bias; a NaN or an infinity stays in its own row."""
    from expert_output_overlap_amd.runtime import LayerNorm

    rnd = gen(5)
    x = rnd(6, 768)
    x[1] = 3.25
    x[3, 5] = float("nan")
    x[4, 700] = float("inf")
    w, b = 1 + 0.1 * rnd(768), rnd(768)
    op = LayerNorm(6, 768, "f32", "f32")
    y = op.forward(x, w, b)
    assert torch.equal(y[1], b) and torch.isnan(y[3]).all() and not torch.isfinite(y[4]).any()
    good = [0, 2, 5]
    ref.within(y[good], *ref.layer_norm(x[good], w, b, 1e-5)["y"], "good rows")


# ---- the shared expert -------------------------------------------------------------------------------------------

def ffn_case(T, d, f, dtype, seed=0):
    rnd = gen(2000 + seed)
    dt = DT[dtype]
    x, res, dy = (rnd(T, d).to(dt) for _ in range(3))
    return x, (rnd(2 * f, d) / d ** 0.5).to(dt), (rnd(d, f) / d ** 0.5).to(dt), res, dy


FFN_SIZES = [(1, 64, 64), (1, 1, 1), (1, 7168, 256), (2, 100, 36), (5, 333, 517), (16, 512, 200), (17, 256, 1408), (31, 65, 8),
             (64, 1024, 512), (65, 128, 320), (100, 8, 520), (129, 72, 1032), (200, 2048, 1408), (255, 320, 257),
             (256, 256, 256), (301, 333, 517), (512, 512, 384), (777, 640, 136), (1030, 264, 648), (2049, 136, 72)]


@pytest.mark.parametrize("T,d,f", FFN_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_ffn(T, d, f, dtype):
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, dy = ffn_case(T, d, f, dtype)
    serve = SharedFFN(T, d, f, dtype, train=False)
    want = ref.shared_ffn(x, wgu, wd, residual=res)
    ref.within(serve.forward(x, wgu, wd, residual=res), *want["y"], ("y + residual", T, d, f))
    op = SharedFFN(T, d, f, dtype)
    want = ref.shared_ffn(x, wgu, wd, residual=res, dy=dy)
    got = {"y": op.forward(x, wgu, wd), "dx": op.backward(dy, x, wgu, wd, residual=res), "dw_gate_up": op.dw_gate_up,
           "dw_down": op.dw_down}
    check(got, want, ("y", "dx", "dw_gate_up", "dw_down"), (T, d, f, dtype))


@pytest.mark.parametrize("T,d,f,dtype", [(4096, 1024, 768, "bf16"), (3, 2048, 5632, "bf16"), (40, 4096, 3000, "bf16"),
                                         (1500, 2000, 1000, "bf16"), (600, 700, 800, "f32"),
                                         (2, 192, 6895, "f32"), (2, 192, 13790, "bf16"), (20, 48, 9001, "bf16"),
                                         (50, 4096, 64, "bf16"), (60, 264, 6000, "f32"), (300, 7168, 520, "bf16")])
def test_shared_ffn_larger(T, d, f, dtype):
    """Sizes where the products split, or fill the device several times; the same call twice gives the same bits."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, dy = ffn_case(T, d, f, dtype, seed=1)
    op = SharedFFN(T, d, f, dtype)
    want = ref.shared_ffn(x, wgu, wd, residual=res, dy=dy)
    got = {"y": op.forward(x, wgu, wd), "dx": op.backward(dy, x, wgu, wd, residual=res), "dw_gate_up": op.dw_gate_up,
           "dw_down": op.dw_down}
    check(got, want, ("y", "dx", "dw_gate_up", "dw_down"), (T, d, f, dtype))
    first = {k: v.clone() for k, v in got.items()}
    op.forward(x, wgu, wd)
    op.backward(dy, x, wgu, wd, residual=res)
    assert all(torch.equal(first[k], got[k]) for k in first)


@pytest.mark.parametrize("T,d,f,dtype", [(1, 256, 512, "bf16"), (48, 200, 100, "bf16"), (300, 512, 256, "bf16"),
                                         (50, 33, 65, "f32")])
def test_shared_ffn_in_place_and_fewer_tokens(T, d, f, dtype):
    """y over the residual, dx over its residual; rows behind the last token stay as they were."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, dy = ffn_case(T, d, f, dtype, seed=2)
    op = SharedFFN(T + 37, d, f, dtype)
    for t in (op.y, op.h, op.gu, op.dgu, op.dx):
        t.fill_(7.0)
    want, wante = ref.shared_ffn(x, wgu, wd, residual=res, dy=dy), ref.shared_ffn(x, wgu, wd, residual=res)
    y = res.clone()
    op.forward(x, wgu, wd, residual=y, y=y)
    ref.within(y, *wante["y"], "y over its residual")
    dx = res.clone()
    op.backward(dy, x, wgu, wd, residual=dx, dx=dx)
    check({"dx": dx, "dw_gate_up": op.dw_gate_up, "dw_down": op.dw_down}, want, ("dx", "dw_gate_up", "dw_down"), "in place")
    for t in (op.h, op.gu, op.dgu):
        assert (t[T:] == 7).all()
    assert (op.y == 7).all() and (op.dx == 7).all()


@pytest.mark.parametrize("d,f", [(100, 36), (7, 9), (104, 41), (65, 8)])
@pytest.mark.parametrize("T,dtype", [(2, "bf16"), (70, "bf16"), (40, "f32")])
def test_shared_ffn_writes_only_its_outputs(T, d, f, dtype):
    """Outputs inside larger buffers: what lies before and behind them stays (odd widths, whose padding has no place)."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, dy = ffn_case(T, d, f, dtype, seed=6)
    op = SharedFFN(T, d, f, dtype)
    wide = []

    def inside(t):
        at = torch.full((t.numel() + 8192,), 7.0, dtype=t.dtype, device="cuda")
        wide.append((at, 4096, t.numel()))
        return at[4096: 4096 + t.numel()].view(t.shape)

    op.y, op.dx, op.dw_gate_up, op.dw_down, op.h, op.gu, op.dgu = (
        inside(t) for t in (op.y, op.dx, op.dw_gate_up, op.dw_down, op.h, op.gu, op.dgu))
    op.forward(x, wgu, wd)
    op.backward(dy, x, wgu, wd, residual=res)
    for at, a, n in wide:
        assert (at[:a] == 7).all() and (at[a + n:] == 7).all()
    want = ref.shared_ffn(x, wgu, wd, residual=res, dy=dy)
    check({"y": op.y, "dx": op.dx, "dw_gate_up": op.dw_gate_up, "dw_down": op.dw_down}, want,
          ("y", "dx", "dw_gate_up", "dw_down"), (T, d, f, dtype))


@pytest.mark.parametrize("T,d,f", [(2, 100, 36), (40, 24, 33), (70, 100, 36), (300, 65, 9), (20, 64, 4), (90, 72, 68)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_ffn_does_not_read_what_it_has_not_written(T, d, f, dtype):
    """Buffers and workspace full of NaN before the calls: the padding of their rows reaches no result."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, dy = ffn_case(T, d, f, dtype, seed=8)
    op = SharedFFN(T, d, f, dtype)
    for t in (op.y, op.h, op.gu, op.dgu, op.dx, op.dw_gate_up, op.dw_down):
        t.fill_(float("nan"))
    if op.workspace is not None:
        op.workspace.fill_(255)
    want = ref.shared_ffn(x, wgu, wd, residual=res, dy=dy)
    got = {"y": op.forward(x, wgu, wd), "dx": op.backward(dy, x, wgu, wd, residual=res), "dw_gate_up": op.dw_gate_up,
           "dw_down": op.dw_down}
    check(got, want, ("y", "dx", "dw_gate_up", "dw_down"), (T, d, f, dtype))


def test_shared_ffn_of_nothing():
    from expert_output_overlap_amd.runtime import SharedFFN

    for dtype in ("bf16", "f32"):
        _, wgu, wd, _, _ = ffn_case(1, 72, 40, dtype)
        op = SharedFFN(4, 72, 40, dtype)
        none = torch.empty(0, 72, device="cuda", dtype=DT[dtype])
        op.dw_gate_up.fill_(3.0)
        op.dw_down.fill_(3.0)
        assert op.forward(none, wgu, wd).shape == (0, 72)
        op.backward(none, none, wgu, wd)
        assert (op.dw_gate_up == 0).all() and (op.dw_down == 0).all()


@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (20, "bf16"), (150, "bf16"), (30, "f32")])
def test_shared_ffn_bad_tokens_stay_in_their_rows(T, dtype):
    """A token of NaN changes no other token's output, nor what lies in buffers that no row of this call owns."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, _ = ffn_case(T, 136, 200, dtype, seed=3)
    op = SharedFFN(T, 136, 200, dtype)
    if op.workspace is not None:
        op.workspace.fill_(255)  # NaN patterns
    y = op.forward(x, wgu, wd, residual=res).clone()
    assert torch.isfinite(y).all()
    if T > 1:
        x[T // 2] = float("nan")
        z = op.forward(x, wgu, wd, residual=res)
        keep = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(z[keep], y[keep]) and torch.isnan(z[T // 2]).all()


@pytest.mark.parametrize("T,d,f", [(5, 100, 36), (40, 64, 41), (70, 100, 36), (300, 65, 9), (300, 72, 41), (40, 128, 1001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_shared_ffn_padding_of_bad_tokens(T, d, f, dtype, bad):
    """h, g | u and dg | du past f are 0 in every row, that of a token that is not finite too."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, _, dy = ffn_case(T, d, f, dtype, seed=14)
    x[T // 2, d // 3] = dy[T // 3, d // 2] = bad
    op = SharedFFN(T, d, f, dtype)
    for t in (op.h, op.gu, op.dgu):
        t.fill_(7.0)
    op.forward(x, wgu, wd)
    op.backward(dy, x, wgu, wd)
    F = op.h.shape[1]
    for t in (op.h, op.gu[:, :F], op.gu[:, F:], op.dgu[:, :F], op.dgu[:, F:]):
        assert (t[:, f:] == 0).all()
    assert not torch.isfinite(op.h[T // 2, :f]).all() and not torch.isfinite(op.dgu[T // 3, :f]).all()


def test_shared_ffn_gradients_against_differences():
    """f32: the backward call against central differences of the forward call, in a few directions.  With a step of 2^-7 the
    difference's own error is the third derivative's 2^-14 / 6 of the loss' size along unit directions, and the forward's
    rounding (2^-22 of the loss' terms) over the step: 2^-12 of the loss' terms together bounds both."""
    from expert_output_overlap_amd.runtime import SharedFFN

    T, d, f = 37, 48, 56
    x, wgu, wd, _, dy = ffn_case(T, d, f, "f32", seed=4)
    op = SharedFFN(T, d, f, "f32")
    op.forward(x, wgu, wd)
    grads = (op.backward(dy, x, wgu, wd).clone(), op.dw_gate_up.clone(), op.dw_down.clone())
    terms = (op.forward(x, wgu, wd).double() * dy.double()).norm().item()
    rnd, h = gen(9), 2.0 ** -7
    for k, grad in enumerate(grads):
        v = rnd(*grad.shape)
        v = v / v.norm()
        at = [[x, wgu, wd], [x, wgu, wd]]
        at[0][k], at[1][k] = at[0][k] + h * v, at[1][k] - h * v
        up, down = ((op.forward(*a).double() * dy.double()).sum().item() for a in at)
        want = (up - down) / (2 * h)
        assert abs((grad.double() * v.double()).sum().item() - want) <= 2.0 ** -12 * (terms + abs(want)) , k


# Sizes that take every tile of the bf16 products, whole and in k-splits, with rows, columns and k that no tile divides; widths
# of whole eights (operands as they are) and others (packed).  tests/test_block_tiles.py holds them to that.
TILE_SIZES = [(13165, 34, 528), (16633, 40, 136), (8503, 199, 144), (3061, 2021, 32), (35, 707, 39), (11205, 1834, 37),
              (17029, 391, 34), (17273, 136, 41), (8203, 136, 212), (3327, 40, 1800), (35, 37, 738), (16655, 132, 148),
              (5521, 129, 2480), (65, 3739, 5512), (259, 2506, 777), (139, 3512, 2937), (443, 7425, 218), (129, 2576, 1144),
              (39, 6559, 133), (35, 797, 1256), (39, 32, 368), (1055, 64, 3816), (665, 5136, 392), (14219, 72, 600),
              (2049, 2056, 1416), (4920, 3304, 8), (10834, 12, 1889), (16487, 4398, 71), (137, 11126, 6352), (130, 6147, 11321)]


@pytest.mark.parametrize("T,d,f", TILE_SIZES)
def test_shared_ffn_tiles(T, d, f):
    """Every tile against the formulas: outputs and workspace inside larger buffers and full of NaN before the calls, y and dx over
    their residuals; the same bits at a second call."""
    from expert_output_overlap_amd.runtime import SharedFFN

    x, wgu, wd, res, dy = ffn_case(T, d, f, "bf16", seed=13)
    op, wide = SharedFFN(T, d, f), []

    def inside(t, fill=float("nan")):
        at = torch.full((t.numel() + 8192,), 7, dtype=t.dtype, device="cuda")
        at[4096: 4096 + t.numel()] = fill
        wide.append((at, 4096, t.numel()))
        return at[4096: 4096 + t.numel()].view(t.shape)

    op.dw_gate_up, op.dw_down, op.h, op.gu, op.dgu = (inside(t) for t in (op.dw_gate_up, op.dw_down, op.h, op.gu, op.dgu))
    y, dx = inside(op.y), inside(op.dx)
    op.workspace = inside(op.workspace, 255)
    wante, want, first = ref.shared_ffn(x, wgu, wd, residual=res), ref.shared_ffn(x, wgu, wd, residual=res, dy=dy), None
    for _ in range(2):
        y.copy_(res)
        dx.copy_(res)
        op.forward(x, wgu, wd, residual=y, y=y)
        op.backward(dy, x, wgu, wd, residual=dx, dx=dx)
        got = {"dx": dx, "dw_gate_up": op.dw_gate_up, "dw_down": op.dw_down, "y": y}
        if first is None:
            check(got, {**want, "y": wante["y"]}, got, (T, d, f))
            for name, v in got.items():  # sums of thousands: the worst case's bound is wide, the norm's is not (4 roundings in a row)
                exact = wante["y"][0] if name == "y" else want[name][0]
                assert (v.double() - exact).norm() <= 4 * 2.0 ** -8 * exact.norm(), (name, T, d, f)
            first = {k: v.clone() for k, v in got.items()}
        assert all(torch.equal(first[k], got[k]) for k in first)
    for at, a, n in wide:
        assert (at[:a] == 7).all() and (at[a + n:] == 7).all()
    for t in (op.h, op.gu[:, : op.gu.shape[1] // 2], op.gu[:, op.gu.shape[1] // 2:], op.dgu[:, : op.dgu.shape[1] // 2],
              op.dgu[:, op.dgu.shape[1] // 2:]):
        assert (t[:, f:] == 0).all()


def test_shared_ffn_of_nothing_with_wide_weights():
    """2^32 elements of dw_gate_up, one more than a launch has threads: they become 0 all the same."""
    from expert_output_overlap_amd.runtime import SharedFFN

    d, f = 65536, 32768
    op = SharedFFN(1, d, f)
    wgu, wd = (torch.empty_like(t) for t in (op.dw_gate_up, op.dw_down))
    none = torch.empty(0, d, device="cuda", dtype=torch.bfloat16)
    op.dw_gate_up.fill_(3.0)
    op.dw_down.fill_(3.0)
    op.backward(none, none, wgu, wd)
    assert not op.dw_gate_up.any() and not op.dw_down.any()


def test_shared_ffn_of_more_pieces_than_a_launch_has_threads():
    """x and dy of an odd width whose packed copies are 2^32 pieces of 16 bytes, zeros but for a few rows (x serves as dy too).
    A sum of 65535 products makes the worst-case bounds as large as the results, so these are held in the norm: at most three
    roundings to bf16 in a row, each 2^-8 at most and of random sign."""
    T, d, f = 262144, 65535, 8
    shape = B.moe_shared_shape(T, d, f, B.MOE_BF16)
    need = B.moe_shared_ffn_workspace_bytes(shape, True)
    if torch.cuda.mem_get_info()[0] < need + 2 * (2 * T * d) + (8 << 30):
        pytest.skip("%d GiB of device memory wanted" % ((need + 4 * T * d >> 30) + 8))
    _, wgu, wd, _, _ = ffn_case(1, d, f, "bf16", seed=9)
    rows = torch.tensor([0, 1, T // 2 + 1, T - 1], device="cuda")
    some = gen(12)(4, d).bfloat16()
    x, dx = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16), torch.empty(T, d, device="cuda", dtype=torch.bfloat16)
    x[rows] = some
    gu, h = torch.zeros(T, 2 * f, device="cuda"), torch.zeros(T, f, device="cuda", dtype=torch.bfloat16)
    gu[rows] = (some.double() @ wgu.double().T).float()
    g, u = gu[rows].double().chunk(2, 1)
    h[rows] = (g * torch.sigmoid(g) * u).bfloat16()
    dw_gate_up, dw_down = torch.empty_like(wgu), torch.empty_like(wd)
    workspace = torch.empty(need, device="cuda", dtype=torch.uint8)
    B.moe_shared_ffn_backward(shape, {"x": x, "w_gate_up": wgu, "w_down": wd, "h": h, "gu": gu, "dy": x,
                                      "dgu_ws": torch.empty(T, 2 * f, device="cuda", dtype=torch.bfloat16), "dx": dx,
                                      "dw_gate_up": dw_gate_up, "dw_down": dw_down}, workspace)
    want = ref.shared_ffn(some, wgu, wd, dy=some)
    for name, got in (("dx", dx[rows]), ("dw_gate_up", dw_gate_up), ("dw_down", dw_down)):
        assert (got.double() - want[name][0]).norm() <= 3 * 2.0 ** -8 * want[name][0].norm(), name
    dx[rows] = 0.0
    assert not any(part.any() for part in dx.split(T // 16))


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("d,f", [(2080, 65536), (2080, 65535), (65536, 2080), (65535, 2080)])
def test_shared_ffn_few_tokens_sum_in_two_levels(T, d, f):
    """f32: sums of up to 8192 products in a wave, the first of them 1 and the others 2^-27.  A running sum loses the others (four
    products at a time reach 2^-25, half of what it can hold): 2^-14 of the result.  Sums of 256 at a time that are added up
    then round 256 + 32 times in a wave, then over eight waves: at most 304 x 2^-24 of the result, 2^-15.7, and silu's 2^-20."""
    from expert_output_overlap_amd.runtime import SharedFFN

    k = torch.arange(max(d, f), device="cuda")
    terms = torch.where((k < 256) & (k % 32 == 0), 1.0, 2.0 ** -27)  # the first of each wave's
    silu = torch.sigmoid(torch.tensor(1.0, dtype=torch.float64)).item()
    wgu, wd = torch.zeros(2 * f, d, device="cuda"), torch.zeros(d, f, device="cuda")
    if f > d:  # h = silu(1) terms, y its sum
        x = torch.zeros(T, d, device="cuda")
        x[:, 0] = 1.0
        wgu[:f, 0], wgu[f:, 0] = 1.0, terms
        wd.fill_(1.0)
    else:  # u the terms' sum, y = h
        x = torch.ones(T, d, device="cuda")
        wgu[:f, 0] = 1.0
        wgu[f:] = terms[:d]
        wd[k[:d], k[:d] % f] = 1.0
    want = torch.full((T, d), silu * terms[:max(d, f)].double().sum().item(), dtype=torch.float64, device="cuda")
    y = SharedFFN(T, d, f, "f32", train=False).forward(x, wgu, wd)
    ref.within(y, want, (304 * ref.E32 + 2.0 ** -20) * want, (T, d, f))


# ---- AdamW -------------------------------------------------------------------------------------------------------

def adam_tensors(sizes, bits, params, grads, seed=0, values=True):
    """Tensors in odd places of shared buffers; steps of very different sizes."""
    from expert_output_overlap_amd.runtime import AdamW

    rnd = gen(3000 + seed)
    got = []
    for i, n in enumerate(sizes):
        def at(dtype, shift):  # an address that is aligned to its elements only
            return torch.zeros(n + 8, device="cuda", dtype=dtype)[shift: shift + n]

        size = 1e-3 * torch.exp(2 * rnd(n))
        t = {"p": at(torch.bfloat16 if params == "bf16" else torch.float32, i % 3), "g": at(DT[grads], i % 2)}
        t["p"].copy_(rnd(n))
        t["g"].copy_(rnd(n) * size)
        if params == "master":
            t["copy"] = at(torch.bfloat16, i % 5)
        t.update(AdamW.states(t["p"], bits))
        if bits == 32:
            t["m"].copy_(rnd(n) * size)
            t["v"].copy_((size * (0.5 + rnd(n).abs())) ** 2)
        elif values:
            t["m_values"], t["root_values"] = at(torch.bfloat16, 1), at(torch.bfloat16, 2)
        t["weight_decay"], t["lr_scale"] = 0.1 * (i % 2), 1.0 - 0.25 * (i % 3)
        got.append(t)
    return got


HYPER = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8)


def adam_want(t, step, scale=1.0, lr=1e-3):
    D = torch.float64
    if t["m"].dtype is torch.uint8:
        m, v = ref.m_values(t["m"], t["m_scale"]), ref.root_values(t["v"], t["v_scale"]).square()
    else:
        m, v = t["m"].to(D), t["v"].to(D)
    return ref.adamw(t["p"].reshape(-1).to(D), t["g"].reshape(-1).to(D), m, v, step, lr * t["lr_scale"], *HYPER["betas"], HYPER["eps"],
                     t["weight_decay"], scale)


def on_codes(value, scale, bits, low, most, floor, e, what, want):
    """8-bit values: half a step of their code's binade off the 64-bit state at most (or up to the smallest code), and the
    scale the smallest at which the block fits."""
    n = want.numel()
    s = ref.power(scale.long() - 127).repeat_interleave(ref.BLOCK)[:n]
    z = want.abs() / s
    # a value that rounds up across a binade is half a step of the lower one off at most, so the binade of z counts
    step = 2.0 ** (torch.floor(torch.log2(z.clamp(min=1e-300))).clamp(min=low) - bits)
    bound = s * step / 2 + e
    if floor:
        bound = torch.where((z > 0) & (z < 2.0 ** low * (1 + 2.0 ** -bits)), s * 2.0 ** low * (1 + 2.0 ** -bits), bound)
    ref.within(value, want, bound, what)
    if n:
        pad = torch.zeros(-n % ref.BLOCK, device="cuda", dtype=torch.float64)
        top = torch.cat([z, pad]).view(-1, ref.BLOCK).amax(1)
        assert (top <= most * (1 + 2.0 ** -20)).all(), what
        least = 16 if floor else 1
        assert ((top > most / 2 * (1 - 2.0 ** -20)) | (scale == least)).all(), what


SIZES = [1, 0, 31, 32, 33, 4096, 4097, 1000, 5, 12289, 64, 100003]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("params,grads", [("master", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_adamw(bits, params, grads):
    from expert_output_overlap_amd.runtime import AdamW

    ts = adam_tensors(SIZES, bits, params, grads)
    op = AdamW(ts, betas=HYPER["betas"], eps=HYPER["eps"])
    clip = torch.tensor([0.37], device="cuda")
    for step in (1, 2, 3):
        scale = 1.0 if step == 1 else float(clip)
        want = [adam_want(t, step, scale) for t in ts]
        op.step(step, HYPER["lr"], grad_scale=None if step == 1 else clip)
        op.read_states()
        for t, ((p, ep), (m, em), (v, ev)) in zip(ts, want):
            tag = (bits, params, grads, step, p.numel())
            ref.within(t["p"], p, ep + ref.half_step(t["p"].dtype) * p.abs(), tag + ("p",))
            if "copy" in t:
                assert torch.equal(t["copy"], t["p"].bfloat16()), tag
            if bits == 32:
                ref.within(t["m"], m, em, tag + ("m",))
                ref.within(t["v"], v, ev, tag + ("v",))
                continue
            mv, rv = ref.m_values(t["m"], t["m_scale"]), ref.root_values(t["v"], t["v_scale"])
            assert torch.equal(t["m_values"].double(), mv) and torch.equal(t["root_values"].double(), rv), tag
            on_codes(mv, t["m_scale"], 3, -6, 448.0, False, em, tag + ("m",), m)
            on_codes(rv, t["v_scale"], 4, -15, 1.875, True, v.sqrt() * 6 * ref.E32, tag + ("root",), v.sqrt())
            assert ((t["v"] > 0) == (v > 0)).all(), tag  # no divisor becomes zero


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_values_that_are_not_finite(bits):
    """They stay where they are: the other elements of their tensor and of their block go on as without them."""
    from expert_output_overlap_amd.runtime import AdamW

    a = adam_tensors([200], bits, "f32", "f32", seed=1, values=False)[0]
    bad = [3, 40, 41]
    for k in ("g",) if bits == 8 else ("g", "m", "v"):
        a[k][bad] = 0.0
    b = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    b["g"][bad] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")
    ok = torch.ones(200, dtype=torch.bool, device="cuda")
    ok[bad] = False
    opa, opb = AdamW([a], betas=HYPER["betas"]), AdamW([b], betas=HYPER["betas"])
    for step in (1, 2):
        opa.step(step, 1e-3)
        opb.step(step, 1e-3)
        assert torch.isnan(b["p"][bad]).all()
        for k in ("p", "m", "v"):
            assert torch.equal(a[k][ok], b[k][ok]), k
        if bits == 8:
            assert ((b["m"][bad] & 0x7F) == 0x7F).all() and (b["v"][bad] == 255).all()
            assert torch.equal(a["m_scale"], b["m_scale"]) and torch.equal(a["v_scale"], b["v_scale"])


def test_adamw_of_tiny_gradients():
    """No eps, and squares among the subnormals: with m and v from one gradient the update is lr.  v = 0.05 (1e-20)^2 = 5e-42
    holds two roundings of 2^-150 = 7e-46 at most, a relative 3e-4 of it and 1.5e-4 of its root; 2e-4 with fp32's own."""
    from expert_output_overlap_amd.runtime import AdamW

    t = {"p": torch.zeros(300, device="cuda"), "g": torch.full((300,), 1e-20, device="cuda")}
    t.update(AdamW.states(t["p"]))
    AdamW([t], betas=HYPER["betas"], eps=0.0).step(1, 1e-3)
    ref.within(t["p"], torch.full((300,), -1e-3, device="cuda", dtype=torch.float64), torch.full((300,), 2e-7, device="cuda", dtype=torch.float64), "tiny")


def test_adamw_step_from_the_device():
    """Step and rate from device numbers give the same parameters as from the host, also for a step near 1 and beta2 near 1
    (up to the rounding of 1 - beta^t, the same formula on both sides: one step of it in the update)."""
    from expert_output_overlap_amd.runtime import AdamW

    for step in (1, 7, 100000):
        ts = [adam_tensors([5000], 32, "f32", "f32", seed=2)[0] for _ in range(2)]
        ops = [AdamW([t], betas=(0.9, 0.9999)) for t in ts]
        before = ts[0]["p"].double()
        ops[0].step(step, 3e-4)
        ops[1].step(torch.tensor([step], device="cuda"), torch.tensor([3e-4], device="cuda"))
        up = (ts[0]["p"].double() - before).abs()
        ref.within(ts[1]["p"], ts[0]["p"].double(), 6 * ref.E32 * up + 2 * ref.E32 * ts[0]["p"].double().abs(), step)
        assert torch.equal(ts[0]["m"], ts[1]["m"]) and torch.equal(ts[0]["v"], ts[1]["v"])


# ---- streams, graphs, all of them together -----------------------------------------------------------------------

def test_captured_and_replayed():
    """Every operator captured into one graph; each replay after new inputs equals the eager calls, with eager work between."""
    from expert_output_overlap_amd.runtime import AdamW, LayerNorm, SharedFFN

    T, d, f = 70, 264, 200
    x, wgu, wd, res, dy = ffn_case(T, d, f, "bf16", seed=5)
    w = torch.ones(d, device="cuda")

    def make():
        norm, ffn = LayerNorm(T, d), SharedFFN(T, d, f)
        p = wgu.float().clone()
        t = {"p": p, "g": ffn.dw_gate_up, "copy": torch.empty_like(wgu), **AdamW.states(p, 8)}
        t["m_values"], t["root_values"] = (torch.zeros(p.numel(), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        opt = AdamW([t])
        step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-3, device="cuda")
        out = {}

        def run():
            n = norm.forward(x, w)
            out["y"] = ffn.forward(n, wgu, wd, residual=res)
            out["dn"] = ffn.backward(dy, n, wgu, wd)
            out["dx"] = norm.backward(out["dn"], x, w, residual=dy)
            step.add_(1)
            opt.step(step, lr)
            opt.read_states()
            out.update(p=p, copy=t["copy"], m=t["m_values"], r=t["root_values"], dw=ffn.dw_down, dweight=norm.dweight)

        return run, out

    make()[0]()
    torch.cuda.synchronize()
    eager, want = make()
    captured, got = make()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured()
    rnd = gen(6)
    for _ in range(4):
        x.copy_(rnd(T, d))
        dy.copy_(rnd(T, d))
        torch.cuda.synchronize()
        graph.replay()
        eager()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(want[k], got[k]), k


def test_two_streams_at_once():
    """Two sets of operators on two streams at the same time give what each gives alone."""
    from expert_output_overlap_amd.runtime import LayerNorm, SharedFFN

    sets = []
    for k, (T, d, f) in enumerate([(300, 512, 768), (5, 2048, 1408)]):
        x, wgu, wd, res, dy = ffn_case(T, d, f, "bf16", seed=7 + k)
        norm, ffn, w = LayerNorm(T, d), SharedFFN(T, d, f), torch.ones(d, device="cuda")

        def run(stream=None, x=x, wgu=wgu, wd=wd, dy=dy, norm=norm, ffn=ffn, w=w):
            n = norm.forward(x, w, stream=stream)
            ffn.forward(n, wgu, wd, stream=stream)
            dn = ffn.backward(dy, n, wgu, wd, stream=stream)
            return [ffn.y, norm.backward(dn, x, w, stream=stream), ffn.dw_gate_up, ffn.dw_down, norm.dweight]

        sets.append((run, [t.clone() for t in run()], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(stream) for run, _, stream in sets]
        torch.cuda.synchronize()
        for g, (_, want, _) in zip(got, sets):
            assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_block_together():
    """Two training steps of a pre-norm MoE block: norm, router, routed experts, combine, shared expert, their backward and
    AdamW in 32 and in 8 bits, against float64 autograd.  Each result has passed at most eight roundings to bf16 in a row
    (n, h, y, combine, sum; dy, dgu, dx, sums), each 2^-8 at most and of random sign: 8 x 2^-8 of its norm."""
    from expert_output_overlap_amd.runtime import AdamW, MoeBlock, MoePath

    R, T_o, G, k, d, f, fs, M = 2, 40, 4, 2, 128, 128, 192, 16
    T, D = R * T_o, torch.float64
    rnd = gen(11)
    w = {"norm_weight": 1 + 0.1 * rnd(d), "norm_bias": 0.1 * rnd(d), "w_gate_up": (rnd(G, 2 * f, d) / d ** 0.5).bfloat16(),
         "w_down": (rnd(G, d, f) / d ** 0.5).bfloat16(), "shared_gate_up": (rnd(2 * fs, d) / d ** 0.5).bfloat16(),
         "shared_down": (rnd(d, fs) / d ** 0.5).bfloat16()}
    router = rnd(G, d) / d ** 0.5
    block = MoeBlock(MoePath(R, T_o, G, G, k, d, f, M), fs)
    ffn, norm, bb = block.shared, block.norm_op, block.path.bwd_buffers()
    grads = {"norm_weight": norm.dweight, "norm_bias": norm.dbias, "w_gate_up": bb["dw_gate_up"], "w_down": bb["dw_down"],
             "shared_gate_up": ffn.dw_gate_up, "shared_down": ffn.dw_down}
    master = {n: t.float().clone() for n, t in w.items()}
    tensors = []
    for n, t in w.items():
        q = {"p": master[n], "g": grads[n], **AdamW.states(t, 8 if t.dim() > 1 else 32)}
        q["weight_decay"] = 0.1 if t.dim() > 1 else 0.0
        if t.dtype is torch.bfloat16:
            q["copy"] = t
        tensors.append(q)
    opt = AdamW(tensors)
    for step in (1, 2):
        x, d_out = rnd(T, d).bfloat16(), rnd(T, d).bfloat16()
        leaf = {n: t.to(D).requires_grad_() for n, t in w.items()}
        xl = x.to(D).requires_grad_()
        # the framework
        n = block.norm(x, w)
        logits = n.float() @ router.T
        out = block.experts(logits, w).clone()
        idx, wt = block.path.topk_idx.long(), block.path.topk_w.to(D)
        dn = block.experts_backward(d_out, w)
        dx = block.norm_backward(dn, x, w, residual=d_out)
        # float64, the routing as it is
        mu = xl.mean(1, keepdim=True)
        nl = (xl - mu) / ((xl - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * leaf["norm_weight"] + leaf["norm_bias"]

        def mlp(rows, gu, down):
            a = rows @ gu.T
            h = gu.shape[0] // 2
            return (torch.nn.functional.silu(a[:, :h]) * a[:, h:]) @ down.T

        want = mlp(nl, leaf["shared_gate_up"], leaf["shared_down"])
        for e in range(G):
            we = (wt * (idx == e)).sum(1, keepdim=True)
            want = want + we * mlp(nl, leaf["w_gate_up"][e], leaf["w_down"][e])
        (want * d_out.to(D)).sum().backward()
        pairs = [("out", out, want.detach()), ("dx", dx, xl.grad + d_out.to(D))]
        pairs += [(name, grads[name].view(t.shape), leaf[name].grad) for name, t in w.items()]
        for name, got, exp in pairs:
            assert (got.to(D) - exp).norm() <= 8 * 2.0 ** -8 * exp.norm(), (step, name)
        before = {name: t.clone() for name, t in master.items()}
        moved = [adam_want({**q, "lr_scale": 1.0}, step) for q in tensors]
        opt.step(step, 1e-3)
        for (name, t), ((p, ep), _, _) in zip(master.items(), moved):
            assert not torch.equal(t, before[name])
            ref.within(t.view(-1), p, ep + ref.E32 * p.abs(), (step, name))
            if w[name].dtype is torch.bfloat16:
                assert torch.equal(w[name], t.bfloat16())
            else:
                w[name].copy_(t)
    assert block.path.status() == B.MOE_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_without_training(dtype):
    """A block made for serving: its output against float64 (roundings as in test_block_together; fp32: 2^-24 each, sums of 128 and
    192 products: 2^-16 of the norm), no gradients, and an output that its calls give again."""
    from expert_output_overlap_amd.runtime import MoeBlock, MoePath

    R, T_o, G, k, d, f, fs, M = 2, 40, 4, 2, 128, 128, 192, 16
    T, D, dt, rnd = R * T_o, torch.float64, DT[dtype], gen(15)
    w = {"norm_weight": 1 + 0.1 * rnd(d), "norm_bias": 0.1 * rnd(d), "w_gate_up": (rnd(G, 2 * f, d) / d ** 0.5).to(dt),
         "w_down": (rnd(G, d, f) / d ** 0.5).to(dt), "shared_gate_up": (rnd(2 * fs, d) / d ** 0.5).to(dt),
         "shared_down": (rnd(d, fs) / d ** 0.5).to(dt)}
    block, x = MoeBlock(MoePath(R, T_o, G, G, k, d, f, M, dtype=dtype), fs, train=False), rnd(T, d).to(dt)
    router = rnd(G, d) / d ** 0.5
    out = block.experts(block.norm(x, w).float() @ router.T, w).clone()
    idx, wt = block.path.topk_idx.long(), block.path.topk_w.to(D)
    n = torch.nn.functional.layer_norm(x.to(D), (d,), w["norm_weight"].to(D), w["norm_bias"].to(D))

    def mlp(gu, down):
        g, u = (n @ gu.to(D).T).chunk(2, 1)
        return (torch.nn.functional.silu(g) * u) @ down.to(D).T

    want = mlp(w["shared_gate_up"], w["shared_down"])
    for e in range(G):
        want = want + (wt * (idx == e)).sum(1, keepdim=True) * mlp(w["w_gate_up"][e], w["w_down"][e])
    assert (out.to(D) - want).norm() <= (8 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -16) * want.norm()
    assert torch.equal(block.experts(block.norm(x, w).float() @ router.T, w), out) and block.path.status() == B.MOE_OK
    with pytest.raises(RuntimeError, match="train"):
        block.experts_backward(out, w)
