"""The operators around the routed experts where offsets pass 32 bits.  All rows but a few are zeros, so that those few give every
result: they stand at the start, behind 2^32 elements and at the end."""
import pytest
import torch

import block_reference as ref
from expert_output_overlap_amd import binding as B
from test_gpu_block import DT, check, ffn_case, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip("%d GiB of device memory wanted" % gib)


def nothing_else(t, rows):
    """t holds zeros but in `rows`."""
    t[rows] = 0.0
    assert not any(part.any() for part in t.split(-(-t.shape[0] // 16)))


@pytest.mark.parametrize("T,d,f,dtype", [(280000, 16384, 64, "bf16"), (280001, 16383, 41, "bf16"), (140000, 64, 16384, "bf16"),
                                         (280000, 16384, 24, "f32"), (140001, 33, 16381, "f32")])
def test_shared_ffn_of_many_tokens(T, d, f, dtype):
    room(130)
    _, wgu, wd, _, _ = ffn_case(1, d, f, dtype, seed=20)
    dt, rows = DT[dtype], torch.tensor([0, 1, T // 2 + 1, (1 << 32) // max(d, 2 * f) + 1, T - 1], device="cuda")
    some = gen(21)(5, d).to(dt)
    shape = B.moe_shared_shape(T, d, f, B.MOE_BF16 if dtype == "bf16" else B.MOE_F32)
    F = B.moe_shared_ffn_row(shape)
    x = torch.zeros(T, d, device="cuda", dtype=dt)
    x[rows] = some
    y, h = torch.empty_like(x), torch.empty(T, F, device="cuda", dtype=dt)
    gu, dgu = torch.empty(T, 2 * F, device="cuda"), torch.empty(T, 2 * F, device="cuda", dtype=dt)
    need = max(B.moe_shared_ffn_workspace_bytes(shape, b) for b in (False, True))
    workspace = torch.empty(need, device="cuda", dtype=torch.uint8)
    B.moe_shared_ffn(shape, x, wgu, wd, None, h, gu, y, workspace)
    dw_gate_up, dw_down = torch.empty_like(wgu), torch.empty_like(wd)
    want = ref.shared_ffn(some, wgu, wd, dy=some)
    got = {"y": y[rows]}
    nothing_else(y, rows)
    del y
    dx = torch.empty_like(x)
    B.moe_shared_ffn_backward(shape, {"x": x, "w_gate_up": wgu, "w_down": wd, "h": h, "gu": gu, "dy": x, "dgu_ws": dgu, "dx": dx,
                                      "dw_gate_up": dw_gate_up, "dw_down": dw_down}, workspace)
    got.update(dx=dx[rows], dw_gate_up=dw_gate_up, dw_down=dw_down)
    check(got, want, ("y", "dx", "dw_gate_up", "dw_down"), (T, d, f, dtype))
    for name, v in got.items():  # at most four roundings to bf16 in a row; an element from elsewhere is off by the norm itself
        assert (v.double() - want[name][0]).norm() <= 4 * 2.0 ** -8 * want[name][0].norm(), name
    nothing_else(dx, rows)


@pytest.mark.parametrize("d,f,dtype", [(24576, 65536, "bf16"), (32768, 65536, "bf16"), (12288, 65536, "f32"), (16385, 65535, "f32")])
def test_shared_ffn_of_one_token_and_large_weights(d, f, dtype):
    """The up projection's rows start 3 and 4 GiB behind the gate's.  Weights of few values, so that they are quickly made."""
    from expert_output_overlap_amd.runtime import SharedFFN

    room(60)
    dt, rnd = DT[dtype], gen(22)
    x = rnd(2, d).to(dt)
    rows, cols = rnd(2 * f, 1) / d ** 0.5, rnd(1, d)
    wgu = rows.to(dt).expand(2 * f, d) * cols.sign().to(dt)
    wd = (rnd(d, 1) / d ** 0.5).to(dt).expand(d, f) * rnd(1, f).sign().to(dt)
    y = SharedFFN(2, d, f, dtype, train=False).forward(x, wgu, wd)
    # the products' sums: g = row . (x . sign), y = row . (h . sign)
    s = (x.double() * cols.sign().double()).sum(1, keepdim=True)
    gu = s * rows.to(dt).double().T
    g, u = gu.chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    exact = (h * wd[0].double().sign()).sum(1, keepdim=True) * (wd[:, :1].double() * wd[0, 0].double().sign()).T
    assert (y.double() - exact).norm() <= (3 * 2.0 ** -8 if dtype == "bf16" else 2.0 ** -12) * exact.norm()


@pytest.mark.parametrize("d,dtype", [(16384, "bf16"), (16381, "f32")])
def test_norm_of_many_rows(d, dtype):
    from expert_output_overlap_amd.runtime import LayerNorm

    room(100)
    T, dt, rnd = 280000, DT[dtype], gen(23)
    rows = torch.tensor([0, 1, T // 2 + 1, (1 << 32) // d + 1, T - 1], device="cuda")
    op = LayerNorm(T, d, dtype)
    x, dy = torch.zeros(T, d, device="cuda", dtype=dt), torch.zeros(T, d, device="cuda", dtype=dt)
    x[rows], dy[rows] = rnd(5, d).to(dt), rnd(5, d).to(dt)
    w, zero = 1 + 0.2 * rnd(d), torch.zeros(d, device="cuda")
    want = ref.layer_norm(x[rows], w, zero, 1e-5, dy[rows])
    y, dx = op.forward(x, w), op.backward(dy, x, w)
    check({"y": y[rows], "dx": dx[rows], "dweight": op.dweight, "dbias": op.dbias}, want, want, (d, dtype))
    nothing_else(y, rows)
    nothing_else(dx, rows)


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_of_a_large_tensor(bits):
    """The last elements of 2^32 + 77 move as the same values in a tensor of their own."""
    from expert_output_overlap_amd.runtime import AdamW

    room(80)
    n, k, rnd = (1 << 32) + 77, 4096 * 2 + 77, gen(24)
    big = {"p": torch.zeros(n, device="cuda", dtype=torch.bfloat16), "g": torch.zeros(n, device="cuda", dtype=torch.bfloat16)}
    big.update(AdamW.states(big["p"], bits))
    small = {"p": rnd(k).bfloat16(), "g": rnd(k).bfloat16()}
    small.update(AdamW.states(small["p"], bits))
    if bits == 8:
        for t in (big, small):
            t["root_values"] = torch.zeros(t["p"].numel(), device="cuda", dtype=torch.bfloat16)
    for name in ("p", "g"):
        big[name][-k:] = small[name]
    ops = [AdamW([t]) for t in (big, small)]
    for step in (1, 2):
        for op in ops:
            op.step(step, 1e-3)
            op.read_states()
        for name, v in small.items():
            assert torch.equal(big[name][-v.numel():], v), (name, step)
    for name in ("p", "m", "v"):
        assert not any(part.any() for part in big[name][:-k].split(1 << 28)), name
