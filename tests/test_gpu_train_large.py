"""The training operators where elements lie further than 2^31 from the first: the last rows against 64 bits."""
import numpy as np
import pytest
import torch

import train_reference as ref
from block_reference import D, E32, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("80 GiB of device memory wanted")
    yield
    torch.cuda.empty_cache()


def repeated(block, rows):
    """A matrix of `rows` rows, the block's again and again."""
    return block.repeat(-(-rows // block.shape[0]), 1)[:rows]


def test_residual_norm_far_rows():
    from expert_output_overlap_amd.runtime import ResidualNorm

    rows, d, k = 131100, 16384, 300  # 2^31 + 5e5 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, h, ds, dn = (repeated(rnd(k, d).bfloat16(), rows) for _ in range(4))
    w = {n: 1 + 0.1 * rnd(d) for n in ("post_weight", "gate", "pre_weight")}
    op = ResidualNorm(rows, d, post="rms", pre="layer")
    s, n = op.forward(x, h, w)
    dx, dh = op.backward(ds, dn, x, h, w)
    last = slice(rows - 40, rows)
    want = ref.residual_norm(x[last], h[last], w, "rms", "layer", 1.0, 1e-5, None, ds[last], dn[last])
    for name, t in (("s", s), ("n", n), ("dx", dx), ("dh", dh)):
        within(t[last], *want[name], name)
        at = rows // k * k - k  # the block's rows give the same bits wherever they are
        assert torch.equal(t[at: at + k], t[:k])


@pytest.mark.parametrize("rows,d,depth", [(131100, 16384, 513 + 16 + 15), (600000, 128, 37 + 15 + 64 + 15), (300000, 4096, 586 + 32 + 15)])
def test_residual_norm_parameter_gradients_of_many_rows(rows, d, depth):
    """Sums over very many rows in fp32, at the depth that they have instead of one addition after another: a group's rows, the groups of a
    workgroup, then every 16th workgroup's sums in each of 16 waves, and those."""
    from expert_output_overlap_amd.runtime import ResidualNorm

    k = 300
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    part = [rnd(k, d).bfloat16() for _ in range(4)]
    x, h, ds, dn = (repeated(t, rows) for t in part)
    w = {n: 1 + 0.1 * rnd(d) for n in ("post_weight", "gate", "pre_weight")}
    op = ResidualNorm(rows, d, post="rms", pre="layer")
    op.forward(x, h, w)
    op.backward(ds, dn, x, h, w)
    px, ph, pds, pdn = (t.to(D) for t in part)
    w1, gate, w2 = (w[n].to(D) for n in ("post_weight", "gate", "pre_weight"))
    zero = torch.zeros_like(px)
    n1, e_n1, _, _ = ref.norm(ph, zero, "rms", 1e-5)
    s = px + gate * n1 * w1
    e_s = (gate * w1).abs() * (e_n1 + 4 * E32 * n1.abs()) + 2 * E32 * (px.abs() + s.abs())
    n2, e_n2, r2, e_r2 = ref.norm(s, e_s, "layer", 1e-5)
    back, e_b = ref.norm_back(pdn * w2, E32 * (pdn * w2).abs(), n2, e_n2, r2, e_r2, "layer")
    total = pds + back
    e_t = e_b + E32 * total.abs()
    times = torch.full((k, 1), rows // k, dtype=D, device="cuda")
    times[: rows % k] += 1
    u1 = (times * total * n1).sum(0)
    e_u1 = (times * ((depth + 3) * E32 * (total * n1).abs() + e_t * n1.abs() + total.abs() * e_n1)).sum(0)
    e_w2 = (times * ((depth + 3) * E32 * (pdn * n2).abs() + pdn.abs() * e_n2)).sum(0)
    for name, value, bound in (("post_weight", gate * u1, gate.abs() * (e_u1 + 2 * E32 * u1.abs())),
                               ("gate", w1 * u1, w1.abs() * (e_u1 + 2 * E32 * u1.abs())),
                               ("pre_weight", (times * pdn * n2).sum(0), e_w2)):
        within(op.grads[name], value, bound + E32 * value.abs(), name)


def test_router_far_rows():
    from expert_output_overlap_amd.runtime import RouterLoss

    G, k, block = 1024, 1, 256
    T = (1 << 21) + block  # 2^31 + 2^18 logits
    g = torch.Generator(device="cuda").manual_seed(2)
    one = torch.randn(block, G, generator=g, device="cuda")
    logits = repeated(one, T)
    idx = torch.topk(one, k).indices.int()
    ids = repeated(idx, T).contiguous()
    op = RouterLoss(T, G, k, z=1e-3, dtype="bf16")
    losses = op.forward(logits, ids).clone()
    dl = op.backward(logits, ids)
    # the gradient is bf16: half a step of it, 2^-8 of each value, belongs to its bound
    counts, want = ref.router_loss(one, idx, 1, float(np.float32(0.01)), float(np.float32(1e-3)), dtype=torch.bfloat16)
    times = T // block
    assert T % block == 0 and torch.equal(op.counts, counts * times) and op.means.tolist() == [1, T]
    within(losses, *want["losses"], "losses")
    # the mean of a batch of equal blocks: each gradient is the block's over their number
    value, bound = want["dlogits"][0] / times, want["dlogits"][1] / times
    for at in (0, T - block):
        within(dl[at: at + block], value, bound + 2 * E32 * value.abs(), at)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grad_norm_far_elements(dtype):
    from expert_output_overlap_amd.runtime import GradNorm

    n = (1 << 31) + 70001
    t = torch.full((n,), 0.5, dtype=dtype, device="cuda")
    t[-1] = 4096.0
    op = GradNorm([{"g": t}])
    want = torch.tensor(0.25 * (n - 1) + 4096.0 ** 2, dtype=D, device="cuda").sqrt()
    within(op.clip(0.5 * want.item())[0], want, 1.001 * E32 * want, "norm")
    f = op.scale.item()
    assert abs(f - 0.5) < 1e-6
    r = torch.finfo(dtype).eps / 2 + E32
    for at in (0, (1 << 31) - 1, 1 << 31, n - 2, n - 1):
        v = (4096.0 if at == n - 1 else 0.5) * f
        assert abs(t[at].item() - v) <= r * v, at
