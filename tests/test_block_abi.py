"""Argument checks of the operators around the routed experts: each refusal happens on the host, before any launch, so these
run without a GPU on made-up addresses."""
import ctypes

import pytest

from expert_output_overlap_amd import binding as B

A = 1 << 30  # made-up device addresses, far apart
P = [A + k * (1 << 28) for k in range(16)]


def refused(rc, words):
    assert rc == B.MOE_EINVAL and words in B.moe_last_error(), (rc, B.moe_last_error())


def norm_shape(**kw):
    v = dict(rows=4, d=64, dtype=B.MOE_BF16, param_dtype=B.MOE_F32, eps=1e-5, x_stride=0, y_stride=0, dx_stride=0)
    return B.moe_norm_shape(**{**v, **kw})


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(d=0), dict(d=B.MOE_NORM_MAX_D + 1), dict(dtype=2), dict(param_dtype=-1),
                                dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x_stride=63), dict(x_stride=1 << 46), dict(rows=1 << 30, y_stride=1 << 20),
                                dict(y_stride=-64), dict(dx_stride=1)])
def test_norm_shapes(kw):
    s = norm_shape(**kw)
    assert B.moe_layer_norm_workspace_bytes(s) == -1
    assert B.lib().moe_layer_norm(ctypes.byref(s), P[0], P[1], P[2], P[3], None, None, None) == B.MOE_EINVAL
    assert B.moe_last_error()


def test_norm_arguments():
    L, s = B.lib(), norm_shape()
    f = lambda x=P[0], w=P[1], b=P[2], y=P[3], m=P[4], r=P[5]: L.moe_layer_norm(ctypes.byref(s), x, w, b, y, m, r, None)
    refused(f(x=None), "null")
    refused(f(y=None), "null")
    refused(f(m=None), "go together")
    refused(f(x=P[0] + 1), "aligned")
    refused(f(w=P[1] + 2), "aligned")
    refused(f(y=P[0] + 64), "overlaps")
    refused(f(y=P[1]), "overlaps")
    refused(f(m=P[3]), "overlaps")
    refused(f(r=P[4] + 8), "overlaps")
    need = B.moe_layer_norm_workspace_bytes(s)
    assert need > 0
    b = lambda **kw: L.moe_layer_norm_backward(ctypes.byref(s), *[kw.get(k, d) for k, d in (
        ("dy", P[0]), ("x", P[1]), ("w", P[2]), ("mean", P[3]), ("rstd", P[4]), ("res", P[5]), ("dx", P[6]), ("dw", P[7]),
        ("db", P[8]), ("ws", P[9]), ("n", need), ("st", None))])
    refused(b(mean=None), "null")
    refused(b(dx=None), "null")
    refused(b(n=need - 1), "too small")
    refused(b(ws=None), "too small")
    refused(b(ws=P[9] + 8), "aligned")
    for kw in (dict(dx=P[1]), dict(dx=P[0] + 2), dict(dx=P[5] + 128), dict(dx=P[2]), dict(dw=P[8]), dict(dw=P[2]), dict(db=P[6]),
               dict(ws=P[0]), dict(ws=P[7])):
        refused(b(**kw), "overlaps")
    assert L.moe_layer_norm(None, P[0], P[1], P[2], P[3], None, None, None) == B.MOE_EINVAL


@pytest.mark.parametrize("at", [-190, -128, -2, 2, 126, 66 + 256, 190 + 256])
def test_norm_rows_between_rows(at):
    """x and y in one buffer of rows of 192 elements, 64 of which each takes: refused where two rows meet."""
    s = norm_shape(rows=16, x_stride=96, y_stride=96)
    refused(B.lib().moe_layer_norm(ctypes.byref(s), P[0], P[1], P[2], P[0] + at, None, None, None), "overlaps")


def test_norm_workspace_grows_with_rows_to_a_limit():
    sizes = [B.moe_layer_norm_workspace_bytes(norm_shape(rows=r, d=7168)) for r in (1, 10, 1000, 10 ** 6, 10 ** 9)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2] <= 64 << 20


def shared_shape(**kw):
    return B.moe_shared_shape(**{**dict(tokens=8, d=64, f=128, dtype=B.MOE_BF16), **kw})


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=(1 << 27) + 1), dict(d=0), dict(d=65537), dict(f=0),
                                dict(f=65537), dict(dtype=3), dict(tokens=1 << 20, f=8200)])
def test_shared_shapes(kw):
    s = shared_shape(**kw)
    assert B.moe_shared_ffn_row(s) == -1
    assert B.moe_shared_ffn_workspace_bytes(s, False) == -1 and B.moe_shared_ffn_workspace_bytes(s, True) == -1
    assert B.lib().moe_shared_ffn(ctypes.byref(s), *P[:8], 0, None) == B.MOE_EINVAL


def test_shared_arguments():
    L, s = B.lib(), shared_shape()
    big = 1 << 27

    def f(**kw):
        return L.moe_shared_ffn(ctypes.byref(s), *[kw.get(k, d) for k, d in (
            ("x", P[0]), ("wgu", P[1]), ("wd", P[2]), ("res", P[3]), ("h", P[4]), ("gu", P[5]), ("y", P[6]), ("ws", P[7]),
            ("n", big), ("st", None))])

    for k in ("x", "wgu", "wd", "h", "y"):
        refused(f(**{k: None}), "null")
    for k, p in (("x", P[0]), ("wgu", P[1]), ("wd", P[2]), ("res", P[3]), ("h", P[4]), ("gu", P[5]), ("y", P[6]), ("ws", P[7])):
        refused(f(**{k: p + 8}), "aligned")
    for other in (P[0], P[1], P[2], P[4], P[5], P[3] + 16):
        refused(f(y=other), "overlaps")
    for kw in (dict(h=P[0]), dict(gu=P[4]), dict(ws=P[1]), dict(ws=P[6])):
        refused(f(**kw), "overlaps")
    s0 = shared_shape(d=100, f=36)
    need = B.moe_shared_ffn_workspace_bytes(s0, False)
    if need:
        refused(L.moe_shared_ffn(ctypes.byref(s0), *P[:8], need - 1, None), "too small")
        refused(L.moe_shared_ffn(ctypes.byref(s0), *P[:7], None, need, None), "too small")

    def b(**kw):
        a = B.moe_shared_bwd_args(**{**dict(zip(B.SHARED_BWD_FIELDS, P)), **kw})
        return L.moe_shared_ffn_backward(ctypes.byref(s), ctypes.byref(a), P[12], big, None)

    for k in B.SHARED_BWD_FIELDS:
        if k != "residual":
            refused(b(**{k: None}), "null")
        refused(b(**{k: P[B.SHARED_BWD_FIELDS.index(k)] + 4}), "aligned")
    at = dict(zip(B.SHARED_BWD_FIELDS, P))
    refused(b(dx=at["x"]), "overlaps")
    refused(b(dx=at["dy"]), "overlaps")
    refused(b(dgu_ws=at["h"]), "overlaps")
    refused(b(dgu_ws=at["gu"] + 16), "overlaps")
    refused(b(dw_down=at["w_down"]), "overlaps")
    refused(b(dw_down=at["dw_gate_up"]), "overlaps")
    assert L.moe_shared_ffn_backward(ctypes.byref(s), None, None, 0, None) == B.MOE_EINVAL


def test_shared_rows_and_workspaces():
    assert [B.moe_shared_ffn_row(shared_shape(f=f)) for f in (1, 8, 517, 1408)] == [8, 8, 520, 1408]
    for backward in (False, True):
        for d, f, dtype in ((7168, 2048, B.MOE_BF16), (100, 36, B.MOE_BF16), (333, 517, B.MOE_BF16), (333, 517, B.MOE_F32)):
            sizes = [B.moe_shared_ffn_workspace_bytes(shared_shape(tokens=t, d=d, f=f, dtype=dtype), backward)
                     for t in (0, 1, 2, 16, 17, 63, 64, 65, 100, 128, 129, 300, 512, 1000, 3000, 20000)]
            assert sizes == sorted(sizes)  # buffers made for the most tokens serve fewer


def adam(**kw):
    v = dict(param=P[0], copy=P[1], grad=P[2], m=P[3], v=P[4], m_scale=None, v_scale=None, m_values=None, root_values=None,
             n=100, param_dtype=B.MOE_F32, grad_dtype=B.MOE_F32, state_bits=32, weight_decay=0.1, lr_scale=1.0, reserved=0)
    return B.moe_adamw_tensor(**{**v, **kw})


def bind(tensors, ws=P[15], n=1 << 20):
    table, plan = (B.moe_adamw_tensor * len(tensors))(*tensors), B.moe_adamw_plan()
    return B.lib().moe_adamw_bind(table, len(tensors), ws, n, ctypes.byref(plan), None)


@pytest.mark.parametrize("kw,words", [
    (dict(n=-1), "elements"), (dict(param_dtype=5), "dtype"), (dict(grad_dtype=-2), "dtype"), (dict(state_bits=16), "bits"),
    (dict(reserved=1), "reserved"), (dict(n=1 << 37), "too many"), (dict(weight_decay=float("nan")), "finite"), (dict(lr_scale=float("inf")), "finite"), (dict(param=None), "null"),
    (dict(grad=None), "null"), (dict(m=None), "null"), (dict(state_bits=8), "scales"), (dict(m_scale=P[5]), "8-bit"),
    (dict(param=P[0] + 2), "aligned"), (dict(m=P[3] + 1), "aligned"), (dict(copy=P[1] + 1), "aligned"),
    (dict(copy=P[0]), "overlaps"), (dict(m=P[2]), "overlaps"), (dict(v=P[3] + 396), "overlaps"), (dict(grad=P[0] + 4), "overlaps"),
])
def test_adamw_tensors(kw, words):
    refused(bind([adam(**kw)]), words)


def test_adamw_plans():
    t = adam()
    refused(bind([t, adam()]), "overlaps")  # the same tensor twice
    other = dict(param=P[5], copy=P[6], m=P[7], v=P[8])
    refused(bind([t, adam(**other)], n=100), "too small")
    refused(bind([t, adam(**other)], ws=None), "too small")
    refused(bind([t], ws=P[15] + 4), "aligned")
    refused(bind([t], ws=P[0]), "overlaps")
    refused(bind([adam(n=0), adam()], ws=P[3]), "overlaps")
    refused(bind([t, adam(**other)], ws=P[7]), "overlaps")
    two = (B.moe_adamw_tensor * 2)(t, adam(**other, n=5000))
    assert B.moe_adamw_workspace_bytes(two) == 256 + 2 * ctypes.sizeof(B.moe_adamw_tensor)
    assert B.moe_adamw_workspace_bytes((B.moe_adamw_tensor * 1)(adam(n=-1))) == -1
    plan = B.moe_adamw_plan()
    assert B.lib().moe_adamw_bind(None, 0, None, 0, ctypes.byref(plan), None) == B.MOE_OK  # no tensors: nothing to do
    assert B.lib().moe_adamw_step(ctypes.byref(plan), ctypes.byref(cfg()), None) == B.MOE_OK


def cfg(**kw):
    return B.moe_adamw_cfg(**{**dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1), **kw})


@pytest.mark.parametrize("kw,words", [
    (dict(lr=-1.0), "lr"), (dict(lr=float("nan")), "lr"), (dict(eps=-1e-8), "eps"), (dict(beta1=1.0), "betas"),
    (dict(beta2=-0.1), "betas"), (dict(beta2=float("nan")), "betas"), (dict(step=0), "step"), (dict(step_dev=P[0] + 4), "aligned"),
])
def test_adamw_steps(kw, words):
    plan = B.moe_adamw_plan(P[15], 1, 1, 0)
    refused(B.lib().moe_adamw_step(ctypes.byref(plan), ctypes.byref(cfg(**kw)), None), words)


def test_adamw_unbound_plan():
    refused(B.lib().moe_adamw_step(None, ctypes.byref(cfg()), None), "plan")
    refused(B.lib().moe_adamw_step(ctypes.byref(B.moe_adamw_plan(None, 3, 1, 0)), ctypes.byref(cfg()), None), "plan")
    refused(B.lib().moe_adamw_read_states(None, None), "plan")


def test_adamw_state_bits():
    import torch

    from expert_output_overlap_amd.runtime import AdamW

    with pytest.raises(ValueError, match="8 or 32"):
        AdamW.states(torch.zeros(4), 16)


@pytest.mark.parametrize("value", [0, 4, 0.5])
def test_adamw_grad_scale_is_a_tensor(value):
    """The factor is read on the device: a number in its place would become an address."""
    import torch

    from expert_output_overlap_amd.runtime import AdamW

    op = AdamW.__new__(AdamW)
    op.device, op.betas, op.eps, op.plan = torch.device("cuda", 0), (0.9, 0.95), 1e-8, B.moe_adamw_plan()  # no tensors
    with pytest.raises(ValueError, match="grad_scale"):
        AdamW.step.__wrapped__(op, 1, 1e-3, grad_scale=value)


@pytest.mark.parametrize("kw", [dict(eps=1e-39), dict(eps=1e-46), dict(eps=2.0 ** -126 * 0.999), dict(eps=1e39), dict(lr=1e39)])
def test_adamw_numbers_that_single_precision_does_not_hold(kw):
    """eps below 2^-126 would be a divisor whose reciprocal is not finite: 0 times it, of an element without gradients, is NaN."""
    refused(B.lib().moe_adamw_step(ctypes.byref(B.moe_adamw_plan()), ctypes.byref(cfg(**kw)), None), "lr and eps")


def test_adamw_smallest_eps():
    plan = B.moe_adamw_plan()  # no tensors: nothing is launched
    for eps in (0.0, 2.0 ** -126):
        assert B.lib().moe_adamw_step(ctypes.byref(plan), ctypes.byref(cfg(eps=eps)), None) == B.MOE_OK


def test_adamw_states_are_single_precision_whatever_the_default():
    import torch

    from expert_output_overlap_amd.runtime import AdamW

    was = torch.get_default_dtype()
    try:
        for dtype in (torch.bfloat16, torch.float64):
            torch.set_default_dtype(dtype)
            assert {t.dtype for t in AdamW.states(torch.zeros(40, dtype=torch.bfloat16)).values()} == {torch.float32}
    finally:
        torch.set_default_dtype(was)


def test_block_works_on_its_paths_device(monkeypatch):
    """Every call of a block runs with its path's device as the current one, the path's own calls among them: they take the
    current device's stream."""
    import contextlib

    import torch

    from expert_output_overlap_amd import runtime
    from expert_output_overlap_amd.runtime import MoeBlock

    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(runtime, "_need", lambda *a, **kw: None)  # no tensors here

    class Op:  # notes the device that is current at each of its calls
        T, G, E_l, d, f, tdtype, out, n = 2, 4, 4, 3, 5, torch.float32, torch.zeros(2, 3), None

        def __getattr__(self, name):
            return lambda *a, **kw: seen.append((name, current[0])) or {"dx": torch.zeros(2, 3)}

    block = MoeBlock.__new__(MoeBlock)
    block.path = block.norm_op = block.shared = Op()
    block.device, block.train = torch.device("cuda", 1), True
    w = dict.fromkeys(("norm_weight", "norm_bias", "w_gate_up", "w_down", "shared_gate_up", "shared_down"))
    block.norm(None, w)
    block.experts(None, w)
    block.experts_backward(None, w)
    block.norm_backward(None, None, w)
    assert {d for _, d in seen} == {1} and {"route", "layout", "ffn", "combine", "backward", "combine_backward"} <= {n for n, _ in seen}
    assert current == [0]


@pytest.mark.parametrize("T,d,f,dtype", [(40, 64, 72, B.MOE_F32), (100, 40, 48, B.MOE_BF16), (33, 100, 36, B.MOE_BF16), (1, 1, 1, B.MOE_F32),
                                         (7, 300, 8, B.MOE_F32), (4096, 7168, 2048, B.MOE_BF16)])
def test_shared_backward_workspace_holds_every_sum(T, d, f, dtype):
    """Sixteen k-splits of all three gradients at once (they lie one after another) and of dH, up to 2^23 sums."""
    d8, f8 = -(-d // 8) * 8, -(-f // 8) * 8
    sums = 16 * max(T * f8, T * d8 + 2 * f8 * d8 + d8 * f8)
    assert B.moe_shared_ffn_workspace_bytes(shared_shape(tokens=T, d=d, f=f, dtype=dtype), True) >= 4 * min(1 << 23, sums)


def test_block_checks_before_it_launches():
    """A batch of fewer rows than the path's, or other tensors than the path's shape: refused before the routed path, whose calls go by
    addresses alone, reads past them."""
    import torch

    from expert_output_overlap_amd.runtime import MoeBlock

    T, G, E, d, f = 6, 4, 2, 8, 16

    class Op:
        def __getattr__(self, name):
            raise AssertionError("called " + name)

    class Path(Op):
        pass

    p = Path()
    p.T, p.G, p.E_l, p.d, p.f, p.tdtype, p.out = T, G, E, d, f, torch.bfloat16, torch.zeros(T, d)
    block = MoeBlock.__new__(MoeBlock)
    block.path, block.norm_op, block.shared, block.device, block.train = p, Op(), Op(), torch.device("cpu"), True
    block.n = torch.zeros(T, d, dtype=torch.bfloat16)
    z = lambda *n, dtype=torch.bfloat16: torch.zeros(*n, dtype=dtype)
    w = {"norm_weight": None, "norm_bias": None, "w_gate_up": z(E, 2 * f, d), "w_down": z(E, d, f), "shared_gate_up": None, "shared_down": None}
    norm, experts, back = (getattr(MoeBlock, k).__wrapped__ for k in ("norm", "experts", "experts_backward"))
    for x in (z(T - 1, d), z(T, d, dtype=torch.float32)):
        with pytest.raises(ValueError, match="x:"):
            norm(block, x, w)
    for logits in (z(T - 1, G, dtype=torch.float32), z(T, G), z(T, G + 1, dtype=torch.float32), z(G, T, dtype=torch.float32).T):
        with pytest.raises(ValueError, match="logits"):
            experts(block, logits, w)
    for call, first in ((experts, z(T, G, dtype=torch.float32)), (back, z(T, d))):
        for k, bad in (("w_gate_up", z(E, f, d)), ("w_down", z(E, d, f, dtype=torch.float32))):
            with pytest.raises(ValueError, match=k):
                call(block, first, {**w, k: bad})
    for d_out in (z(T - 1, d), z(T, d, dtype=torch.float32), z(T, 2 * d)[:, :d]):
        with pytest.raises(ValueError, match="d_out"):
            back(block, d_out, w)
    block.train = False
    with pytest.raises(RuntimeError, match="train"):
        back(block, z(T, d), w)
