"""Argument checks of the training operators: each refusal happens on the host, before any launch, so these run without a GPU
on made-up addresses."""
import ctypes

import pytest

from expert_output_overlap_amd import binding as B

A = 1 << 30  # made-up device addresses, far apart
P = [A + k * (1 << 28) for k in range(24)]
INF, NAN = float("inf"), float("nan")


def refused(rc, words):
    assert rc == B.MOE_EINVAL and words in B.moe_last_error(), (rc, B.moe_last_error())


# ---- the norms around a block ------------------------------------------------------------------------------------

def res_shape(**kw):
    v = dict(rows=4, d=64, dtype=B.MOE_BF16, param_dtype=B.MOE_F32, post=B.MOE_NORM_RMS, pre=B.MOE_NORM_LAYER, eps=1e-5,
             residual_scale=1.0)
    return B.moe_residual_norm_shape(**{**v, **kw})


PARAMS = dict(zip(B.RESIDUAL_PARAMS, P[10:16]))
ARGS = dict(zip(("x", "h", "s", "n", "stats"), P))
BWD = dict(zip(B.RESIDUAL_BWD_POINTERS, P[:7] + P[16:22]))


def res(shape=None, params=None, **kw):
    p = B.moe_residual_norm_params(**(PARAMS if params is None else params))
    a = B.moe_residual_norm_args(**{**ARGS, **kw})
    return B.lib().moe_residual_norm(ctypes.byref(shape or res_shape()), ctypes.byref(p), ctypes.byref(a), None)


def res_bwd(shape=None, params=None, ws=P[22], nbytes=1 << 27, **kw):
    p = B.moe_residual_norm_params(**(PARAMS if params is None else params))
    a = B.moe_residual_norm_bwd_args(**{**BWD, **kw})
    return B.lib().moe_residual_norm_backward(ctypes.byref(shape or res_shape()), ctypes.byref(p), ctypes.byref(a), ws, nbytes, None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(d=0), dict(d=B.MOE_NORM_MAX_D + 1), dict(dtype=2), dict(param_dtype=-1),
                                dict(post=3), dict(pre=-1), dict(eps=0.0), dict(eps=NAN), dict(eps=INF),
                                dict(residual_scale=NAN), dict(residual_scale=INF)])
def test_residual_shapes(kw):
    s = res_shape(**kw)
    assert B.moe_residual_norm_workspace_bytes(s) == -1
    assert res(s) == B.MOE_EINVAL and res_bwd(s) == B.MOE_EINVAL


def test_residual_arguments():
    L = B.lib()
    assert L.moe_residual_norm(None, None, None, None) == B.MOE_EINVAL
    s, p, a = res_shape(), B.moe_residual_norm_params(), B.moe_residual_norm_args(**ARGS)
    refused(L.moe_residual_norm(ctypes.byref(s), None, ctypes.byref(a), None), "null")
    refused(L.moe_residual_norm(ctypes.byref(s), ctypes.byref(p), None, None), "null")
    for k in ("x", "h", "s"):
        refused(res(**{k: None}), "null")
        refused(res(**{k: ARGS[k] + 1}), "aligned")
    refused(res(n=None), "only then")
    refused(res(stats=P[4] + 8), "16-byte")
    for k in B.RESIDUAL_PARAMS:
        refused(res(params={**PARAMS, k: PARAMS[k] + 2}), "aligned")
    for k in ("x_stride", "h_stride", "s_stride", "n_stride"):
        refused(res(**{k: 63}), "stride")
        refused(res(**{k: -64}), "stride")
        refused(res(**{k: 1 << 46}), "stride")
    none = res_shape(pre=B.MOE_NORM_NONE)
    refused(res(none, {**PARAMS, "pre_weight": None, "pre_bias": None}), "only then")
    refused(res(none, n=None), "is none")
    refused(res(res_shape(post=B.MOE_NORM_NONE)), "is none")


@pytest.mark.parametrize("kw", [dict(s=P[0] + 64), dict(n=P[2]), dict(n=P[2] + 64), dict(stats=P[2]), dict(s=P[10]), dict(n=P[14]),
                                dict(s=P[15]), dict(s=P[0]), dict(n=P[1]), dict(stats=P[0]),
                                dict(s=P[0], stats=None, x_stride=96), dict(n=P[1], stats=None, n_stride=128)])
def test_residual_overlaps(kw):
    """Also x and h of a training forward, which the backward reads."""
    refused(res(**kw), "overlaps")


def test_residual_backward_arguments():
    need = B.moe_residual_norm_workspace_bytes(res_shape())
    assert need > 0
    for k in ("x", "h", "stats", "dx", "dh"):
        refused(res_bwd(**{k: None}), "null")
    refused(res_bwd(dn=None), "only then")
    none = res_shape(pre=B.MOE_NORM_NONE)
    no_pre = {**PARAMS, "pre_weight": None, "pre_bias": None}
    refused(res_bwd(none, no_pre), "only then")
    refused(res_bwd(none, no_pre, dn=None), "is none")
    refused(res_bwd(none, no_pre, dn=None, ds=None, d_pre_weight=None, d_pre_bias=None), "null")
    refused(res_bwd(res_shape(post=B.MOE_NORM_NONE), {**PARAMS, "post_weight": None, "post_bias": None}), "is none")
    for k in ("ds", "dn", "x", "h", "dx", "dh", "d_post_weight", "d_gate", "d_row_gate"):
        refused(res_bwd(**{k: BWD[k] + 1}), "aligned")
    refused(res_bwd(stats=P[4] + 4), "16-byte")
    refused(res_bwd(ws=P[22] + 8), "16-byte")
    refused(res_bwd(nbytes=need - 1), "too small")
    refused(res_bwd(ws=None), "too small")
    for k in ("ds", "dn", "x", "h", "dx", "dh"):
        refused(res_bwd(**{k + "_stride": 63}), "stride")
    at = BWD
    for kw in (dict(dx=at["x"]), dict(dh=at["h"]), dict(dh=at["dx"]), dict(dx=at["ds"] + 2), dict(dx=at["ds"], dx_stride=70),
               dict(dx=at["stats"]), dict(d_gate=at["d_post_weight"]), dict(d_gate=PARAMS["gate"]), dict(d_row_gate=at["dh"]),
               dict(ws=at["dx"]), dict(ws=at["d_gate"]), dict(dx=PARAMS["row_gate"])):
        refused(res_bwd(**kw), "overlaps")


def test_residual_workspace_grows_with_rows_to_a_limit():
    sizes = [B.moe_residual_norm_workspace_bytes(res_shape(rows=r, d=7168)) for r in (1, 10, 1000, 10 ** 6, 10 ** 9)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2] <= 128 << 20


# ---- the router's losses -----------------------------------------------------------------------------------------

def router_shape(**kw):
    return B.moe_router_shape(**{**dict(tokens=8, experts=16, top_k=2, sequences=2, dtype=B.MOE_F32, balance=0.01, z=0.001), **kw})


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=1 << 30), dict(tokens=(1 << 30) + 2, top_k=1), dict(experts=0), dict(experts=1025), dict(top_k=0),
                                dict(top_k=17), dict(experts=4, top_k=5), dict(sequences=0), dict(sequences=-1),
                                dict(sequences=1 << 27), dict(dtype=2), dict(balance=NAN), dict(z=INF)])
def test_router_shapes(kw):
    s = router_shape(**kw)
    assert B.moe_router_loss_workspace_bytes(s) == -1
    assert B.lib().moe_router_loss(ctypes.byref(s), *P[:7], 1 << 20, None) == B.MOE_EINVAL
    assert B.lib().moe_router_backward(ctypes.byref(s), *P[:8], None) == B.MOE_EINVAL


@pytest.mark.parametrize("sequences", [(1 << 30) + 1, (1 << 31) - 512, (1 << 31) - 4, (1 << 31) - 1])
def test_router_sequences_that_the_kernels_cannot_count(sequences):
    """One expert leaves the product below 2^31; the kernels step over the sequences in 32 bits, by up to 512 and from up to 2^30."""
    s = router_shape(tokens=8, experts=1, top_k=1, sequences=sequences)
    assert B.moe_router_loss_workspace_bytes(s) == -1
    refused(B.lib().moe_router_loss(ctypes.byref(s), *P[:7], 1 << 60, None), "sequences")
    refused(B.lib().moe_router_backward(ctypes.byref(s), *P[:8], None), "sequences")
    assert B.moe_router_loss_workspace_bytes(router_shape(tokens=8, experts=1, top_k=1, sequences=1 << 30)) > 0


def test_router_arguments():
    L, s = B.lib(), router_shape()
    need = B.moe_router_loss_workspace_bytes(s)
    names = ("logits", "topk_idx", "spans", "counts", "means", "losses", "ws")
    at = dict(zip(names, P))

    def f(s=s, n=need, **kw):
        return L.moe_router_loss(ctypes.byref(s), *[kw.get(k, at[k]) for k in names], n, None)

    for k in names:
        if k != "spans":
            refused(f(**{k: None}), "too small" if k == "ws" else "null")
        refused(f(**{k: at[k] + 2}), "aligned")
    refused(f(n=need - 1), "too small")
    refused(f(router_shape(tokens=7), spans=None), "multiple")
    for kw in (dict(counts=P[0]), dict(counts=P[1] + 8), dict(means=P[3] + 4), dict(losses=P[4] + 4), dict(losses=P[2]),
               dict(ws=P[3]), dict(ws=P[0])):
        refused(f(**kw), "overlaps")
    bnames = ("logits", "topk_idx", "spans", "counts", "means", "d_loss", "d_weights", "dlogits")
    bat = dict(zip(bnames, P))

    def b(s=s, **kw):
        return L.moe_router_backward(ctypes.byref(s), *[kw.get(k, bat[k]) for k in bnames], None)

    for k in bnames:
        if k not in ("spans", "d_loss", "d_weights"):
            refused(b(**{k: None}), "null")
        refused(b(**{k: bat[k] + 2}), "aligned")
    refused(b(router_shape(tokens=7), spans=None), "multiple")
    for other in bnames[:-1]:
        refused(b(dlogits=bat[other]), "overlaps")


# ---- the gradient norm -------------------------------------------------------------------------------------------

def grads(*rows):
    table = (B.moe_grad_tensor * len(rows))()
    for q, kw in zip(table, rows):
        for k, v in {**dict(grad=P[0], out=None, n=100, grad_dtype=B.MOE_F32, out_dtype=0), **kw}.items():
            setattr(q, k, v)
    return table


@pytest.mark.parametrize("kw", [dict(n=-1), dict(n=1 << 41), dict(grad_dtype=2), dict(out=P[1], out_dtype=7), dict(grad=None),
                                dict(grad=P[0] + 2), dict(out=P[1] + 2, out_dtype=B.MOE_F32),
                                dict(out=P[1] + 1, out_dtype=B.MOE_BF16), dict(n=1 << 40)])
def test_grad_tensors(kw):
    t = grads(kw)
    assert B.moe_grad_workspace_bytes(t) == -1
    plan = B.moe_grad_plan()
    assert B.lib().moe_grad_bind(t, 1, P[5], 1 << 27, ctypes.byref(plan), None) == B.MOE_EINVAL


def test_grad_arguments():
    L, plan, t = B.lib(), B.moe_grad_plan(), grads({}, dict(grad=P[1], out=P[2], out_dtype=B.MOE_BF16))
    need = B.moe_grad_workspace_bytes(t)
    assert need > 0
    bind = lambda t=t, ws=P[5], n=need, plan=ctypes.byref(plan): L.moe_grad_bind(t, len(t), ws, n, plan, None)
    refused(bind(plan=None), "null")
    refused(bind(ws=None), "too small")
    refused(bind(n=need - 1), "too small")
    refused(bind(ws=P[5] + 8), "16-byte")
    for rows in ([{}, {}], [{}, dict(grad=P[0] + 396)], [dict(out=P[0])], [dict(out=P[0], out_dtype=B.MOE_F32)],
                 [dict(out=P[1], out_dtype=1), dict(grad=P[1] + 100)], [dict(grad=P[5])], [dict(out=P[5] + 16, out_dtype=1)]):
        refused(bind(grads(*rows), n=1 << 20), "overlaps")
    assert B.moe_grad_workspace_bytes(grads(dict(grad=None, n=0))) >= 0
    # not bound
    refused(L.moe_grad_norm(None, 1.0, 1.0, P[6], P[7], None), "not bound")
    bad = B.moe_grad_plan(None, 3, 1, 0)
    refused(L.moe_grad_norm(ctypes.byref(bad), 1.0, 1.0, P[6], P[7], None), "not bound")
    refused(L.moe_grad_clip(ctypes.byref(bad), P[7], None), "not bound")
    ok = B.moe_grad_plan(P[5], 1, 1, 0)
    norm = lambda m=1.0, f=1.0, a=P[6], b=P[7]: L.moe_grad_norm(ctypes.byref(ok), m, f, a, b, None)
    for m in (0.0, -1.0, NAN, 1e39):
        refused(norm(m=m), "max_norm")
    for f in (0.0, -1.0, NAN, INF, 1e39, 1e-60):
        refused(norm(f=f), "factor")
    refused(norm(a=None), "null")
    refused(norm(b=None), "null")
    refused(norm(a=P[6] + 2), "aligned")
    refused(norm(a=P[7]), "overlaps")
    refused(L.moe_grad_clip(ctypes.byref(ok), None, None), "null")
    refused(L.moe_grad_clip(ctypes.byref(ok), P[7] + 1, None), "aligned")


@pytest.mark.parametrize("chunks", [0, 1, 3, 5000])
def test_grad_numbers_in_the_plans_workspace(chunks):
    """Its records hold the addresses that the next call reads and writes."""
    L, plan = B.lib(), B.moe_grad_plan(P[5], chunks, 1, 0)
    t = grads(*([dict(n=chunks * 8192)] if chunks else []))
    end = P[5] + B.moe_grad_workspace_bytes(t)
    for at in {P[5], P[5] + 4, (P[5] + end) // 8 * 4, end - 4}:
        refused(L.moe_grad_norm(ctypes.byref(plan), 1.0, 1.0, at, P[7], None), "workspace")
        refused(L.moe_grad_norm(ctypes.byref(plan), 1.0, 1.0, P[7], at, None), "workspace")
        refused(L.moe_grad_clip(ctypes.byref(plan), at, None), "workspace")


@pytest.mark.parametrize("experts", [1, 64, 1024])
@pytest.mark.parametrize("sequences", [1, 3, 40, 255, 256, 3000])
def test_router_workspace_serves_fewer_tokens(experts, sequences):
    """A workspace of the largest call holds every smaller one's."""
    sizes = [B.moe_router_loss_workspace_bytes(router_shape(tokens=sequences * t, experts=experts, top_k=1, sequences=sequences))
             for t in (0, 1, 7, 16, 100, 1000, 5000, 20000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def test_dynamic_lds_is_aligned_to_its_vector_accesses():
    """Dynamic LDS starts behind a kernel's static LDS, at its own type's alignment unless it is declared with more."""
    import glob
    import os
    import re

    seen = 0
    for path in glob.glob(os.path.join(os.path.dirname(B.__file__), "csrc", "*.hip")):
        text = open(path).read()
        for m in re.finditer(r"extern __shared__ (__align__\((\d+)\) )?[\w ]+? (\w+)\[\];", text):
            body = text[m.end(): text.find("extern __shared__", m.end())]
            if re.search(r"\(const float4\*\)\(%s|\(float4\*\)\(%s" % (m.group(3), m.group(3)), body):
                assert int(m.group(2) or 4) >= 16, (path, m.group(0))
                seen += 1
    assert seen > 0
