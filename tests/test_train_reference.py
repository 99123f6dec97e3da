"""The 64-bit references of the training operators against autograd (no GPU)."""
import pytest
import torch

import train_reference as ref

D = torch.float64


def rnd(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=D)


@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("pre", ["none", "layer", "rms"])
def test_residual_norm_is_autograds(post, pre):
    r, T, d, eps, rho = rnd(1), 5, 12, 1e-5, 0.7
    names = ([] if post == "none" else ["post_weight", "post_bias"]) + ["gate"] + ([] if pre == "none" else ["pre_weight", "pre_bias"])
    leaf = {n: r(d).requires_grad_() for n in names}
    leaf.update(x=r(T, d).requires_grad_(), h=r(T, d).requires_grad_(), row_gate=r(T).requires_grad_())
    w = {n: leaf[n].detach() for n in names}

    def norm(v, kind, where):
        if kind == "none":
            return v
        if kind == "layer":
            v = v - v.mean(1, keepdim=True)
        return v / (v.square().mean(1, keepdim=True) + eps).sqrt() * leaf[where + "_weight"] + leaf[where + "_bias"]

    s = rho * leaf["x"] + leaf["row_gate"][:, None] * leaf["gate"] * norm(leaf["h"], post, "post")
    n = norm(s, pre, "pre")
    ds, dn = r(T, d), r(T, d) if pre != "none" else None
    loss = (s * ds).sum() + (0 if dn is None else (n * dn).sum())
    loss.backward()
    got = ref.residual_norm(leaf["x"].detach(), leaf["h"].detach(), w, post, pre, rho, eps, leaf["row_gate"].detach(), ds, dn)
    want = {"s": s, "dx": leaf["x"].grad, "dh": leaf["h"].grad, **{k: leaf[k].grad for k in names + ["row_gate"]}}
    if pre != "none":
        want["n"] = n
    assert set(got) == set(want)
    for k, v in want.items():
        assert (got[k][0] - v).abs().max() <= 1e-11 * (1 + v.abs().max()), k


@pytest.mark.parametrize("padded", [False, True])
def test_router_loss_is_autograds(padded):
    r, T, G, k, S, a, b = rnd(2), 30, 7, 3, 5, 0.3, 0.2
    logits = r(T, G)
    logits[4, 2] = -float("inf")
    idx = torch.topk(logits, k).indices
    spans = torch.tensor([[0, 4], [4, 4], [5, 11], [12, 29], [29, 29]]) if padded else None
    leaf = logits.clone().requires_grad_()
    p, lse = torch.softmax(leaf, 1), torch.logsumexp(leaf, 1)
    rows = ref.rows_of(spans, T, S)
    live = [(x, y) for x, y in rows if y > x]
    N = sum(y - x for x, y in live)
    B = Z = 0.0
    inside = torch.zeros(T, dtype=torch.bool)
    for x, y in live:
        f = torch.bincount(idx[x:y].reshape(-1), minlength=G).to(D) * G / ((y - x) * k)
        B = B + (f * p[x:y].mean(0)).sum() / len(live)
        Z = Z + lse[x:y].square().sum() / N
        inside[x:y] = True
    dw = r(T, k)
    (1.7 * (a * B + b * Z) + (p.gather(1, idx) * dw)[inside].sum()).backward()
    counts, got = ref.router_loss(logits, idx, S, a, b, spans, dw, 1.7)
    assert counts.sum() == N * k and (padded or (counts.sum(1) == T // S * k).all())
    for want, value in ((torch.stack([a * B + b * Z, B, Z]), got["losses"][0]), (leaf.grad, got["dlogits"][0])):
        assert (value - want).abs().max() <= 1e-12


def test_grad_norm_is_the_norm_of_all():
    g = [rnd(3)(n).float() for n in (1, 10, 1000)]
    norm, scale = ref.grad_norm(g, 2.0, 0.5)
    want = 0.5 * torch.linalg.vector_norm(torch.cat(g).double())
    assert torch.isclose(norm, want) and torch.isclose(scale, 0.5 * 2.0 / (want + 1e-6))
    assert ref.grad_norm(g, 1e9, 0.5)[1] == 0.5 and ref.grad_norm([], 1.0, 1.0) == (0.0, 1.0)
