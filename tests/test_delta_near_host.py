"""Host-only: the tolerances that the gated delta rule's outputs and gradients are held to let none of these pass:
zeros, the wrong sign, a segment's map or a term of a gradient left out."""
import pytest
import torch

from tests import delta_near, delta_ref

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
SHAPES = [(1, 1, 1, 64, 64), (3, 2, 2, 64, 128), (65, 1, 2, 128, 64), (200, 1, 2, 128, 128)]


def _inputs(L, hk, hv, dk, dv, dtype, rate=0.05):
    g = torch.Generator().manual_seed(L + dk)
    n = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    ins = [t.to(dtype) for t in (unit(n(L, hk, dk)), unit(n(L, hk, dk)), n(L, hv, dv), -torch.rand(L, hv, generator=g) * rate,
                                 torch.sigmoid(n(L, hv)))]
    return ins, n(hv, dk, dv), n(L, hv, dv).to(dtype), n(hv, dk, dv)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_zeros_and_wrong_signs_are_found(shape, dtype):
    L, hk, hv, dk, dv = shape
    ins, h0, do, dhT = _inputs(*shape, dtype)
    want = delta_near.check(*ins, h0, dk ** -0.5, dtype, do, dhT)
    assert set(want) == set(delta_near.NAMES)
    for name, (w, tol) in want.items():
        size = delta_near.heads(name, w).norm(dim=1)
        assert (tol <= size / 16).all(), (name, tol / size)
        assert delta_near.off(name, w, w, tol) == 0
        assert delta_near.off(name, torch.zeros_like(w), w, tol) > 10 and delta_near.off(name, -w, w, tol) > 20, name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_map_left_out_is_found(dtype):
    """S = E + d S0 behind the second of three segments of 64, for E + d S0 + F S0."""
    ins, h0, do, dhT = _inputs(192, 1, 2, 64, 64, dtype, 1e-3)
    want = delta_near.check(*ins, h0, 0.125, dtype, do, dhT)
    q, k, v, g, b = (t.to(F64) for t in ins)
    part = lambda s, h: delta_ref.scan(*(t[s] for t in (q, k, v, g, b)), h, 0.125)[:2]
    first, second, third = slice(0, 64), slice(64, 128), slice(128, 192)
    o1, h1 = part(first, h0.to(F64))
    o2, _ = part(second, h1[-1])
    end = part(second, None)[1][-1] + torch.exp(g[second].sum(0))[:, None, None] * h1[-1]
    o3, h3 = part(third, end)
    assert delta_near.off("hT", h3[-1], *want["hT"]) > 10
    assert delta_near.off("o", torch.cat([o1, o2, o3]), *want["o"]) > 10


def _scan(q, k, v, g, beta, h, scale, k_miss, g_miss):
    """The recurrence, with the keys and decays of what a write misses given apart."""
    o = []
    for t in range(v.shape[0]):
        m = v[t] - torch.einsum("hkv,hk->hv", torch.exp(g_miss[t])[:, None, None] * h, k_miss[t])
        h = torch.exp(g[t])[:, None, None] * h + torch.einsum("hk,hv->hkv", k[t], beta[t][:, None] * m)
        o.append(scale * torch.einsum("hkv,hk->hv", h, q[t]))
    return torch.stack(o), h


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_term_of_a_gradient_left_out_is_found(dtype):
    """dk without the keys' part in what a write misses, dg without the decays' part in it."""
    ins, h0, do, dhT = _inputs(100, 2, 2, 64, 64, dtype)
    want = delta_near.check(*ins, h0, 0.125, dtype, do, dhT)
    for left in (None, "dk", "dg"):
        x = [t.to(F64).requires_grad_(True) for t in ins]
        o, h = _scan(*x, h0.to(F64), 0.125, x[1].detach() if left == "dk" else x[1], x[3].detach() if left == "dg" else x[3])
        d = dict(zip(("dq", "dk", "dv", "dg", "dbeta"), torch.autograd.grad(
            (o * do.to(F64)).sum() + (h * dhT.to(F64)).sum(), x)))
        for name, t in d.items():
            e = delta_near.off(name, t, *want[name])
            assert e > 10 if name == left else e < 1e-3, (left, name, e)
