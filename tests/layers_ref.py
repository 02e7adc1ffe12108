"""Plain 64-bit forms of the gated recurrence, the q/k norms with rotary
positions and causal attention, on the CPU, with the error bounds that the
tests hold the kernels to.

A rounding to type t is off by at most U[t] relative (half a step)."""
from __future__ import annotations

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F64 = torch.float64


def f64(t):
    return None if t is None else t.detach().to("cpu", F64)


def worst(got, ref, bound):
    """max over elements of |got - ref| / bound (0 / 0 is 0)."""
    g, r = f64(got), ref.to(F64)
    assert g.shape == r.shape, (g.shape, r.shape)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), "NaN in other places"
    inf = torch.isinf(r)
    assert torch.equal(g[inf], r[inf]) and not torch.isinf(g[~inf]).any(), "infinities differ"
    ok = torch.isfinite(r)
    if not ok.any():
        return 0.0
    d = (g - r).abs()[ok]
    b = bound.expand_as(r)[ok]
    return float(torch.where(d == 0, torch.zeros_like(d), d / b.clamp(min=1e-300)).max())


# --------------------------------------------------------------------------
# gated recurrence
def gated(x, r, i, decay, h0=None, c=8.0, cu=None):
    """(y, hT) token by token; differentiable.  x [B, T, D] or [T, D] with cu."""
    a = torch.exp(-c * torch.nn.functional.softplus(decay, threshold=1e9) * torch.sigmoid(r))
    b = torch.sqrt(-torch.expm1(2 * torch.log(a))) * torch.sigmoid(i) * x
    if cu is None:
        h = h0 if h0 is not None else torch.zeros_like(b[:, 0])
        ys = []
        for t in range(x.shape[1]):
            h = a[:, t] * h + b[:, t]
            ys.append(h)
        return torch.stack(ys, 1), h
    ys, ends = [], []
    for s in range(len(cu) - 1):
        h = h0[s] if h0 is not None else torch.zeros_like(b[0])
        for t in range(cu[s], cu[s + 1]):
            h = a[t] * h + b[t]
            ys.append(h)
        ends.append(h)
    y = torch.stack(ys) if ys else x[:0]
    return y, torch.stack(ends)


def gated_grads(x, r, i, decay, dy, h0=None, dhT=None, c=8.0, cu=None):
    v = dict(x=f64(x), r=f64(r), i=f64(i), decay=f64(decay))
    if h0 is not None:
        v["h0"] = f64(h0)
    v = {k: t.clone().requires_grad_(True) for k, t in v.items()}
    y, hT = gated(v["x"], v["r"], v["i"], v["decay"], v.get("h0"), c, cu)
    loss = (y * f64(dy)).sum()
    if dhT is not None:
        loss = loss + (hT * f64(dhT)).sum()
    g = torch.autograd.grad(loss, list(v.values()), allow_unused=True)
    return dict(zip(v, (torch.zeros_like(t) if d is None else d for t, d in zip(v.values(), g))))


def gated_bound(ref, amax, T, dtype):
    """Each step's a is off by at most 2^-20 relative in fp32 (its logarithm a
    product of three roundings and three hardware functions of 1 ulp, times
    at most 8; the exponential 1 ulp) and each b by 2^-20; both pass through
    min(T, 1 / (1 - amax)) steps.  Then one rounding to the type."""
    span = min(T, 1.0 / max(1e-9, 1.0 - amax))
    scale = ref.abs().amax(0, keepdim=True).clamp(min=float(ref.abs().mean()) + 1e-30)
    return 2.0 ** -20 * (span + 2) * scale + (U[dtype] if dtype != torch.float32 else 0.0) * ref.abs()


# --------------------------------------------------------------------------
# q/k norms and rotation
def qk_one(v, pos, w, eps, base, rot, half):
    """One of q, k: v [T, H, D] fp64 -> rotated, by complex products."""
    n = rot // 2
    u = v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps)
    if w is not None:
        u = u * w
    if n == 0:
        return u
    phi = pos.to(F64)[:, None] * torch.tensor([base ** (-2.0 * j / rot) for j in range(n)], dtype=F64)
    turn = torch.polar(torch.ones_like(phi), phi)[:, None]
    if half:
        z = torch.complex(u[..., :n], u[..., n:rot]) * turn
        return torch.cat([z.real, z.imag, u[..., rot:]], -1)
    z = torch.complex(u[..., 0:rot:2], u[..., 1:rot:2]) * turn
    return torch.cat([torch.stack([z.real, z.imag], -1).flatten(-2), u[..., rot:]], -1)


# --------------------------------------------------------------------------
# attention: one sequence, all heads
def attn(q, k, v, scale):
    """fp64 (o, lse, p): q [Lq, Hq, D], k and v [Lk, Hk, D]."""
    Lq, Hq, D = q.shape
    Lk, Hk = k.shape[:2]
    kk, vv = (t.repeat_interleave(Hq // Hk, 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, kk) * scale
    hidden = torch.arange(Lk)[None, :] > torch.arange(Lq)[:, None] + (Lk - Lq)
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1) if Lk else torch.full((Hq, Lq), -math.inf, dtype=F64)
    p = torch.exp(s - torch.where(torch.isinf(lse) & (lse < 0), torch.zeros_like(lse), lse)[..., None])
    p = torch.where(hidden, torch.zeros_like(p), p)
    return _weighted(p, vv, hidden), lse.t(), p


def _weighted(p, vv, hidden):
    """sum_j p_ij v_j over the keys that i sees (a hidden key's value is not
    multiplied by its zero weight)."""
    fine = torch.where(torch.isfinite(vv), vv, torch.zeros_like(vv))
    o = torch.einsum("hij,jhd->ihd", p, fine)
    if not torch.isfinite(vv).all():
        for j, h, d in torch.nonzero(~torch.isfinite(vv)).tolist():
            o[~hidden[:, j], h, d] += vv[j, h, d]
    return o


def attn_bound(q, k, v, o, p, scale, dtype):
    """Scores: D products and sums in fp32, off by D 2^-24 of the sum of
    absolute products; weights by that plus 2^-21, rounded to the type before
    the product with v; the result rounded once more."""
    G = q.shape[1] // k.shape[1]
    ka, va = (t.abs().repeat_interleave(G, 1) for t in (k, v))
    ds = 2.0 ** -24 * (q.shape[2] + 8) * abs(scale) * torch.einsum("ihd,jhd->hij", q.abs(), ka)
    rel = ds + 2.0 ** -20 + (U[dtype] if dtype == torch.bfloat16 else 2.0 ** -24 * (k.shape[0] + 8))
    b = torch.einsum("hij,jhd->ihd", p * rel, va) + \
        o.abs() * torch.einsum("hij->ih", p * (ds + 2.0 ** -20))[..., None]
    return b + U[dtype] * o.abs() + 1e-30


def attn_grads(q, k, v, do, scale, dtype):
    """((dq, dk, dv), bounds) of one sequence.  The bounds: scores as above;
    weights and ds rounded to the type (by u of each) before the products;
    D_i = <o_i, do_i> from an o that is off by attn_bound; results rounded."""
    G = q.shape[1] // k.shape[1]
    kk, vv = (t.repeat_interleave(G, 1) for t in (k, v))
    o, _, p = attn(q, k, v, scale)
    dp = torch.einsum("ihd,jhd->hij", do, vv)
    D = (o * do).sum(-1).t()[..., None]
    ds = p * (dp - D)
    fold = lambda t: t.view(t.shape[0], t.shape[1] // G, G, t.shape[2]).sum(2)
    dq = scale * torch.einsum("hij,jhd->ihd", ds, kk)
    dk = fold(scale * torch.einsum("hij,ihd->jhd", ds, q))
    dv = fold(torch.einsum("hij,ihd->jhd", p, do))
    n = q.shape[2] + max(q.shape[0], k.shape[0]) * G + 16
    e = 2.0 ** -24 * n
    u = U[dtype] if dtype == torch.bfloat16 else e
    a = lambda t: t.abs()
    srel = 2.0 ** -24 * (q.shape[2] + 8) * abs(scale) * torch.einsum("ihd,jhd->hij", a(q), a(kk)) + 2.0 ** -20
    dpa = torch.einsum("ihd,jhd->hij", a(do), a(vv))
    ob = attn_bound(q, k, v, o, p, scale, dtype)
    Db = (ob * a(do)).sum(-1).t()[..., None] + e * (a(o) * a(do)).sum(-1).t()[..., None]
    pb = p * (srel + u)
    dsb = a(ds) * (srel + u) + p * (e * dpa + Db)
    bq = abs(scale) * (torch.einsum("hij,jhd->ihd", dsb + e * a(ds), a(kk)))
    bk = fold(abs(scale) * torch.einsum("hij,ihd->jhd", dsb + e * a(ds), a(q)))
    bv = fold(torch.einsum("hij,ihd->jhd", pb + e * p, a(do)))
    r = U[dtype]
    return (dq, dk, dv), (bq + r * a(dq) + 1e-30, bk + r * a(dk) + 1e-30, bv + r * a(dv) + 1e-30)
