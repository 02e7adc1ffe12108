"""The gated delta rule in 64 bits, on the CPU, token by token, with its adjoint, and the bounds that the
tests hold the kernels to.

The bounds are norms per sequence and head.  A product in fp32 of n terms is off by at most n 2^-24
|A| |B| (Frobenius).  A chunk of 64 tokens chains K S, T R and K^T U, n <= 128 each; K of 64 keys of
length <= 1 has a norm of at most 8 and T, here, of kappa, which is computed.  So a chunk's state is off
by at most 3 * 128 * 2^-24 * 8 kappa of |S| + |U|, and as later tokens only shrink a difference (a decay
<= 1, and 1 - beta k k^T for beta <= 2 and |k| <= 1), the chunks' errors add up.  The gradients' chain is
its mirror image; each gradient is then one more sum of products of those.  Outputs in bf16 also pass
operands of two bf16 parts (2^-16 each) and one rounding, U[bf16]."""
from __future__ import annotations

import torch

from tests.layers_ref import F64, U, f64


def scan(q, k, v, g, beta, h0, scale):
    """One sequence: q, k [L, Hk, Dk], v [L, Hv, Dv], g, beta [L, Hv], h0 [Hv, Dk, Dv] or None.  Returns
    (o, states [L + 1, Hv, Dk, Dv], miss [L, Hv, Dv]); differentiable."""
    L, hv = v.shape[:2]
    n = hv // k.shape[1]
    h = h0 if h0 is not None else torch.zeros(hv, k.shape[2], v.shape[2], dtype=F64)
    o, hs, ms = [], [h], []
    for t in range(L):
        kt, qt = (x[t].repeat_interleave(n, 0) for x in (k, q))
        h = torch.exp(g[t])[:, None, None] * h
        m = v[t] - torch.einsum("hkv,hk->hv", h, kt)
        h = h + torch.einsum("hk,hv->hkv", kt, beta[t][:, None] * m)
        o.append(scale * torch.einsum("hkv,hk->hv", h, qt))
        hs.append(h)
        ms.append(m)
    z = torch.zeros(0, hv, v.shape[2], dtype=F64)
    return (torch.stack(o) if o else z), torch.stack(hs), (torch.stack(ms) if ms else z)


def kappa(k, g, beta, hv):
    """The largest norm of (1 + A)^-1 over chunks and heads."""
    n, worst = hv // k.shape[1], 1.0
    for c in range(0, k.shape[0], 64):
        kk, G = k[c:c + 64].repeat_interleave(n, 1), g[c:c + 64].clamp(min=-128).cumsum(0)
        for h in range(hv):
            E = (kk[:, h] @ kk[:, h].t()) * torch.exp((G[:, None, h] - G[None, :, h]).clamp(max=0))
            A = torch.tril(E, -1) * beta[c:c + 64, h][:, None]
            worst = max(worst, float(torch.linalg.matrix_norm(torch.linalg.inv(torch.eye(len(A), dtype=F64) + A), 2)))
    return worst


def check(q, k, v, g, beta, h0, scale, dtype, do=None, dhT=None):
    """{name: (value, bound)} for one sequence; gradients where do is given.  Inputs on any device."""
    ins = [f64(t) for t in (q, k, v, g, beta)]
    H0 = f64(h0)
    grads = do is not None
    if grads:
        ins = [t.clone().requires_grad_(True) for t in ins]
        H0 = None if H0 is None else H0.clone().requires_grad_(True)
    Q, K, V, Gt, B = ins
    hv, dv = V.shape[1:]
    n = hv // K.shape[1]
    o, hs, ms = scan(Q, K, V, Gt, B, H0, scale)
    hT = hs[-1]
    if grads:
        leaves = ins + ([] if H0 is None else [H0])
        loss = (o * f64(do)).sum() + (0 if dhT is None else (hT * f64(dhT)).sum())
        d = torch.autograd.grad(loss, leaves, allow_unused=True)
        d = [torch.zeros_like(x) if y is None else y for x, y in zip(leaves, d)]
    Q, K, V, Gt, B, o, hs, ms, hT = (t.detach() for t in (Q, K, V, Gt, B, o, hs, ms, hT))
    chunks = (V.shape[0] + 63) // 64 + 1
    kap = kappa(K, Gt, B, hv)
    e = 3 * 128 * 2.0 ** -24 * 8 * kap * chunks
    S = hs.flatten(2).norm(dim=2).amax(0)                                  # [Hv]
    u = B[..., None] * ms
    W = torch.stack([u[c:c + 64].norm(dim=(0, 2)) for c in range(0, max(1, u.shape[0]), 64)]).amax(0) if len(u) else S * 0
    size = S + W                                                          # of a chunk's state and writes
    two = 2.0 ** -15 if dtype == torch.bfloat16 else 0.0
    qn = Q.norm(dim=-1).amax() if len(Q) else torch.tensor(0.0)
    out = {"hT": (hT, (e * size + 1e-30)[:, None, None]),
           "o": (o, U[dtype] * o.abs() + abs(scale) * qn * ((e + two * kap * 8) * size)[None, :, None] + 1e-30)}
    if not grads:
        return out
    # the adjoint's sizes: dS of every token
    dS = torch.zeros_like(hs[0]) if dhT is None else f64(dhT)
    big = dS.flatten(1).norm(dim=1)
    dc = f64(do)
    for t in reversed(range(V.shape[0])):
        kt, qt = (x[t].repeat_interleave(n, 0) for x in (K, Q))
        dS = dS + scale * torch.einsum("hk,hv->hkv", qt, dc[t])
        big = torch.maximum(big, dS.flatten(1).norm(dim=1))
        du = torch.einsum("hkv,hk->hv", dS, kt)
        dS = torch.exp(Gt[t])[:, None, None] * (dS - torch.einsum("hk,hv->hkv", kt, B[t][:, None] * du))
    O = torch.stack([dc[c:c + 64].norm(dim=(0, 2)) for c in range(0, max(1, len(dc)), 64)]).amax(0) * abs(scale) * qn * 8 \
        if len(dc) else big * 0
    dsize = big + O
    # each gradient is a sum of products of two of these; their errors are those of both
    f = 4 * (e + two * kap * 8)
    prod = size * dsize
    bk = (f * kap * prod).view(-1, n).sum(1)[None, :, None]
    r = U[dtype]
    names = ("dq", "dk", "dv", "dg", "dbeta")
    bounds = (bk / max(float(qn), 1e-30) + r * d[0].abs(), bk + r * d[1].abs(),
              (f * kap * dsize)[None, :, None] + r * d[2].abs(),
              # a sum of up to 64 rows' terms
              64 * (f * kap * prod)[None] + r * d[3].abs(), 8 * (f * kap * prod)[None] + r * d[4].abs())
    for name, val, b in zip(names, d, bounds):
        out[name] = (val, b + 1e-30)
    if H0 is not None:
        out["dh0"] = (d[5], (4 * e * kap * dsize + 1e-30)[:, None, None])
    return out
