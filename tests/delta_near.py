"""The gated delta rule of one sequence in 64 bits, on the CPU, and how far each output and gradient of the kernels
may be from it: a norm for each head.

What bounds an error:
  * the recurrence token by token in fp32, whose own error e32 is measured on the same inputs.  Of a product of
    sums of three bf16 parts those below 2^-24 are left out, where a product in fp32 is off by half of 2^-24: 6
    times as much at most, with the chunk's inverse 8;
  * U[dtype] of what is rounded to it;
  * by chance e32 may be small (a sequence of one token).  So a product's operands' rounding is added, of the
    norms of what is multiplied: 8 2^-24 of |A| |B| for three parts (their pairs below 2^-24 and a sum's
    roundings), 6 2^-16 for up to six products of two parts in a row, which in bf16 calls o, dq, dk, dg and
    dbeta pass through.
The norms, with M, D the largest of the states and of their gradients, U, O, R those of a chunk's u, do and
dr = dv / beta, kappa that of the chunk's inverse, K, Q the spectral norms of its keys and queries and P the norm of
scale Q K^T on and below the diagonal:
  o: scale Q M + P U       hT: kappa (M + K U)       dh0: kappa (D + scale Q O + beta K R)       dv: kappa beta R
  dq: scale O M + scale O U K       dk: scale O U Q + 2 beta R U K + beta R M + U D
  dbeta, of a row: |dr| (|v| + |k| M + sum over the rows before it of |k.k'| |u'|)
dg is a sum over the rows behind it in the chunk of q.dq, k.dk and v.dv, whose errors are independent."""
from __future__ import annotations

import torch

from tests import delta_ref
from tests.layers_ref import F64, U

NAMES = ("o", "hT", "dq", "dk", "dv", "dg", "dbeta", "dh0")


def plain(ins, h0, scale, do, dhT, t):
    """(o, hT, dq, dk (of value heads), dv, dg, dbeta, dh0), states [L + 1, ...], u [L, Hv, Dv] of the recurrence in
    type t; q and k already repeated for value heads."""
    x = [y.to(t, copy=True).requires_grad_(True) for y in (*ins, h0)]
    o, hs, ms = delta_ref.scan(*x, scale)
    loss = (o * do.to(t)).sum() + (hs[-1] * dhT.to(t)).sum()
    d = torch.autograd.grad(loss, x)
    return [o.detach(), hs[-1].detach(), *d], hs.detach(), (x[4][..., None] * ms).detach()


def heads(name, t):
    """[heads, everything else] of an output."""
    t = t.detach().to("cpu", F64)
    return t.flatten(1) if name in ("hT", "dh0") else t.transpose(0, 1).flatten(1)


def check(q, k, v, g, beta, h0, scale, dtype, do, dhT):
    """{name: (value, tolerance of the norm of each head)} for one sequence of at least one token; inputs of any
    device, of a head's value heads as the library takes them."""
    q, k, v, g, beta, h0, do, dhT = (t.detach().cpu() for t in (q, k, v, g, beta, h0, do, dhT))
    L, hv = v.shape[:2]
    group = hv // k.shape[1]
    wide = lambda t: t.repeat_interleave(group, 1)
    g = g.float().clamp(min=-1000.0)   # (-inf has no product with 0)
    ins = (wide(q), wide(k), v, g, beta)
    want, hs, us = plain(ins, h0, scale, do, dhT, F64)
    near = plain(ins, h0, scale, do, dhT, torch.float32)[0]
    Q, K, V, B, DO = (t.to(F64) for t in (ins[0], ins[1], v, beta, do))
    # the adjoint's states, from the last to the first
    dS = dhT.to(F64)
    D = dS.flatten(1).norm(dim=1)
    dr = torch.zeros_like(V)
    G = g.to(F64)
    for t in reversed(range(L)):
        dS = dS + scale * Q[t][:, :, None] * DO[t][:, None, :]
        D = torch.maximum(D, dS.flatten(1).norm(dim=1))
        dr[t] = torch.einsum("hkv,hk->hv", dS, K[t])
        dS = torch.exp(G[t])[:, None, None] * (dS - K[t][:, :, None] * (B[t][:, None] * dr[t])[:, None, :])
    cut = range(0, L, 64)
    most = lambda f: torch.stack([f(slice(c, c + 64)) for c in cut]).amax(0)
    M = hs.flatten(2).norm(dim=2).amax(0)
    W, O, R = (most(lambda c: t[c].norm(dim=(0, 2))) for t in (us, DO, dr))
    spec = lambda t: most(lambda c: torch.linalg.matrix_norm(t[c].transpose(0, 1), 2))
    K2, Q2, bm = spec(K), spec(Q), B.abs().amax(0)
    P = abs(scale) * most(lambda c: torch.linalg.matrix_norm((Q[c].transpose(0, 1) @ K[c].permute(1, 2, 0).contiguous()).tril()))
    pairs = torch.cat([torch.einsum("hij,jh->ih", (K[c].transpose(0, 1) @ K[c].permute(1, 2, 0).contiguous()).abs().tril(-1),
                                    us[c].norm(dim=2)) for c in (slice(c, c + 64) for c in cut)])
    kap = delta_ref.kappa(k.to(F64), G, B, hv)
    p = abs(scale) * O * W
    n = len(cut) ** 0.5
    size = {"o": n * (abs(scale) * Q2 * M + P * W), "hT": kap * (M + K2 * W),
            "dh0": kap * (D + abs(scale) * Q2 * O + bm * K2 * R), "dv": kap * n * bm * R,
            "dq": n * (abs(scale) * O * M + p * K2), "dk": n * (p * Q2 + 2 * bm * R * W * K2 + bm * R * M + W * D),
            "dbeta": (dr.norm(dim=2) * (V.norm(dim=2) + K.norm(dim=2) * M + pairs)).norm(dim=0)}
    rows = Q.norm(dim=2) * want[2].norm(dim=2) + K.norm(dim=2) * want[3].norm(dim=2) + 2 * V.norm(dim=2) * want[4].norm(dim=2)
    behind = torch.stack([rows[t:t // 64 * 64 + 64].pow(2).sum(0) for t in range(L)]).sum(0).sqrt()
    out = {}
    for name, w, x in zip(NAMES, want, near):
        e = 2.0 ** -16 * 6 if dtype == torch.bfloat16 and name in ("o", "dq", "dk", "dg", "dbeta") else 2.0 ** -24 * 8
        tol = 8 * (heads(name, x) - heads(name, w)).norm(dim=1) + e * (behind if name == "dg" else size[name])
        if name in ("dq", "dk"):   # the value heads' sum, in order
            w = w.unflatten(1, (-1, group)).sum(2)
            tol = tol.view(-1, group).sum(1) + 2.0 ** -24 * group * heads(name, w).norm(dim=1)
        if name not in ("hT", "dh0"):
            tol = tol + U[dtype] * heads(name, w).norm(dim=1)
        out[name] = (w, tol + 1e-30)
    return out


def off(name, got, want, tol):
    """The largest of the heads' errors, of their tolerance."""
    return float(((heads(name, got) - heads(name, want)).norm(dim=1) / tol).max())
