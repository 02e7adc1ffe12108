"""The norms around a block in 64 bits, on the CPU, with the error bounds that the tests hold the kernels
to.  A rounding to type t is off by at most U[t] relative (half a step)."""
from __future__ import annotations

import torch

from tests.layers_ref import F64, U, f64


def forward(x, y, gate, wy, scale, wn, eps, act, raw):
    """Everything on the way, as a dict; differentiable."""
    one = torch.ones((), dtype=F64)
    wy, scale, wn = (one if w is None else w for w in (wy, scale, wn))
    iy = one if raw else 1 / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps)
    u = y * iy
    if gate is None:
        a = torch.ones_like(y)
    else:
        a = {"linear": lambda g: g, "sigmoid": torch.sigmoid, "silu": lambda g: g * torch.sigmoid(g)}[act](gate)
    z = u * wy
    t = scale * a * z
    h = x + t
    ih = 1 / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + eps)
    return dict(iy=iy, u=u, a=a, z=z, t=t, h=h, ih=ih, n=h * ih * wn)


def check(x, y, gate, wy, scale, wn, eps, act, raw, dtype, dh, dn):
    """{name: (value, bound)} of the outputs and, where dh or dn is given, of the gradients.

    In fp32: a norm is off by at most 2^-20 of itself (a sum of squares taken in parts of at most 16, 64
    and 16 terms, and the hardware's root, 1 ulp); act(g) by 2^-21 (1 + |g|) relative for the product with
    1.44 |g| in the exponent; products and sums by 2^-24 each.  Then one rounding to the type."""
    X, Y, G, WY, SC, WN = (f64(t) for t in (x, y, gate, wy, scale, wn))
    leaves = {k: v.clone().requires_grad_(True) for k, v in
              (("x", X), ("y", Y), ("gate", G), ("y_weight", WY), ("scale", SC), ("n_weight", WN)) if v is not None}
    get = leaves.get
    f = forward(get("x"), get("y"), get("gate"), get("y_weight"), get("scale"), get("n_weight"), eps, act, raw)
    v = {k: t.detach() for k, t in f.items()}
    one = torch.ones((), dtype=F64)
    WY, SC, WN = (one if w is None else w for w in (WY, SC, WN))
    ga = torch.zeros_like(X) if G is None else G.abs()
    et = 2.0 ** -20 + 2.0 ** -21 * (1 + ga)
    mean = lambda t: t.mean(-1, keepdim=True)
    bh = et * v["t"].abs() + 2.0 ** -23 * (v["h"].abs() + v["t"].abs())
    r = v["ih"] * torch.sqrt(mean(bh * bh)) + 2.0 ** -20   # of rms(h), relative
    u = U[dtype]
    out = {"h": (v["h"], bh + u * v["h"].abs() + 1e-30),
           "n": (v["n"], WN.abs() * v["ih"] * bh + v["n"].abs() * (r + u + 2.0 ** -22) + 1e-30)}
    if dh is None and dn is None:
        return out
    loss = 0.0
    if dh is not None:
        loss = loss + (f["h"] * f64(dh)).sum()
    if dn is not None:
        loss = loss + (f["n"] * f64(dn)).sum()
    d = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)))
    d = {k: torch.zeros_like(leaves[k]) if t is None else t for k, t in d.items()}
    m = v["h"] * v["ih"]
    bm = v["ih"] * bh + m.abs() * r
    bH = 2.0 ** -23 * d["x"].abs()
    if dn is not None:
        gm = f64(dn) * WN
        c = mean((gm * m).abs())
        bH = bH + v["ih"] * (gm.abs() * (r + 2.0 ** -21) + bm * c + m.abs() * (mean(gm.abs() * bm) + c * (2 * r + 2.0 ** -19)))
    dH = d["x"].abs()
    out["dx"] = (d["x"], bH + u * dH + 1e-30)
    k = (SC * v["a"] * WY).abs()
    gu = dH * k
    bg = k * bH + gu * et
    au = v["u"].abs()
    by = bg + (0 if raw else au * mean(bg * au) + au * mean(gu * au) * 2.0 ** -18 + gu * 2.0 ** -20)
    out["dy"] = (d["y"], v["iy"] * by + u * d["y"].abs() + 1e-30)
    if gate is not None:
        s = torch.sigmoid(G)
        da = {"linear": torch.ones_like(G), "sigmoid": s * (1 - s), "silu": s * (1 + G * (1 - s))}[act].abs()
        sz = (SC * v["z"]).abs()
        out["dgate"] = (d["gate"], sz * (da * bH + dH * 2.0 ** -20 * (1 + ga)) + d["gate"].abs() * (et + u) + 1e-30)
    # sums over rows: of a workgroup one after the other (at least 256 of them), then of the workgroups
    n = 2.0 ** -24 * (x.shape[0] / 256 + 300)
    rows = (bH * (v["a"] * v["u"]).abs() + dH * (v["a"] * v["u"]).abs() * (et + n)).sum(0)
    if wy is not None:
        out["dy_weight"] = (d["y_weight"], rows * SC.abs() + 1e-30)
    if scale is not None:
        out["dscale"] = (d["scale"], rows * WY.abs() + 1e-30)
    if wn is not None:
        out["dn_weight"] = (d["n_weight"], torch.zeros_like(d["n_weight"]) + 1e-30 if dn is None else
                            (f64(dn).abs() * (bm + m.abs() * (n + 2.0 ** -22))).sum(0) + 1e-30)
    return out
