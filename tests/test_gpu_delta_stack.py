"""Blocks of the gated delta rule as a stack runs them: the norms before and after a block with its gate and
residual scale, its queries and keys brought to length 1, the scan over a packed prompt, and one token after
another from where it ended."""
import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import block_ref, delta_ref
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _near(name, a, b, tol):
    e = float((a.double().cpu() - b.double().cpu()).norm() / b.double().norm())
    say(f"  {name}: {e:.2e}")
    assert e <= tol, (name, e)


class Stack:
    """Two blocks: n -> q, k, v, g, beta and a gate by one product; the scan; a product; the norms."""

    def __init__(self, dtype, seed, hk=2, hv=4, dk=64, dv=64, width=200, layers=2):
        gen = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen)
        self.hk, self.hv, self.dk, self.dv, self.width = hk, hv, dk, dv, width
        self.at = [0, hk * dk, 2 * hk * dk, 2 * hk * dk + hv * dv]
        self.at += [self.at[-1] + hv, self.at[-1] + 2 * hv]
        cols = self.at[-1] + 8   # (rows of a multiple of 8)
        cols -= cols % 8
        w = lambda a, b: (n(a, b) * a ** -0.5).to(dtype).cuda()
        self.layers = [dict(a=w(width, cols), gate=w(width, width), out=w(hv * dv, width),
                            wq=torch.full((dk,), dk ** -0.5).cuda(), wk=torch.full((dk,), dk ** -0.5).cuda(),
                            wy=(0.5 + torch.rand(width, generator=gen)).cuda(), sc=(0.2 * n(width)).cuda(),
                            wn=(0.5 + torch.rand(width, generator=gen)).cuda()) for _ in range(layers)]

    def split(self, p):
        q, k, v, g, b = (p[:, s:e] for s, e in zip(self.at, self.at[1:]))
        heads = lambda t, h: t.unflatten(1, (h, -1))
        return (heads(q, self.hk), heads(k, self.hk), heads(v, self.hv),
                -torch.nn.functional.softplus(g.float() - 3).to(g.dtype), torch.sigmoid(b))

    def unit(self, q, k, L):
        at = torch.zeros(q.shape[0], dtype=torch.int32, device=q.device)
        return m3.qk_norm_rope(q, k, at, L["wq"], L["wk"], rotary_dim=0)

    def run(self, x, n, states, cu=None):
        """A prompt (cu) or one token a sequence; states advance."""
        for i, L in enumerate(self.layers):
            q, k, v, g, b = self.split(n @ L["a"])
            q, k = self.unit(q, k, L)
            if cu is None:
                o = m3.delta_step(states[i], q, k, v, g, b)
            else:
                o, states[i], _ = m3.delta_scan(q, k, v, g, b, h0=states[i], cu_seqlens=cu)
            x, n = m3.block_norm(x, o.flatten(1) @ L["out"], n @ L["gate"], L["wy"], L["sc"], L["wn"],
                                 flags=m3.M3_GATE_SIGMOID)
        return x, n

    def states(self, S):
        return [torch.zeros(S, self.hv, self.dk, self.dv, device="cuda") for _ in self.layers]


@pytest.mark.parametrize("dtype,tol", [(F32, 2e-5), (BF16, 3e-2)])
def test_prompt_then_steps_equals_longer_prompt(dtype, tol):
    lengths, steps = [130, 0, 70], 3
    st = Stack(dtype, 1)
    gen = torch.Generator().manual_seed(2)
    whole = [n + steps for n in lengths]
    x = [torch.randn(n, st.width, generator=gen).to(dtype).cuda() for n in whole]
    offs = lambda ls: torch.tensor([0] + torch.tensor(ls).cumsum(0).tolist(), dtype=torch.int32).cuda()
    norm = lambda t: m3.block_norm(t, torch.zeros_like(t), n_weight=torch.ones(st.width, device="cuda"))[1]
    every = torch.cat(x)
    sa = st.states(3)
    ya, na = st.run(every, norm(every), sa, offs(whole))
    short = torch.cat([t[:n] for t, n in zip(x, lengths)])
    sb = st.states(3)
    yb, _ = st.run(short, norm(short), sb, offs(lengths))
    ends = offs(whole)[1:].long()
    _near("prompt", yb, torch.cat([t[:n] for t, n in zip(ya.split(whole), lengths)]), tol)
    for s in range(steps):
        t = torch.stack([a[n + s] for a, n in zip(x, lengths)])
        y, n = st.run(t, norm(t), sb)
        _near(f"step {s}", y, ya[ends - steps + s], tol)
    for a, b in zip(sb, sa):
        _near("state", a, b, tol)


def test_gradients_through_a_block():
    """block_norm -> length 1 -> scan -> block_norm, backwards through the library's calls, against the 64-bit
    definitions differentiated together."""
    lengths, hk, hv, dk, dv = [70, 0, 31], 1, 2, 64, 64
    T, width = 101, 2 * 64 + 2 * 64
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    x, y0, gate, mix = n(T, width), n(T, width), n(T, width), n(hv * dv, width) / 8
    g, b = -torch.nn.functional.softplus(n(T, hv) - 2), torch.sigmoid(n(T, hv))
    wy, sc, wn, wq, wk = (0.5 + torch.rand(m, generator=gen).cuda() for m in (width, width, width, dk, dk))
    wq, wk, eps = wq * dk ** -0.5, wk * dk ** -0.5, 1e-6
    dh, dn = n(T, width), n(T, width)
    cu = torch.tensor([0, 70, 70, 101], dtype=torch.int32).cuda()
    at = torch.zeros(T, dtype=torch.int32).cuda()
    cut = lambda t: (t[:, :64].unflatten(1, (1, 64)), t[:, 64:128].unflatten(1, (1, 64)), t[:, 128:].unflatten(1, (2, 64)))

    h1, n1 = m3.block_norm(x, y0, gate, wy, sc, wn, eps, m3.M3_GATE_SILU)
    q, k, v = cut(n1)
    qu, ku = m3.qk_norm_rope(q, k, at, wq, wk, eps, rotary_dim=0)
    o, _, st = m3.delta_scan(qu, ku, v, g, b, cu_seqlens=cu, want_states=True)
    y1 = o.flatten(1) @ mix
    h2, n2 = m3.block_norm(h1, y1, gate, wy, sc, wn, eps, m3.M3_GATE_SIGMOID)

    B2 = m3.block_norm_backward(h1, y1, dh, dn, gate, wy, sc, wn, eps, m3.M3_GATE_SIGMOID)
    D = m3.delta_scan_backward(qu, ku, v, g, b, (B2["y"] @ mix.t()).view(T, hv, dv).contiguous(), st, cu_seqlens=cu)
    Q = m3.qk_norm_rope_backward(q, k, at, D["q"], D["k"], wq, wk, eps, rotary_dim=0)
    dn1 = torch.cat([Q["q"].flatten(1), Q["k"].flatten(1), D["v"].flatten(1)], 1)
    B1 = m3.block_norm_backward(x, y0, B2["x"], dn1, gate, wy, sc, wn, eps, m3.M3_GATE_SILU)

    names = ("x", "y0", "gate", "wy", "sc", "wn", "wq", "wk", "g", "b")
    leaves = [ref.f64(t).requires_grad_(True) for t in (x, y0, gate, wy, sc, wn, wq, wk, g, b)]
    X, Y, G, WY, SC, WN, WQ, WK, GT, BT = leaves
    f1 = block_ref.forward(X, Y, G, WY, SC, WN, eps, "silu", False)
    a, c, vv = cut(f1["n"])
    unit = lambda t, w: ref.qk_one(t, at.cpu(), w, eps, 10000.0, 0, False)
    a, c = unit(a, WQ), unit(c, WK)
    offs = cu.tolist()
    od = torch.cat([delta_ref.scan(a[s:e], c[s:e], vv[s:e], GT[s:e], BT[s:e], None, dk ** -0.5)[0]
                    for s, e in zip(offs, offs[1:]) if e > s])
    f2 = block_ref.forward(f1["h"], od.flatten(1) @ ref.f64(mix), G, WY, SC, WN, eps, "sigmoid", False)
    # five fp32 operators in a row, each within about 2e-6 of its size
    _near("h", h2, f2["h"].detach(), 1e-5)
    _near("n", n2, f2["n"].detach(), 1e-5)
    want = dict(zip(names, torch.autograd.grad((f2["h"] * ref.f64(dh)).sum() + (f2["n"] * ref.f64(dn)).sum(), leaves)))
    got = dict(x=B1["x"], y0=B1["y"], gate=B1["gate"] + B2["gate"], wy=B1["y_weight"] + B2["y_weight"],
               sc=B1["scale"] + B2["scale"], wn=B1["n_weight"] + B2["n_weight"], wq=Q["q_weight"], wk=Q["k_weight"],
               g=D["g"], b=D["beta"])
    for k in names:
        _near("d" + k, got[k], want[k], 1e-5)


def test_steps_of_a_captured_stack():
    """Decode steps of the whole stack, captured once and replayed with eager work between, have the eager bits;
    two captured stacks on streams of their own keep theirs."""
    S = 5
    graphs = []
    for seed in (11, 12):
        st = Stack(BF16, seed)
        gen = torch.Generator().manual_seed(seed)
        toks = torch.randn(4, S, st.width, generator=gen).to(BF16).cuda()
        x, held = toks[0].clone(), st.states(S)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            st.run(x, x, [h.clone() for h in held])   # (the products' libraries are loaded)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                y, n = st.run(x, x, held)
        torch.cuda.synchronize()
        for h in held:
            h.zero_()
        graphs.append((st, toks, x, held, s, g, y))
    eager = [[] for _ in graphs]
    for (st, toks, *_), out in zip(graphs, eager):
        states = st.states(S)
        for t in toks:
            out.append((st.run(t, t, states)[0].clone(), [h.clone() for h in states]))
    torch.cuda.synchronize()
    for i in range(4):
        for st, toks, x, held, s, g, y in graphs:
            with torch.cuda.stream(s):
                x.copy_(toks[i])
                g.replay()
        torch.cuda.synchronize()
        for (st, toks, x, held, s, g, y), out in zip(graphs, eager):
            assert torch.equal(y, out[i][0]) and all(torch.equal(a, b) for a, b in zip(held, out[i][1])), i


def test_on_a_given_stream():
    st = Stack(BF16, 21)
    gen = torch.Generator().manual_seed(22)
    L = st.layers[0]
    x, n = (torch.randn(300, st.width, generator=gen).to(BF16).cuda() for _ in range(2))
    q, k, v, g, b = st.split(n @ L["a"])
    q, k = st.unit(q, k, L)
    cu = torch.tensor([0, 100, 300], dtype=torch.int32).cuda()
    do = torch.randn(v.shape, generator=gen).to(BF16).cuda()
    h = torch.randn(300, st.hv, st.dk, st.dv, generator=gen).cuda()

    def run(stream):
        o, hT, states = m3.delta_scan(q, k, v, g, b, cu_seqlens=cu, want_states=True, stream=stream)
        d = m3.delta_scan_backward(q, k, v, g, b, do, states, cu_seqlens=cu, stream=stream)
        hs = h.clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        y = m3.delta_step(hs, q, k, v, g, b, stream=stream)
        r = m3.block_norm(x, n, n, L["wy"], L["sc"], L["wn"], flags=m3.M3_GATE_SILU, stream=stream)
        e = m3.block_norm_backward(x, n, x, n, n, L["wy"], L["sc"], L["wn"], flags=m3.M3_GATE_SILU, stream=stream)
        return [o, hT, y, hs, *r] + [t for t in (*d.values(), *e.values()) if t is not None]

    want = run(None)
    torch.cuda.synchronize()
    got = run(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
