"""The layers of a hybrid stack run together over one packed batch, with one
set of offsets, and go on token by token from where the prompt ended."""
import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from linear_recurrent_sequence_mamba_amd import inputs as I
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _near(name, a, b, tol):
    """Two evaluations in bf16: their difference over the size of the result."""
    e = float((a.double() - b.double()).norm() / b.double().norm())
    say(f"  {name}: {e:.2e}")
    assert e <= tol, (name, e)


def test_prompt_then_steps_equals_longer_prompt():
    lengths = [130, 1, 77]
    T, S = sum(lengths), len(lengths)
    Hq, Hk, D = 4, 2, 64
    width = Hq * D
    g = torch.Generator().manual_seed(21)
    n = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()
    # the projections a stack would compute, given here for every token of
    # the longer prompt; the shorter one leaves out each sequence's last
    cu = torch.tensor([0, 130, 131, 208], dtype=torch.int32).cuda()
    short = [v - 1 for v in lengths]
    keep = torch.ones(T, dtype=torch.bool)
    keep[[129, 130, 207]] = False
    cus = torch.tensor([0, 129, 129, 205], dtype=torch.int32).cuda()
    w = I.Workload("hy", 31, 1, T, 4, 64, 128, 1, 64, "bf16")
    d = {k: (None if v is None else v.cuda()) for k, v in I.packed_inputs(w, lengths, h0="normal").items()}
    qkv = n(T, (Hq + 2 * Hk) * D)
    gates = n(T, 3 * width)
    decay = torch.linspace(-6, -2, width).cuda()
    wq, wk = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")

    def positions(ls):
        return torch.cat([torch.arange(v) for v in ls]).int().cuda()

    def prompt(rows, offsets, ls):
        # Mamba-3 scan
        c = {k: d[k][rows].contiguous() for k in ("x", "dt", "lam", "theta", "B", "C")}
        ym, hm = m3.scan_prefill_varlen(offsets, c["x"], c["dt"], d["A"], c["lam"], c["theta"], c["B"], c["C"],
                                        h0=d["h0"])
        # attention, its values scaled by what the scan gave
        p = qkv[rows]
        q, k, v = (p[:, a * D:b * D].view(p.shape[0], -1, D) for a, b in
                   ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        qr, kr = m3.qk_norm_rope(q, k, positions(ls), wq, wk)
        o, lse = m3.attn_prefill_varlen(qr, kr, v, offsets, offsets)
        # gated recurrence over the attention's output
        x = (o.reshape(-1, width).float() + ym.reshape(-1, width).float() * 0.1).to(BF16)
        gg = gates[rows]
        y, h, _ = m3.gated_scan(x, gg[:, width:2 * width], gg[:, 2 * width:], decay, cu_seqlens=offsets)
        return ym, hm, kr, v, y, h

    every = torch.arange(T).cuda()
    ym, hm, kr, v, y, h = prompt(every, cu, lengths)
    rows = every[keep.cuda()]
    ym1, hm1, kr1, v1, y1, h1 = prompt(rows, cus, short)
    _near("y of the shorter prompt", y1, y[rows], 1e-2)

    # the last token of each sequence as a step
    last = torch.tensor([129, 130, 207]).cuda()
    prev = torch.tensor([128, 0, 206]).cuda()
    first = torch.tensor([False, True, False]).cuda()
    xp, Bp = d["x"][prev].clone(), d["B"][prev].clone()
    xp[first] = 0
    Bp[first] = 0
    yt = m3.decode_step(hm1, d["x"][last].contiguous(), d["B"][last].contiguous(), d["C"][last].contiguous(),
                        d["dt"][last].contiguous(), d["A"], d["lam"][last].contiguous(),
                        d["theta"][last].contiguous(), x_prev=xp, B_prev=Bp)
    _near("scan step", yt, ym[last], 3e-4)
    _near("scan state", hm1, hm, 3e-4)
    cap = 140
    ck, cv = (torch.full((S, cap, Hk, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    off = cus.tolist()
    for s in range(S):
        ck[s, :short[s]] = kr1[off[s]:off[s + 1]]
        cv[s, :short[s]] = v1[off[s]:off[s + 1]]
    p = qkv[last]
    pos = torch.tensor(short, dtype=torch.int32).cuda()
    qr, kn = m3.qk_norm_rope(p[:, :Hq * D].view(S, Hq, D), p[:, Hq * D:(Hq + Hk) * D].view(S, Hk, D), pos, wq, wk)
    assert torch.equal(kn, kr[last])
    at = pos.long()
    ck[torch.arange(S), at] = kn
    cv[torch.arange(S), at] = p[:, (Hq + Hk) * D:].view(S, Hk, D)
    o, _ = m3.attn_decode(qr, ck, cv, pos + 1)
    x = (o.reshape(S, width).float() + yt.reshape(S, width).float() * 0.1).to(BF16)
    gg = gates[last]
    ys = m3.gated_step(h1, x, gg[:, width:2 * width], gg[:, 2 * width:], decay)
    _near("gated step", ys, y[last], 1e-2)
    _near("gated state", h1, h, 1e-2)


def test_gradients_through_the_layers():
    """norm + rotation -> attention -> gated recurrence, backwards through the
    library's calls, against the 64-bit definitions differentiated together."""
    lengths, Hq, Hk, D = [40, 25], 2, 1, 64
    T, width, cu = 65, 128, [0, 40, 65]
    g = torch.Generator().manual_seed(22)
    n = lambda *s: torch.randn(*s, generator=g).cuda()
    q, k, v = n(T, Hq, D), n(T, Hk, D), n(T, Hk, D)
    r, i, dy = n(T, width), n(T, width), n(T, width)
    decay = torch.linspace(-5, -1, width).cuda()
    wq, wk = (0.5 + torch.rand(D, generator=g)).cuda(), (0.5 + torch.rand(D, generator=g)).cuda()
    pos = torch.cat([torch.arange(m) for m in lengths]).int().cuda()
    cut = torch.tensor(cu, dtype=torch.int32).cuda()
    qr, kr = m3.qk_norm_rope(q, k, pos, wq, wk)
    o, lse = m3.attn_prefill_varlen(qr, kr, v, cut, cut)
    y, _, st = m3.gated_scan(o.view(T, width), r, i, decay, cu_seqlens=cut, want_states=True)
    dg = m3.gated_scan_backward(o.view(T, width), r, i, decay, dy, st, cu_seqlens=cut)
    dq, dk, dv = m3.attn_prefill_varlen_backward(qr, kr, v, o, lse, dg["x"].view(T, Hq, D), cut, cut)
    dn = m3.qk_norm_rope_backward(q, k, pos, dq, dk, wq, wk)
    leaves = [ref.f64(t).requires_grad_(True) for t in (q, k, v, wq, wk, r, i, decay)]
    a, b, c, x, z, rr, ii, dd = leaves
    qd = ref.qk_one(a, pos.cpu(), x, 1e-6, 10000.0, D, False)
    kd = ref.qk_one(b, pos.cpu(), z, 1e-6, 10000.0, D, False)
    od = torch.cat([ref.attn(qd[s:e], kd[s:e], c[s:e], D ** -0.5)[0] for s, e in zip(cu, cu[1:])])
    yd, _ = ref.gated(od.reshape(T, width), rr, ii, dd, None, 8.0, cu)
    want = torch.autograd.grad((yd * ref.f64(dy)).sum(), leaves)
    got = (dn["q"], dn["k"], dv, dn["q_weight"], dn["k_weight"], dg["r"], dg["i"], dg["decay"])
    # four fp32 operators in a row, each within about 1e-6 of its size
    _near("y", y.cpu(), yd.detach(), 1e-5)
    for name, u, w in zip(("q", "k", "v", "wq", "wk", "r", "i", "decay"), got, want):
        _near("d" + name, u.cpu(), w, 1e-5)


def test_layers_on_two_streams_at_once():
    """Calls of two streams share the chip, tiles of two scans in flight
    together among them; each has the bits that it has alone."""
    def work(seed):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g).to(BF16).cuda()
        T, Hq, Hk, D = 2600, 8, 2, 64
        cu = torch.tensor([0, 700, 703, 2600], dtype=torch.int32).cuda()
        q, k, v, do = n(T, Hq, D), n(T, Hk, D), n(T, Hk, D), n(T, Hq, D)
        x, r, i, dy = (n(T, Hq * D) for _ in range(4))
        decay, pos = torch.linspace(-6, -2, Hq * D).cuda(), torch.arange(T, dtype=torch.int32).cuda()
        cache, lens = n(3, 1500, Hk, D), torch.tensor([1500, 0, 77], dtype=torch.int32).cuda()

        def run():
            y, hT, st = m3.gated_scan(x, r, i, decay, cu_seqlens=cu, want_states=True)
            d = m3.gated_scan_backward(x, r, i, decay, dy, st, cu_seqlens=cu)
            qr, kr = m3.qk_norm_rope(q, k, pos)
            o, lse = m3.attn_prefill_varlen(qr, kr, v, cu, cu)
            return [y, hT, d["x"], d["decay"], o, lse,
                    *m3.attn_prefill_varlen_backward(qr, kr, v, o, lse, do, cu, cu),
                    *m3.attn_decode(q[:3], cache, cache, lens)]
        return run

    runs = [work(41), work(42)]
    want = [[t.clone() for t in f()] for f in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for n in range(4):
        got = []
        for s, f in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, o)), n
