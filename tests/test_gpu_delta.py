"""The gated delta rule: the scan over dense and packed prompts, its gradients and one step, against the
recurrence token by token in 64 bits."""
import math

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import delta_ref
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _check(name, got, want, bound):
    w = ref.worst(got, want, bound)
    say(f"  {name}: {w:.4f} of its bound")
    assert w <= 1.0, (name, w)


def _rel(got, want):
    return float((ref.f64(got) - want).norm() / want.norm().clamp(min=1e-300))


def _inputs(rows, hk, hv, dk, dv, dtype, seed, strided=False, batch=1, same=0.0):
    """same: how much of one direction all keys share."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    q, k = unit(n(rows, hk, dk)), unit((1 - same) * n(rows, hk, dk) + same * n(1, hk, dk) * math.sqrt(dk))
    v = n(rows, hv, dv)
    gt = -torch.exp(torch.rand(hv, generator=g) * 5 - 5.5) * torch.nn.functional.softplus(n(rows, hv))
    beta = torch.sigmoid(n(rows, hv))
    if strided:   # columns of one projection's rows
        w = [hk * dk, hk * dk, hv * dv, hv, hv]
        at = [sum(w[:i]) for i in range(6)]
        p = torch.cat([t.reshape(rows, -1) for t in (q, k, v, gt, beta)] + [n(rows, 8 - at[5] % 8)], 1).to(dtype).cuda()
        q, k, v, gt, beta = (p[:, a:a + x] for a, x in zip(at, w))
        q, k, v = q.unflatten(1, (hk, dk)), k.unflatten(1, (hk, dk)), v.unflatten(1, (hv, dv))
    else:
        q, k, v, gt, beta = (t.to(dtype).cuda() for t in (q, k, v, gt, beta))
    return q, k, v, gt, beta, n(batch, hv, dk, dv).cuda(), n(rows, hv, dv).to(dtype).cuda(), n(batch, hv, dk, dv).cuda()


def _run(case, dtype, lengths, ins, given, tail=0):
    """Packed run of the lengths (with rows behind the last sequence), every sequence checked by itself."""
    q, k, v, g, b, h0, do, dhT = ins
    scale = q.shape[-1] ** -0.5
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    cu = torch.tensor(off, dtype=torch.int32).cuda()
    h = h0 if "h" in given else None
    dT = dhT if "T" in given else None
    o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h, dhT=dT, cu_seqlens=cu)
    o2, hT2, _ = m3.delta_scan(q, k, v, g, b, h0=h, cu_seqlens=cu)
    torch.cuda.synchronize()
    keep = slice(0, off[-1])
    assert torch.equal(o[keep], o2[keep]) and torch.equal(hT, hT2)
    worst = {}
    for s in range(len(lengths)):
        c = slice(off[s], off[s + 1])
        if lengths[s] == 0:
            assert torch.equal(hT[s], h0[s] if h is not None else torch.zeros_like(hT[s]))
            if h is not None:
                assert torch.equal(d["h0"][s], dhT[s] if dT is not None else torch.zeros_like(dhT[s]))
            continue
        want = delta_ref.check(q[c], k[c], v[c], g[c], b[c], None if h is None else h[s], scale, dtype, do[c],
                               None if dT is None else dT[s])
        got = {"o": o[c], "hT": hT[s], "dq": d["q"][c], "dk": d["k"][c], "dv": d["v"][c], "dg": d["g"][c],
               "dbeta": d["beta"][c], "dh0": None if h is None else d["h0"][s]}
        for name, (val, bound) in want.items():
            _check(f"{name} of sequence {s}", got[name], val, bound)
            worst[name] = max(worst.get(name, 0.0), _rel(got[name], val))
    say(f"  {case} {dtype}: relative errors " + ", ".join("%s %.1e" % p for p in worst.items()))


CASES = [  # lengths, Hk, Hv, Dk, Dv, what is given of h0 and dhT, strided, shared direction of the keys
    ([1], 1, 1, 64, 64, "hT", False, 0.0), ([2, 1, 0, 3], 2, 2, 64, 128, "", False, 0.0),
    ([63, 64, 65], 1, 2, 128, 64, "hT", True, 0.0), ([0, 130, 1], 1, 3, 128, 128, "h", False, 0.0),
    ([200], 2, 2, 64, 64, "T", True, 0.3), ([17, 100, 0, 0, 33], 2, 4, 128, 64, "hT", False, 0.1),
    ([257], 1, 1, 128, 128, "hT", False, 0.5), ([129, 64], 3, 3, 64, 128, "hT", True, 0.0)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_packed_scan_and_gradients(case, dtype):
    lengths, hk, hv, dk, dv, given, strided, same = case
    ins = _inputs(sum(lengths), hk, hv, dk, dv, dtype, sum(lengths) + dk + dv, strided, len(lengths), same)
    _run(case, dtype, lengths, ins, given)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequences_in_segments(dtype):
    """Long enough for several segments of a sequence, a short one and an empty one beside it."""
    for lengths, hk, hv, dk, dv in (([2500, 0, 70, 1200], 1, 2, 64, 64), ([2243], 1, 1, 128, 128),
                                    ([20] * 7 + [0, 3000, 1, 64] + [33] * 5, 1, 1, 64, 128)):
        rows = sum(lengths)
        q, k, v, g, b, h0, do, dhT = _inputs(rows, hk, hv, dk, dv, dtype, rows, False, len(lengths))
        g = (g.float() * 0.05).to(dtype)   # what is at the start is still there at the end
        _run(("long", lengths), dtype, lengths, (q, k, v, g, b, h0, do, dhT), "hT")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dense_equals_packed(dtype):
    B, T, hk, hv, dk, dv = 3, 150, 1, 2, 128, 64
    q, k, v, g, b, h0, do, dhT = _inputs(B * T, hk, hv, dk, dv, dtype, 4, True, B)
    cu = torch.arange(0, B * T + 1, T, dtype=torch.int32).cuda()
    o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
    f = lambda t: t.unflatten(0, (B, T))
    od, hd, sd = m3.delta_scan(f(q), f(k), f(v), f(g), f(b), h0=h0, want_states=True)
    dd = m3.delta_scan_backward(f(q), f(k), f(v), f(g), f(b), f(do), sd, h0=h0, dhT=dhT)
    assert torch.equal(od.flatten(0, 1), o) and torch.equal(hd, hT)
    for n in d:
        assert torch.equal(dd[n].reshape(d[n].shape), d[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 2, 64, 64, 300), (2, 2, 128, 128, 200), (1, 3, 128, 64, 700), (2, 4, 64, 128, 129),
                                   (1, 1, 64, 64, 2100)])
def test_as_near_as_the_recurrence_in_32_bits(shape, dtype):
    """The error (a norm) against that of the recurrence token by token in fp32.

    Of a product of sums of three parts the terms from 2^-24 on are left out, three of them, where a product in
    fp32 is off by half of 2^-24 at most: 6 times as much.  With the chunk's inverse and 1.3 for its norm: 8.  In
    bf16 a result is rounded once more, U, and P, U and what reaches the gradients of q and k have two parts,
    2^-16 of a product each, of at most six products that they pass through.  dg is a sum over the rows behind it
    in the chunk of differences of q.dq, k.dk and v.dv, which are each off as dq, dk and dv are before their
    rounding."""
    hk, hv, dk, dv, L = shape
    q, k, v, g, b, h0, do, dhT = _inputs(L, hk, hv, dk, dv, dtype, 40 + L, False, 1)
    scale = dk ** -0.5
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
    got = [o, hT[0]] + [d[n] for n in ("q", "k", "v", "g", "beta")] + [d["h0"][0]]

    def plain(t):
        ins = [x.cpu().to(t).requires_grad_(True) for x in (q, k, v, g, b, h0[0])]
        y, hs, _ = delta_ref.scan(*ins, scale)
        loss = (y * do.cpu().to(t)).sum() + (hs[-1] * dhT[0].cpu().to(t)).sum()
        return [y.detach(), hs[-1].detach()] + list(torch.autograd.grad(loss, ins))

    want, near = plain(torch.float64), plain(F32)
    names = ("o", "hT", "dq", "dk", "dv", "dg", "dbeta", "dh0")
    size = lambda t: ref.f64(t).flatten(1).norm(dim=1)
    rows = size(q) * size(want[2]) + size(k) * size(want[3]) + 2 * size(v) * size(want[4])
    behind = torch.stack([rows[t:t // 64 * 64 + 64].pow(2).sum() for t in range(L)]).sqrt().norm()
    for n, x, w, p in zip(names, got, want, near):
        whole = float(w.norm())
        tol = 8 * float((p.double() - w).norm()) + (0 if n in ("hT", "dh0") else ref.U[dtype] * whole)
        if dtype == BF16 and n not in ("hT", "dh0", "dv"):
            tol += 6 * 2.0 ** -16 * (whole if n != "dg" else float(behind))
        if n == "dg":
            tol += 8 * 2.0 ** -24 * float(behind)
        e = float((ref.f64(x) - w).norm())
        say(f"  {n}: {e / whole:.1e}, in 32 bits {float((p.double() - w).norm()) / whole:.1e}, {e / tol:.2f} of its bound")
        assert e <= tol, (n, e, tol)


def test_the_state_goes_on_in_place():
    """hT may be h0, also where a sequence is cut into segments, which run at once."""
    import ctypes
    lib = m3.library()
    for B, T, hk, hv, dk, dv, lengths in ((2, 4096, 1, 1, 64, 64, None), (3, 4300, 1, 2, 128, 128, [4000, 0, 300])):
        rows = T if lengths else B * T
        q, k, v, g, b, h0, _, _ = _inputs(rows, hk, hv, dk, dv, BF16, 50, False, B)
        g = (g.float() * 0.02).to(BF16)   # what is at the start is still there at the end
        cu = torch.tensor([0, 4000, 4000, 4300], dtype=torch.int32).cuda() if lengths else None
        f = (lambda t: t) if lengths else (lambda t: t.unflatten(0, (B, T)))
        o, hT, _ = m3.delta_scan(*(f(t) for t in (q, k, v, g, b)), h0=h0, cu_seqlens=cu)
        dims = m3.m3_delta_dims(B, T, hk, hv, dk, dv, m3.M3_BF16, dk ** -0.5, 0, 0, 0, 0, 0)
        p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
        ws = torch.empty(lib.m3_delta_scan_workspace_size(ctypes.byref(dims), int(cu is not None)), dtype=torch.uint8,
                         device="cuda")
        y, h = torch.empty_like(v), h0.clone()
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        for n in range(3):
            h.copy_(h0)
            assert lib.m3_delta_scan(ctypes.byref(dims), p(cu), p(q), p(k), p(v), p(g), p(b), p(h), p(y), p(h), None,
                                     p(ws), ws.numel(), s) == 0
            torch.cuda.synchronize()
            assert torch.equal(h, hT) and torch.equal(y, o.reshape(y.shape)), (B, n)
        assert not torch.equal(hT, m3.delta_scan(*(f(t) for t in (q, k, v, g, b)), cu_seqlens=cu)[1])


@pytest.mark.parametrize("shape", [(2, 2100, 1, 1, 64, 128), (1, 3000, 1, 2, 128, 128)])
def test_dense_prompts_in_segments(shape):
    B, T, hk, hv, dk, dv = shape
    for dtype in (F32, BF16):
        q, k, v, g, b, h0, do, dhT = _inputs(B * T, hk, hv, dk, dv, dtype, 60, True, B)
        g = (g.float() * 0.05).to(dtype)
        f = lambda t: t.unflatten(0, (B, T))
        o, hT, st = m3.delta_scan(f(q), f(k), f(v), f(g), f(b), h0=h0, want_states=True)
        d = m3.delta_scan_backward(f(q), f(k), f(v), f(g), f(b), f(do), st, h0=h0, dhT=dhT)
        for s in range(B):
            c = slice(s * T, (s + 1) * T)
            want = delta_ref.check(q[c], k[c], v[c], g[c], b[c], h0[s], dk ** -0.5, dtype, do[c], dhT[s])
            got = {"o": o[s], "hT": hT[s], "dq": d["q"][s], "dk": d["k"][s], "dv": d["v"][s], "dg": d["g"][s],
                   "dbeta": d["beta"][s], "dh0": d["h0"][s]}
            for n, (val, bound) in want.items():
                _check(n, got[n], val, bound)


@pytest.mark.parametrize("heads,each", [(40, 1), (35, 2)])
@pytest.mark.parametrize("dk", [64, 128])
def test_more_chunks_and_heads_than_workgroups(dk, heads, each):
    """Gradients whose workgroups go on from one chunk and head to the next, past slots that no chunk takes."""
    lengths, dv = [700, 0, 0, 64, 1, 299], 64
    q, k, v, g, b, h0, do, dhT = _inputs(sum(lengths), heads, heads * each, dk, dv, BF16, 70 + dk, False, len(lengths))
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    cu = torch.tensor(off, dtype=torch.int32).cuda()
    o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
    for s, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(d["h0"][s], dhT[s])
            continue
        c = slice(off[s], off[s + 1])
        for h in (0, 7, 23, heads - 1):
            y, x = slice(h, h + 1), slice(h * each, (h + 1) * each)
            want = delta_ref.check(q[c, y], k[c, y], v[c, x], g[c, x], b[c, x], h0[s, x], dk ** -0.5, BF16, do[c, x],
                                   dhT[s, x])
            got = {"o": o[c, x], "hT": hT[s, x], "dq": d["q"][c, y], "dk": d["k"][c, y], "dv": d["v"][c, x],
                   "dg": d["g"][c, x], "dbeta": d["beta"][c, x], "dh0": d["h0"][s, x]}
            for name, (val, bound) in want.items():
                _check(f"{name} of sequence {s}, head {h}", got[name], val, bound)
                assert name == "dg" or _rel(got[name], val) <= 2 * ref.U[BF16], (name, s, h)


def test_strong_gates():
    """Decays of 0 (-inf and far below), no decay, no write, and writes of twice the miss."""
    L, hk, hv, dk, dv = 140, 1, 2, 64, 64
    for dtype in (F32, BF16):
        q, k, v, g, b, h0, do, dhT = _inputs(L, hk, hv, dk, dv, dtype, 8)
        g[5, 0], g[70, 0], g[100, 1] = -200.0, float("-inf"), -90.0
        g[110:120, 1], b[20:30, 0], b[60:66, 1], b[128, 0] = 0.0, 0.0, 2.0, 1.0
        g[64:100, 1] = -20.0
        cu = torch.tensor([0, L], dtype=torch.int32).cuda()
        o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True)
        d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
        want = delta_ref.check(q, k, v, g.float().clamp(min=-1000.0), b, h0[0], dk ** -0.5, dtype, do, dhT[0])
        got = {"o": o, "hT": hT[0], "dq": d["q"], "dk": d["k"], "dv": d["v"], "dg": d["g"], "dbeta": d["beta"],
               "dh0": d["h0"][0]}
        for n, (val, bound) in want.items():
            _check(n, got[n], val, bound)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (3, 2, 4, 128, 64), (2, 1, 3, 64, 128), (5, 2, 2, 128, 128)])
def test_step_and_a_prompt_taken_in_pieces(shape, dtype):
    """A step is the scan over one token; a scan over two pieces is the scan over both."""
    B, hk, hv, dk, dv = shape
    T = 67
    q, k, v, g, b, h0, _, _ = _inputs(B * T, hk, hv, dk, dv, dtype, 5, False, B)
    q, k, v, g, b = (t.unflatten(0, (B, T)) for t in (q, k, v, g, b))
    o, hT, _ = m3.delta_scan(q, k, v, g, b, h0=h0)
    cut = lambda t, a, e: t[:, a:e].contiguous()
    p = [cut(t, 0, 66) for t in (q, k, v, g, b)]
    o1, h1, _ = m3.delta_scan(*p, h0=h0)
    h = h1.clone()
    y = m3.delta_step(h, *(t[:, 66] for t in (q, k, v, g, b)))
    for s in range(B):
        want = delta_ref.check(q[s, 66:], k[s, 66:], v[s, 66:], g[s, 66:], b[s, 66:], h1[s], dk ** -0.5, dtype)
        _check("step o", y[s][None], *want["o"])
        _check("step h", h[s], *want["hT"])
        both = delta_ref.check(q[s], k[s], v[s], g[s], b[s], h0[s], dk ** -0.5, dtype)
        _check("pieces o", torch.cat([o1[s], y[s][None]]), *both["o"])
        _check("pieces h", h[s], *both["hT"])
        _check("whole o", o[s], *both["o"])


def test_rows_behind_and_between_are_left():
    q, k, v, g, b, h0, do, dhT = _inputs(100, 1, 1, 64, 64, BF16, 6, False, 2)
    cu = torch.tensor([10, 40, 81], dtype=torch.int32).cuda()
    import ctypes
    lib = m3.library()
    dims = m3.m3_delta_dims(2, 100, 1, 1, 64, 64, m3.M3_BF16, 0.125, 0, 0, 0, 0, 0)
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    ws = torch.empty(lib.m3_delta_scan_workspace_size(ctypes.byref(dims), 1), dtype=torch.uint8, device="cuda")
    o, hT = torch.full_like(v, 7.0), torch.empty_like(h0)
    st = torch.empty((100 // 64 + 2, 1, m3.m3_delta_state_floats(64, 64)), device="cuda")
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.m3_delta_scan(ctypes.byref(dims), p(cu), p(q), p(k), p(v), p(g), p(b), p(h0), p(o), p(hT), p(st), p(ws),
                             ws.numel(), s) == 0
    out = [torch.full_like(t, 7.0) for t in (q, k, v, g, b)]
    ws = torch.empty(lib.m3_delta_scan_backward_workspace_size(ctypes.byref(dims), 1), dtype=torch.uint8, device="cuda")
    assert lib.m3_delta_scan_backward(ctypes.byref(dims), p(cu), p(q), p(k), p(v), p(g), p(b), p(st), p(do), p(dhT),
                                      *(p(t) for t in out), None, p(ws), ws.numel(), s) == 0
    torch.cuda.synchronize()
    for t in [o] + out:
        assert (t[:10] == 7).all() and (t[81:] == 7).all() and torch.isfinite(t).all()
    want = delta_ref.check(q[10:40], k[10:40], v[10:40], g[10:40], b[10:40], h0[0], 0.125, BF16)
    _check("o", o[10:40], *want["o"])


def test_batches_without_rows_and_offsets_that_do_not_rise():
    """Sequences that are all empty leave every row and pass their states on; offsets that fall, are negative or
    behind the rows keep within the buffers (their results are unspecified), and the next call is right."""
    T, H = 3000, 2
    q, k, v, g, b, h0, do, dhT = _inputs(T, H, H, 64, 64, BF16, 17, False, 5)
    cu = lambda *o: torch.tensor(o, dtype=torch.int32).cuda()

    def run(c):
        o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=c, want_states=True)
        return o, hT, m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=c)

    for at in (0, 64, T):
        _, hT, d = run(cu(*[at] * 6))
        assert torch.equal(hT, h0) and torch.equal(d["h0"], dhT)
    good = cu(0, 1300, 1300, 2800, 2900, T)
    want = run(good)
    for bad in ((2000, 100, 2900, 50, 3000, 0), (-7, 5000, -1, 2 ** 31 - 1, -2 ** 31, 3000), (0, 3000, 0, 3000, 0, 3000)):
        run(cu(*bad))
        torch.cuda.synchronize()
    got = run(good)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(got[2][n], want[2][n]) for n in want[2])


def test_nan_stays_in_its_sequence_and_head():
    lengths = [70, 130, 64]
    q, k, v, g, b, h0, do, dhT = _inputs(264, 2, 4, 64, 64, BF16, 7, False, 3)
    cu = torch.tensor([0, 70, 200, 264], dtype=torch.int32).cuda()
    run = lambda: (lambda r: (r[0], r[1], m3.delta_scan_backward(q, k, v, g, b, do, r[2], h0=h0, dhT=dhT, cu_seqlens=cu)))(
        m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True))
    o, hT, d = run()
    v[160, 1, 3], k[10, 1, 0], g[263, 3] = float("nan"), float("inf"), float("nan")
    o2, hT2, d2 = run()
    ok = torch.ones(264, 4, dtype=torch.bool)
    ok[70:200, 1], ok[:70, 2:], ok[200:, 3] = False, False, False
    ok = ok.cuda()
    assert torch.equal(o[ok], o2[ok]) and torch.isnan(o2[199, 1]).any()
    # (before the chunk of the NaN, the same)
    assert torch.equal(o[70:134], o2[70:134])
    for n in ("v", "g", "beta"):
        assert torch.equal(d[n][ok], d2[n][ok]), n
    okk = ok.view(264, 2, 2).all(2)
    for n in ("q", "k"):
        assert torch.equal(d[n][okk], d2[n][okk]), n
    assert torch.equal(hT[0, :2], hT2[0, :2]) and torch.equal(hT[1, [0, 2, 3]], hT2[1, [0, 2, 3]])


def test_gradients_against_differences():
    L, hk, hv, dk, dv = 75, 1, 2, 64, 64
    q, k, v, g, b, h0, do, dhT = _inputs(L, hk, hv, dk, dv, F32, 9)
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True)[2]
    d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
    ins = [ref.f64(t) for t in (q, k, v, g, b, h0[0])]
    gen = torch.Generator().manual_seed(2)
    for i, n in enumerate(("q", "k", "v", "g", "beta", "h0")):
        way = torch.randn(ins[i].shape, generator=gen, dtype=torch.float64) * ins[i].abs().mean()

        def loss(e):
            x = [t + e * way if j == i else t for j, t in enumerate(ins)]
            o, hs, _ = delta_ref.scan(*x, dk ** -0.5)
            return float((o * ref.f64(do)).sum() + (hs[-1] * ref.f64(dhT[0])).sum())

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        terms = ref.f64(d[n]).reshape(way.shape) * way
        # a difference of 1e-4 is off by 1e-8 / 6 of a third derivative; the kernels by 1e-5 of the terms
        assert abs(slope - float(terms.sum())) <= 1e-5 * float(terms.abs().sum()), n


def test_equal_bits_replayed_and_on_two_streams():
    def work(seed):
        rows = 2700
        q, k, v, g, b, h0, do, dhT = _inputs(rows, 1, 2, 64, 64, BF16, seed, True, 3)
        cu = torch.tensor([0, 2400, 2400, 2700], dtype=torch.int32).cuda()
        hs = h0.clone()

        def run():
            o, hT, st = m3.delta_scan(q, k, v, g, b, h0=h0, cu_seqlens=cu, want_states=True)
            d = m3.delta_scan_backward(q, k, v, g, b, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
            h = hs.clone()
            y = m3.delta_step(h, q[:3], k[:3], v[:3], g[:3], b[:3])
            return [o, hT, y, h] + [d[n] for n in ("q", "k", "v", "g", "beta", "h0")]
        return run, v

    (r1, v1), (r2, _) = work(31), work(32)
    want = [[t.clone() for t in r()] for r in (r1, r2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, r in zip(streams, (r1, r2)):
            with torch.cuda.stream(s):
                got.append(r())
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert all(torch.equal(a, c) for a, c in zip(w, o))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = r1()
    for n in range(3):
        v1.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, r1())), n


def test_offsets_that_pass_32_bits():
    """Rows so far apart that their addresses pass 4 GiB."""
    T, ld = 300, (1 << 23)
    p = torch.empty(T * ld, dtype=BF16, device="cuda").view(T, ld)
    q, k, v, g, b, h0, do, dhT = _inputs(T, 1, 1, 64, 64, BF16, 13)
    big = []
    for i, t in enumerate((q, k, v, g, b)):
        c = p[:, 64 * i:64 * i + t[0].numel()]
        c.copy_(t.reshape(T, -1))
        big.append(c.unflatten(1, t.shape[1:]) if t.dim() == 3 else c)
    cu = torch.tensor([0, 130, T], dtype=torch.int32).cuda()
    h2 = h0.repeat(2, 1, 1, 1)
    a = m3.delta_scan(q, k, v, g, b, h0=h2, cu_seqlens=cu, want_states=True)
    c = m3.delta_scan(*big, h0=h2, cu_seqlens=cu, want_states=True)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    da = m3.delta_scan_backward(q, k, v, g, b, do, a[2], h0=h2, cu_seqlens=cu)
    dc = m3.delta_scan_backward(*big, do, c[2], h0=h2, cu_seqlens=cu)
    assert all(torch.equal(da[n], dc[n]) for n in da)


def test_states_that_pass_32_bits():
    """What is saved, and the gradients of the states, past 2^31 elements: the last sequence of many against a
    call of its own, whose sums are grouped by segments (so: near, not equal)."""
    B, T, H, dk, dv = 65, 4096, 32, 128, 64
    g = torch.Generator(device="cuda").manual_seed(90)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF16)
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1)
    q, k, v, do = unit(n(B, T, H, dk)), unit(n(B, T, H, dk)), n(B, T, H, dv), n(B, T, H, dv)
    gt, b = -torch.nn.functional.softplus(n(B, T, H) - 3), torch.sigmoid(n(B, T, H))
    dhT = torch.randn(B, H, dk, dv, generator=g, device="cuda")
    o, hT, st = m3.delta_scan(q, k, v, gt, b, want_states=True)
    assert st.numel() > 2 ** 31
    d = m3.delta_scan_backward(q, k, v, gt, b, do, st, h0=dhT, dhT=dhT)   # (h0: only that its gradient is wanted)
    x = [t[-1:].contiguous() for t in (q, k, v, gt, b, do, dhT)]
    o1, hT1, st1 = m3.delta_scan(*x[:5], want_states=True)
    d1 = m3.delta_scan_backward(*x[:5], x[5], st1, h0=x[6], dhT=x[6])
    pairs = dict(o=(o, o1), hT=(hT, hT1), **{i: (d[i], d1[i]) for i in ("q", "k", "v", "g", "beta", "h0")})
    for name, (many, one) in pairs.items():
        e = float((many[-1].double() - one[0].double()).norm() / one.double().norm())
        say(f"  {name}: {e:.1e}")
        assert e <= (1e-5 if one.dtype == F32 else 2 * ref.U[BF16]), name


def test_refused_tensors():
    q, k, v, g, b, h0, do, dhT = _inputs(10, 1, 2, 64, 64, BF16, 3)
    cu = torch.tensor([0, 10], dtype=torch.int32).cuda()
    run = lambda **o: m3.delta_scan(*(o.get(n, t) for n, t in zip("qkvgb", (q, k, v, g, b))), h0=o.get("h0", h0),
                                    cu_seqlens=o.get("cu", cu))
    run()
    for bad in (dict(q=q.cpu()), dict(q=q.float()), dict(g=g.float()), dict(b=b[:, :1]), dict(v=v[:9]), dict(k=k[..., :32]),
                dict(h0=h0.half()), dict(h0=h0[..., :32]), dict(cu=cu.long()), dict(cu=cu[:1]),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)[..., ::2])):
        with pytest.raises((ValueError, TypeError)):
            run(**bad)
    for bad in (dict(q=q[..., :32].contiguous(), k=k[..., :32].contiguous(), h0=None),        # Dk = 32
                dict(q=torch.cat([q] * 3, 1), k=torch.cat([k] * 3, 1))):                       # 2 heads on 3
        with pytest.raises(m3.M3Error):
            run(**bad)
    with pytest.raises(ValueError):
        m3.delta_step(h0, q[:1], k[:1], v[:1], g[:1], b[:1], o=torch.empty(1, 2, 64, device="cuda"))
    with pytest.raises(ValueError):
        m3.delta_scan_backward(q, k, v, g, b, do, torch.zeros(1, 2, 64, 64, device="cuda"), cu_seqlens=cu)
    x = torch.zeros(2, 20, 1, 64, dtype=BF16, device="cuda")[:, :10]
    with pytest.raises(ValueError):
        m3.delta_scan(x, x, x, x[..., 0], x[..., 0])
