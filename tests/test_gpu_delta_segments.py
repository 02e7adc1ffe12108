"""The gated delta rule where its segments' maps carry the states: slow decays, keys that overwrite the state in
one segment and hardly touch it in the next, against the recurrence in 64 bits."""
import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import delta_ref
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
def test_states_through_maps_keep_32_bits(dk, dv, dtype):
    """Three segments of 512 tokens and one of 40.  The decay of a segment is about exp(-0.3); the second and the
    third overwrite their state (d S + F S cancels), the last writes 40 tokens and the first hardly anything, so
    that an error of the state that the maps give reaches hT, and one of its gradient dh0.

    The recurrence in fp32 rounds the state twice a token, the chunks once for each of their few products, of sums
    that keep 24 bits of each operand, and a map once more: no more than twice the recurrence's error."""
    L = 3 * 512 + 40
    g = torch.Generator().manual_seed(dk + dv)
    n = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    q, k, v = unit(n(L, 2, dk)), unit(n(L, 2, dk)), n(L, 2, dv)
    gt = -torch.rand(L, 2, generator=g) * 1.2e-3
    b = torch.sigmoid(n(L, 2) + 1)
    b[:512] *= 0.02
    q, k, v, gt, b, do = (t.to(dtype) for t in (q, k, v, gt, b, n(L, 2, dv)))
    h0, dhT = n(2, dk, dv), 4 * n(2, dk, dv)
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    dev = [t.cuda() for t in (q, k, v, gt, b)]
    start = h0[None].cuda()
    _, hT, st = m3.delta_scan(*dev, h0=start, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(*dev, do.cuda(), st, h0=start, dhT=dhT[None].cuda(), cu_seqlens=cu)

    def plain(t):
        ins = [x.to(t).requires_grad_(True) for x in (q, k, v, gt, b, h0)]
        y, hs, _ = delta_ref.scan(*ins, dk ** -0.5)
        loss = (y * do.to(t)).sum() + (hs[-1] * dhT.to(t)).sum()
        return hs[-1].detach(), torch.autograd.grad(loss, ins[-1])[0]

    want, near = plain(torch.float64), plain(F32)
    for name, x, w, p in zip(("hT", "dh0"), (hT[0], d["h0"][0]), want, near):
        size = w.flatten(1).norm(dim=1)
        e = (ref.f64(x) - w).flatten(1).norm(dim=1)
        tol = 2 * (p.double() - w).flatten(1).norm(dim=1)
        say(f"  {name}: {[f'{a:.1e}' for a in (e / size).tolist()]}, in 32 bits {[f'{a:.1e}' for a in (tol / 2 / size).tolist()]}")
        assert (e <= tol).all(), (name, e, tol)


def _packed(lengths, hk, hv, dk, dv, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    T = sum(lengths)
    off = [0]
    for m in lengths:
        off.append(off[-1] + m)
    ins = [t.to(dtype) for t in (unit(n(T, hk, dk)), unit(n(T, hk, dk)), n(T, hv, dv), -torch.rand(T, hv, generator=g) * 4e-3,
                                 torch.sigmoid(n(T, hv)))]
    return ins, n(len(lengths), hv, dk, dv), off, n(T, hv, dv).to(dtype), n(len(lengths), hv, dk, dv)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 2, 64, 128), (1, 1, 128, 128)])
def test_few_long_sequences_among_many(shape, dtype):
    """More sequences than segments: long ones among them, one next to the other and with empty ones between, have
    the results that they have alone, also where hT is h0."""
    hk, hv, dk, dv = shape
    lengths = [1] * 200 + [2500] + [0] * 90 + [3] * 150 + [1800, 1300] + [2] * 60 + [0] * 5
    ins, h0, off, do, dhT = _packed(lengths, hk, hv, dk, dv, dtype, dk + dv)
    dev = [t.cuda() for t in ins]
    start, end, cu = h0.cuda(), dhT.cuda(), torch.tensor(off, dtype=torch.int32).cuda()
    o, hT, st = m3.delta_scan(*dev, h0=start, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(*dev, do.cuda(), st, h0=start, dhT=end, cu_seqlens=cu)
    for s, L in enumerate(lengths):
        if L == 0:
            assert torch.equal(hT[s].cpu(), h0[s]) and torch.equal(d["h0"][s].cpu(), dhT[s])
        if L == 0 or s % 61 and L < 1000:
            continue

        def plain(t):
            x = [y[off[s]:off[s + 1]].to(t) for y in ins] + [h0[s].to(t).requires_grad_(True)]
            y, hs, _ = delta_ref.scan(*x, dk ** -0.5)
            loss = (y * do[off[s]:off[s + 1]].to(t)).sum() + (hs[-1] * dhT[s].to(t)).sum()
            return y.detach(), hs[-1].detach(), torch.autograd.grad(loss, x[-1])[0]

        want, near = plain(torch.float64), plain(F32)
        for name, x, w, p in zip(("o", "hT", "dh0"), (o[off[s]:off[s + 1]], hT[s], d["h0"][s]), want, near):
            # (the recurrence's error, of a short sequence at least half a step of each element; and o's rounding,
            # in bf16 after operands of two parts)
            tol = 2 * float((p.double() - w).norm()) + 2.0 ** -24 * float(w.norm())
            tol += (ref.U[dtype] * (1 + 2.0 ** -6) if name == "o" else 0) * float(w.norm())
            e = float((ref.f64(x) - w).norm())
            assert e <= tol, (s, L, name, e, tol)
    # in place
    import ctypes
    lib = m3.library()
    dims = m3.m3_delta_dims(len(lengths), sum(lengths), hk, hv, dk, dv, m3.dtype_code(dtype), dk ** -0.5, 0, 0, 0, 0, 0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    ws = torch.empty(lib.m3_delta_scan_workspace_size(ctypes.byref(dims), 1), dtype=torch.uint8, device="cuda")
    y, h = torch.empty_like(dev[2]), start.clone()
    assert lib.m3_delta_scan(ctypes.byref(dims), p(cu), *(p(t) for t in dev), p(h), p(y), p(h), None, p(ws), ws.numel(),
                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert torch.equal(h, hT) and torch.equal(y, o)


def test_more_heads_of_sequences_than_a_launch_for_each():
    """So many empty sequences that a workgroup for each 16 columns of each of their heads would pass 2^32 threads,
    and long ones at their ends."""
    B, hv, dk, dv, L = 70000, 32, 128, 128, [4000, 2000]
    q, k, v, g, b = (t.cuda() for t in _packed(L, 1, hv, dk, dv, BF16, 5)[0])
    cu = torch.full((B + 1,), L[0], dtype=torch.int32)
    cu[0], cu[-1] = 0, sum(L)
    o = m3.delta_scan(q, k, v, g, b, cu_seqlens=cu.cuda(), want_hT=False)[0]
    for s, c in ((0, slice(0, L[0])), (1, slice(L[0], sum(L)))):
        one = torch.tensor([0, L[s]], dtype=torch.int32).cuda()
        want = m3.delta_scan(q[c], k[c], v[c], g[c], b[c], cu_seqlens=one)[0]
        # (sums are grouped by other segments)
        e = float((o[c].double() - want.double()).norm() / want.double().norm())
        say(f"  {s}: {e:.1e}")
        assert e <= 2.0 ** -8


def test_a_captured_batch_takes_other_offsets():
    """The launches depend on sizes alone: a step captured once runs any offsets within its rows and sequences."""
    S, T, hk, hv, dk, dv = 40, 6000, 1, 2, 64, 64
    ins, h0, _, do, dhT = _packed([T], hk, hv, dk, dv, BF16, 31)
    dev = [t.cuda() for t in ins]
    g = torch.Generator().manual_seed(32)
    h0, dhT = (torch.randn(S, hv, dk, dv, generator=g).cuda() for _ in range(2))
    do = do.cuda()
    batches = [[150] * 40, [6000] + [0] * 39, [0] * 20 + [2000, 1, 3000] + [17] * 17, [5] * 39 + [3333], [0] * 40]
    offsets = [torch.tensor([0] + torch.tensor(b).cumsum(0).tolist(), dtype=torch.int32).cuda() for b in batches]
    cu = offsets[0].clone()

    def run(c):
        o, hT, st = m3.delta_scan(*dev, h0=h0, cu_seqlens=c, want_states=True)
        d = m3.delta_scan_backward(*dev, do, st, h0=h0, dhT=dhT, cu_seqlens=c)
        return dict(o=o, hT=hT, **{"d" + n: t for n, t in d.items()})

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(cu)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = run(cu)
    for b, c in list(zip(batches, offsets)) * 2:
        cu.copy_(c)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = run(c)
        n = sum(b)
        for name, w in want.items():
            x = out[name]
            assert torch.equal(x, w) if name in ("hT", "dh0") else torch.equal(x[:n], w[:n]), (b[:3], name)
