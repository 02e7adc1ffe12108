"""The gated linear recurrence (scan, packed scan, step, gradients) against
its definition in 64 bits, token by token."""
import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
C = 8.0


def _inputs(rows, D, dtype, seed, nseq, strided=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    if strided:
        p = n(*rows, 3 * D + 8).to(dtype).cuda()
        x, r, i = p[..., :D], p[..., D + 8:2 * D + 8], p[..., 2 * D + 8:]
    else:
        x, r, i = (n(*rows, D).to(dtype).cuda() for _ in range(3))
    # a full gate decays to 0.5 .. 0.99 per step
    a = 0.5 + 0.49 * torch.rand(D, generator=g)
    decay = torch.log(torch.expm1(-torch.log(a.double()) / C)).float().cuda()
    h0 = n(nseq, D).cuda()
    return x, r, i, decay, h0


def _amax(r, decay):
    return float(torch.exp(-C * torch.nn.functional.softplus(ref.f64(decay)) *
                           torch.sigmoid(ref.f64(r).clamp(min=-30))).max())


def _check(name, got, want, bound):
    w = ref.worst(got, want, bound)
    say(f"  {name}: {w:.3f} of its bound")
    assert w <= 1.0, (name, w)


def _flat(t):
    return t.reshape(-1, t.shape[-1])


def _grad_bound(want, amax, T, dtype):
    # h and g each carry the scan's error; their products and the three
    # gate derivatives add a few roundings
    return 3 * ref.gated_bound(want, amax, T, dtype) + (ref.U[dtype] * want.abs())


DENSE = [(1, 1, 64), (2, 2, 1), (1, 127, 65), (3, 128, 64), (1, 129, 130), (2, 300, 63), (1, 1000, 96),
         (1, 2700, 20)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D", DENSE)
def test_scan_and_gradients(B, T, D, dtype):
    for strided, use_h0 in ((False, True), (D % 8 == 0, False)):
        say(f"gated B={B} T={T} D={D} {dtype} strided={strided} h0={use_h0}")
        x, r, i, decay, h0 = _inputs((B, T), D, dtype, 100 + T, B, strided)
        h0 = h0 if use_h0 else None
        y, hT, st = m3.gated_scan(x, r, i, decay, h0=h0, c=C, want_states=True)
        torch.cuda.synchronize()
        wy, wh = ref.gated(ref.f64(x), ref.f64(r), ref.f64(i), ref.f64(decay), ref.f64(h0), C)
        am = _amax(r, decay)
        _check("y", _flat(y), _flat(wy), ref.gated_bound(_flat(wy), am, T, dtype))
        _check("hT", hT, wh, ref.gated_bound(_flat(wy), am, T, F32).amax(0))
        assert st.shape == (B, (T + 127) // 128, D)
        for k in range(st.shape[1]):
            want = wy[:, 128 * k - 1] if k else (torch.zeros(B, D) if h0 is None else ref.f64(h0))
            _check(f"state {k}", st[:, k], want.double(),
                   ref.gated_bound(_flat(wy), am, T, F32).amax(0) + 1e-30)
        g = torch.Generator().manual_seed(7)
        dy = torch.randn(B, T, D, generator=g).to(dtype).cuda()
        dhT = torch.randn(B, D, generator=g).cuda() if use_h0 else None
        d = m3.gated_scan_backward(x, r, i, decay, dy, st, h0=h0, dhT=dhT, c=C)
        torch.cuda.synchronize()
        want = ref.gated_grads(x, r, i, decay, dy, h0, dhT, C)
        for k in ("x", "r", "i"):
            _check("d" + k, _flat(d[k]), _flat(want[k]), _grad_bound(_flat(want[k]), am, T, dtype))
        # the sum of B T terms, each as dr (which is the term times 1 - sigmoid)
        sr = torch.sigmoid(ref.f64(r))
        terms = _flat(want["r"] / (1 - sr)).abs()
        ratio = torch.sigmoid(ref.f64(decay)) / torch.nn.functional.softplus(ref.f64(decay))
        _check("ddecay", d["decay"], want["decay"],
               ratio * (_grad_bound(terms, am, T, F32).sum(0) + 2.0 ** -22 * terms.sum(0)) + 1e-30)
        if use_h0:
            _check("dh0", d["h0"], want["h0"], _grad_bound(want["h0"], am, T, F32) +
                   2.0 ** -20 * (min(T, 100) + 2) * want["h0"].abs().mean())


LENGTHS = [[1], [0, 5, 0, 0, 1, 127, 0], [128, 1, 128, 255], [700, 3, 1, 1, 40], [0, 0, 300],
           [2500, 3, 700], [1] * 150 + [0] * 40 + [2] * 33]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_packed(lengths, dtype):
    D, S = 70, len(lengths)
    lead, tail = 3, 5   # rows that no sequence covers
    T = sum(lengths) + lead + tail
    say(f"gated packed {lengths} {dtype}")
    x, r, i, decay, h0 = _inputs((T,), D, dtype, 5, S)
    for t in (x, r, i):   # what is there must not matter
        t[:lead] = float("nan")
        t[T - tail:] = float("inf")
    cu = [lead]
    for n in lengths:
        cu.append(cu[-1] + n)
    cut = torch.tensor(cu, dtype=torch.int32).cuda()
    y0 = torch.full((T, D), -77.0, dtype=dtype, device="cuda")
    y, hT, st = _raw_scan(x, r, i, decay, h0, cut, y0)
    wy, wh = ref.gated(ref.f64(x), ref.f64(r), ref.f64(i), ref.f64(decay), ref.f64(h0), C, cu)
    am, n = _amax(r[lead:T - tail], decay), max(lengths)
    assert (y[:lead] == -77).all() and (y[T - tail:] == -77).all()
    body = y[lead:T - tail]
    bound = ref.gated_bound(wy, am, n, dtype)
    _check("y", body, wy, bound)
    _check("hT", hT, wh, ref.gated_bound(wy, am, n, F32).amax(0) * torch.ones(S, 1) + 1e-30)
    for s in range(S):
        if not lengths[s]:
            assert torch.equal(hT[s], h0[s])
    g = torch.Generator().manual_seed(8)
    dy = torch.randn(T, D, generator=g).to(dtype).cuda()
    dy[:lead] = float("nan")
    dy[T - tail:] = float("nan")
    dhT = torch.randn(S, D, generator=g).cuda()
    d = m3.gated_scan_backward(x, r, i, decay, dy, st, h0=h0, dhT=dhT, c=C, cu_seqlens=cut)
    torch.cuda.synchronize()
    off = [v - lead for v in cu]
    part = lambda t: t[lead:T - tail]
    want = ref.gated_grads(part(x), part(r), part(i), decay, part(dy), h0, dhT, C, off)
    for k in ("x", "r", "i"):
        _check("d" + k, part(d[k]), want[k], _grad_bound(want[k], am, n, dtype))
    terms = (want["r"] / (1 - torch.sigmoid(ref.f64(part(r))))).abs()
    ratio = torch.sigmoid(ref.f64(decay)) / torch.nn.functional.softplus(ref.f64(decay))
    _check("ddecay", d["decay"], want["decay"],
           ratio * (_grad_bound(terms, am, n, F32).sum(0) + 2.0 ** -22 * terms.sum(0)) + 1e-30)
    _check("dh0", d["h0"], want["h0"], _grad_bound(want["h0"], am, n, F32) +
           2.0 ** -20 * (min(n, 100) + 2) * want["h0"].abs().mean())


def _raw_scan(x, r, i, decay, h0, cu, y):
    """m3_gated_scan into a y that is there already."""
    import ctypes
    T, D = x.shape
    S = cu.numel() - 1
    d = m3.m3_gated_dims(S, T, D, m3.dtype_code(x.dtype), C, 0, 0, 0, 0)
    lib = m3.library()
    ws = torch.empty(lib.m3_gated_scan_workspace_size(ctypes.byref(d), 1), dtype=torch.uint8,
                     device="cuda").fill_(255)
    hT = torch.empty(S, D, device="cuda")
    st = torch.empty((T + 127) // 128, D, device="cuda")
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    e = lib.m3_gated_scan(ctypes.byref(d), p(cu), p(x), p(r), p(i), p(decay), p(h0), p(y), p(hT),
                          p(st), p(ws), ws.numel(),
                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert e == 0
    torch.cuda.synchronize()
    return y, hT, st


def test_packed_with_thousands_of_sequences():
    """More offsets than one workgroup's memory holds, most windows with many."""
    g = torch.Generator().manual_seed(31)
    test_packed(torch.randint(0, 4, (9000,), generator=g).tolist(), BF16)


@pytest.mark.parametrize("S", [3, 700, 8192, 8193, 20000])
def test_any_offsets_are_cleaned(S):
    """Offsets in any order give the bits of the cleaned ones, gradients too."""
    T, D = 3000, 33
    x, r, i, decay, h0 = _inputs((T,), D, F32, 9, S)
    g = torch.Generator().manual_seed(S)
    rise = torch.sort(torch.randint(0, T, (S + 1,), generator=g))[0]
    bad = rise + torch.randint(-300, 30, (S + 1,), generator=g) * (torch.rand(S + 1, generator=g) < 0.2)
    good = bad.clamp(0, T).cummax(0)[0]
    bad, good = bad.to(torch.int32).cuda(), good.to(torch.int32).cuda()
    dhT = torch.randn(S, D, generator=g).cuda()
    body = slice(int(good[0]), int(good[-1]))
    res = []
    for cu in (bad, good):
        y, hT, st = m3.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=cu, want_states=True)
        d = m3.gated_scan_backward(x, r, i, decay, x, st, h0=h0, dhT=dhT, cu_seqlens=cu)
        res.append([y[body], hT, d["x"][body], d["r"][body], d["i"][body], d["decay"], d["h0"]])
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(*res))
    empty = (good[1:] == good[:-1])
    assert torch.equal(res[0][1][empty], h0[empty]) and torch.equal(res[0][6][empty], dhT[empty])


def test_offsets_that_do_not_rise_are_cleaned():
    T, D = 300, 64
    x, r, i, decay, h0 = _inputs((T,), D, F32, 9, 4)
    bad = torch.tensor([-5, 120, 40, 1000, 7], dtype=torch.int32).cuda()
    good = torch.tensor([0, 120, 120, 300, 300], dtype=torch.int32).cuda()
    a = m3.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=bad, want_states=True)
    b = m3.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=good, want_states=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_nan_stays_in_its_sequence():
    D, cu = 64, [0, 100, 200, 500]
    x, r, i, decay, h0 = _inputs((500,), D, BF16, 10, 3)
    cut = torch.tensor(cu, dtype=torch.int32).cuda()
    y, hT, st = m3.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=cut, want_states=True)
    dy = torch.randn(500, D, device="cuda").to(BF16)
    d = m3.gated_scan_backward(x, r, i, decay, dy, st, h0=h0, cu_seqlens=cut)
    x2, dy2 = x.clone(), dy.clone()
    x2[150, 3] = float("nan")
    x2[151, 4] = float("inf")
    dy2[150, 5] = float("nan")
    y2, hT2, st2 = m3.gated_scan(x2, r, i, decay, h0=h0, cu_seqlens=cut, want_states=True)
    d2 = m3.gated_scan_backward(x2, r, i, decay, dy2, st2, h0=h0, cu_seqlens=cut)
    for a, b in [(y, y2)] + [(d[k], d2[k]) for k in ("x", "r", "i")]:
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[200:], b[200:])
    assert torch.equal(y[:150], y2[:150])
    assert torch.isnan(y2[150:200, 3]).all() and torch.isinf(y2[151:200, 4]).all()
    assert torch.equal(hT[0], hT2[0]) and torch.equal(hT[2], hT2[2])
    assert torch.equal(d["h0"][0], d2["h0"][0]) and torch.equal(d["h0"][2], d2["h0"][2])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_at_their_ends(dtype):
    """Closed and open gates, tiny and huge decays: finite results, equal to
    the definition where it is finite."""
    B, T, D = 1, 140, 6
    x, r, i, _, h0 = _inputs((B, T), D, dtype, 11, B)
    decay = torch.tensor([-100.0, -20.0, -14.0, 0.0, 30.0, 5.0], device="cuda")
    r[:, 10] = -200.0     # a = 1 exactly
    r[:, 11] = 200.0
    r[:, 12] = -float("inf")
    i[:, 13] = -200.0
    i[:, 14] = 200.0
    y, hT, st = m3.gated_scan(x, r, i, decay, h0=h0, c=C, want_states=True)
    dy = torch.ones_like(x)
    d = m3.gated_scan_backward(x, r, i, decay, dy, st, h0=h0, c=C)
    torch.cuda.synchronize()
    wy, _ = ref.gated(ref.f64(x), ref.f64(r).clamp(min=-700), ref.f64(i), ref.f64(decay), ref.f64(h0), C)
    _check("y", _flat(y), _flat(wy), ref.gated_bound(_flat(wy), 1.0, T, dtype) + 1e-30)
    for k in ("x", "r", "i", "decay", "h0"):
        assert torch.isfinite(d[k]).all(), k
    assert (d["r"][:, 10] == 0).all() and (d["r"][:, 12] == 0).all()
    # dx and di have no singular point: they follow the definition everywhere
    want = ref.gated_grads(x, r.clamp(min=-700), i, decay, dy, h0, None, C)
    _check("dx", _flat(d["x"]), _flat(want["x"]), _grad_bound(_flat(want["x"]), 1.0, T, dtype) + 1e-30)
    _check("di", _flat(d["i"]), _flat(want["i"]), _grad_bound(_flat(want["i"]), 1.0, T, dtype) + 1e-30)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 64, 77])
def test_steps_continue_a_scan(D, dtype):
    B, T = 3, 140
    x, r, i, decay, h0 = _inputs((B, T), D, dtype, 12, B)
    y, hT, _ = m3.gated_scan(x, r, i, decay, h0=h0, c=C)
    _, h, _ = m3.gated_scan(x[:, :100].contiguous(), r[:, :100].contiguous(),
                            i[:, :100].contiguous(), decay, h0=h0, c=C)
    wy, wh = ref.gated(ref.f64(x), ref.f64(r), ref.f64(i), ref.f64(decay), ref.f64(h0), C)
    bound = ref.gated_bound(_flat(wy), _amax(r, decay), T, dtype)
    ys = []
    for t in range(100, T):
        ys.append(m3.gated_step(h, x[:, t].contiguous(), r[:, t].contiguous(), i[:, t].contiguous(),
                                decay, c=C))
    torch.cuda.synchronize()
    _check("y", _flat(torch.stack(ys, 1)), _flat(wy[:, 100:]), bound.view(B, T, D)[:, 100:].reshape(-1, D))
    _check("h", h, wh, ref.gated_bound(_flat(wy), _amax(r, decay), T, F32).amax(0))


def test_step_takes_cut_rows():
    B, D = 5, 64
    p = torch.randn(B, 3 * D, device="cuda").to(BF16)
    decay, h = torch.randn(D, device="cuda"), torch.randn(B, D, device="cuda")
    cut = [p[:, k * D:(k + 1) * D] for k in range(3)]
    h1, h2 = h.clone(), h.clone()
    a = m3.gated_step(h1, *cut, decay)
    b = m3.gated_step(h2, *(t.contiguous() for t in cut), decay)
    assert torch.equal(a, b) and torch.equal(h1, h2)


def test_equal_calls_give_equal_bits_and_hT_may_be_h0():
    x, r, i, decay, h0 = _inputs((2, 700), 96, BF16, 13, 2)
    y, hT, st = m3.gated_scan(x, r, i, decay, h0=h0, want_states=True)
    dy = torch.randn(2, 700, 96, device="cuda").to(BF16)
    d = m3.gated_scan_backward(x, r, i, decay, dy, st, h0=h0)
    for _ in range(3):
        y2, hT2, st2 = m3.gated_scan(x, r, i, decay, h0=h0, want_states=True)
        d2 = m3.gated_scan_backward(x, r, i, decay, dy, st2, h0=h0)
        assert torch.equal(y, y2) and torch.equal(hT, hT2) and torch.equal(st, st2)
        assert all(torch.equal(d[k], d2[k]) for k in d)
    import ctypes
    h = h0.clone()
    dims = m3.m3_gated_dims(2, 700, 96, m3.M3_BF16, 8.0, 0, 0, 0, 0)
    lib = m3.library()
    ws = torch.empty(lib.m3_gated_scan_workspace_size(ctypes.byref(dims), 0), dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    assert lib.m3_gated_scan(ctypes.byref(dims), None, p(x), p(r), p(i), p(decay), p(h), p(y2), p(h),
                             None, p(ws), ws.numel(),
                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert torch.equal(h, hT) and torch.equal(y2, y)


def _in_place(x, r, i, decay, h0, cu):
    """The scan with hT written over h0."""
    import ctypes
    D, dt = x.shape[-1], m3.M3_BF16 if x.dtype == BF16 else m3.M3_F32
    dims = ctypes.byref(m3.m3_gated_dims(h0.shape[0], x.shape[-2], D, dt, 8.0, 0, 0, 0, 0))
    lib, h, y = m3.library(), h0.clone(), torch.empty_like(x)
    ws = torch.empty(lib.m3_gated_scan_workspace_size(dims, cu is not None), dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())
    assert lib.m3_gated_scan(dims, p(cu), p(x), p(r), p(i), p(decay), p(h), p(y), p(h), None, p(ws),
                             ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    return y, h


@pytest.mark.parametrize("B,T", [(1, 600), (3, 1900), (2, 5000)])
def test_hT_over_h0_in_every_tile_count(B, T):
    """Every tile of the first group has read h0 before the last one writes
    hT: with fewer tiles than a group, within the second, and beyond."""
    x, r, i, decay, h0 = _inputs((B, T), 1000, BF16, 21, B)
    h0 = h0 * 100   # a tile that took the new state for the old one would show
    y, hT, _ = m3.gated_scan(x, r, i, decay, h0=h0)
    for _ in range(5):
        y2, h = _in_place(x, r, i, decay, h0, None)
        assert torch.equal(h, hT) and torch.equal(y2, y)


def test_hT_over_h0_packed():
    lengths = [700, 0, 1, 255, 1044]
    x, r, i, decay, h0 = _inputs((sum(lengths),), 1000, BF16, 22, len(lengths))
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    y, hT, _ = m3.gated_scan(x, r, i, decay, h0=h0, cu_seqlens=cu)
    for _ in range(5):
        y2, h = _in_place(x, r, i, decay, h0, cu)
        assert torch.equal(h, hT) and torch.equal(y2, y)


def test_graphs_and_streams():
    """Two captured graphs, replayed in turn with eager work between, and a
    call on another stream, all equal the eager result."""
    x, r, i, decay, h0 = _inputs((1, 1500), 128, BF16, 14, 1)
    dy = torch.randn(1, 1500, 128, device="cuda").to(BF16)

    def once():
        y, hT, st = m3.gated_scan(x, r, i, decay, h0=h0, want_states=True)
        d = m3.gated_scan_backward(x, r, i, decay, dy, st, h0=h0)
        return [y, hT, d["x"], d["r"], d["i"], d["decay"], d["h0"]]

    want = [t.clone() for t in once()]
    graphs = []
    for _ in range(2):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            once()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = once()
        graphs.append((g, out))
    for n in range(4):
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), n
        once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, hT, _ = m3.gated_scan(x, r, i, decay, h0=h0, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(hT, want[1])
