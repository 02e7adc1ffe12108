"""The norms around a block with its gate and residual scale, and the gradients, against the definition in
64 bits."""
import ctypes

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import block_ref
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6
FLAGS = {None: 0, "linear": 0, "sigmoid": m3.M3_GATE_SIGMOID, "silu": m3.M3_GATE_SILU}
NAMES = dict(dx="x", dy="y", dgate="gate", dy_weight="y_weight", dscale="scale", dn_weight="n_weight")


def _inputs(T, W, dtype, act, weights, cut, seed):
    """cut: 0 dense rows, else rows of a tensor that is `cut` elements wider, so that three are cut out."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    size = torch.rand(T, 1, generator=g) * 3 + 0.1
    if cut:
        p = torch.zeros(T, 3 * W + cut)
        at = [0, (W + 7) // 8 * 8, (2 * W + 15) // 8 * 8]
        for k in range(3):
            p[:, at[k]:at[k] + W] = n(T, W) * (size if k == 1 else 1)
        p = p.to(dtype).cuda()
        x, y, gate = (p[:, a:a + W] for a in at)
    else:
        x, y, gate = n(T, W).to(dtype).cuda(), (n(T, W) * size).to(dtype).cuda(), n(T, W).to(dtype).cuda()
    w = [(0.5 + torch.rand(W, generator=g)).cuda() for _ in range(3)] if weights else [None] * 3
    w[1] = None if w[1] is None else w[1] * torch.where(torch.rand(W, generator=g) < 0.1, 0.0, 1.0).cuda()
    return x, y, (None if act is None else gate), w, n(T, W).to(dtype).cuda(), n(T, W).to(dtype).cuda()


def _check(name, got, want, bound):
    w = ref.worst(got, want, bound)
    say(f"  {name}: {w:.3f} of its bound")
    assert w <= 1.0, (name, w)


CASES = [  # T, W, act, raw, weights, cut, what is given of dh and dn
    (1, 1, "silu", False, True, 0, "hn"), (1, 8, None, False, False, 0, "hn"),
    (3, 64, "sigmoid", False, True, 16, "hn"), (7, 100, "silu", True, True, 0, "n"),
    (5, 513, "linear", False, True, 24, "hn"), (300, 1021, "silu", False, True, 0, "hn"),
    (1100, 72, "sigmoid", False, False, 8, "h"), (2, 4096, "silu", False, True, 0, "hn"),
    (600, 2048, None, True, True, 0, "hn"), (9, 8192, "silu", False, True, 13, "hn"),
    (3, 8200, "sigmoid", False, True, 0, "n"), (2, 16384, "linear", False, True, 0, "hn"),
    (5, 12001, "silu", False, True, 0, "hn"), (2100, 520, "silu", False, True, 16, "hn")]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_block_norm_and_gradients(case, dtype):
    T, W, act, raw, weights, cut, given = case
    say(f"block norm {case} {dtype}")
    x, y, gate, (wy, sc, wn), dh, dn = _inputs(T, W, dtype, act, weights, cut, T + W)
    dh, dn = (dh if "h" in given else None), (dn if "n" in given else None)
    kw = dict(gate=gate, y_weight=wy, scale=sc, n_weight=wn, eps=EPS, flags=FLAGS[act] | (m3.M3_BLOCK_RAW if raw else 0))
    h, n = m3.block_norm(x, y, **kw)
    d = m3.block_norm_backward(x, y, dh, dn, **kw)
    torch.cuda.synchronize()
    want = block_ref.check(x, y, gate, wy, sc, wn, EPS, act, raw, dtype, dh, dn)
    got = {"h": h, "n": n, **{k: d[v] for k, v in NAMES.items()}}
    for name, (v, b) in want.items():
        _check(name, got[name], v, b)
    assert all(got[k] is None for k in got if k not in want)


def test_gradients_against_differences():
    """One direction of all inputs at once, by central differences of the 64-bit form."""
    T, W = 6, 40
    x, y, gate, (wy, sc, wn), dh, dn = _inputs(T, W, F32, "silu", True, 0, 3)
    d = m3.block_norm_backward(x, y, dh, dn, gate=gate, y_weight=wy, scale=sc, n_weight=wn, flags=m3.M3_GATE_SILU)
    ins = [ref.f64(t) for t in (x, y, gate, wy, sc, wn)]
    g = torch.Generator().manual_seed(9)
    way = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in ins]

    def loss(e):
        f = block_ref.forward(*(t + e * w for t, w in zip(ins, way)), 1e-6, "silu", False)
        return float((f["h"] * ref.f64(dh)).sum() + (f["n"] * ref.f64(dn)).sum())

    e = 1e-5
    slope = (loss(e) - loss(-e)) / (2 * e)
    got = sum(float((ref.f64(d[k]) * w).sum()) for k, w in zip(("x", "y", "gate", "y_weight", "scale", "n_weight"), way))
    # the difference is off by e^2 / 6 of a third derivative, far below 1e-6 of the slope's terms
    size = sum(float((ref.f64(d[k]) * w).abs().sum()) for k, w in zip(("x", "y", "gate", "y_weight", "scale", "n_weight"), way))
    assert abs(slope - got) <= 1e-5 * size, (slope, got, size)


def test_infinities_and_nan_stay_in_their_row():
    T, W = 700, 256
    x, y, gate, (wy, sc, wn), dh, dn = _inputs(T, W, BF16, "silu", True, 0, 5)
    kw = dict(gate=gate, y_weight=wy, scale=sc, n_weight=wn, flags=m3.M3_GATE_SILU)
    clean = m3.block_norm(x, y, **kw)
    dclean = m3.block_norm_backward(x, y, dh, dn, **kw)
    x2, y2, g2 = x.clone(), y.clone(), gate.clone()
    x2[3, 7], y2[300, 0], g2[699, 255] = float("inf"), float("nan"), float("-inf")
    kw["gate"] = g2
    got, d = m3.block_norm(x2, y2, **kw), m3.block_norm_backward(x2, y2, dh, dn, **kw)
    keep = [t for t in range(T) if t not in (3, 300, 699)]
    for a, b in zip(clean, got):
        assert torch.equal(a[keep], b[keep])
    for k in ("x", "y", "gate"):
        assert torch.equal(dclean[k][keep], d[k][keep]), k
    assert torch.isinf(got[0][3, 7]) and torch.isnan(got[1][300]).all() and torch.isnan(got[0][699, 255])


def test_equal_bits_in_place_and_replayed():
    T, W = 900, 1032
    x, y, gate, (wy, sc, wn), dh, dn = _inputs(T, W, BF16, "sigmoid", True, 0, 6)
    kw = dict(gate=gate, y_weight=wy, scale=sc, n_weight=wn, flags=m3.M3_GATE_SIGMOID)
    h, n = m3.block_norm(x, y, **kw)
    d = m3.block_norm_backward(x, y, dh, dn, **kw)
    d2 = m3.block_norm_backward(x, y, dh, dn, **kw)
    assert all(torch.equal(d[k], d2[k]) for k in d)
    # h over x
    dims = m3.m3_block_dims(T, W, m3.M3_BF16, m3.M3_GATE_SIGMOID, 1e-6, 0, 0, 0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    x2, n2 = x.clone(), torch.empty_like(n)
    assert m3.library().m3_block_norm(ctypes.byref(dims), p(x2), p(y), p(gate), p(wy), p(sc), p(wn), p(x2), p(n2),
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert torch.equal(x2, h) and torch.equal(n2, n)
    # without n
    assert torch.equal(m3.block_norm(x, y, want_n=False, **kw)[0], h)
    # a captured step, replayed over changing inputs with eager work between
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gh, gn = m3.block_norm(x, y, **kw)
            gd = m3.block_norm_backward(x, y, dh, dn, **kw)
    for k in range(3):
        x.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eh, en = m3.block_norm(x, y, **kw)
        ed = m3.block_norm_backward(x, y, dh, dn, **kw)
        assert torch.equal(gh, eh) and torch.equal(gn, en), k
        assert all(torch.equal(gd[n], ed[n]) for n in gd), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", [(600, 5473, "silu", False, 0, "hn"), (300, 6001, "sigmoid", True, 0, "n"),
                                  (300, 8192, "silu", False, 0, "h"), (530, 9001, "silu", False, 0, "hn"),
                                  (290, 12345, None, False, 21, "n"), (270, 8208, "linear", True, 0, "h"),
                                  (270, 16000, "silu", False, 0, "hn"), (3, 16383, "silu", False, 0, "hn")])
def test_wide_rows_several_to_a_workgroup(case, dtype):
    T, W, act, raw, cut, given = case
    test_block_norm_and_gradients((T, W, act, raw, True, cut, given), dtype)


@pytest.mark.parametrize("W", [4097, 9001, 12352])
def test_wide_rows_in_place(W):
    for dtype in (F32, BF16):
        x, y, gate, (wy, sc, wn), _, _ = _inputs(540, W, dtype, "silu", True, 0, W)
        h, n = m3.block_norm(x, y, gate, wy, sc, wn, flags=m3.M3_GATE_SILU)
        dims = m3.m3_block_dims(540, W, m3.dtype_code(dtype), m3.M3_GATE_SILU, 1e-6, 0, 0, 0)
        p = lambda t: ctypes.c_void_p(t.data_ptr())
        for over in (0, 1):
            ins = [x.clone(), y.clone()]
            n2 = torch.empty_like(n)
            assert m3.library().m3_block_norm(ctypes.byref(dims), p(ins[0]), p(ins[1]), p(gate), p(wy), p(sc), p(wn),
                                              p(ins[over]), p(n2), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
            torch.cuda.synchronize()
            assert torch.equal(ins[over], h) and torch.equal(n2, n) and torch.equal(ins[1 - over], (y, x)[over])


def test_two_streams_and_refused_tensors():
    runs = []
    for seed in (11, 12):
        x, y, gate, (wy, sc, wn), dh, dn = _inputs(400, 777, F32, "silu", True, 0, seed)
        kw = dict(gate=gate, y_weight=wy, scale=sc, n_weight=wn, flags=m3.M3_GATE_SILU)
        runs.append(lambda x=x, y=y, dh=dh, dn=dn, kw=kw: [*m3.block_norm(x, y, **kw), *(
            t for t in m3.block_norm_backward(x, y, dh, dn, **kw).values())])
    want = [[t.clone() for t in f()] for f in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = []
        for s, f in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, o))
    x, y, gate, (wy, sc, wn), dh, dn = _inputs(4, 64, BF16, "silu", True, 0, 1)
    for bad in (dict(gate=gate.cpu()), dict(gate=gate[:, :32]), dict(y_weight=wy.double()), dict(scale=sc[:63]),
                dict(gate=gate.t().contiguous().t()), dict(n_weight=wn.cpu())):
        with pytest.raises(ValueError):
            m3.block_norm(x, y, **bad)
    with pytest.raises(ValueError):
        m3.block_norm(x, y.float())
    with pytest.raises(TypeError):
        m3.block_norm(x.half(), y.half())
    with pytest.raises(m3.M3Error):
        m3.block_norm_backward(x, y, None, None)
    with pytest.raises(m3.M3Error):
        m3.block_norm(torch.zeros(4, 72, dtype=BF16, device="cuda")[:, 1:65], y)   # not on 16 bytes
    with pytest.raises(m3.M3Error):
        m3.block_norm(x[:0], y[:0])
    with pytest.raises(m3.M3Error):
        m3.block_norm(*(torch.zeros(1, 16385, device="cuda") for _ in range(2)))
