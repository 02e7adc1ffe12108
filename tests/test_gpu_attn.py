"""Causal attention over packed sequences, its gradients and the one-token
form over a cache, against the definition in 64 bits."""
import ctypes
import math

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _check(name, got, want, bound):
    w = ref.worst(got, want, bound)
    say(f"  {name}: {w:.3f} of its bound")
    assert w <= 1.0, (name, w)


def _offsets(n):
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    return cu


def _dev(cu):
    return torch.tensor(cu, dtype=torch.int32).cuda()


def _inputs(Tq, Tk, Hq, Hk, D, dtype, seed, strided=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    if strided:
        pq = n(Tq, (Hq + 1) * D).to(dtype).cuda()
        pk = n(Tk, 2 * Hk * D + 8).to(dtype).cuda()
        return (pq[:, D:].view(Tq, Hq, D), pk[:, :Hk * D].view(Tk, Hk, D),
                pk[:, Hk * D + 8:].view(Tk, Hk, D), n(Tq, Hq, D).to(dtype).cuda())
    return (n(Tq, Hq, D).to(dtype).cuda(), n(Tk, Hk, D).to(dtype).cuda(),
            n(Tk, Hk, D).to(dtype).cuda(), n(Tq, Hq, D).to(dtype).cuda())


def _all(q, k, v, do, nq, nk, scale, dtype):
    """Outputs, gradients and bounds over all sequences, in 64 bits."""
    cq, ck = _offsets(nq), _offsets(nk)
    parts = []
    for s in range(len(nq)):
        a, b = (ref.f64(t[cq[s]:cq[s + 1]]) for t in (q, do))
        c, d = (ref.f64(t[ck[s]:ck[s + 1]]) for t in (k, v))
        o, lse, p = ref.attn(a, c, d, scale)
        g, gb = ref.attn_grads(a, c, d, b, scale, dtype)
        parts.append((o, ref.attn_bound(a, c, d, o, p, scale, dtype), lse, *g, *gb))
    return [torch.cat(t) for t in zip(*parts)]


CASES = [  # queries and keys of each sequence, Hq, Hk, D
    ([1], [1], 1, 1, 64), ([5, 0, 1, 70], [5, 3, 1, 70], 4, 2, 64),
    ([128, 129], [128, 129], 2, 1, 128), ([63, 200], [300, 200], 8, 1, 128),
    ([40, 33], [10, 0], 3, 3, 64), ([1, 1, 1], [33, 64, 65], 10, 2, 128),
    ([257], [321], 5, 1, 64), ([0, 0, 2], [0, 4, 2], 2, 2, 128)]


def _many(n, seed):
    """n sequences of up to 40 queries; some are empty, some go on from more keys."""
    g = torch.Generator().manual_seed(seed)
    nq = torch.randint(0, 41, (n,), generator=g).tolist()
    more = torch.randint(-5, 60, (n,), generator=g).clamp(min=0).tolist()
    return nq, [a + b for a, b in zip(nq, more)]


# few queries of many keys, whose keys are split over workgroups
CASES += [([2], [3000], 16, 2, 64), ([1, 5, 0, 9], [2600, 1500, 0, 700], 4, 2, 128),
          ([90, 70], [1100, 1300], 3, 3, 64)]
# groups of 32 and 12 heads; more sequences than a wave has lanes; as many; sequences of several tiles that are
# taken in the order of their work
CASES += [([5, 40, 3], [9, 40, 70], 32, 1, 64), ([9, 70], [9, 200], 24, 2, 128),
          (*_many(70, 1), 4, 2, 64), (*_many(64, 2), 40, 4, 64), (*_many(64, 3), 3, 1, 128),
          ([130, 400, 0, 257], [600, 400, 9, 300], 4, 2, 64), ([129, 300, 20], [129, 300, 700], 2, 2, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES)
def test_prompt_and_gradients(case, dtype):
    nq, nk, Hq, Hk, D = case
    for strided in (False, True):
        say(f"attn {case} {dtype} strided={strided}")
        tail = 3   # rows behind the last sequence
        Tq, Tk = sum(nq) + tail, sum(nk) + tail
        q, k, v, do = _inputs(Tq, Tk, Hq, Hk, D, dtype, Tq, strided)
        for t in (q, k, v, do):
            t[t.shape[0] - tail:] = float("nan")
        scale = D ** -0.5
        cq, ck = _dev(_offsets(nq)), _dev(_offsets(nk))
        o, lse = m3.attn_prefill_varlen(q, k, v, cq, ck)
        dq, dk, dv = m3.attn_prefill_varlen_backward(q, k, v, o, lse, do, cq, ck)
        torch.cuda.synchronize()
        wo, bo, wl, wq, wk, wv, bq, bk, bv = _all(q, k, v, do, nq, nk, scale, dtype)
        n, m = Tq - tail, Tk - tail
        _check("o", o[:n], wo, bo)
        # a score: D fp32 sums of products; the logarithm of their sum 2^-20
        amax = float(scale * D * 16)
        _check("lse", lse[:n], wl, torch.tensor(2.0 ** -24 * (D + 8) * amax + 2.0 ** -19 * 8))
        _check("dq", dq[:n], wq, bq)
        _check("dk", dk[:m], wk, bk)
        _check("dv", dv[:m], wv, bv)


def test_rows_behind_the_last_sequence_stay():
    q, k, v, do = _inputs(200, 200, 2, 1, 64, BF16, 3)
    cu = _dev([0, 100, 150])
    o = torch.full_like(q, 7.0)
    lse = torch.full((200, 2), 7.0, device="cuda")
    d = m3.m3_attn_dims(2, 200, 200, 2, 1, 64, m3.M3_BF16, 0.125, 0, 0, 0, 0, 0, 0, 0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    lib = m3.library()
    assert lib.m3_attn_prefill_varlen(ctypes.byref(d), p(cu), p(cu), p(q), p(k), p(v), p(o), p(lse), None, 0, s) == 0
    g = [torch.full_like(t, 7.0) for t in (q, k, v)]
    ws = torch.empty(lib.m3_attn_prefill_varlen_backward_workspace_size(ctypes.byref(d)), dtype=torch.uint8,
                     device="cuda")
    assert lib.m3_attn_prefill_varlen_backward(
        ctypes.byref(d), p(cu), p(cu), p(q), p(k), p(v), p(o), p(lse), p(do), *(p(t) for t in g), p(ws),
        ws.numel(), s) == 0
    torch.cuda.synchronize()
    for t in (o, lse, *g):
        assert (t[150:] == 7).all() and not (t[:150] == 7).all(-1).any()


def test_few_queries_of_many_keys():
    """The keys split over workgroups: rows that no sequence covers stay, NaN of
    what a query does not see as well, and replays of a graph keep the bits."""
    Hq, Hk, D, nk = 4, 2, 64, [3000, 2500]
    q, k, v, _ = _inputs(12, 5510, Hq, Hk, D, BF16, 31)
    cq, ck = _dev([2, 5, 9]), _dev([5, 3005, 5505])
    k[:5] = v[:5] = float("nan")
    v[3004, 0] = float("inf")   # the last key of the first sequence: its last query alone sees it
    o, lse = torch.full_like(q, 7.0), torch.full((12, Hq), 7.0, device="cuda")
    d = m3.m3_attn_dims(2, 12, 5510, Hq, Hk, D, m3.M3_BF16, 0.125, *[0] * 7)
    lib = m3.library()
    n = lib.m3_attn_prefill_varlen_workspace_size(ctypes.byref(d))
    assert n > 16
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN
    p = lambda t: ctypes.c_void_p(t.data_ptr())

    def run():
        assert lib.m3_attn_prefill_varlen(ctypes.byref(d), p(cq), p(ck), p(q), p(k), p(v), p(o), p(lse), p(ws), n,
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    run()
    torch.cuda.synchronize()
    for t in (o, lse):
        assert (t[:2] == 7).all() and (t[9:] == 7).all()
    assert torch.isinf(o[4, :2]).all() and torch.isfinite(o[2:4]).all() and torch.isfinite(o[5:9]).all()
    assert torch.isfinite(o[4, 2:]).all() and torch.isfinite(lse[2:9]).all()
    want = [o.clone(), lse.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        o.fill_(7.0)
        lse.fill_(7.0)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_offsets_outside_the_rows_touch_nothing_else():
    """Offsets that do not rise or leave the rows: no row outside the buffers
    is touched (guard rows around them stay), and the call returns."""
    T, H, D = 100, 2, 64
    guard = lambda: torch.full((T + 20, H, D), 5.0, dtype=BF16, device="cuda")
    q, k, v, do = _inputs(T, T, H, H, D, BF16, 4)
    bufs = [guard() for _ in range(4)]
    o, dq, dk, dv = (b[10:10 + T] for b in bufs)
    lse = torch.zeros(T, H, device="cuda")
    lib = m3.library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for cu in ([-7, 50, 400], [90, 10, 100], [100, 100, 0], [0, 500, 20]):
        c = _dev(cu)
        d = m3.m3_attn_dims(2, T, T, H, H, D, m3.M3_BF16, 0.125, 0, 0, 0, 0, 0, 0, 0)
        ws = torch.empty(lib.m3_attn_prefill_varlen_backward_workspace_size(ctypes.byref(d)),
                         dtype=torch.uint8, device="cuda")
        assert lib.m3_attn_prefill_varlen(ctypes.byref(d), p(c), p(c), p(q), p(k), p(v), p(o), p(lse), None, 0, s) == 0
        assert lib.m3_attn_prefill_varlen_backward(
            ctypes.byref(d), p(c), p(c), p(q), p(k), p(v), p(o), p(lse), p(do), p(dq), p(dk), p(dv), p(ws),
            ws.numel(), s) == 0
        torch.cuda.synchronize()
    for b in bufs:
        assert (b[:10] == 5).all() and (b[10 + T:] == 5).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_infinities_and_nan_reach_only_who_sees_them(D, dtype):
    n, Hq, Hk = [150, 90], 2, 1
    q, k, v, _ = _inputs(240, 240, Hq, Hk, D, dtype, 6)
    v[70, 0, 3] = float("nan")
    v[100, 0, 9] = float("inf")
    v[149, 0, D - 1] = -float("inf")
    k[120, 0, 1] = float("nan")
    k[239] = float("inf")
    cu = _dev(_offsets(n))
    o, lse = m3.attn_prefill_varlen(q, k, v, cu, cu)
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[~torch.isfinite(t)] = 0.5
    o2, lse2 = m3.attn_prefill_varlen(q, k2, v2, cu, cu)
    torch.cuda.synchronize()
    # before a special value nothing changes; the second sequence has only
    # its last query's own key
    assert torch.equal(o[:70], o2[:70]) and torch.equal(lse[:120], lse2[:120])
    assert torch.equal(o[150:239], o2[150:239]) and torch.equal(lse[150:239], lse2[150:239])
    keep = [d for d in range(D) if d not in (3, 9)]
    assert torch.equal(o[70:120][..., keep], o2[70:120][..., keep])
    assert torch.isnan(o[70:120, :, 3]).all()
    assert torch.equal(o[70:100, :, 9], o2[70:100, :, 9])
    assert (o[100:120, :, 9] == float("inf")).all()
    assert torch.isnan(o[120:150]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_a_sequence_with_nan_stay_there(dtype):
    n, Hq, Hk, D = [70, 45, 130], 4, 2, 64
    q, k, v, do = _inputs(245, 245, Hq, Hk, D, dtype, 16)
    cu = _dev(_offsets(n))
    o, lse = m3.attn_prefill_varlen(q, k, v, cu, cu)
    g = m3.attn_prefill_varlen_backward(q, k, v, o, lse, do, cu, cu)
    for t in (q, k, v, do):
        t[70:115] = float("nan")
    o2, lse2 = m3.attn_prefill_varlen(q, k, v, cu, cu)
    g2 = m3.attn_prefill_varlen_backward(q, k, v, o2, lse2, do, cu, cu)
    torch.cuda.synchronize()
    for a, b in zip((o, lse, *g), (o2, lse2, *g2)):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[115:], b[115:])
        assert torch.isnan(b[70:115]).all()


def test_a_masked_score_of_any_size():
    """Scores far below and above what fp32's exponential holds."""
    q, k, v, _ = _inputs(100, 100, 1, 1, 64, F32, 7)
    k = k * torch.logspace(-3, 3, 100, device="cuda")[:, None, None]
    cu = _dev([0, 100])
    o, lse = m3.attn_prefill_varlen(q, k, v, cu, cu)
    wo, wl, p = ref.attn(ref.f64(q), ref.f64(k), ref.f64(v), 0.125)
    _check("o", o, wo, ref.attn_bound(ref.f64(q), ref.f64(k), ref.f64(v), wo, p, 0.125, F32))
    assert torch.isfinite(lse).all()


def _decode_ref(q, k, v, lengths, scale, dtype):
    outs = []
    for s, n in enumerate(lengths):
        a, c, d = ref.f64(q[s:s + 1]), ref.f64(k[s, :n]), ref.f64(v[s, :n])
        o, lse, p = ref.attn(a, c, d, scale)
        outs.append((o, ref.attn_bound(a, c, d, o, p, scale, dtype), lse))
    return [torch.cat(t) for t in zip(*outs)]


DECODE = [  # lengths, cap, Hq, Hk, D
    ([0, 1, 31, 32, 33], 40, 4, 2, 64), ([700, 5, 1500], 1500, 8, 1, 128),
    ([2000], 2100, 3, 3, 64), ([513], 513, 40, 1, 64), ([64, 1000, 0, 3], 1030, 33, 1, 128)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", DECODE)
def test_decode(case, dtype):
    lengths, cap, Hq, Hk, D = case
    S = len(lengths)
    say(f"decode {case} {dtype}")
    g = torch.Generator().manual_seed(cap)
    q = torch.randn(S, Hq, D, generator=g).to(dtype).cuda()
    kv = torch.randn(S, cap + 2, 2, Hk, D, generator=g).to(dtype).cuda()
    for s, n in enumerate(lengths):   # the rest of a cache is not read
        kv[s, n:] = float("nan")
    k, v = kv[:, :cap, 0], kv[:, :cap, 1]
    o, lse = m3.attn_decode(q, k, v, torch.tensor(lengths, dtype=torch.int32).cuda())
    o2, lse2 = m3.attn_decode(q, k.contiguous(), v.contiguous(), torch.tensor(lengths, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    scale = D ** -0.5
    wo, bo, wl = _decode_ref(q, k, v, lengths, scale, dtype)
    _check("o", o, wo, bo)
    _check("lse", lse, wl, torch.tensor(2.0 ** -24 * (D + 8) * scale * D * 16 + 2.0 ** -19 * 8))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_of_many_sequences(dtype):
    """More sequences and heads than 2^15 together; some of them checked."""
    S, cap, Hq, Hk, D = 600, 70, 64, 8, 64
    g = torch.Generator().manual_seed(S)
    q = torch.randn(S, Hq, D, generator=g).to(dtype).cuda()
    k, v = (torch.randn(S, cap, Hk, D, generator=g).to(dtype).cuda() for _ in range(2))
    lengths = torch.randint(0, cap + 1, (S,), generator=g).tolist()
    o, lse = m3.attn_decode(q, k, v, torch.tensor(lengths, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for s in (0, 1, 299, 511, 512, 513, 598, 599):
        one = slice(s, s + 1)
        wo, bo, wl = _decode_ref(q[one], k[one], v[one], lengths[one], D ** -0.5, dtype)
        _check("o", o[one], wo, bo)
        _check("lse", lse[one], wl, torch.tensor(2.0 ** -24 * (D + 8) * D ** 0.5 * 16 + 2.0 ** -19 * 8))


def test_decode_lengths_are_clamped():
    q = torch.randn(2, 2, 64, device="cuda")
    k, v = torch.randn(2, 50, 1, 64, device="cuda"), torch.randn(2, 50, 1, 64, device="cuda")
    t = lambda *n: torch.tensor(n, dtype=torch.int32).cuda()
    a, b = m3.attn_decode(q, k, v, t(-4, 900)), m3.attn_decode(q, k, v, t(0, 50))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0][0] == 0).all() and torch.isinf(a[1][0]).all()


def test_decode_offsets_beyond_32_bits():
    """A cache of 2^31 and more elements: nearly all weight on its last row."""
    Hk, D = 8, 128
    n = (1 << 21) + 77
    k = torch.zeros(1, n, Hk, D, dtype=BF16, device="cuda")
    v = torch.zeros(1, n, Hk, D, dtype=BF16, device="cuda")
    q = torch.ones(1, Hk, D, dtype=BF16, device="cuda")
    k[0, -1] = 20.0 / D
    val = torch.randn(Hk, D, device="cuda").to(BF16)
    v[0, -1] = val
    o, lse = m3.attn_decode(q, k, v, torch.tensor([n], dtype=torch.int32).cuda(), scale=1.0)
    torch.cuda.synchronize()
    e = math.exp(float(ref.f64(k[0, -1, 0]).sum()))
    w = e / (e + n - 1)
    _check("o", o[0], ref.f64(val) * w, 2 * 2.0 ** -8 * ref.f64(val).abs() + 1e-30)
    assert abs(float(lse[0, 0]) - math.log(e + n - 1)) <= 1e-4


def test_one_token_prompt_equals_decode():
    """A single query at the end of a cache through both calls."""
    q, k, v, _ = _inputs(1, 900, 4, 2, 128, F32, 12)
    o, lse = m3.attn_prefill_varlen(q, k, v, _dev([0, 1]), _dev([0, 900]))
    o2, lse2 = m3.attn_decode(q, k[None], v[None], torch.tensor([900], dtype=torch.int32).cuda())
    wo, wl, p = ref.attn(ref.f64(q), ref.f64(k), ref.f64(v), 128 ** -0.5)
    b = ref.attn_bound(ref.f64(q), ref.f64(k), ref.f64(v), wo, p, 128 ** -0.5, F32)
    _check("prompt", o, wo, b)
    _check("decode", o2, wo, b)


def test_equal_bits_graphs_and_streams():
    q, k, v, do = _inputs(500, 500, 8, 2, 64, BF16, 8)
    cu = _dev([0, 300, 301, 500])
    cache = torch.randn(2, 2000, 2, 64, device="cuda").to(BF16)
    ln = torch.tensor([1999, 7], dtype=torch.int32).cuda()

    def once():
        o, lse = m3.attn_prefill_varlen(q, k, v, cu, cu)
        g = m3.attn_prefill_varlen_backward(q, k, v, o, lse, do, cu, cu)
        return [o, lse, *g, *m3.attn_decode(q[:2], cache, cache, ln)]

    want = [t.clone() for t in once()]
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(once(), want))
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
    for _ in range(3):
        for g, out in graphs:
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = m3.attn_prefill_varlen(q, k, v, cu, cu, stream=s)
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def _tail_specials(v, s, n, D):
    """Infinities of both signs and NaN in the last rows of a cache's values."""
    v[s, n - 1, 0, 3] = float("inf")
    v[s, n - 1, -1, D - 1] = -float("inf")
    if n > 1:
        v[s, n - 2, 0, 9] = float("nan")
        v[s, n - 2, 0, 40] = float("inf")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_infinite_values_in_a_cache_that_ends_inside_a_tile(D, dtype):
    """The last row is there once: what is loaded for the rest of its tile must
    not turn an infinity into NaN.  Whole tiles, one row, and caches that are
    split over workgroups among them."""
    Hq, Hk = 6, 2
    for lengths, cap in (([1, 33, 64, 95, 2, 31], 96), ([1500, 513, 1026], 1500)):
        S = len(lengths)
        g = torch.Generator().manual_seed(cap + D)
        q = torch.randn(S, Hq, D, generator=g).to(dtype).cuda()
        k, v = (torch.randn(S, cap, Hk, D, generator=g).to(dtype).cuda() for _ in range(2))
        for s, n in enumerate(lengths):
            _tail_specials(v, s, n, D)
        o, lse = m3.attn_decode(q, k, v, torch.tensor(lengths, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        wo, bo, wl = _decode_ref(q, k, v, lengths, D ** -0.5, dtype)
        _check("o", o, wo, bo)
        _check("lse", lse, wl, torch.tensor(2.0 ** -24 * (D + 8) * D ** 0.5 * 16 + 2.0 ** -19 * 8))


def _of_sequence(q, k, v, do, o, lse, grads, a, c, dtype):
    """Rows a of queries and c of keys against the definition."""
    scale = q.shape[-1] ** -0.5
    x, y, z, w = ref.f64(q[a]), ref.f64(k[c]), ref.f64(v[c]), ref.f64(do[a])
    wo, wl, p = ref.attn(x, y, z, scale)
    (wq, wk, wv), (bq, bk, bv) = ref.attn_grads(x, y, z, w, scale, dtype)
    _check("o", o[a], wo, ref.attn_bound(x, y, z, wo, p, scale, dtype))
    _check("lse", lse[a], wl, torch.tensor(2.0 ** -24 * (q.shape[-1] + 8) * q.shape[-1] ** 0.5 * 16 + 2.0 ** -19 * 8))
    for n, got, want, b in (("dq", grads[0][a], wq, bq), ("dk", grads[1][c], wk, bk), ("dv", grads[2][c], wv, bv)):
        _check(n, got, want, b)


def test_rows_times_heads_beyond_2_to_28():
    """2^34 and more elements of q: sequences at both ends and in the middle."""
    torch.cuda.empty_cache()   # 110 GB
    n, Hq, D, L = (1 << 23) + 1000, 32, 64, 200
    q = torch.empty(n, Hq, D, dtype=BF16, device="cuda")
    for r in range(0, n, 1 << 18):
        q[r:r + (1 << 18)].normal_()
    k, v = torch.randn(n, 1, D, device="cuda").to(BF16), torch.randn(n, 1, D, device="cuda").to(BF16)
    cut = list(range(0, n, L)) + [n]
    cu = _dev(cut)
    o, lse = m3.attn_prefill_varlen(q, k, v, cu, cu)
    g = m3.attn_prefill_varlen_backward(q, k, v, o, lse, q, cu, cu)
    torch.cuda.synchronize()
    for s in (0, 1, len(cut) // 2, len(cut) - 3, len(cut) - 2):
        rows = slice(cut[s], cut[s + 1])
        say(f"sequence {s}: rows {rows.start}..{rows.stop}")
        _of_sequence(q, k, v, q, o, lse, g, rows, rows, BF16)


def test_keys_of_more_than_2_to_34_elements():
    """The last sequence's keys lie behind 2^34 elements of a sequence that has
    no query, whose gradients are 0."""
    torch.cuda.empty_cache()   # 140 GB
    n0, L, H, D = (1 << 24) - 100, 201, 16, 64
    k, v = (torch.empty(n0 + L, H, D, dtype=BF16, device="cuda") for _ in range(2))
    k[n0:].normal_()
    v[n0:].normal_()
    q, do = torch.randn(70, H, D, device="cuda").to(BF16), torch.randn(70, H, D, device="cuda").to(BF16)
    cq, ck = _dev([0, 0, 70]), _dev([0, n0, n0 + L])
    o, lse = m3.attn_prefill_varlen(q, k, v, cq, ck)
    g = m3.attn_prefill_varlen_backward(q, k, v, o, lse, do, cq, ck)
    torch.cuda.synchronize()
    for t in g[1:]:
        assert not t[:5000].any() and not t[n0 - 5000:n0].any()
    _of_sequence(q, k, v, do, o, lse, g, slice(0, 70), slice(n0, n0 + L), BF16)


# 64 sequences of 40 heads: more workgroups than are taken in the order of their
# work (counted in test_layers_host.py)
MANY_Q, MANY_K = _many(60, 2)
MANY_Q, MANY_K = [300, 0, 257, 130] + MANY_Q, [400, 3, 257, 100] + MANY_K
MANY_HEADS = 40, [40, 8]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hk", MANY_HEADS[1])
def test_few_sequences_in_more_workgroups_than_are_ranked(Hk, dtype):
    test_prompt_and_gradients((MANY_Q, MANY_K, MANY_HEADS[0], Hk, 64), dtype)
