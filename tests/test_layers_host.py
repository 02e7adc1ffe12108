"""Host-only checks of the gated recurrence, the q/k norms and the attention
calls: what they refuse, before anything is launched, and the 64-bit
references that the GPU tests use."""
import ctypes
import re
import os

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import layers_ref as ref

C = 8.0
F32 = torch.float32
OK, NULL, SHAPE, DTYPE, UNSUP, ALIGN, WS = range(7)
P16 = ctypes.c_void_p(4096)     # aligned, never dereferenced
P_MIS = ctypes.c_void_p(4104)
P_ODD = ctypes.c_void_p(4098)
BIG = 1 << 50


def _gdims(**kw):
    base = dict(batch=2, seqlen=300, width=64, dtype=m3.M3_BF16, c=8.0, ld_x=0, ld_r=0, ld_i=0, ld_g=0)
    base.update(kw)
    return m3.m3_gated_dims(*base.values())


def _qdims(**kw):
    base = dict(tokens=10, nheads_q=4, nheads_k=2, headdim=64, rotary_dim=64, dtype=m3.M3_BF16, flags=0,
                eps=1e-6, base=1e4, ld_q=0, ld_k=0, ld_dq=0, ld_dk=0)
    base.update(kw)
    return m3.m3_qk_dims(*base.values())


def _adims(**kw):
    base = dict(nseq=2, tokens_q=100, tokens_k=100, nheads_q=4, nheads_k=2, headdim=64, dtype=m3.M3_BF16,
                scale=0.1, ld_q=0, ld_k=0, ld_v=0, ld_o=0, ld_do=0, stride_k=0, stride_v=0)
    base.update(kw)
    return m3.m3_attn_dims(*base.values())


def _call(fn, d, names, required, over, ws=True):
    args = {n: (P16 if n in required else None) for n in names}
    args.update({k: v for k, v in over.items() if k in args})
    a = list(args.values())
    if ws:
        a += [over.get("ws", P16), over.get("ws_bytes", BIG)]
    return getattr(m3.library(), fn)(None if d is None else ctypes.byref(d), *a, None)


def _scan(d, **o):
    return _call("m3_gated_scan", d, ("cu", "x", "r", "i", "decay", "h0", "y", "hT", "states"),
                 ("x", "r", "i", "decay", "y"), o)


def _scan_bwd(d, **o):
    return _call("m3_gated_scan_backward", d,
                 ("cu", "x", "r", "i", "decay", "h0", "states", "dy", "dhT", "dx", "dr", "di", "ddecay", "dh0"),
                 ("x", "r", "i", "decay", "states", "dy", "dx", "dr", "di", "ddecay"), o)


def _step(d, **o):
    return _call("m3_gated_step", d, ("h", "x", "r", "i", "decay", "y"), ("h", "x", "r", "i", "decay", "y"), o,
                 ws=False)


def _qk(d, **o):
    return _call("m3_qk_norm_rope", d, ("q", "k", "wq", "wk", "pos", "qo", "ko"), ("q", "k", "pos", "qo", "ko"), o,
                 ws=False)


def _qk_bwd(d, **o):
    return _call("m3_qk_norm_rope_backward", d,
                 ("q", "k", "wq", "wk", "pos", "gq", "gk", "dq", "dk", "dwq", "dwk"),
                 ("q", "k", "pos", "gq", "gk", "dq", "dk"), o)


def _attn(d, **o):
    return _call("m3_attn_prefill_varlen", d, ("cuq", "cuk", "q", "k", "v", "o", "lse"),
                 ("cuq", "cuk", "q", "k", "v", "o"), o)


def _attn_bwd(d, **o):
    n = ("cuq", "cuk", "q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")
    return _call("m3_attn_prefill_varlen_backward", d, n, n, o)


def _decode(d, **o):
    return _call("m3_attn_decode", d, ("len", "q", "k", "v", "o", "lse"), ("len", "q", "k", "v", "o"), o)


def test_header_declares_and_the_library_exports():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "m3ssm.h")).read(), flags=re.S)
    for n in ("m3_gated_scan", "m3_gated_scan_backward", "m3_gated_step", "m3_qk_norm_rope",
              "m3_qk_norm_rope_backward", "m3_attn_prefill_varlen", "m3_attn_prefill_varlen_workspace_size", "m3_attn_prefill_varlen_backward",
              "m3_attn_decode", "m3_gated_scan_workspace_size", "m3_gated_scan_backward_workspace_size",
              "m3_qk_norm_rope_backward_workspace_size", "m3_attn_prefill_varlen_backward_workspace_size",
              "m3_attn_decode_workspace_size"):
        assert re.search(r"\b" + n + r"\s*\(", src) and hasattr(m3.library(), n), n


def test_struct_sizes_match_the_header():
    """ctypes lays the dims out as the C compiler does (fields in the
    header's order; 8-byte fields aligned)."""
    assert ctypes.sizeof(m3.m3_gated_dims) == 56 and m3.m3_gated_dims.ld_x.offset == 24
    assert ctypes.sizeof(m3.m3_qk_dims) == 72 and m3.m3_qk_dims.base.offset == 32
    assert ctypes.sizeof(m3.m3_attn_dims) == 88 and m3.m3_attn_dims.ld_q.offset == 32


def test_gated_refusals():
    for call in (_scan, _scan_bwd, _step):
        assert call(None) == NULL
        assert call(_gdims(batch=0)) == SHAPE
        assert call(_gdims(width=0)) == SHAPE
        assert call(_gdims(c=0.0)) == SHAPE
        assert call(_gdims(c=float("nan"))) == SHAPE
        assert call(_gdims(c=float("inf"))) == SHAPE
        assert call(_gdims(ld_r=63)) == SHAPE
        assert call(_gdims(ld_g=-64)) == SHAPE
        assert call(_gdims(dtype=2)) == DTYPE
        for n in ("x", "r", "i", "decay"):
            assert call(_gdims(), **{n: None}) == NULL
            assert call(_gdims(), **{n: P_MIS}) == ALIGN
    for call in (_scan, _scan_bwd):
        assert call(_gdims(seqlen=0)) == SHAPE
        assert call(_gdims(batch=1 << 20, seqlen=1 << 20, width=1 << 20)) == SHAPE   # grid
        assert call(_gdims(), cu=P_ODD) == ALIGN
        assert call(_gdims(), h0=P_MIS) == ALIGN
        assert call(_gdims(), ws=None) == WS
        assert call(_gdims(), ws=P_MIS) == ALIGN
    assert _scan(_gdims(), y=None) == NULL
    for n in ("states", "dy", "dx", "dr", "di", "ddecay"):
        assert _scan_bwd(_gdims(), **{n: None}) == NULL
    assert _step(_gdims(), h=None) == NULL
    size = m3.library().m3_gated_scan_workspace_size
    for packed in (0, 1):
        n = size(ctypes.byref(_gdims()), packed)
        assert n > 0
        assert _scan(_gdims(), ws_bytes=n - 1, cu=P16 if packed else None) == WS
        nb = m3.library().m3_gated_scan_backward_workspace_size(ctypes.byref(_gdims()), packed)
        assert nb > n and _scan_bwd(_gdims(), ws_bytes=nb - 1, cu=P16 if packed else None) == WS
    assert size(ctypes.byref(_gdims(seqlen=0)), 0) == 0 and size(None, 0) == 0


def test_qk_refusals():
    for call in (_qk, _qk_bwd):
        assert call(None) == NULL
        for bad in (dict(tokens=0), dict(nheads_q=0), dict(nheads_k=-1), dict(rotary_dim=66), dict(rotary_dim=-2),
                    dict(rotary_dim=7), dict(flags=2), dict(eps=-1.0), dict(eps=float("nan")), dict(base=0.0),
                    dict(base=float("inf")), dict(ld_q=255), dict(ld_k=127), dict(ld_dq=8)):
            assert call(_qdims(**bad)) == SHAPE, bad
        assert call(_qdims(dtype=7)) == DTYPE
        for D in (8, 48, 96, 512):
            assert call(_qdims(headdim=D, rotary_dim=0)) == UNSUP
        assert call(_qdims(ld_q=260)) == ALIGN
        assert call(_qdims(), pos=P_ODD) == ALIGN
        for n in ("q", "k", "pos"):
            assert call(_qdims(), **{n: None}) == NULL
        for n in ("q", "k", "wq", "wk"):
            assert call(_qdims(), **{n: P_MIS}) == ALIGN
    assert _qk(_qdims(), qo=None) == NULL
    for n in ("gq", "gk", "dq", "dk"):
        assert _qk_bwd(_qdims(), **{n: None}) == NULL
    n = m3.library().m3_qk_norm_rope_backward_workspace_size(ctypes.byref(_qdims()))
    assert n > 0 and _qk_bwd(_qdims(), ws_bytes=n - 1) == WS and _qk_bwd(_qdims(), ws=None) == WS
    assert m3.library().m3_qk_norm_rope_backward_workspace_size(ctypes.byref(_qdims(tokens=0))) == 0


def test_attn_refusals():
    for call in (_attn, _attn_bwd, _decode):
        assert call(None) == NULL
        for bad in (dict(nseq=0), dict(tokens_k=0), dict(nheads_q=0), dict(nheads_k=0), dict(nheads_q=5),
                    dict(nheads_q=2, nheads_k=4), dict(scale=float("nan")), dict(scale=float("inf")),
                    dict(ld_q=248), dict(ld_k=120), dict(ld_v=-8), dict(ld_o=8), dict(ld_do=8),
                    dict(stride_k=-8), dict(ld_q=1 << 24), dict(ld_v=1 << 24)):
            assert call(_adims(**bad)) == SHAPE, bad
        assert call(_adims(dtype=-1)) == DTYPE
        for D in (32, 96, 256):
            assert call(_adims(headdim=D)) == UNSUP
        assert call(_adims(ld_q=260)) == ALIGN
        assert call(_adims(stride_v=4)) == ALIGN
        for n in ("q", "k", "v", "o"):
            assert call(_adims(), **{n: None}) == NULL
            assert call(_adims(), **{n: P_MIS}) == ALIGN
    for call in (_attn, _attn_bwd):
        assert call(_adims(tokens_q=0)) == SHAPE
        assert call(_adims(), cuq=None) == NULL and call(_adims(), cuk=None) == NULL
        assert call(_adims(), cuq=P_ODD) == ALIGN and call(_adims(), cuk=P_ODD) == ALIGN
    assert _decode(_adims(), len=None) == NULL and _decode(_adims(), len=P_ODD) == ALIGN
    for n in ("lse", "do", "dq", "dk", "dv"):
        assert _attn_bwd(_adims(), **{n: None}) == NULL
    lib = m3.library()
    n = lib.m3_attn_prefill_varlen_backward_workspace_size(ctypes.byref(_adims()))
    assert n > 0 and _attn_bwd(_adims(), ws_bytes=n - 1) == WS and _attn_bwd(_adims(), ws=None) == WS
    long = _adims(tokens_k=100000)
    n = lib.m3_attn_decode_workspace_size(ctypes.byref(long))
    assert n > 16 and _decode(long, ws_bytes=n - 1) == WS and _decode(long, ws=None) == WS
    assert lib.m3_attn_decode_workspace_size(ctypes.byref(_adims(headdim=96))) == 0
    few = _adims(tokens_q=8, tokens_k=100000)
    n = lib.m3_attn_prefill_varlen_workspace_size(ctypes.byref(few))
    assert n > 16 and _attn(few, ws_bytes=n - 1) == WS and _attn(few, ws=None) == WS
    assert lib.m3_attn_prefill_varlen_workspace_size(ctypes.byref(_adims())) == 16
    assert lib.m3_attn_prefill_varlen_workspace_size(ctypes.byref(_adims(headdim=96))) == 0


def test_attn_refuses_scales_that_are_not_positive():
    """A masked score is -inf before its scale, and the maximum is taken of
    the products: neither holds for a scale of zero or below."""
    for s in (0.0, -0.125, 1e-39):
        d = _adims(scale=s)
        assert _attn(d) == SHAPE and _attn_bwd(d) == SHAPE and _decode(d) == SHAPE, s


def test_sizes_beyond_the_struct_are_refused():
    """More rows than an int32 holds must not wrap round to fewer."""
    for v in (2 ** 31, 2 ** 32 + 5, -2 ** 33):
        with pytest.raises(ValueError, match="seqlen"):
            m3._dims(m3.m3_gated_dims, 1, v, 64, m3.M3_BF16, 8.0, 0, 0, 0, 0)
    with pytest.raises(ValueError, match="flags"):
        m3._dims(m3.m3_qk_dims, 1, 4, 2, 64, 64, m3.M3_BF16, -1, 1e-6, 1e4, 0, 0, 0, 0)
    d, _ = m3._dims(m3.m3_gated_dims, 1, 2 ** 31 - 1, 64, m3.M3_BF16, 8, 0, 0, 0, 0)
    assert d.seqlen == 2 ** 31 - 1 and d.c == 8.0


def test_counts_near_the_end_of_an_int_are_refused():
    """A loop or a tile count past the last row must not overflow."""
    n = 2 ** 31 - 5
    assert _qk(_qdims(tokens=n)) == SHAPE and _qk_bwd(_qdims(tokens=n)) == SHAPE
    assert m3.library().m3_qk_norm_rope_backward_workspace_size(ctypes.byref(_qdims(tokens=n))) == 0
    assert _attn(_adims(tokens_q=n)) == SHAPE and _attn(_adims(tokens_k=n)) == SHAPE
    assert _decode(_adims(tokens_k=n)) == SHAPE
    for k in (dict(seqlen=n, width=1), dict(width=n), dict(batch=n, width=1)):
        assert _scan(_gdims(**k)) == SHAPE and _scan_bwd(_gdims(**k)) == SHAPE, k
    assert _step(_gdims(batch=n, width=1)) == SHAPE


def test_decode_takes_large_batches():
    lib = m3.library()
    size = lambda **k: lib.m3_attn_decode_workspace_size(ctypes.byref(_adims(tokens_k=4096, nheads_q=64, nheads_k=8, **k)))
    assert size(nseq=512) > 0 and size(nseq=4096) > 0 and size(nseq=200000) > 0
    assert size(nseq=1 << 20) == 0   # 2^26 workgroups


def test_helpers_refuse_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        m3.gated_scan(z(1, 4, 8), z(1, 4, 8), z(1, 4, 8), z(8))
    with pytest.raises(ValueError):
        m3.gated_step(z(1, 8), z(1, 8), z(1, 8), z(1, 8), z(8))
    with pytest.raises(ValueError):
        m3.qk_norm_rope(z(4, 2, 64), z(4, 1, 64), z(4, dtype=torch.int32))
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        m3.attn_prefill_varlen(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), cu, cu)
    with pytest.raises(ValueError):
        m3.attn_decode(z(1, 2, 64), z(1, 4, 1, 64), z(1, 4, 1, 64), cu[:1])


def test_row_strides():
    """What counts as token rows cut out of wider rows."""
    t = torch.zeros(3, 5, 24)
    assert m3._rows("x", t, (3, 5, 24), F32) == 0   # dense
    assert m3._rows("x", t[..., 8:16], (3, 5, 8), F32) == 24
    assert m3._rows("q", t[:, 1:3], (3, 2, 24), F32) == 120
    assert m3._rows("q", t[:, 0], (3, 24), F32) == 120
    assert m3._rows("x", t[:, :1, :8], (3, 1, 8), F32) == 120
    assert m3._rows("x", t[:1, :1, :8], (1, 1, 8), F32) in (0, 24, 120)
    for bad in (t[:, :4], t.transpose(1, 2), t[..., ::2], t[:, :, :1].expand(3, 5, 24), t[:1, :1].expand(3, 5, 24)):
        with pytest.raises(ValueError):
            m3._rows("x", bad, bad.shape, F32)
    with pytest.raises(ValueError):
        m3._rows("x", t, (3, 5, 23), F32)
    with pytest.raises(ValueError):
        m3._rows("x", t, (3, 5, 24), torch.bfloat16)


def test_reference_gradients_against_differences():
    """The 64-bit gradients that the tests use against central differences."""
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    v = dict(x=n(7, 2), r=n(7, 2), i=n(7, 2), decay=n(2), h0=n(3, 2))
    dy, dhT, cu = n(7, 2), n(3, 2), [0, 4, 4, 7]
    d = ref.gated_grads(v["x"], v["r"], v["i"], v["decay"], dy, v["h0"], dhT, C, cu)

    def loss(**k):
        y, hT = ref.gated(k["x"], k["r"], k["i"], k["decay"], k["h0"], C, cu)
        return float((y * dy).sum() + (hT * dhT).sum())

    for k in v:
        for e in range(v[k].numel()):
            up, dn = ({**v, k: v[k].clone()} for _ in range(2))
            up[k].view(-1)[e] += 1e-6
            dn[k].view(-1)[e] -= 1e-6
            diff = (loss(**up) - loss(**dn)) / 2e-6
            assert abs(diff - float(d[k].reshape(-1)[e])) <= 1e-7 * (1 + abs(diff)), (k, e)


def test_reference_gradients_against_differentiation():
    """The formulas that the tests' gradients use against torch's."""
    g = torch.Generator().manual_seed(9)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    q, k, v, do = n(6, 4, 8), n(9, 2, 8), n(9, 2, 8), n(6, 4, 8)
    (dq, dk, dv), _ = ref.attn_grads(q, k, v, do, 0.3, F32)
    w = [t.clone().requires_grad_(True) for t in (q, k, v)]
    want = torch.autograd.grad((ref.attn(*w, 0.3)[0] * do).sum(), w)
    for a, b in zip((dq, dk, dv), want):
        assert float((a - b).abs().max()) <= 1e-12


class _StreamOf:
    """What the helpers look at in a stream."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.cuda_stream = 0


def test_a_stream_of_another_device_is_refused():
    """The call would go to the tensors' device, on a stream that the caller did
    not name."""
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        m3._on(0, _StreamOf("cuda:1"))
    assert isinstance(m3._on(1, _StreamOf("cuda:1")), m3._Switch)


def test_attention_takes_what_its_launches_hold():
    """Rows times heads beyond 2^28 and keys of more than 2^34 elements: a grid
    has a workgroup for 128 rows and a head, and fewer where heads share one."""
    lib = m3.library()
    size = lambda **k: lib.m3_attn_prefill_varlen_workspace_size(ctypes.byref(_adims(**k)))
    back = lambda **k: lib.m3_attn_prefill_varlen_backward_workspace_size(ctypes.byref(_adims(**k)))
    for k in (dict(tokens_q=(1 << 23) + 1, nheads_q=32, nheads_k=1), dict(tokens_q=1 << 26, nheads_q=8),
              dict(tokens_q=9000000, tokens_k=9000000, nheads_q=32, nheads_k=8),
              dict(tokens_k=(1 << 24) + 64, nheads_q=16, nheads_k=16, headdim=128)):
        assert size(**k) > 0, k
        rows = k.get("tokens_q", 100) * k["nheads_q"]
        assert back(**k) >= 8 * rows, k
    # 2^24 workgroups of 256 threads are more than a launch counts
    assert size(tokens_q=1 << 27, nheads_q=16) == 0 and back(tokens_k=1 << 27, nheads_q=16) == 0


FREQ_CPP = """
#include "rope_freq.h"
extern "C" void table(double base, int rot, double* f) { m3::rope_freq(base, rot, f); }
"""


@pytest.mark.parametrize("rot", [2, 18, 32, 64, 128, 256])
def test_rotary_frequencies(rot, tmp_path):
    """Turns a position, base^(-2 j / rot) / (2 pi), against 50 digits.  In half
    steps of fp64: 1 / (2 pi) one, two powers two each (one step of the math
    library), two products one each, and an exponent off by one turns the power
    by its logarithm, y = (2 j / rot) |ln base|."""
    import subprocess
    from decimal import Decimal, localcontext
    src, out = tmp_path / "t.cpp", tmp_path / "t.so"
    src.write_text(FREQ_CPP)
    csrc = os.path.join(os.path.dirname(m3.LIB_PATH), "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", csrc, str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.table.argtypes = [ctypes.c_double, ctypes.c_int, ctypes.c_void_p]
    for base in (0.5, 1.0, 100.0, 1e4, 5e5, 1e6):
        f = (ctypes.c_double * 128)()
        lib.table(base, rot, f)
        with localcontext() as c:
            c.prec = 60
            two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
            for j in range(rot // 2):
                y = Decimal(2 * j) / Decimal(rot) * Decimal(base).ln()
                want = (-y).exp() / two_pi
                err = abs(Decimal(f[j]) - want) / want * 2 ** 53
                assert err <= 7 + abs(y), (base, rot, j, float(err))


GRID_CPP = """
#include "attn.h"
extern "C" long long workgroups(int Tq, int S, int Hq, int Hk) { return m3::attn_query_workgroups(Tq, S, Hq, Hk); }
extern "C" int ranked(int seqs) { return seqs ? m3::kRankedSeqs : m3::kRankedWorkgroups; }
"""


def test_attention_cases_reach_both_orders_of_work(tmp_path):
    """Tiles of queries are taken by work up to a number of workgroups and by a
    search beyond: the GPU tests have several sequences on both sides."""
    import subprocess
    from tests import test_gpu_attn as t
    src, out = tmp_path / "t.cpp", tmp_path / "t.so"
    src.write_text(GRID_CPP)
    csrc = os.path.join(os.path.dirname(m3.LIB_PATH), "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", csrc, "-I",
                    "/opt/rocm/include", str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.workgroups.restype = ctypes.c_longlong
    assert lib.workgroups(16384, 5, 32, 8) == (16384 // 32 + 5) * 8 and lib.workgroups(1, 1, 3, 1) == 3
    seqs, most = lib.ranked(1), lib.ranked(0)
    for Hk in t.MANY_HEADS[1]:
        assert 1 < len(t.MANY_Q) <= seqs
        assert lib.workgroups(sum(t.MANY_Q) + 3, len(t.MANY_Q), t.MANY_HEADS[0], Hk) > most
    by_work = [c for c in t.CASES if 1 < len(c[0]) <= seqs and max(c[0]) > 128 and
               lib.workgroups(sum(c[0]) + 3, len(c[0]), c[2], c[3]) <= most]
    assert len(by_work) >= 3
