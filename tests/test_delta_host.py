"""Host-only checks of the gated delta rule: what the calls refuse, before anything is launched, the sizes
of workspaces, and the 64-bit reference that the GPU tests use."""
import ctypes
import os
import re

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import delta_ref

OK, NULL, SHAPE, DTYPE, UNSUP, ALIGN, WS = range(7)
P16 = ctypes.c_void_p(4096)     # aligned, never dereferenced
P_MIS = ctypes.c_void_p(4104)
P_ODD = ctypes.c_void_p(4097)
P2 = ctypes.c_void_p(4098)
BIG = 1 << 50
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCAN = ("cu", "q", "k", "v", "g", "beta", "h0", "o", "hT", "states")
BACK = ("cu", "q", "k", "v", "g", "beta", "states", "d_o", "dhT", "dq", "dk", "dv", "dg", "dbeta", "dh0")
STEP = ("h", "q", "k", "v", "g", "beta", "o")


def _dims(**kw):
    base = dict(batch=2, seqlen=100, nheads_k=2, nheads_v=4, headdim_k=64, headdim_v=128, dtype=m3.M3_BF16,
                scale=0.125, ld_q=0, ld_k=0, ld_v=0, ld_g=0, ld_beta=0)
    base.update(kw)
    return m3.m3_delta_dims(*base.values())


def _call(fn, d, names, optional, over, ws=True):
    a = [over.get(n, None if n in optional else P16) for n in names]
    if ws:
        a += [over.get("ws", P16), over.get("ws_bytes", BIG)]
    return getattr(m3.library(), fn)(None if d is None else ctypes.byref(d), *a, None)


def _scan(d, **o):
    return _call("m3_delta_scan", d, SCAN, ("cu", "h0", "hT", "states"), o)


def _back(d, **o):
    return _call("m3_delta_scan_backward", d, BACK, ("cu", "dhT", "dh0"), o)


def _step(d, **o):
    return _call("m3_delta_step", d, STEP, (), o, False)


CALLS = ((_scan, SCAN, ("cu", "h0", "hT", "states")), (_back, BACK, ("cu", "dhT", "dh0")), (_step, STEP, ()))


def test_header_declares_and_the_library_exports():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "m3ssm.h")).read(), flags=re.S)
    for n in ("m3_delta_scan", "m3_delta_scan_workspace_size", "m3_delta_scan_backward",
              "m3_delta_scan_backward_workspace_size", "m3_delta_step"):
        assert re.search(r"\b" + n + r"\s*\(", src) and hasattr(m3.library(), n), n
    assert ctypes.sizeof(m3.m3_delta_dims) == 72 and m3.m3_delta_dims.ld_q.offset == 32
    assert re.search(r"#define M3_DELTA_CHUNK %d\b" % m3.M3_DELTA_CHUNK, src)
    expr = re.search(r"#define M3_DELTA_STATE_FLOATS\(dk, dv\) (.*)", src).group(1)
    for dk in (64, 128):
        for dv in (64, 128):
            assert eval(expr, {"dk": dk, "dv": dv}) == m3.m3_delta_state_floats(dk, dv)


@pytest.mark.parametrize("call,names,optional", CALLS)
def test_refusals(call, names, optional):
    assert call(None) == NULL
    bad = [dict(batch=0), dict(batch=-1), dict(batch=0x7fffffff), dict(nheads_k=0), dict(nheads_v=0), dict(nheads_v=3),
           dict(headdim_k=0), dict(headdim_v=-64), dict(scale=float("nan")), dict(scale=float("inf")), dict(ld_q=120),
           dict(ld_k=-128), dict(ld_v=504), dict(ld_g=3), dict(ld_beta=3), dict(ld_g=1 << 24), dict(ld_q=1 << 24),
           dict(nheads_k=1 << 18, nheads_v=1 << 18), dict(batch=1 << 30)]
    if call is not _step:
        bad += [dict(seqlen=0), dict(seqlen=-5), dict(seqlen=0x7fffffff), dict(seqlen=0x7fff0000, nheads_v=8),
                dict(batch=1 << 12, seqlen=1 << 16, nheads_v=4)]
    for b in bad:
        assert call(_dims(**b)) == SHAPE, b
    assert call(_dims(dtype=2)) == DTYPE
    for b in (dict(headdim_k=32), dict(headdim_k=96), dict(headdim_v=256), dict(headdim_v=1)):
        assert call(_dims(**b)) == UNSUP, b
    for b in (dict(ld_q=132), dict(ld_k=129), dict(ld_v=516)):
        assert call(_dims(**b)) == ALIGN, b
    for n in names:
        if n not in optional:
            assert call(_dims(), **{n: None}) == NULL, n
        if n == "cu":
            assert call(_dims(), cu=P2) == ALIGN
        elif n in ("g", "beta"):   # their elements' alignment
            assert call(_dims(), **{n: P_ODD}) == ALIGN
            assert call(_dims(dtype=m3.M3_F32), **{n: P2}) == ALIGN
        else:
            assert call(_dims(), **{n: P_MIS}) == ALIGN, n


def test_workspaces():
    """A call with less than its workspace is refused; sizes cover every chunk's matrix (scan) or state gradients
    (backward), and 0 stands for dims that no call takes."""
    lib = m3.library()
    for call, size in ((_scan, lib.m3_delta_scan_workspace_size), (_back, lib.m3_delta_scan_backward_workspace_size)):
        assert call(_dims(), ws=None) == WS
        assert call(_dims(), ws=P_MIS) == ALIGN
        for packed in (0, 1):
            need = size(ctypes.byref(_dims()), packed)
            over = {"cu": P16} if packed else {}
            assert need > 0 and call(_dims(), ws_bytes=need - 1, **over) == WS
            assert size(ctypes.byref(_dims(headdim_k=32)), packed) == 0 and size(None, packed) == 0
        for B in (1, 2, 7, 300):
            for T in (1, 63, 64, 65, 511, 512, 513, 5000, 16384, 100001):
                for hv in (1, 8, 32):
                    for packed in (0, 1):
                        slots = T // 64 + B if packed else B * -(-T // 64)
                        if slots * hv >= 1 << 22:
                            continue
                        dims = _dims(batch=B, seqlen=T, nheads_k=1, nheads_v=hv)
                        least = slots * hv * 4 * (4096 + 320 if call is _scan else (64 + 64) * 128)
                        # segments: states and maps of them, of which there are at most an eighth of the chunks
                        # and one for each sequence
                        most = least + (slots // 8 + B) * hv * (64 * (4 * 128 + 6 * 64) + 16)
                        assert least <= size(ctypes.byref(dims), packed) <= most, (B, T, hv, packed)


def test_reference_is_the_closed_form_of_one_and_two_tokens():
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    q, k, v, gt, b, h0 = n(2, 1, 4), n(2, 1, 4), n(2, 2, 3), -n(2, 2).abs(), n(2, 2).sigmoid(), n(2, 4, 3)
    o, hs, ms = delta_ref.scan(q, k, v, gt, b, h0, 0.5)
    S = h0
    for t in range(2):
        for h in range(2):
            M = torch.exp(gt[t, h]) * (torch.eye(4, dtype=torch.float64) - b[t, h] * torch.outer(k[t, 0], k[t, 0]))
            want = M @ S[h] + b[t, h] * torch.outer(k[t, 0], v[t, h])
            assert torch.allclose(hs[t + 1, h], want, rtol=1e-12, atol=1e-12)
            assert torch.allclose(o[t, h], 0.5 * q[t, 0] @ want, rtol=1e-12, atol=1e-12)
        S = hs[t + 1]
