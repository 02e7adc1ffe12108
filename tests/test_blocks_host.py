"""Host-only checks of the norms around a block: what the calls refuse, before anything is launched, and the
64-bit reference that the GPU tests use."""
import ctypes
import re
import os

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import block_ref

OK, NULL, SHAPE, DTYPE, UNSUP, ALIGN, WS = range(7)
P16 = ctypes.c_void_p(4096)     # aligned, never dereferenced
P_MIS = ctypes.c_void_p(4104)
BIG = 1 << 50
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _dims(**kw):
    base = dict(tokens=10, width=64, dtype=m3.M3_BF16, flags=0, eps=1e-6, ld_x=0, ld_y=0, ld_gate=0)
    base.update(kw)
    return m3.m3_block_dims(*base.values())


def _call(fn, d, names, required, over, ws):
    a = [over.get(n, P16 if n in required else None) for n in names]
    if ws:
        a += [over.get("ws", P16), over.get("ws_bytes", BIG)]
    return getattr(m3.library(), fn)(None if d is None else ctypes.byref(d), *a, None)


def _fwd(d, **o):
    return _call("m3_block_norm", d, ("x", "y", "gate", "wy", "sc", "wn", "h", "n"), ("x", "y", "h"), o, False)


BWD = ("x", "y", "gate", "wy", "sc", "wn", "dh", "dn", "dx", "dy", "dgate", "dwy", "dsc", "dwn")


def _bwd(d, **o):
    return _call("m3_block_norm_backward", d, BWD, ("x", "y", "dh", "dn", "dx", "dy"), o, True)


def test_header_declares_and_the_library_exports():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "m3ssm.h")).read(), flags=re.S)
    for n in ("m3_block_norm", "m3_block_norm_backward", "m3_block_norm_backward_workspace_size"):
        assert re.search(r"\b" + n + r"\s*\(", src) and hasattr(m3.library(), n), n
    assert ctypes.sizeof(m3.m3_block_dims) == 48 and m3.m3_block_dims.ld_x.offset == 24


def test_refusals():
    for call in (_fwd, _bwd):
        assert call(None) == NULL
        for bad in (dict(tokens=0), dict(tokens=-1), dict(tokens=0x7fffffff), dict(width=0), dict(eps=-1.0),
                    dict(eps=float("nan")), dict(eps=float("inf")), dict(flags=8), dict(flags=3), dict(ld_x=63),
                    dict(ld_y=-64), dict(ld_gate=1)):
            assert call(_dims(**bad)) == SHAPE, bad
        assert call(_dims(dtype=2)) == DTYPE
        assert call(_dims(width=16385)) == UNSUP
        for n in ("x", "y"):
            assert call(_dims(), **{n: None}) == NULL
        for n in ("x", "y", "gate", "wy", "sc", "wn"):
            assert call(_dims(), **{"dgate": P16, n: P_MIS}) == ALIGN
    assert _fwd(_dims(), h=None) == NULL
    assert _fwd(_dims(), n=P_MIS) == ALIGN
    for n in ("dx", "dy"):
        assert _bwd(_dims(), **{n: None}) == NULL
    assert _bwd(_dims(), dh=None, dn=None) == NULL
    assert _bwd(_dims(), gate=P16) == NULL            # a gate without room for its gradient
    for n in ("dh", "dn", "dx", "dy", "dwy", "dsc", "dwn", "ws"):
        assert _bwd(_dims(), **{n: P_MIS}) == ALIGN
    assert _bwd(_dims(), ws=None) == WS
    size = m3.library().m3_block_norm_backward_workspace_size
    need = size(ctypes.byref(_dims()))
    assert need > 0 and _bwd(_dims(), ws_bytes=need - 1) == WS
    assert size(ctypes.byref(_dims(width=0))) == 0 and size(None) == 0


def test_workspace_holds_every_launch():
    """Two rows of the width for each workgroup: at least one a row up to 256 rows, never more than rows."""
    size = m3.library().m3_block_norm_backward_workspace_size
    for T in (1, 2, 255, 256, 4097, 1 << 20):
        for W in (1, 63, 64, 513, 1021, 4096, 8192, 8193, 16384):
            n = size(ctypes.byref(_dims(tokens=T, width=W)))
            assert n % (8 * W) == 0 and min(T, 256) <= n // (8 * W) <= T


def test_arguments_match_the_header():
    """The binding passes as many arguments as the header declares."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "m3ssm.h")).read(), flags=re.S)
    lib = m3.library()
    seen = 0
    for name, args in re.findall(r"\b(m3_\w+)\s*\(([^()]*)\)\s*;", src):
        fn = getattr(lib, name)
        if fn.argtypes is not None:
            assert len(fn.argtypes) == (0 if args.strip() == "void" else len(args.split(","))), name
            seen += 1
    assert seen > 20


@pytest.mark.parametrize("act", [None, "linear", "sigmoid", "silu"])
def test_reference_gradients_are_those_of_differences(act):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x, y, gate, w = n(3, 10), n(3, 10), n(3, 10), [n(10) for _ in range(3)]
    dh, dn = n(3, 10), n(3, 10)
    want = block_ref.check(x, y, None if act is None else gate, *w, 1e-6, act, False, torch.float32, dh, dn)

    def loss(t):
        f = block_ref.forward(t["x"], t["y"], t.get("gate"), t["y_weight"], t["scale"], t["n_weight"], 1e-6, act, False)
        return float((f["h"] * dh).sum() + (f["n"] * dn).sum())

    ins = dict(x=x, y=y, y_weight=w[0], scale=w[1], n_weight=w[2])
    if act is not None:
        ins["gate"] = gate
    for k, key in (("x", "dx"), ("y", "dy"), ("gate", "dgate"), ("y_weight", "dy_weight"), ("scale", "dscale"),
                   ("n_weight", "dn_weight")):
        if k not in ins:
            continue
        way = n(*ins[k].shape)
        e = 1e-6
        up, down = ({**ins, k: ins[k] + s * e * way} for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * e)
        assert abs(slope - float((want[key][0] * way).sum())) <= 1e-6 * (1 + abs(slope)), k
