"""The gated delta rule's outputs and gradients, each head of each sequence by its norm, against the recurrence in 64
bits: short and ragged batches, sequences in segments (several of them, dense ones, every size of a state), strong
gates."""
import ctypes
import math

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import delta_near
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _inputs(rows, hk, hv, dk, dv, dtype, seed, batch, same=0.0, slow=False):
    """same: how much of one direction all keys share; slow: decays that leave some of the start at the end."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    q, k = unit(n(rows, hk, dk)), unit((1 - same) * n(rows, hk, dk) + same * n(1, hk, dk) * math.sqrt(dk))
    v = n(rows, hv, dv)
    rate = torch.exp(torch.rand(hv, generator=g) * 5 - 5.5) * (0.02 if slow else 1.0)
    gt, beta = -rate * torch.nn.functional.softplus(n(rows, hv)), torch.sigmoid(n(rows, hv))
    ins = [t.to(dtype).cuda() for t in (q, k, v, gt, beta)]
    return ins, n(batch, hv, dk, dv).cuda(), n(rows, hv, dv).to(dtype).cuda(), n(batch, hv, dk, dv).cuda()


def _in_segments(dims, packed):
    lib = m3.library()
    slots = dims.seqlen // 64 + dims.batch if packed else dims.batch * -(-dims.seqlen // 64)
    return lib.m3_delta_scan_workspace_size(ctypes.byref(dims), packed) > 4 * (4096 + 320) * slots * dims.nheads_v


def _check(got, s, c, ins, h0, do, dhT, scale, dtype, worst):
    want = delta_near.check(*(t[c] for t in ins), h0[s], scale, dtype, do[c], dhT[s])
    for name, (w, tol) in want.items():
        e = delta_near.off(name, got[name][s] if name in ("hT", "dh0") else got[name][c], w, tol)
        worst[name] = max(worst.get(name, 0.0), e)
        assert e <= 1.0, (name, s, e)


def _run(lengths, hk, hv, dk, dv, dtype, segments, same=0.0, gates=None, slow=False):
    rows = sum(lengths)
    ins, h0, do, dhT = _inputs(rows, hk, hv, dk, dv, dtype, rows + dk + dv, len(lengths), same, slow)
    if gates is not None:
        gates(ins[3], ins[4])
    dims = m3.m3_delta_dims(len(lengths), rows, hk, hv, dk, dv, m3.dtype_code(dtype), 1.0, 0, 0, 0, 0, 0)
    assert _in_segments(dims, 1) == segments
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    cu = torch.tensor(off, dtype=torch.int32).cuda()
    o, hT, st = m3.delta_scan(*ins, h0=h0, cu_seqlens=cu, want_states=True)
    d = m3.delta_scan_backward(*ins, do, st, h0=h0, dhT=dhT, cu_seqlens=cu)
    got = dict(o=o, hT=hT, **{"d" + n: t for n, t in d.items()})
    worst = {}
    for s, n in enumerate(lengths):
        if n:
            _check(got, s, slice(off[s], off[s + 1]), ins, h0, do, dhT, dk ** -0.5, dtype, worst)
    say("  of their tolerance: " + ", ".join("%s %.2f" % p for p in worst.items()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", [
    ([1], 1, 1, 64, 64, 0.0), ([2, 1, 0, 3], 2, 2, 64, 128, 0.0), ([63, 64, 65], 1, 2, 128, 64, 0.0),
    ([0, 130, 1], 1, 3, 128, 128, 0.0), ([200], 2, 2, 64, 64, 0.3), ([17, 100, 0, 0, 33], 2, 4, 128, 64, 0.1),
    ([257], 1, 1, 128, 128, 0.5), ([129, 64], 3, 3, 64, 128, 0.0), ([70, 300], 1, 4, 64, 64, 0.0),
    ([70, 300], 1, 2, 64, 128, 0.0), ([5, 190], 2, 4, 128, 128, 0.0), ([5, 190], 2, 2, 128, 64, 0.2)])
def test_short_sequences(case, dtype):
    _run(*case[:5], dtype, False, case[5])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", [
    ([1900, 0, 70, 1700], 1, 2, 64, 64), ([1450], 1, 1, 128, 128), ([900, 1100], 1, 2, 128, 128), ([1700], 1, 1, 128, 64),
    ([20] * 5 + [0, 2300, 1, 64] + [33] * 3, 1, 1, 64, 128), ([1100, 1600], 1, 2, 64, 128), ([1300, 1500], 2, 2, 128, 64)])
def test_sequences_in_segments(case, dtype):
    _run(*case, dtype, True, slow=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_longer_sequence_whole(dtype):
    _run([20] * 5 + [0, 1600, 1, 64] + [33] * 3, 1, 1, 64, 128, dtype, False, slow=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 1500, 1, 1, 64, 128, True), (1, 1500, 1, 2, 128, 128, True),
                                   (3, 1100, 1, 1, 128, 64, False), (3, 1700, 1, 1, 128, 64, True)])
def test_dense_prompts(shape, dtype):
    """Whole and in segments."""
    B, T, hk, hv, dk, dv, segments = shape
    ins, h0, do, dhT = _inputs(B * T, hk, hv, dk, dv, dtype, T + dv, B, 0.0, True)
    dims = m3.m3_delta_dims(B, T, hk, hv, dk, dv, m3.dtype_code(dtype), 1.0, 0, 0, 0, 0, 0)
    assert _in_segments(dims, 0) == segments
    f = lambda t: t.unflatten(0, (B, T))
    o, hT, st = m3.delta_scan(*(f(t) for t in ins), h0=h0, want_states=True)
    d = m3.delta_scan_backward(*(f(t) for t in ins), f(do), st, h0=h0, dhT=dhT)
    got = dict(o=o.flatten(0, 1), hT=hT, **{"d" + n: t if n == "h0" else t.flatten(0, 1) for n, t in d.items()})
    worst = {}
    for s in range(B):
        _check(got, s, slice(s * T, (s + 1) * T), ins, h0, do, dhT, dk ** -0.5, dtype, worst)
    say("  of their tolerance: " + ", ".join("%s %.2f" % p for p in worst.items()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_strong_gates(dk, dv, dtype):
    """Decays of 0 (-inf and far below), no decay, no write, and writes of twice the miss."""
    def gates(g, b):
        g[5, 0], g[70, 0], g[100, 1] = -200.0, float("-inf"), -90.0
        g[110:120, 1], b[20:30, 0], b[60:66, 1], b[128, 0] = 0.0, 0.0, 2.0, 1.0
        g[64:100, 1] = -20.0
    _run([140], 1, 2, dk, dv, dtype, False, gates=gates)
