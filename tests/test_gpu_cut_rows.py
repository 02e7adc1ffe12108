"""Outputs written into columns of wider rows, through the library's own calls:
the bits of the dense call, and nothing else of the buffer touched."""
import ctypes

import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
MARK = -77.0


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ws(n):
    """A workspace full of NaN, with room behind it that must stay."""
    return torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")


def _wide(rows, width, dtype, before, behind):
    """Rows of `width` inside a buffer of marks: (buffer, the view, elements from
    row to row).  `before` and `behind` are columns, multiples of 8."""
    buf = torch.full((rows, before + (width + 7) // 8 * 8 + behind), MARK, dtype=dtype, device="cuda")
    return buf, buf[:, before:before + width], buf.shape[1]


def _same(buf, view, want, rows=slice(None)):
    """The view's rows have the bits wanted, all else is as it was."""
    assert torch.equal(view[rows], want.reshape(want.shape[0], -1)[rows])
    view[rows] = MARK
    assert (buf == MARK).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D,packed", [(1, 1, 64, False), (2, 300, 70, False), (3, 129, 1, False),
                                          (4, 700, 70, True), (3, 130, 200, True)])
def test_gated_gradients(B, T, D, packed, dtype):
    g = torch.Generator().manual_seed(T + D)
    rows = T if packed else B * T
    n = lambda *s: torch.randn(*s, generator=g)
    x, r, i, dy = (n(rows, D).to(dtype).cuda() for _ in range(4))
    decay, h0, dhT = n(D).cuda() - 4, n(B, D).cuda(), n(B, D).cuda()
    cu, live = None, slice(None)
    if packed:   # rows before and behind the sequences, one of them empty
        cut = [5, 5, T // 3, T - 9] if B == 3 else [5, 140, 140, 141, T - 9]
        cu, live = torch.tensor(cut, dtype=torch.int32).cuda(), slice(cut[0], cut[-1])
    shape = (T, D) if packed else (B, T, D)
    v = lambda t: t.view(shape)
    _, _, st = m3.gated_scan(v(x), v(r), v(i), decay, h0=h0, cu_seqlens=cu, want_states=True)
    want = m3.gated_scan_backward(v(x), v(r), v(i), decay, v(dy), st, h0=h0, dhT=dhT, cu_seqlens=cu)
    ld = (D + 7) // 8 * 8 + 24
    out = [_wide(rows, D, dtype, 8, 16) for _ in range(3)]
    d = m3.m3_gated_dims(B, T, D, m3.dtype_code(dtype), 8.0, 0, 0, 0, ld)
    assert all(o[2] == ld for o in out)
    lib = m3.library()
    size = lib.m3_gated_scan_backward_workspace_size(ctypes.byref(d), int(packed))
    ws, dd, dh = _ws(size), torch.empty(D, device="cuda"), torch.empty(B, D, device="cuda")
    assert lib.m3_gated_scan_backward(
        ctypes.byref(d), _p(cu), _p(x), _p(r), _p(i), _p(decay), _p(h0), _p(st), _p(dy), _p(dhT),
        *(_p(o[1]) for o in out), _p(dd), _p(dh), _p(ws), size, _stream()) == 0
    torch.cuda.synchronize()
    for (buf, view, _), k in zip(out, "xri"):
        _same(buf, view, want[k].reshape(rows, D), live)
    assert torch.equal(dd, want["decay"]) and torch.equal(dh, want["h0"]) and (ws[size:] == 255).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,half", [(1, 2, 1, 32, 32, False), (37, 5, 2, 64, 64, True),
                                                (600, 3, 3, 128, 18, True), (9, 2, 1, 256, 256, False)])
def test_qk_norm_gradients(T, Hq, Hk, D, rot, half, dtype):
    g = torch.Generator().manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    q, k, gq, gk = n(T, Hq, D), n(T, Hk, D), n(T, Hq, D), n(T, Hk, D)
    wq, wk = (torch.rand(D, generator=g).cuda() + 0.5 for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32).cuda() * 1000
    flags = m3.M3_ROPE_HALF if half else 0
    want = m3.qk_norm_rope_backward(q, k, pos, gq, gk, wq, wk, rotary_dim=rot, flags=flags)
    # one buffer, as the gradient of one projection: dq and dk beside each other
    wide = (Hq + Hk) * D + 24
    buf = torch.full((T, wide), MARK, dtype=dtype, device="cuda")
    dq, dk = buf[:, 8:8 + Hq * D], buf[:, 16 + Hq * D:16 + (Hq + Hk) * D]
    d = m3.m3_qk_dims(T, Hq, Hk, D, rot, m3.dtype_code(dtype), flags, 1e-6, 1e4, 0, 0, wide, wide)
    lib = m3.library()
    size = lib.m3_qk_norm_rope_backward_workspace_size(ctypes.byref(d))
    ws, dwq, dwk = _ws(size), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    assert lib.m3_qk_norm_rope_backward(ctypes.byref(d), _p(q), _p(k), _p(wq), _p(wk), _p(pos), _p(gq), _p(gk),
                                        _p(dq), _p(dk), _p(dwq), _p(dwk), _p(ws), size, _stream()) == 0
    torch.cuda.synchronize()
    assert torch.equal(dq, want["q"].view(T, -1)) and torch.equal(dk, want["k"].view(T, -1))
    dq.fill_(MARK)
    dk.fill_(MARK)
    assert (buf == MARK).all() and (ws[size:] == 255).all()
    assert torch.equal(dwq, want["q_weight"]) and torch.equal(dwk, want["k_weight"])


PROMPTS = [  # queries and keys of each sequence, Hq, Hk, D; the second splits its keys
    ([150, 0, 31], [150, 4, 60], 4, 2, 64), ([2, 5], [3000, 2100], 4, 2, 128), ([130], [130], 5, 1, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", PROMPTS)
def test_attention_prompt_and_gradients(case, dtype):
    nq, nk, Hq, Hk, D = case
    tail = 2
    Tq, Tk = sum(nq) + tail, sum(nk) + tail
    g = torch.Generator().manual_seed(Tk)
    n = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    q, k, v = n(Tq, Hq, D), n(Tk, Hk, D), n(Tk, Hk, D)
    cq, ck = (torch.tensor([0] + t).cumsum(0).to(torch.int32).cuda() for t in (nq, nk))
    o, lse = m3.attn_prefill_varlen(q, k, v, cq, ck)
    buf, view, ld = _wide(Tq, Hq * D, dtype, 16, 40)
    d = m3.m3_attn_dims(len(nq), Tq, Tk, Hq, Hk, D, m3.dtype_code(dtype), D ** -0.5, 0, 0, 0, ld, 0, 0, 0)
    lib = m3.library()
    size = lib.m3_attn_prefill_varlen_workspace_size(ctypes.byref(d))
    assert (size > 16) == (max(nk) > 2500)
    ws, lse2 = _ws(size), torch.full((Tq, Hq), MARK, device="cuda")
    assert lib.m3_attn_prefill_varlen(ctypes.byref(d), _p(cq), _p(ck), _p(q), _p(k), _p(v), _p(view), _p(lse2),
                                      _p(ws), size, _stream()) == 0
    torch.cuda.synchronize()
    live = slice(0, Tq - tail)
    assert torch.equal(lse2[live], lse[live]) and (lse2[Tq - tail:] == MARK).all() and (ws[size:] == 255).all()
    _same(buf, view, o, live)
    # o and its gradient as columns of wider rows, of different widths
    do = n(Tq, Hq, D)
    want = m3.attn_prefill_varlen_backward(q, k, v, o, lse, do, cq, ck)
    cut = []
    for t, before, behind in ((o, 8, 0), (do, 24, 8)):
        w = torch.full((Tq, before + Hq * D + behind), float("nan"), dtype=dtype, device="cuda")
        w[:, before:before + Hq * D] = t.view(Tq, -1)
        cut.append(w[:, before:before + Hq * D].view(Tq, Hq, D))
    got = m3.attn_prefill_varlen_backward(q, k, v, cut[0], lse, cut[1], cq, ck)
    torch.cuda.synchronize()
    for a, b, rows in zip(got, want, (Tq, Tk, Tk)):
        assert torch.equal(a[:rows - tail], b[:rows - tail])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cap,Hq,Hk,D", [(70, 4, 2, 64), (1800, 6, 2, 128), (1100, 40, 1, 64)])
def test_attention_decode(cap, Hq, Hk, D, dtype):
    """o and the workspace are the caller's."""
    S = 3
    g = torch.Generator().manual_seed(cap)
    n = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    q, k, v = n(S, Hq, D), n(S, cap, Hk, D), n(S, cap, Hk, D)
    ln = torch.tensor([cap, 0, cap // 2 + 1], dtype=torch.int32).cuda()
    o, lse = m3.attn_decode(q, k, v, ln)
    d = m3.m3_attn_dims(S, 0, cap, Hq, Hk, D, m3.dtype_code(dtype), D ** -0.5, *[0] * 7)
    size = m3.library().m3_attn_decode_workspace_size(ctypes.byref(d))
    assert (size > 16) == (cap > 512)
    buf, view, _ = _wide(S, Hq * D, dtype, 8, 8)
    ws = _ws(size)
    for _ in range(2):   # the workspace of one call serves the next
        o2, lse2 = m3.attn_decode(q, k, v, ln, o=view.view(S, Hq, D), ws=ws[:size])
        torch.cuda.synchronize()
        assert o2.data_ptr() == view.data_ptr() and torch.equal(lse2, lse) and (ws[size:] == 255).all()
        _same(buf, view, o)
    if size > 16:
        with pytest.raises(m3.M3Error, match="WORKSPACE"):
            m3.attn_decode(q, k, v, ln, ws=ws[:size - 16])
