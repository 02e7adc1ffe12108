"""Norms of queries and keys with the position rotation, and the gradients,
against the definition in 64 bits (complex rotations, differentiated)."""
import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3
from tests import layers_ref as ref
from tests.util import say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def _check(name, got, want, bound):
    w = ref.worst(got, want, bound)
    say(f"  {name}: {w:.3f} of its bound")
    assert w <= 1.0, (name, w)


def _inputs(T, Hq, Hk, D, dtype, seed, far, strided):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    if strided:
        p = n(T, (Hq + 2 * Hk) * D).to(dtype).cuda()
        q, k = p[:, :Hq * D].view(T, Hq, D), p[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    else:
        q, k = n(T, Hq, D).to(dtype).cuda(), n(T, Hk, D).to(dtype).cuda()
    wq, wk = (0.5 + torch.rand(D, generator=g)).cuda(), (0.5 + torch.rand(D, generator=g)).cuda()
    pos = torch.randint(-far, far, (T,), generator=g).int().cuda() if far else torch.arange(T).int().cuda()
    return q, k, wq, wk, pos, n(T, Hq, D).to(dtype).cuda(), n(T, Hk, D).to(dtype).cuda()


def _bound(u, rot, half, dtype):
    """A pair's length is off by 2^-20 of itself (norm: a sum of at most 256
    squares in 16 parts, a square root, a quotient; two products) and its
    direction by at most 2e-6 (a turn reduced in fp64 and rounded to fp32:
    2^-25 turns; the hardware sine and cosine 3e-7); then one rounding."""
    n, b = rot // 2, u.abs().clone()
    if n:
        x, y = (u[..., :n], u[..., n:rot]) if half else (u[..., 0:rot:2], u[..., 1:rot:2])
        l = torch.sqrt(x * x + y * y)
        b[..., :rot] = torch.cat([l, l], -1) if half else torch.stack([l, l], -1).flatten(-2)
    return (2.0 ** -20 + 2e-6) * b + ref.U[dtype] * u.abs() + 1e-30


CASES = [  # T, Hq, Hk, D, rot, half, far, strided
    (1, 1, 1, 32, 32, False, 0, False), (5, 3, 1, 64, 64, True, 0, True),
    (7, 8, 2, 128, 128, False, 1 << 30, True), (130, 5, 4, 64, 18, True, 100000, False),
    (33, 2, 2, 256, 64, True, 2147483647, True), (9, 1, 3, 128, 0, False, 0, False),
    (64, 7, 1, 32, 10, False, 1000000, True), (3000, 2, 1, 64, 32, True, 0, False),
    (5000, 1, 1, 128, 128, True, 50000, False)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", CASES)
def test_norm_rotation_and_gradients(case, dtype):
    T, Hq, Hk, D, rot, half, far, strided = case
    for weights in (True, False):
        say(f"qk {case} {dtype} weights={weights}")
        q, k, wq, wk, pos, gq, gk = _inputs(T, Hq, Hk, D, dtype, T + D, far, strided)
        if not weights:
            wq = wk = None
        kw = dict(q_weight=wq, k_weight=wk, eps=EPS, rotary_dim=rot, flags=m3.M3_ROPE_HALF if half else 0)
        qo, ko = m3.qk_norm_rope(q, k, pos, **kw)
        d = m3.qk_norm_rope_backward(q, k, pos, gq, gk, **kw)
        torch.cuda.synchronize()
        assert weights or (d["q_weight"] is None and d["k_weight"] is None)
        for n, v, w, o, g in (("q", q, wq, qo, gq), ("k", k, wk, ko, gk)):
            vv = ref.f64(v).requires_grad_(True)
            ww = (torch.ones(D, dtype=torch.float64) if w is None else ref.f64(w)).requires_grad_(True)
            u = ref.qk_one(vv, pos.cpu(), ww, EPS, 10000.0, rot, half)
            _check(n, o, u.detach(), _bound(u.detach(), rot, half, dtype))
            dv, dw = torch.autograd.grad(u, [vv, ww], ref.f64(g))
            # dv = inv (gw - u mean(gw u)): both terms off by the bound of a
            # rotated pair, the mean by that of a sum of D
            inv = 1 / torch.sqrt(vv.detach().pow(2).mean(-1, keepdim=True) + EPS)
            gw = ref.f64(g).abs().amax(-1, keepdim=True) * ww.detach().abs().max()
            un = vv.detach().abs() * inv
            b = inv * gw * (1 + un * un.mean(-1, keepdim=True)) * 2 * (2.0 ** -19 + 4e-6)
            _check("d" + n, d[n], dv, b + ref.U[dtype] * dv.abs() + 1e-30)
            if weights:
                terms = (ref.f64(g).abs().amax(-1, keepdim=True) * 1.5 * un).sum((0, 1))
                _check("dw" + n, d[n + "_weight"], dw, (2.0 ** -19 + 4e-6) * terms)


def test_in_place_and_equal_bits():
    q, k, wq, wk, pos, gq, gk = _inputs(300, 6, 2, 128, BF16, 1, 0, False)
    kw = dict(q_weight=wq, k_weight=wk, eps=EPS)
    qo, ko = m3.qk_norm_rope(q, k, pos, **kw)
    d = m3.qk_norm_rope_backward(q, k, pos, gq, gk, **kw)
    for _ in range(3):
        d2 = m3.qk_norm_rope_backward(q, k, pos, gq, gk, **kw)
        assert all(torch.equal(d[n], d2[n]) for n in d)
    import ctypes
    dims = m3.m3_qk_dims(300, 6, 2, 128, 128, m3.M3_BF16, 0, EPS, 10000.0, 0, 0, 0, 0)
    q2, k2 = q.clone(), k.clone()
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    assert m3.library().m3_qk_norm_rope(ctypes.byref(dims), p(q2), p(k2), p(wq), p(wk), p(pos), p(q2), p(k2),
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_rows_of_zeros_and_nan_stay_alone():
    q, k, wq, wk, pos, gq, gk = _inputs(20, 4, 4, 64, F32, 2, 0, False)
    qo, ko = m3.qk_norm_rope(q, k, pos, q_weight=wq, k_weight=wk)
    q2 = q.clone()
    q2[3, 1] = 0.0
    q2[4, 2, 5] = float("nan")
    qz, kz = m3.qk_norm_rope(q2, k, pos, q_weight=wq, k_weight=wk)
    assert (qz[3, 1] == 0).all() and torch.isnan(qz[4, 2]).all()
    keep = torch.ones(20, 4, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[4, 2] = False
    assert torch.equal(qz[keep], qo[keep]) and torch.equal(kz, ko)
    assert torch.isnan(m3.qk_norm_rope(q2, k, pos, eps=0.0)[0][3, 1]).all()


def test_gradient_against_differences():
    """The kernel's own gradients against central differences of its outputs."""
    q, k, wq, wk, pos, gq, gk = _inputs(2, 2, 1, 32, F32, 3, 0, False)
    kw = dict(q_weight=wq, k_weight=wk, rotary_dim=16, flags=m3.M3_ROPE_HALF)
    d = m3.qk_norm_rope_backward(q, k, pos, gq, gk, **kw)
    loss = lambda a: float((m3.qk_norm_rope(a, k, pos, **kw)[0].double() * gq.double()).sum())
    h = 2.0 ** -8   # truncation h^2 |f'''| / 6, rounding 2^-20 |loss terms| / h
    for e in range(0, q.numel(), 7):
        up, dn = q.clone(), q.clone()
        up.view(-1)[e] += h
        dn.view(-1)[e] -= h
        assert abs((loss(up) - loss(dn)) / (2 * h) - float(d["q"].view(-1)[e])) <= 4e-3


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("half", [False, True])
def test_far_positions_of_many_pairs(half, dtype):
    """All 128 pairs of the widest head, at positions up to the ends of an int."""
    test_norm_rotation_and_gradients((65, 2, 1, 256, 256, half, 2147483647, False), dtype)
