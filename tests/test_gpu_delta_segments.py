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
