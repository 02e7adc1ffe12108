"""The norms around a block where a row holds what is not finite, for every way that rows are taken."""
import pytest
import torch

from linear_recurrent_sequence_mamba_amd import binding as m3

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [72, 1021, 4096, 5473, 8192, 9001, 12352, 16384])
def test_without_dn_the_stream_is_of_no_weight(W, dtype):
    """h only reaches n, so with dn = 0 no gradient depends on x, whatever it holds."""
    g = torch.Generator().manual_seed(W)
    n = lambda *s: torch.randn(*s, generator=g)
    x, y, gate, dh = (n(5, W).to(dtype).cuda() for _ in range(4))
    w = [(0.5 + torch.rand(W, generator=g)).cuda() for _ in range(3)]
    for raw in (0, m3.M3_BLOCK_RAW):
        kw = dict(gate=gate, y_weight=w[0], scale=w[1], n_weight=w[2], flags=m3.M3_GATE_SILU | raw)
        want = m3.block_norm_backward(torch.zeros_like(x), y, dh, None, **kw)
        assert torch.equal(want["x"], dh) and not want["n_weight"].any()
        x2 = x.clone()
        x2[0, W // 2], x2[1, 0], x2[3, W - 1] = float("inf"), float("nan"), float("-inf")
        got = m3.block_norm_backward(x2, y, dh, None, **kw)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, raw)
