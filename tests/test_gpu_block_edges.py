"""The feed-forward block without tokens: empty results, and gradients of zero
(not what their memory held)."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import block

pytestmark = pytest.mark.gpu


def _dirty():
    """Memory handed out next is not zero."""
    junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]
    del junk


def test_no_tokens():
    d, f = 256, 384
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    net = block.GatedFeedForward(r(2 * f, d), r(d, f), r(d), r(d))
    x = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    y, saved = net.forward(x, training=True)
    assert y.shape == (0, d)
    _dirty()
    g = net.backward(x, saved)
    assert g.x.shape == (0, d) and g.up.shape == (2 * f, d) and g.down.shape == (d, f)
    assert not g.up.any() and not g.down.any() and not g.norm_weight.any() and not g.norm_bias.any()
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("rows", [0, 256])
def test_experts_without_tokens(rows):
    """No rows at all, or nothing but padding."""
    d, f, groups = 256, 128, 3
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    net = block.GatedExperts(r(groups, 2 * f, d), r(groups, d, f))
    q, sf = dg.quantize_fp8(r(rows, d), 1)
    index = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    dy = torch.full((rows, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    y, kept = net.forward(q, sf, index, training=True)
    assert y.shape == (rows, d)
    _dirty()
    ks = torch.tensor([0, rows, 0], dtype=torch.int32, device="cuda")
    dx, d_up, d_down = net.backward(dy, q, sf, kept, index, ks)
    assert dx.shape == (rows, d) and not d_up.any() and not d_down.any()
    masked = net.decode(torch.zeros(groups, 0, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                        torch.zeros(groups, 1, 0, dtype=torch.int32, device="cuda"),
                        torch.zeros(groups, dtype=torch.int32, device="cuda"))
    assert masked.shape == (groups, 0, d)
    assert dg.get_device_error()[0] == 0
