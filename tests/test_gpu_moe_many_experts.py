"""The layer as models with 256 experts have it, at full width: many experts hit, mostly by a token or a few each."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import test_gpu_moe_few_tokens as M

pytestmark = pytest.mark.gpu
D, F, E, K = 7168, 2048, 256, 8


@pytest.fixture(scope="module")
def layer():
    """(up, up_sf, down, down_sf), 11.3 GB, and a router."""
    g = torch.Generator(device="cuda").manual_seed(0)
    out = None
    for e in range(E):
        up = torch.randn(1, 2 * F, D, generator=g, device="cuda") * D ** -0.5
        down = torch.randn(1, D, F, generator=g, device="cuda") * F ** -0.5
        one = dg.quantize_fp8(up, 128) + dg.quantize_fp8(down, 128)
        if out is None:
            out = [torch.empty((E,) + v.shape[1:], dtype=v.dtype, device="cuda") for v in one]
        for to, v in zip(out, one):
            raw = torch.uint8 if v.element_size() == 1 else v.dtype
            to.view(raw)[e] = v.view(raw)[0]
    return tuple(out), M.gate(E, D)


class OneByOne:
    """The weights' values in 64 bits, an expert's at a time."""

    def __init__(self, q, sf):
        self.q, self.sf, self.shape = q, sf, q.shape

    def __getitem__(self, e):
        return dg.dequantize_fp8(self.q[e:e + 1], self.sf[e:e + 1], torch.float32)[0].double()


@pytest.mark.parametrize("t", [1, 8, 16, 32, 64])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_experts_at_full_width(layer, monkeypatch, t, score):
    w, r = layer
    x, c = M.tokens(t, D), M.tokens(t, D, seed=5)
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3)).cuda() if score == "sigmoid" else None
    got = dg.fp8_moe_few_tokens(x, r, *w, K, router_bias=b, score=score, scale=2.5, c=c)
    monkeypatch.setattr(M, "values", OneByOne)
    M.check(got, M.reference(x, r, w, K, bias=b, score=score, scale=2.5, c=c))
    again = dg.fp8_moe_few_tokens(x, r, *w, K, router_bias=b, score=score, scale=2.5, c=c)
    assert torch.equal(got.y, again.y) and torch.equal(got.weights, again.weights)
