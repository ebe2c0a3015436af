"""Calls on an explicit stream that is not the current one: their copies,
workspaces and results follow that stream's order, while the current stream is
busy with work that they must not wait for or be waited on by."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg

pytestmark = pytest.mark.gpu

BUSY = 20_000_000  # clock cycles, about 10 ms


def _bits(out):
    return [t.view(torch.uint8) for t in out if t is not None]


def test_quantising_a_strided_input():
    x = torch.randn(512, 300, device="cuda").t()  # [300, 512], columns innermost
    s = torch.cuda.Stream()
    for dtype in (torch.bfloat16, torch.float32):
        y = x.to(dtype)
        assert not y.is_contiguous()
        want = dg.quantize_fp8(y.contiguous(), 1)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)  # the current stream: a copy made there would come too late
        got = dg.quantize_fp8(y, 1, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_bits(got), _bits(want)))
        again = dg.quantize_fp8(y, 1, stream=s.cuda_stream)  # a raw handle
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_bits(again), _bits(want)))
