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


def _operators():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, w, b = r(256, 512).to(torch.bfloat16), r(512), r(512)
    n = dg.layer_norm(x, w, b, out_format="fp8")
    up, up_sf = dg.quantize_fp8(r(512, 512), 128)
    experts, experts_sf = dg.quantize_fp8(r(2, 512, 512), 128)
    h = dg.fp8_gated_gemm_nt(n.y, n.sf, up, up_sf, out_format="fp8", checkpoint=True)
    index = torch.tensor([0] * 128 + [1] * 128, dtype=torch.int32).cuda()
    counts = torch.tensor([128, 128], dtype=torch.int32).cuda()
    xm, xm_sf = dg.quantize_fp8(x.view(2, 128, 512), 1)
    dh = r(256, 256).to(torch.bfloat16)
    return {
        "save": lambda s: dg.quantize_fp8(x, 1, stream=s),
        "restore": lambda s: (dg.dequantize_fp8(n.y, n.sf, stream=s),),
        "use": lambda s: dg.requantize_fp8_cols(n.y, n.sf, stream=s),
        "gated": lambda s: dg.fp8_gated_gemm_nt(n.y, n.sf, up, up_sf, out_format="fp8", checkpoint=True, stream=s),
        "gated, contiguous": lambda s: dg.m_grouped_fp8_gated_gemm_nt_contiguous(n.y, n.sf, experts, experts_sf, index,
                                                                                 stream=s),
        "gated, masked": lambda s: dg.m_grouped_fp8_gated_gemm_nt_masked(xm, xm_sf, experts, experts_sf, counts, stream=s),
        "gated backward": lambda s: dg.fp8_gated_backward(dh, h.checkpoint, h.checkpoint_sf, stream=s),
        "layer norm": lambda s: dg.layer_norm(x, w, b, stream=s),
        "layer norm backward": lambda s: dg.layer_norm_backward(x, x, w, n.mean, n.rstd, stream=s),
    }


def test_results_are_not_in_memory_the_current_stream_still_writes():
    calls = _operators()
    s = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in _bits(call(None))]
        torch.cuda.synchronize()
        # released here, but written on the current stream only after its pause
        torch.cuda._sleep(BUSY)
        junk = [torch.empty_like(t).fill_(0x55) for t in want for _ in range(4)]
        del junk
        got = call(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_bits(got), want)), name


def test_results_released_early_are_not_handed_out_under_the_callers_stream():
    """A result read on the caller's stream and released while that read is still
    waiting: the call's stream does not get its memory back before."""
    s = torch.cuda.Stream()
    x = torch.randn(1024, 512, device="cuda").to(torch.bfloat16)
    w = torch.ones(512, device="cuda")
    want = dg.layer_norm(x, w).y.clone()
    torch.cuda.synchronize()
    r = dg.layer_norm(x, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    kept = r.y.clone()  # on the caller's stream, after the pause
    del r
    for _ in range(8):
        with torch.cuda.stream(s):
            torch.empty_like(x).fill_(7)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


@pytest.mark.parametrize("handle", [False, True])
def test_a_stream_of_the_current_device_by_object_or_handle(handle):
    calls = _operators()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for name, call in calls.items():
        got = _bits(call(s.cuda_stream if handle else s))
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, _bits(call(None)))), name
        assert all(torch.equal(a, b) for a, b in zip(_bits(call(0)), _bits(call(None)))), name  # the default stream


def test_the_products_on_an_explicit_stream():
    """New results and the binding's own workspace, while the current stream is busy."""
    g = torch.Generator().manual_seed(8)
    q, sf = dg.quantize_fp8(torch.randn(256, 512, generator=g).cuda(), 1)
    qb, sfb = dg.quantize_fp8(torch.randn(256, 512, generator=g).cuda(), 128)
    e, sfe = dg.quantize_fp8(torch.randn(2, 256, 512, generator=g).cuda(), 128)
    xm, sfm = dg.quantize_fp8(torch.randn(2, 128, 512, generator=g).cuda(), 1)
    index = torch.tensor([0] * 128 + [1] * 128, dtype=torch.int32).cuda()
    counts = torch.tensor([128, 128], dtype=torch.int32).cuda()
    xc, sfc = dg.quantize_fp8_cols(torch.randn(256, 128, generator=g).cuda())
    calls = {
        "dense": lambda s: dg.fp8_gemm_nt(q, sf, qb, sfb, stream=s),
        "contiguous": lambda s: dg.m_grouped_fp8_gemm_nt_contiguous(q, sf, e, sfe, index, stream=s),
        "masked": lambda s: dg.m_grouped_fp8_gemm_nt_masked(xm, sfm, e, sfe, counts, stream=s),
        "k-grouped": lambda s: dg.k_grouped_fp8_gemm_tn_contiguous(xc, sfc, xc, sfc, counts, stream=s),
    }
    s = torch.cuda.Stream()
    for name, call in calls.items():
        want = call(None).clone()
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        junk = [torch.empty_like(want).fill_(7) for _ in range(4)]
        del junk
        got = call(s)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name
    assert dg.get_device_error()[0] == 0
