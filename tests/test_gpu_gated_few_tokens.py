"""The gated product of one to four tokens with 8-bit results, whose CTAs tell
one another their columns' maxima, where there is the least time between their
start and the first maximum sent."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [1, 2, 4])
@pytest.mark.parametrize("f,k", [(128, 128), (2048, 128), (2048, 512)])
def test_short_k_many_times(m, f, k):
    """One step over K, launches back to back: every one gives what the tiled
    kernel's 129-row call gives for the same tokens, code for code, up to sums
    that round the other way (K this short: none)."""
    g = torch.Generator().manual_seed(m + f + k)
    # small whole numbers: every sum is exact in any order
    x = torch.randint(-8, 9, (129, k), generator=g).float()
    w = torch.randint(-4, 5, (2 * f, k), generator=g).float() / 64
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    qw, sw = dg.quantize_fp8(w.cuda(), 128)
    want = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True)
    few, few_sf = dg.quantize_fp8(x[:m].contiguous().cuda(), 1)
    got = [dg.fp8_gated_gemm_nt(few, few_sf, qw, sw, out_format="fp8", checkpoint=True) for _ in range(50)]
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r.checkpoint.view(torch.uint8), want.checkpoint.view(torch.uint8)[:m])
        assert torch.equal(r.checkpoint_sf[:, :m], want.checkpoint_sf[:, :m])
        assert torch.equal(r.h.view(torch.uint8), want.h.view(torch.uint8)[:m])
        assert torch.equal(r.h_sf[:, :m], want.h_sf[:, :m])


@pytest.mark.parametrize("m", [1, 2, 3, 40, 200])
@pytest.mark.parametrize("f,sms", [(2048, 20), (256, 20), (2048, 128), (640, 1)])
def test_a_limit_of_the_sms_is_kept(m, f, sms, monkeypatch, capfd):
    """No form of the product launches more CTAs than the SMs it may use."""
    k = 512
    g = torch.Generator().manual_seed(m + f)
    x = torch.randint(-8, 9, (m, k), generator=g).float()
    w = torch.randint(-4, 5, (2 * f, k), generator=g).float() / 64
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    qw, sw = dg.quantize_fp8(w.cuda(), 128)
    want = dg.fp8_gated_gemm_nt(q, sf, qw, sw)
    monkeypatch.setenv("DG_PRINT_CONFIGS", "1")
    dg.set_num_sms(sms)
    try:
        for out_format in ("bf16", "fp8"):
            capfd.readouterr()
            got = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format=out_format)
            line, = [x for x in capfd.readouterr().err.splitlines() if "gated" in x]
            assert int(line.split("grid=")[1].split()[0]) <= sms, line
            if out_format == "bf16":
                assert torch.equal(got.h, want.h)  # whole numbers: exact in any order up to the activation
    finally:
        dg.set_num_sms(0)
    assert dg.get_device_error()[0] == 0
