"""Sums of products of 8-bit integers that cancel, on each kernel's path."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import test_gpu_int8 as I

pytestmark = pytest.mark.gpu
# tokens and channels that reach the streaming kernel, the one with swapped roles (64 and 128 tokens), single tiles and
# pairs of CTAs
PATHS = [(3, 72), (20, 200), (64, 200), (300, 2000), (64, 10000), (2048, 2048)]


def cancelling(m, n, k):
    """a of one sign, b's second half the first's negative but for a few codes: sums of up to k 2^13 that leave little."""
    g = torch.Generator().manual_seed(m + n + k)
    a = torch.randint(100, 128, (m, 1), generator=g, dtype=torch.int32).expand(m, k)
    half = torch.randint(64, 128, (n, k // 2), generator=g, dtype=torch.int32)
    other = -half + torch.randint(-1, 2, (n, k // 2), generator=g, dtype=torch.int32)
    return a.to(torch.int8).cuda(), torch.cat([half, other], 1).clamp_(-128, 127).to(torch.int8).cuda()


@pytest.mark.parametrize("m,n", PATHS)
@pytest.mark.parametrize("k", [48, 512, 1024])
def test_short_sums_are_exact(m, n, k):
    """Up to 1024 columns no sum of some of the products is above 2^24, so FP32 holds each: the integer, rounded once."""
    for a, b in [cancelling(m, n, k), (I.codes(m, k), I.codes(n, k, 1))]:
        one = torch.ones(max(m, n), device="cuda")
        for dtype in (torch.bfloat16, torch.float16):
            # (FP16 ends at 65504; a power of two scales exactly)
            sa = one[:m] if dtype == torch.bfloat16 else one[:m] * 2.0 ** -9
            got = dg.int8_gemm_nt(a, sa, b, one[:n], out_dtype=dtype)
            want = (a.double() @ b.double().t() * float(sa[0])).to(dtype)
            assert torch.equal(got, want)
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("m,n", PATHS)
@pytest.mark.parametrize("k", [1040, 8192])
def test_long_sums_that_cancel(m, n, k):
    """Beyond, off by FP32's roundings of the partial sums: as far as the bound by the sum of magnitudes allows, however
    little is left of it."""
    a, b = cancelling(m, n, k)
    sa, sb = I.scales(m), I.scales(n, 1)
    I.check(dg.int8_gemm_nt(a, sa, b, sb), a, sa, b, sb)


@pytest.mark.parametrize("m,n", PATHS)
def test_scales_of_any_size(m, n):
    """A token's scale up to 2^96 and a channel's that undoes it: the sum times the first stays below 2^128."""
    k = 256
    a, b = I.codes(m, k), I.codes(n, k, 1)
    for power in (-120, -60, 60, 96):
        sa, sb = I.scales(m) * 2.0 ** power, I.scales(n, 1) * 2.0 ** -power
        I.check(dg.int8_gemm_nt(a, sa, b, sb), a, sa, b, sb)
