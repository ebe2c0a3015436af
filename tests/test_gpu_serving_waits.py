"""A layer of experts whose wait at the barrier over the grid runs out: the call ends, says where, and the next is right."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import test_gpu_moe_few_tokens as M

pytestmark = pytest.mark.gpu
DG_ERR_DEVICE_TIMEOUT, SITE_BARRIER = 5, 20


# 16 tokens: finishing warps take units by turns; 40: they share each. Of the first product there are at most 8 units, 4 MB
# of weights each, so that nearly all CTAs come to the barrier at once and wait there for more than the limit.
@pytest.mark.parametrize("t", [16, 40])
def test_the_barrier_gives_up(t):
    d, f, e, k = 65536, 128, 2, 2
    w, x, r = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d)
    call = lambda: dg.fp8_moe_few_tokens(x, r, *w, k).y  # noqa: E731
    want = call().clone()
    assert dg.get_device_error()[0] == 0
    for _ in range(3):
        dg.set_wait_timeout_ns(1)
        try:
            call()
            status, word = dg.get_device_error()
        finally:
            dg.set_wait_timeout_ns(2_000_000_000)
        assert status == DG_ERR_DEVICE_TIMEOUT and word >> 8 & 0xFFFF == SITE_BARRIER
        assert torch.equal(call(), want) and dg.get_device_error()[0] == 0
