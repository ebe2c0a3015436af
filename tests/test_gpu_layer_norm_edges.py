"""Layer norm where its formula meets infinities: rows without spread at eps = 0."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [1, 37, 128, 2048, 2049, 7168, 20480, 70001])
def test_rows_without_spread_at_eps_0(cols, dtype):
    """rstd = 1 / sqrt(0) is infinite, whichever kernel the width takes; its neighbours are not touched."""
    x = torch.zeros(5, cols, dtype=dtype)
    x[1] = 2.0
    x[3, 0] = 1.0 if cols > 1 else 0.0
    r = dg.layer_norm(x.cuda(), torch.ones(cols, device="cuda"), eps=0.0)
    flat = [0, 1, 2, 4] + ([3] if cols == 1 else [])
    assert torch.isinf(r.rstd[flat]).all() and (r.rstd[flat] > 0).all()
    assert torch.equal(r.mean.cpu()[[0, 1, 2, 4]], torch.tensor([0.0, 2.0, 0.0, 0.0]))
    if cols > 1:
        var = (x[3].double() - x[3].double().mean()).square().mean()
        assert abs(float(r.rstd[3]) * float(var.sqrt()) - 1) < 2.0 ** -20
