"""The gated backward pass at gates whose square is past FP32: act' is 0 or 1
there to every digit, whatever the intermediate terms do."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import _fp8ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("power", [7, 12, 60, 62, 64, 70, 100, 118])
def test_derivative_of_large_gates(activation, power):
    """g = +-1.5 2^power from the checkpoint's scale, u = 1, dh small powers of
    two: dg = dh for positive g and 0 for negative, du = dh g or 0, exactly."""
    m, f = 130, 128
    codes = torch.full((m, 2 * f), 0x38, dtype=torch.uint8)  # 1
    codes[:, :f] = 0x3C                                      # 1.5
    codes[:, 1:f:2] = 0xBC                                   # -1.5
    words = torch.zeros(1, 132, 4, dtype=torch.uint8)
    words[0, :m, 0] = 127 + power
    words[0, :m, 1] = 127
    dh = torch.exp2(-torch.arange(m * f).reshape(m, f).remainder(5).float()).to(torch.bfloat16)
    r = dg.fp8_gated_backward(dh.cuda(), codes.cuda().view(torch.float8_e4m3fn), words.view(torch.int32).squeeze(-1).cuda(),
                              activation=activation)
    d = dh.double().numpy()
    up = np.arange(f) % 2 == 0
    want = np.concatenate([np.where(up, d, 0.0), np.where(up, d * 1.5 * 2.0 ** power, 0.0)], 1)
    got = R.row_values(r.q.view(torch.uint8).cpu().numpy(), r.sf.cpu().numpy())
    # dh 1.5 2^power has at most 2 significant bits, so its codes are exact
    assert np.array_equal(got, want)
    columns = R.codes_to_values(r.q_cols.view(torch.uint8).cpu().numpy()) * R.col_scales(r.sf_cols.cpu().numpy(), 256, 2 * f)
    assert np.array_equal(columns[:m], want) and not columns[m:].any()
