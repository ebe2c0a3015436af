"""Layer norm at its edges: rows without spread at eps = 0, rows too wide for the
ring, loud channels and large means, and what lies around its results."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import _lib, feedforward
import test_gpu_layer_norm as L

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


# Rows too wide for the ring and not for registers (more than 16384 columns in
# 16 bits, 13312 in FP32), the last piece of a thread partly or wholly past the row.
WIDE = [(torch.bfloat16, 3, 16640), (torch.bfloat16, 5, 24704), (torch.float16, 6, 20480), (torch.float16, 1, 32768),
        (torch.bfloat16, 2, 16392), (torch.float32, 3, 13440), (torch.float32, 5, 14976), (torch.float32, 2, 16384),
        (torch.float32, 3, 13316)]


@pytest.mark.parametrize("out_format", ["same", "fp8"])
@pytest.mark.parametrize("dtype,rows,cols", WIDE)
def test_wide_rows(dtype, rows, cols, out_format):
    if out_format == "fp8" and cols % 128:
        pytest.skip("8-bit results have whole groups")
    x, w, b, _ = L._inputs(rows, cols, dtype, rows + cols)
    L._check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=L.EPS, out_format=out_format), x, w, b)
    L._check_forward(dg.layer_norm(x.cuda(), w.cuda(), eps=L.EPS, out_format=out_format), x, w, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (40, 9), (300, 255), (300, 2047), (60, 4414), (20, 7167), (9, 7168), (2, 70001)])
@pytest.mark.parametrize("at", [0, 1, 2, 5, 8])
def test_nothing_around_the_results_is_written(dtype, rows, cols, at):
    """y and dx at every kind of offset inside a larger buffer, mean and rstd
    and the column sums likewise: what lies around them stays, bit for bit."""
    x, w, b, dy = L._inputs(rows, cols, dtype, rows + cols + at)
    xd, wd, bd, dyd = x.cuda(), w.cuda(), b.cuda(), dy.cuda()
    lib, code = _lib.lib(), feedforward._DTYPES[dtype]
    room = 16

    def guarded(n, kind, skip):
        big = torch.full((room + skip + n + room,), 7.0, dtype=kind, device="cuda")
        return big, big[room + skip:room + skip + n]

    def intact(big, part, skip):
        return bool((big[:room + skip] == 7).all()) and bool((big[room + skip + part.numel():] == 7).all())

    stream = torch.cuda.current_stream().cuda_stream
    y, mean, rstd = guarded(rows * cols, dtype, at), guarded(rows, torch.float32, at), guarded(rows, torch.float32, at)
    assert lib.dg_layer_norm(xd.data_ptr(), code, wd.data_ptr(), bd.data_ptr(), 0, y[1].data_ptr(), None,
                             mean[1].data_ptr(), rstd[1].data_ptr(), rows, cols, cols, L.EPS, stream) == 0
    r = dg.LayerNormOutput(y[1].view(rows, cols), None, mean[1], rstd[1])
    L._check_forward(r, x, w, b)
    dx, dw, db = guarded(rows * cols, dtype, at), guarded(cols, torch.float32, at), guarded(cols, torch.float32, at)
    need = feedforward._backward_workspace(cols, dg.get_num_sms())
    ws = torch.full((need // 4 + 2 * room,), 7.0, device="cuda")
    assert lib.dg_layer_norm_backward(dyd.data_ptr(), xd.data_ptr(), code, wd.data_ptr(), 0, mean[1].data_ptr(),
                                      rstd[1].data_ptr(), dx[1].data_ptr(), dw[1].data_ptr(), db[1].data_ptr(),
                                      ws[room:].data_ptr(), need, rows, cols, cols, cols, stream) == 0
    L._check_backward((dx[1].view(rows, cols), dw[1], db[1]), x, w, dy, r)
    for big, part in (y, mean, rstd, dx, dw, db):
        assert intact(big, part, at)
    assert bool((ws[:room] == 7).all()) and bool((ws[room + need // 4:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [40, 256, 1001, 2048, 7168, 16384])
def test_one_loud_channel(dtype, cols):
    """A value a thousand to a million times the others, wherever it lies: the
    others keep their digits (the bound is that of any row)."""
    at = [c for c in (0, 1, 2, 3, 5, 8, 15, 16, 31, 33, 64, 200, 511, 1000, 2047, 7000) if c < cols]
    x, w, b, _ = L._inputs(len(at) * 3, cols, torch.float32, cols, mean=0.0)
    for i, c in enumerate(at):
        for j, loud in enumerate((1e3, -3e4, 1e6)):
            x[3 * i + j, c] = loud
    x = x.to(dtype)
    L._check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=L.EPS), x, w, b)


@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5, 33, 65, 66, 67, 96, 130, 513, 1025, 2049, 4100, 7169])
def test_a_large_mean_at_any_width(cols):
    """Rows whose mean is 2^12 times their spread, also where a warp's first
    values are partly past the row's end."""
    x, w, b, _ = L._inputs(9, cols, torch.float32, cols, mean=0.0)
    x += 4096.0 * torch.arange(1, 10)[:, None]
    L._check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=L.EPS), x, w, b)
