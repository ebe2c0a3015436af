"""8-bit checkpoints on the GPU: saving from BF16, restoring, and the
requantisation over columns, bit for bit against the oracle's quantiser (the
arithmetic is exact: a power of two times the number, rounded once)."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import oracle
import _fp8ref as R

pytestmark = pytest.mark.gpu


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _spread(rows, cols, seed):
    """Activations whose channels and rows differ by powers of two, with zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(3 * torch.randn(1, cols, generator=g))
    x = x * torch.exp2(2 * torch.randn(rows, 1, generator=g))
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    return x


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 384), (130, 512), (77, 1152), (513, 640)])
def test_save_is_the_oracles_quantisation(rows, cols):
    x = _spread(rows, cols, 7 * rows + cols).to(torch.bfloat16)
    x[0, :128] = 0
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    oq, oe, _ = oracle.quantize(x.float().numpy(), 1)
    assert np.array_equal(_bytes(q), oq)
    assert np.array_equal(sf.cpu().numpy(), oracle.pack_ue8m0(oe, rows, 1))


def test_save_in_groups_and_into_given_tensors():
    x = torch.stack([_spread(5, 256, s) for s in range(3)]).to(torch.bfloat16)
    out = (torch.empty(3, 5, 256, dtype=torch.float8_e4m3fn, device="cuda"),
           torch.empty(dg.sf_packed_shape(5, 256, 3), dtype=torch.int32, device="cuda"))
    q, sf = dg.quantize_fp8(x.cuda(), 1, out=out)
    assert q.data_ptr() == out[0].data_ptr()
    for g in range(3):
        oq, oe, _ = oracle.quantize(x[g].float().numpy(), 1)
        assert np.array_equal(_bytes(q[g]), oq)
        assert np.array_equal(sf[g].cpu().numpy(), oracle.pack_ue8m0(oe, 5, 1))


def test_save_of_extreme_values():
    """Subnormals, the largest BF16 numbers and powers of two at the scale rule's edges."""
    v = torch.tensor([0.0, 2.0 ** -133, 2.0 ** -126, 3.3e38, -3.3e38, 448.0, 449.0, 2.0 ** -9 * 448, 1.75, 1.7578125])
    x = torch.zeros(len(v), 128)
    x[:, 5] = v
    x = x.to(torch.bfloat16)
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    oq, oe, _ = oracle.quantize(x.float().numpy(), 1)
    assert np.array_equal(_bytes(q), oq)
    assert np.array_equal(sf.cpu().numpy(), oracle.pack_ue8m0(oe, len(v), 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 640)])
def test_restore_gives_the_values_exactly(rows, cols, dtype):
    q, sf = dg.quantize_fp8(_spread(rows, cols, 3).cuda(), 1)
    x = dg.dequantize_fp8(q, sf, dtype=dtype)
    want = R.row_values(_bytes(q), sf.cpu().numpy())
    assert x.dtype == dtype and np.array_equal(x.double().cpu().numpy(), want)


@pytest.mark.parametrize("rows,cols", [(1, 128), (128, 256), (129, 384), (640, 128), (1000, 1152)])
def test_use_requantises_the_saved_values(rows, cols):
    q, sf = dg.quantize_fp8(_spread(rows, cols, rows).cuda(), 1)
    qc, sfc = dg.requantize_fp8_cols(q, sf)
    v = np.zeros(((rows + 127) // 128 * 128, cols), dtype=np.float32)
    v[:rows] = R.row_values(_bytes(q), sf.cpu().numpy())  # exact in FP32
    oq, oe, _ = oracle.quantize_cols(v)
    assert np.array_equal(_bytes(qc), oq)
    assert np.array_equal(sfc.cpu().numpy(), dg_pack_cols(oe, cols))


def dg_pack_cols(e, cols):
    """Exponents [blocks, cols] -> packed words [ceil(blocks/4), cols]."""
    blocks = e.shape[0]
    b = np.zeros(((blocks + 3) // 4 * 4, cols), dtype=np.uint8)
    b[:blocks] = (e + 127).astype(np.uint8)
    return np.ascontiguousarray(b.reshape(-1, 4, cols).transpose(0, 2, 1)).view(np.int32)[..., 0]


def test_use_over_a_wide_range_of_row_scales():
    """Rows whose scales lie up to 2^60 apart inside one block of 128: a
    column whose only non-zero entry is in a quiet row keeps its digits."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(256, 256, generator=g)
    x *= torch.exp2(torch.randint(-30, 31, (256, 1), generator=g).float())
    x[:, 3] = 0
    x[17, 3] = 2.0 ** -40
    x[:, 4] = 0
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    qc, sfc = dg.requantize_fp8_cols(q, sf)
    oq, oe, _ = oracle.quantize_cols(R.row_values(_bytes(q), sf.cpu().numpy()).astype(np.float32))
    assert np.array_equal(_bytes(qc), oq)
    assert np.array_equal(sfc.cpu().numpy(), dg_pack_cols(oe, 256))


def test_use_ignores_padding_rows_whatever_they_hold():
    rows, cols = 384, 256
    q, sf = dg.quantize_fp8(_spread(rows, cols, 9).cuda(), 1)
    index = torch.zeros(rows, dtype=torch.int32)
    index[100:128] = -1
    index[128:256] = -1
    index[300:] = -1
    q.view(torch.uint8)[index.cuda() < 0] = 0x7F  # NaN
    sf[:, :rows][:, index.cuda() < 0] = -1
    qc, sfc = dg.requantize_fp8_cols(q, sf, m_indices=index.cuda())
    live = index.numpy() >= 0
    v = np.zeros((rows, cols), dtype=np.float32)
    v[live] = R.row_values(_bytes(q), sf.cpu().numpy())[live]
    oq, oe, _ = oracle.quantize_cols(v)
    assert np.array_equal(_bytes(qc), oq)
    assert np.array_equal(sfc.cpu().numpy(), dg_pack_cols(oe, cols))


def test_use_feeds_the_weight_gradient_product():
    """dW = dY^T X with X from its checkpoint, on the K-grouped GEMM: the FP64
    product of the operands' values, within FP32 accumulation."""
    rows, m, n = 200, 128, 256
    g = torch.Generator().manual_seed(2)
    dy = torch.zeros(256, m)
    dy[:rows] = torch.randn(rows, m, generator=g)
    q, sf = dg.quantize_fp8(_spread(rows, n, 4).to(torch.bfloat16).cuda(), 1)
    qx, sx = dg.requantize_fp8_cols(q, sf)
    qd, sd = dg.quantize_fp8_cols(dy.cuda())
    d = dg.k_grouped_fp8_gemm_tn_contiguous(qd, sd, qx, sx, torch.tensor([256], dtype=torch.int32, device="cuda"))[0]
    a = R.codes_to_values(_bytes(qd)) * R.col_scales(sd.cpu().numpy(), 256, m)
    b = R.codes_to_values(_bytes(qx)) * R.col_scales(sx.cpu().numpy(), 256, n)
    err = np.abs(d.double().cpu().numpy() - a.T @ b)
    # 256 products summed in FP32: each of at most 256 partial sums rounded by 2^-23 of the sum of magnitudes
    assert (err <= 2.0 ** -15 * (np.abs(a).T @ np.abs(b))).all()


def test_on_a_side_stream():
    x = _spread(300, 512, 1).to(torch.bfloat16).cuda()
    want = dg.quantize_fp8(x, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, sf = dg.quantize_fp8(x, 1, stream=s)
    qc, sfc = dg.requantize_fp8_cols(q, sf, stream=s)
    s.synchronize()
    ref = dg.requantize_fp8_cols(*want)
    assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(sf, want[1])
    assert torch.equal(qc.view(torch.uint8), ref[0].view(torch.uint8)) and torch.equal(sfc, ref[1])


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        dg.quantize_fp8(x, 128)
    with pytest.raises(ValueError):
        dg.quantize_fp8(x, 1, packed=False)
    with pytest.raises(dg.DGError):
        dg.quantize_fp8(x[:, :100].contiguous(), 1)
    q, sf = dg.quantize_fp8(x, 1)
    with pytest.raises(ValueError):
        dg.requantize_fp8_cols(q, sf[:, :2])
    with pytest.raises(ValueError):
        dg.requantize_fp8_cols(q, sf, m_indices=torch.zeros(5, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        dg.requantize_fp8_cols(q, sf, m_indices=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        dg.dequantize_fp8(q, sf, dtype=torch.float16)
    with pytest.raises(ValueError):
        dg.requantize_fp8_cols(q.cpu(), sf)


@pytest.mark.parametrize("spread", [0, 4, 15, 16, 30])
def test_use_at_the_edges_of_exact_halves(spread):
    """Rows whose scales lie `spread` powers of two apart, and columns that hold
    nothing but the smallest codes (their scale is 2^17 below the rows')."""
    g = torch.Generator().manual_seed(spread)
    codes = torch.randint(0, 0x7F, (300, 256), generator=g, dtype=torch.uint8)
    codes |= torch.randint(0, 2, codes.shape, generator=g, dtype=torch.uint8) * 128
    codes[:, 5] = 1                     # 2^-9
    codes[:, 6] = 0
    codes[7, 6] = 0x83                  # one subnormal in an empty column
    codes[:, 9] = 0x7E                  # 448
    e = torch.randint(-20, -20 + spread + 1, (300, 2), generator=g)
    words = torch.zeros(1, 300, 4, dtype=torch.uint8)
    words[0, :, :2] = (e + 127).to(torch.uint8)
    sf = words.view(torch.int32).squeeze(-1)
    q = codes.cuda().view(torch.float8_e4m3fn)
    qc, sfc = dg.requantize_fp8_cols(q, sf.cuda())
    v = np.zeros((384, 256), dtype=np.float32)
    v[:300] = R.row_values(codes.numpy(), sf.numpy())
    oq, oe, _ = oracle.quantize_cols(v)
    assert np.array_equal(_bytes(qc), oq)
    assert np.array_equal(sfc.cpu().numpy(), dg_pack_cols(oe, 256))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(5, 640), (131, 1152)])
def test_restored_into_memory_on_16_bytes(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows)
    q, sf = dg.quantize_fp8(torch.randn(rows, cols, generator=g).to(torch.bfloat16).cuda(), 1)
    skip = 128 // torch.finfo(dtype).bits  # 16 bytes
    room = torch.full((skip + rows * cols + skip,), 7.0, dtype=dtype, device="cuda")
    out = room[skip:skip + rows * cols].view(rows, cols)
    assert out.data_ptr() % 32 == 16
    dg.dequantize_fp8(q, sf, dtype=dtype, out=out)
    assert torch.equal(out, dg.dequantize_fp8(q, sf, dtype=dtype))
    assert (room[:skip] == 7).all() and (room[-skip:] == 7).all()
