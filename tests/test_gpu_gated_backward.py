"""The gated product's backward pass from its 8-bit checkpoint against the
formulas in FP64, and against central differences of the forward formula."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import _fp8ref as R

pytestmark = pytest.mark.gpu

# FP32 arithmetic against the exact result, relative to |dh u| (dg), |dh|
# (du) and |u| (h): the logistic function carries about 2^-21 (fast
# exponential, whose argument's rounding grows with |g|, and reciprocal), and
# 1 - s in act' loses digits for large g while its factor grows like g^3 in
# the tanh form.
SLACK = 2.0 ** -18


def _np(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy()


def _inputs(m, f, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    gu = torch.randn(m, 2 * f, generator=g) * torch.exp2(spread * torch.randn(m, 1, generator=g))
    dh = (torch.randn(m, f, generator=g) * 2.0 ** -8 * torch.exp2(torch.randn(m, 1, generator=g))).to(torch.bfloat16)
    q, sf = dg.quantize_fp8(gu.cuda(), 1)
    return dh, q, sf


def _check(r, dh, q, sf, live, activation, diff=False):
    m, f = dh.shape
    kept = R.row_values(_np(q), _np(sf))
    d = dh.double().numpy().copy()
    kept[~live] = 0
    d[~live] = 0
    g, u = kept[:, :f], kept[:, f:]
    if diff:  # act' by central differences, error about step^2 and 2^-52 / step
        step = 2.0 ** -13
        da = (R.act(g + step, activation) - R.act(g - step, activation)) / (2 * step)
    else:
        da = R.act_grad(g, activation)
    a = R.act(g, activation)
    value = np.concatenate([d * u * da, d * a], 1)
    grow = 1 + np.abs(g) ** 3
    slack = SLACK * np.concatenate([np.abs(d * u) * grow, np.abs(d) * np.abs(g) * (1 + np.abs(g))], 1)
    sh = SLACK * np.abs(u) * np.abs(g) * (1 + np.abs(g))
    if diff:
        slack[:, :f] += np.abs(d * u) * 2.0 ** -20
    R.check_codes(_np(r.q), np.repeat(R.unpack_rows(_np(r.sf), m, 2 * f), 128, 1), 1, value, slack, "rows")
    assert not R.unused_bytes(_np(r.sf), m, 2 * f // 128).any()
    m128 = (m + 127) // 128 * 128
    pad = lambda x: np.concatenate([x, np.zeros((m128 - m, x.shape[1]))])  # noqa: E731
    R.check_codes(_np(r.q_cols), R.col_scales(_np(r.sf_cols), m128, 2 * f), 0, pad(value), pad(slack), "columns")
    R.check_codes(_np(r.h_cols), R.col_scales(_np(r.h_sf_cols), m128, f), 0, pad(a * u), pad(sh), "h")
    for w, c in ((r.sf_cols, 2 * f), (r.h_sf_cols, f)):
        assert not R.unused_bytes(_np(w), c, m128 // 128).any()


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,f", [(1, 128), (77, 384), (128, 128), (200, 256), (641, 640)])
def test_against_the_formula(m, f, activation):
    dh, q, sf = _inputs(m, f, 10 * m + f)
    r = dg.fp8_gated_backward(dh.cuda(), q, sf, activation=activation)
    _check(r, dh, q, sf, np.ones(m, dtype=bool), activation)


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
def test_against_differences(activation):
    dh, q, sf = _inputs(150, 256, 3)
    r = dg.fp8_gated_backward(dh.cuda(), q, sf, activation=activation)
    _check(r, dh, q, sf, np.ones(150, dtype=bool), activation, diff=True)


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
def test_large_gates(activation):
    """Gates up to a few hundred: the exponential overflows or vanishes."""
    dh, q, sf = _inputs(130, 128, 8, spread=4.0)
    r = dg.fp8_gated_backward(dh.cuda(), q, sf, activation=activation)
    _check(r, dh, q, sf, np.ones(130, dtype=bool), activation)


def test_padding_rows_count_as_zero_whatever_they_hold():
    m, f = 512, 256
    dh, q, sf = _inputs(m, f, 4)
    index = torch.zeros(m, dtype=torch.int32)
    index[90:128] = -1
    index[128:256] = 1
    index[256:384] = -1  # a whole block
    index[500:] = -1
    dead = index < 0
    dh[dead] = float("nan")
    dh[300] = float("inf")
    q.view(torch.uint8)[dead.cuda()] = 0x7F
    sf[:, :m][:, dead.cuda()] = -1
    r = dg.fp8_gated_backward(dh.cuda(), q, sf, m_indices=index.cuda())
    _check(r, dh, q, sf, ~dead.numpy(), "silu")


def test_strided_dh_and_side_stream():
    m, f = 200, 256
    dh, q, sf = _inputs(m, f, 6)
    wide = torch.zeros(m, f + 12, dtype=torch.bfloat16, device="cuda")
    wide[:, 4:4 + f] = dh.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = dg.fp8_gated_backward(wide[:, 4:4 + f], q, sf, stream=s)
    s.synchronize()
    _check(r, dh, q, sf, np.ones(m, dtype=bool), "silu")


def test_no_rows():
    e = lambda *s, t=torch.float8_e4m3fn: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    r = dg.fp8_gated_backward(e(0, 128, t=torch.bfloat16), e(0, 256), e(1, 0, t=torch.int32))
    assert r.q.shape == (0, 256) and r.q_cols.shape == (0, 256) and r.h_cols.shape == (0, 128)


def test_same_bits_every_time():
    dh, q, sf = _inputs(700, 512, 5)
    a = dg.fp8_gated_backward(dh.cuda(), q, sf)
    for _ in range(3):
        b = dg.fp8_gated_backward(dh.cuda(), q, sf)
        assert all(np.array_equal(_np(x), _np(y)) for x, y in zip(a, b))


def test_refusals():
    dh, q, sf = _inputs(8, 256, 1)
    dh = dh.cuda()
    with pytest.raises(ValueError):
        dg.fp8_gated_backward(dh, q, sf, activation="relu")
    with pytest.raises(TypeError):
        dg.fp8_gated_backward(dh.float(), q, sf)
    with pytest.raises(ValueError):
        dg.fp8_gated_backward(dh[:, :128], q, sf)
    with pytest.raises(ValueError):
        dg.fp8_gated_backward(dh, q, sf[:, :4])
    with pytest.raises(ValueError):
        dg.fp8_gated_backward(dh.t().contiguous().t(), q, sf)
    with pytest.raises(ValueError):
        dg.fp8_gated_backward(dh, q, sf, m_indices=torch.zeros(9, dtype=torch.int32, device="cuda"))
    odd = torch.zeros(8, 257, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dg.DGError):  # row stride of 257 elements
        dg.fp8_gated_backward(odd[:, :256], q, sf)
    with pytest.raises(dg.DGError):  # F % 128
        q2, sf2 = dg.quantize_fp8(torch.zeros(8, 384, device="cuda"), 1)
        dg.fp8_gated_backward(dh[:, :192], q2, sf2)
