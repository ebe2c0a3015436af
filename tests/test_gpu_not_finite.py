"""Infinities and NaN in live rows: one rule for the scales wherever codes are
written.  The group's maximum passes over NaN, which becomes the code NaN; an
infinity gives the scale 2^127 and the code +-448."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import _fp8ref as R

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _np(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy()


def _rule(v):
    """Codes and scale bytes of float64 rows by the rule, groups of 128."""
    g = v.reshape(v.shape[0], -1, 128)
    a = np.where(np.isnan(g), 0, np.abs(g)).max(2)
    e = np.zeros(a.shape, dtype=int)
    for i in np.ndindex(a.shape):
        if a[i] == np.inf:
            e[i] = 127
        elif a[i] > 0:
            e[i] = next(k for k in range(-127, 128) if 448 * 2.0 ** k >= a[i])
    q = g / np.exp2(e.astype(float))[:, :, None]
    grid = R.TABLE[:127]
    at = np.searchsorted(grid, np.minimum(np.abs(q), 448))
    low, high = grid[np.maximum(at - 1, 0)], grid[np.minimum(at, 126)]
    mid = np.minimum(np.abs(q), 448)
    up = (high - mid < mid - low) | ((high - mid == mid - low) & (at % 2 == 0))
    code = np.where(up, at, np.maximum(at - 1, 0)).astype(np.uint8) | np.where(np.signbit(q), 0x80, 0).astype(np.uint8)
    code[np.isnan(q)] = 0x7F
    return code.reshape(v.shape), (e + 127).astype(np.uint8)


def _scale_bytes(words, rows, cols):
    b = np.ascontiguousarray(_np(words)).view(np.uint8).reshape(words.shape[0], words.shape[1], 4)
    return b.transpose(1, 0, 2).reshape(words.shape[1], -1)[:rows, :cols // 128]


def _check(q, words, value, what):
    code, byte = _rule(value)
    assert np.array_equal(_scale_bytes(words, *value.shape), byte), what + " scales"
    got = _np(q).copy()
    got[(got & 0x7F) == 0x7F] = 0x7F  # either NaN
    assert np.array_equal(got, code), what + " codes"


def test_save_follows_the_rule_of_the_fp32_quantiser():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 512, generator=g).to(torch.bfloat16)
    x[0, 5], x[1, 200], x[1, 201] = INF, -INF, 3e38
    x[2, 300], x[3, :128], x[4, :] = NAN, NAN, NAN
    x[5, 1], x[5, 2] = NAN, INF
    x[6, 7] = 3.3e38
    x[7, :128] = 0
    x[7, 3] = NAN
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    q32, sf32 = dg.quantize_fp8(x.float().cuda(), 1)
    assert np.array_equal(_np(q), _np(q32)) and torch.equal(sf, sf32)
    _check(q, sf, x.double().numpy(), "save")


@pytest.mark.parametrize("decode", ["1", "2", "0"])
@pytest.mark.parametrize("k", [128, 1024])
@pytest.mark.parametrize("m", [1, 2, 4, 5, 33, 129])
def test_gated_product(m, k, decode, monkeypatch):
    """Ones everywhere, so that g = u = K exactly and h = K^2; Wg's second
    block of rows has the scale 2^127 and overflows, two weights and a token are
    NaN.  Every kernel of the dense form."""
    monkeypatch.setenv("DG_DECODE", decode)
    f = 384
    one = lambda *s: torch.full(s, 0x38, dtype=torch.uint8)  # noqa: E731
    x, w = one(m, k), one(2 * f, k)
    w[5, 3] = 0x7F          # Wg
    w[f + 300, 0] = 0x7F    # Wu
    if m > 1:
        x[m - 1, 7] = 0x7F
    sf = torch.full(dg.sf_packed_shape(m, k), 0x7F7F7F7F, dtype=torch.int32)
    sw = torch.full(dg.sf_packed_shape(2 * f, k), 0x7F7F7F7F, dtype=torch.int32)
    sw[:, 128:256] = int(np.array([0xFEFEFEFE], dtype=np.uint32).view(np.int32)[0])
    if k == 128:
        sf[:, :] = 0x7F
        sw &= 0xFF
    sf[:, m:] = 0
    fp8 = lambda t: t.cuda().view(torch.float8_e4m3fn)  # noqa: E731
    r = dg.fp8_gated_gemm_nt(fp8(x), sf.cuda(), fp8(w), sw.cuda(), out_format="fp8", checkpoint=True)
    assert dg.get_device_error()[0] == 0
    gu = np.full((m, 2 * f), float(k))
    gu[:, 128:256] = INF    # K 2^127 is past FP32
    gu[:, 5] = gu[:, f + 300] = NAN
    if m > 1:
        gu[m - 1] = NAN
    h = gu[:, :f] * gu[:, f:]  # silu(K) is K to FP32's last bit
    _check(r.checkpoint, r.checkpoint_sf, gu, "checkpoint")
    _check(r.h, r.h_sf, h, "h")


def test_gated_product_contiguous_and_masked():
    m, k, f = 128, 256, 128
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-8, 9, (m, k), generator=g).float()
    w = torch.randint(-4, 5, (1, 2 * f, k), generator=g).float() / 64
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    qw, sw = dg.quantize_fp8(w.cuda(), 128)
    qw.view(torch.uint8)[0, 9, 0] = 0x7F
    q.view(torch.uint8)[77, 5] = 0x7F
    want = dg.fp8_gated_gemm_nt(q, sf, qw[0], sw[0], out_format="fp8", checkpoint=True)
    clean = dg.quantize_fp8(w.cuda(), 128)[0]
    fine = dg.fp8_gated_gemm_nt(q, sf, clean[0], sw[0], out_format="fp8", checkpoint=True)
    # one NaN among the weights: the other columns keep a scale of their own maximum
    v = R.codes_to_values(_np(fine.checkpoint)) * np.repeat(R.unpack_rows(_np(fine.checkpoint_sf), m, 2 * f), 128, 1)
    v[:, 9] = NAN
    got = R.codes_to_values(_np(want.checkpoint)) * np.repeat(R.unpack_rows(_np(want.checkpoint_sf), m, 2 * f), 128, 1)
    rows = np.arange(m) != 77
    keep = np.arange(2 * f) != 9
    assert np.isnan(got[rows][:, 9]).all() and np.isnan(got[77]).all()
    # the same scale except where column 9 held the group's maximum, then finer
    assert (np.abs(got - v)[rows][:, keep] <= np.abs(v)[rows][:, keep] * 2.0 ** -3 + 2.0 ** -9).all()
    index = torch.zeros(m, dtype=torch.int32).cuda()
    a = dg.m_grouped_fp8_gated_gemm_nt_contiguous(q, sf, qw, sw, index, out_format="fp8", checkpoint=True)
    b = dg.m_grouped_fp8_gated_gemm_nt_masked(q.view(torch.uint8).view(1, m, k).view(torch.float8_e4m3fn), sf.unsqueeze(0),
                                              qw, sw, torch.tensor([m], dtype=torch.int32).cuda(), out_format="fp8")
    assert np.array_equal(_np(a.h), _np(want.h)) and torch.equal(a.h_sf, want.h_sf)
    assert np.array_equal(_np(a.checkpoint), _np(want.checkpoint)) and torch.equal(a.checkpoint_sf, want.checkpoint_sf)
    assert np.array_equal(_np(b.h[0]), _np(want.h)) and torch.equal(b.h_sf[0], want.h_sf)


def test_gated_backward():
    """g = 0 and u = 1: dg = dh / 2 exactly, du = h = 0 but where dh is not finite (0 inf = NaN)."""
    m, f = 130, 128
    gu = torch.zeros(m, 2 * f)
    gu[:, f:] = 1
    q, sf = dg.quantize_fp8(gu.cuda(), 1)
    g = torch.Generator().manual_seed(4)
    dh = torch.randint(-30, 31, (m, f), generator=g).to(torch.bfloat16)
    dh[3, 10], dh[7, 20], dh[129, 1] = INF, NAN, -INF
    r = dg.fp8_gated_backward(dh.cuda(), q, sf)
    d = dh.double().numpy()
    value = np.concatenate([d / 2, d * 0.0], 1)
    _check(r.q, r.sf, value, "rows")
    pad = np.zeros((256, 2 * f))
    pad[:m] = value
    code, byte = _rule(np.ascontiguousarray(pad.T))
    assert np.array_equal(_scale_bytes(r.sf_cols, 2 * f, 256), byte)
    got = _np(r.q_cols).copy()
    got[(got & 0x7F) == 0x7F] = 0x7F
    assert np.array_equal(got & 0x7F, code.T & 0x7F)  # du's zeros have dh's sign
    assert not (_np(r.h_cols) & 0x7F).any()


def test_use():
    """Codes whose scale 2^127 stands for infinities, and NaN codes, in live rows."""
    codes = torch.full((256, 128), 0x38, dtype=torch.uint8)
    words = torch.full((1, 256), 0x7F, dtype=torch.int32)
    codes[3, 7] = 0x7F
    codes[200, :] = 0x7F
    words[0, 20] = 254
    codes[20, :] = 0
    codes[20, 9] = 0x7E
    q = codes.cuda().view(torch.float8_e4m3fn)
    qc, sfc = dg.requantize_fp8_cols(q, words.cuda())
    with np.errstate(over="ignore"):
        v = R.row_values(codes.numpy(), words.numpy()).astype(np.float32).astype(np.float64)
    assert np.isinf(v[20, 9])
    code, byte = _rule(np.ascontiguousarray(v.T))
    assert np.array_equal(_scale_bytes(sfc, 128, 256), byte)
    got = _np(qc).copy()
    got[(got & 0x7F) == 0x7F] = 0x7F
    assert np.array_equal(got, code.T)
