"""The gated feed-forward product (dense, contiguous, masked) against the
formula in FP64 on the operands' exact values."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import _fp8ref as R

pytestmark = pytest.mark.gpu

BF16_U = 2.0 ** -8     # half a unit in the last place of BF16, relative
ACT = 2.0 ** -18       # the activation's FP32 arithmetic, relative (its argument's rounding grows with |g|)


def _np(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy()


def _operands(rows, f, k, seed, groups=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randn(rows, 1, generator=g))
    w = torch.randn(*((groups,) if groups else ()), 2 * f, k, generator=g) * 1.5 * k ** -0.5
    q, sf = dg.quantize_fp8(x.cuda(), 1)
    qw, sw = dg.quantize_fp8(w.cuda(), 128)
    return q, sf, qw, sw


def _weights(qw, sw):
    """Exact values of the weights: the packed words hold one scale a row and K block."""
    if qw.dim() == 2:
        return R.row_values(_np(qw), _np(sw))
    return np.stack([R.row_values(_np(qw[i]), _np(sw[i])) for i in range(qw.shape[0])])


def _reference(x, w, activation):
    """h, [g | u] and how far FP32 accumulation may put each off: one rounding
    or truncation of the partial sum a 32-deep step, at most 2^-23 of the sum
    of magnitudes each, and as much again inside the step."""
    f = w.shape[0] // 2
    gu, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    s = mag * (w.shape[1] // 32) * 2.0 ** -22
    g, u = gu[:, :f], gu[:, f:]
    a = R.act(g, activation)
    h = a * u
    sh = 1.2 * s[:, :f] * np.abs(u) + (np.abs(a) + 1.2 * s[:, :f]) * s[:, f:] + ACT * np.abs(h) * (1 + np.abs(g)) \
        + ACT * np.abs(g * u) * 2.0 ** -6
    return h, gu, sh, s


def _check(out, x, w, activation, what="", h_rows=None):
    """h (and the checkpoint, where kept) of rows x; h_rows: those rows of the result."""
    h, gu, sh, s = _reference(x, w, activation)
    pick = slice(None) if h_rows is None else h_rows
    if out.h_sf is None:
        err = np.abs(out.h.float().double().cpu().numpy()[pick] - h)
        assert (err <= BF16_U * np.abs(h) + sh).all(), "%s: %.3g" % (what, (err - BF16_U * np.abs(h) - sh).max())
    else:
        rows, f = out.h.shape
        sc = np.repeat(R.unpack_rows(_np(out.h_sf), rows, f), 128, 1)[pick]
        R.check_codes(_np(out.h)[pick], sc, 1, h, sh, what + " h")
    if out.checkpoint is not None:
        rows, f2 = out.checkpoint.shape
        sc = np.repeat(R.unpack_rows(_np(out.checkpoint_sf), rows, f2), 128, 1)[pick]
        R.check_codes(_np(out.checkpoint)[pick], sc, 1, gu, s, what + " checkpoint")


DENSE = [(1, 128, 128), (1, 2048, 1152), (2, 8, 256), (5, 1000, 640), (33, 384, 512), (64, 256, 2048), (127, 128, 384),
         (128, 512, 1024), (129, 640, 256), (333, 136, 1536), (700, 1152, 768)]


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,f,k", DENSE)
def test_dense_bf16(m, f, k, activation):
    q, sf, qw, sw = _operands(m, f, k, m + f + k)
    out = dg.fp8_gated_gemm_nt(q, sf, qw, sw, activation=activation)
    assert out.h_sf is None and out.checkpoint is None
    _check(out, R.row_values(_np(q), _np(sf)), _weights(qw, sw), activation)
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("out_format,checkpoint", [("fp8", False), ("fp8", True), ("bf16", True)])
@pytest.mark.parametrize("m,f,k", [c for c in DENSE if c[1] % 128 == 0])
def test_dense_8_bit_results(m, f, k, out_format, checkpoint):
    q, sf, qw, sw = _operands(m, f, k, m + f + k + 1)
    out = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format=out_format, checkpoint=checkpoint)
    _check(out, R.row_values(_np(q), _np(sf)), _weights(qw, sw), "silu")
    for words, blocks in ((out.h_sf, f // 128), (out.checkpoint_sf, 2 * f // 128)):
        if words is not None:
            assert not R.unused_bytes(_np(words), m, blocks).any()
    assert dg.get_device_error()[0] == 0


def test_8_bit_result_is_the_next_products_operand():
    """The codes and scales go straight into fp8_gemm_nt."""
    m, f, k, n = 200, 256, 512, 128
    q, sf, qw, sw = _operands(m, f, k, 3)
    out = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8")
    wd, sd = dg.quantize_fp8(torch.randn(n, f, generator=torch.Generator().manual_seed(1)).cuda(), 128)
    y = dg.fp8_gemm_nt(out.h, out.h_sf, wd, sd).double().cpu().numpy()
    a, b = R.row_values(_np(out.h), _np(out.h_sf)), R.row_values(_np(wd), _np(sd))
    assert (np.abs(y - a @ b.T) <= BF16_U * np.abs(a @ b.T) + 2.0 ** -18 * (np.abs(a) @ np.abs(b).T)).all()


def test_strided_operands_and_given_results():
    m, f, k = 150, 256, 384
    q, sf, qw, sw = _operands(m, f, k, 4)
    aw = torch.zeros(m, k + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    aw[:, :k].copy_(q)
    bw = torch.zeros(2 * f, k + 32, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    bw[:, :k].copy_(qw)
    d = torch.full((m, f + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = dg.fp8_gated_gemm_nt(aw[:, :k], sf, bw[:, :k], sw, d=d[:, :f])
    assert out.h.data_ptr() == d.data_ptr() and bool((d[:, f:] == 7).all())
    _check(out, R.row_values(_np(q), _np(sf)), _weights(qw, sw), "silu")


def test_zero_rows_and_a_side_stream():
    q, sf, qw, sw = _operands(140, 128, 256, 5)
    q.view(torch.uint8)[3] = 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True, stream=s)
    s.synchronize()
    assert not _np(out.h)[3].any() and (R.unpack_rows(_np(out.h_sf), 140, 128)[3] == 1).all()
    _check(out, R.row_values(_np(q), _np(sf)), _weights(qw, sw), "silu")
    e = dg.fp8_gated_gemm_nt(q[:0], torch.empty(1, 0, dtype=torch.int32, device="cuda"), qw, sw)
    assert e.h.shape == (0, 128)


def _layout(counts):
    index, spans = [], []
    for g, c in enumerate(counts):
        spans.append((g, len(index), c))
        index += [g] * c + [-1] * (-c % 128)
    return torch.tensor(index, dtype=torch.int32), spans


def _prefilled(shape, kind):
    """A result whose untouched parts can be told: codes 0x55 / words 0x55555555 / BF16 of a given pattern."""
    if kind == "codes":
        return torch.full(shape, 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    if kind == "words":
        return torch.full(shape, 0x55555555, dtype=torch.int32, device="cuda")
    return torch.full(shape, 0x7F3C, dtype=torch.int16, device="cuda").view(torch.bfloat16)


@pytest.mark.parametrize("out_format,checkpoint", [("bf16", False), ("fp8", False), ("fp8", True)])
@pytest.mark.parametrize("counts,f,k", [([100, 28], 128, 256), ([1, 0, 300, 128], 384, 640), ([5], 256, 128),
                                        ([129, 1, 500], 512, 896)])
def test_contiguous(counts, f, k, out_format, checkpoint):
    index, spans = _layout(counts)
    m = len(index)
    q, sf, qw, sw = _operands(m, f, k, m + f + k, groups=len(counts))
    dead = (index < 0)
    q.view(torch.uint8)[dead.cuda()] = 0x7F  # NaN in the padding
    d = (_prefilled((m, f), "codes"), _prefilled(dg.sf_packed_shape(m, f), "words")) if out_format == "fp8" else \
        _prefilled((m, f), "bf16")
    kept = (_prefilled((m, 2 * f), "codes"), _prefilled(dg.sf_packed_shape(m, 2 * f), "words")) if checkpoint else False
    out = dg.m_grouped_fp8_gated_gemm_nt_contiguous(q, sf, qw, sw, index.cuda(), d=d, out_format=out_format,
                                                    checkpoint=kept)
    x, w = R.row_values(_np(q), _np(sf)), _weights(qw, sw)
    for g, row, c in spans:
        if c:
            rows = np.arange(row, row + c)
            _check(out, x[rows], w[g], "silu", "expert %d" % g, rows)
    dn = dead.numpy()
    if out_format == "fp8":
        assert (_np(out.h)[dn] == 0x55).all() and (_np(out.h_sf)[:, dn] == 0x55555555).all()
    else:
        assert (out.h.view(torch.int16).cpu().numpy()[dn] == 0x7F3C).all()
    if checkpoint:
        assert (_np(out.checkpoint)[dn] == 0x55).all() and (_np(out.checkpoint_sf)[:, dn] == 0x55555555).all()
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("out_format", ["bf16", "fp8"])
@pytest.mark.parametrize("counts,cap,f,k", [([77, 0], 128, 256, 256), ([1, 5, 9], 9, 128, 384), ([200, 256, 0, 129], 256, 384, 512),
                                            ([1], 1, 640, 1280)])
def test_masked(counts, cap, f, k, out_format):
    g = len(counts)
    ops = [_operands(cap, f, k, 7 * i + cap + f) for i in range(g)]
    q, qw = (torch.stack([o[i].view(torch.uint8) for o in ops]).view(torch.float8_e4m3fn) for i in (0, 2))
    sf, sw = (torch.stack([o[i] for o in ops]) for i in (1, 3))
    d = (_prefilled((g, cap, f), "codes"), _prefilled(dg.sf_packed_shape(cap, f, g), "words")) \
        if out_format == "fp8" else _prefilled((g, cap, f), "bf16")
    out = dg.m_grouped_fp8_gated_gemm_nt_masked(q, sf, qw, sw, torch.tensor(counts, dtype=torch.int32, device="cuda"),
                                                d=d, out_format=out_format, expected_m=max(1, sum(counts) // g))
    for i, c in enumerate(counts):
        one = dg.GatedOutput(out.h[i], None if out.h_sf is None else out.h_sf[i], None, None)
        if c:
            _check(one, R.row_values(_np(q[i]), _np(sf[i]))[:c], R.row_values(_np(qw[i]), _np(sw[i])), "silu",
                   "expert %d" % i, np.arange(c))
        if out_format == "fp8":
            assert (_np(one.h)[c:] == 0x55).all() and (_np(one.h_sf)[:, c:] == 0x55555555).all()
        else:
            assert (one.h.view(torch.int16).cpu().numpy()[c:] == 0x7F3C).all()
    assert dg.get_device_error()[0] == 0


def test_bad_counts_and_indices_are_reported():
    q, sf, qw, sw = _operands(128, 128, 128, 1, groups=2)
    index = torch.zeros(128, dtype=torch.int32)
    index[64:] = 1  # a second expert inside a block of 128 rows
    d = _prefilled((128, 128), "bf16")
    out = dg.m_grouped_fp8_gated_gemm_nt_contiguous(q, sf, qw, sw, index.cuda(), d=d)
    assert dg.get_device_error()[0] == 6
    assert (out.h.view(torch.int16).cpu().numpy()[64:] == 0x7F3C).all()
    qm, sm = q.view(torch.uint8).reshape(1, 128, 128).view(torch.float8_e4m3fn), sf.reshape(1, 1, 128)
    dg.m_grouped_fp8_gated_gemm_nt_masked(qm, sm, qw[:1], sw[:1], torch.tensor([200], dtype=torch.int32, device="cuda"))
    assert dg.get_device_error()[0] == 6
    assert dg.get_device_error()[0] == 0


def test_same_bits_every_time():
    q, sf, qw, sw = _operands(300, 512, 1024, 6)
    a = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True)
    for _ in range(3):
        b = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True)
        assert all(np.array_equal(_np(x), _np(y)) for x, y in zip(a, b))


def test_in_a_graph_with_programmatic_launch():
    q, sf, qw, sw = _operands(40, 256, 512, 2)
    want = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8")
    d = (torch.empty_like(want.h), torch.empty_like(want.h_sf))
    dg.set_pdl(True)
    try:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            dg.fp8_gated_gemm_nt(q, sf, qw, sw, d=d, out_format="fp8")
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dg.fp8_gated_gemm_nt(q, sf, qw, sw, d=d, out_format="fp8")
            dg.fp8_gated_gemm_nt(q, sf, qw, sw, d=d, out_format="fp8")
        d[0].view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
    finally:
        dg.set_pdl(False)
    assert np.array_equal(_np(d[0]), _np(want.h)) and np.array_equal(_np(d[1]), _np(want.h_sf))


def test_a_load_that_never_lands_ends_the_launch_by_itself():
    q, sf, qw, sw = _operands(256, 256, 512, 9)
    want = dg.fp8_gated_gemm_nt(q, sf, qw, sw)
    torch.cuda.synchronize()
    dg.set_wait_timeout_ns(20_000_000)
    dg.debug_set_drop_load(2)
    try:
        dg.fp8_gated_gemm_nt(q, sf, qw, sw)
        assert dg.get_device_error()[0] == 5
    finally:
        dg.debug_set_drop_load(0)
        dg.set_wait_timeout_ns(2_000_000_000)
    again = dg.fp8_gated_gemm_nt(q, sf, qw, sw)
    assert dg.get_device_error()[0] == 0 and torch.equal(again.h, want.h)


def test_refusals():
    q, sf, qw, sw = _operands(8, 136, 256, 1)
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8")   # F = 136 has no whole groups
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf, qw, sw, checkpoint=True)
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf, qw, sw, activation="tanh")
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp16")
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf, qw[:, :128], sw)
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf[:, :4], qw, sw)
    with pytest.raises(TypeError):
        dg.fp8_gated_gemm_nt(q.float(), sf, qw, sw)
    with pytest.raises(ValueError):
        dg.fp8_gated_gemm_nt(q, sf, qw, sw, d=torch.empty(8, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dg.DGError):                              # F % 8
        qo, so = dg.quantize_fp8(torch.zeros(20, 256, device="cuda"), 128)
        dg.fp8_gated_gemm_nt(q, sf, qo, so)
    q3, s3, qw3, sw3 = _operands(100, 128, 128, 1, groups=2)
    with pytest.raises(dg.DGError):                              # m_sum % 128
        dg.m_grouped_fp8_gated_gemm_nt_contiguous(q3, s3, qw3, sw3, torch.zeros(100, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        dg.m_grouped_fp8_gated_gemm_nt_contiguous(q3, s3, qw3, sw3, torch.zeros(99, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("out_format,checkpoint", [("bf16", False), ("fp8", True)])
@pytest.mark.parametrize("m,f,k", [(1, 128, 128), (1, 2048, 7168), (1, 384, 16512), (2, 640, 7168), (2, 256, 1024),
                                   (3, 128, 7168), (4, 384, 1920), (3, 1024, 640), (17, 256, 4224), (32, 2048, 512), (33, 128, 1408),
                                   (64, 384, 2048), (65, 256, 896), (100, 1024, 640), (128, 128, 256)])
def test_few_tokens_agree_with_the_tiled_kernel(m, f, k, out_format, checkpoint, monkeypatch):
    """The kernels for one to four tokens, for a few (K split over clusters) and
    the tiled one, each against FP64; K ranges that do and do not divide among
    the CTAs."""
    q, sf, qw, sw = _operands(m, f, k, m + f + k + 2)
    x, w = R.row_values(_np(q), _np(sf)), _weights(qw, sw)
    for decode in ("1", "2", "0"):
        monkeypatch.setenv("DG_DECODE", decode)
        _check(dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format=out_format, checkpoint=checkpoint), x, w, "silu")
        assert dg.get_device_error()[0] == 0


def test_few_tokens_with_a_load_that_never_lands():
    q, sf, qw, sw = _operands(5, 256, 2048, 9)
    want = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True)
    torch.cuda.synchronize()
    dg.set_wait_timeout_ns(20_000_000)
    dg.debug_set_drop_load(1)
    try:
        dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True)
        assert dg.get_device_error()[0] == 5
    finally:
        dg.debug_set_drop_load(0)
        dg.set_wait_timeout_ns(2_000_000_000)
    again = dg.fp8_gated_gemm_nt(q, sf, qw, sw, out_format="fp8", checkpoint=True)
    assert dg.get_device_error()[0] == 0
    assert all(np.array_equal(_np(x), _np(y)) for x, y in zip(again, want))



@pytest.mark.parametrize("m", [1, 2, 4])
def test_one_to_four_strided_tokens(m):
    """Row strides of A, W and h other than their widths, F not a multiple of
    the 16 columns of a CTA."""
    f, k = 200, 640
    q, sf, qw, sw = _operands(m, f, k, 40 + m)
    aw = torch.full((m, k + 48), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    aw[:, :k].copy_(q)
    bw = torch.full((2 * f, k + 16), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    bw[:, :k].copy_(qw)
    d = torch.full((m, f + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = dg.fp8_gated_gemm_nt(aw[:, :k], sf, bw[:, :k], sw, d=d[:, :f], activation="gelu_tanh")
    assert bool((d[:, f:] == 7).all())
    _check(out, R.row_values(_np(q), _np(sf)), _weights(qw, sw), "gelu_tanh")
