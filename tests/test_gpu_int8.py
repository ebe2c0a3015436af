"""Products of 8-bit integers and their quantiser against the formulas in 64 bits."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg

pytestmark = pytest.mark.gpu
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def codes(rows, k, seed=0, lo=-128):
    g = torch.Generator().manual_seed(seed + rows * 7 + k)
    return torch.randint(lo, 128, (rows, k), generator=g, dtype=torch.int32).to(torch.int8).cuda()


def scales(n, seed=0):
    g = torch.Generator().manual_seed(seed + n)
    return (torch.exp2(torch.randn(n, generator=g)) / 4096).cuda()


def check(got, a, sa, b, sb, c=None):
    """Half a step of the result's type (FP16: and half of its smallest), and FP32 sums: at most 2^-23 of the sum of
    magnitudes a step of the tensor cores' (16 columns), and three FP32 roundings."""
    p = a.double() @ b.double().t()
    size = a.double().abs() @ b.double().abs().t()
    s = sa.double()[:, None] * sb.double()
    want = p * s + (0 if c is None else c.double())
    steps = a.shape[1] / 16 + 16
    off = size * s * steps * 2.0 ** -23 + want.abs() * (torch.finfo(got.dtype).eps / 2 + 2.0 ** -22)
    if got.dtype == FP16:
        off = off + 2.0 ** -25
    far = (got.double() - want).abs()
    assert (far <= off).all(), float((far / off).max())
    assert dg.get_device_error()[0] == 0


GEMM = [(1, 8, 16), (1, 7168, 2048), (2, 1, 128), (3, 17, 144), (8, 100, 256), (9, 128, 112), (16, 4096, 1024), (31, 33, 1040),
        (33, 1000, 528), (64, 4096, 7168), (64, 16, 16), (65, 64, 64), (65, 1, 16), (100, 129, 80), (128, 256, 512),
        (129, 300, 1552), (200, 2112, 1024), (333, 1001, 1552), (1000, 200, 48), (2048, 3000, 640), (4096, 4096, 1024)]


@pytest.mark.parametrize("m,n,k", GEMM)
@pytest.mark.parametrize("dtype,with_c", [(BF16, True), (FP16, False)])
def test_sizes(m, n, k, dtype, with_c):
    a, b, sa, sb = codes(m, k), codes(n, k, 1), scales(m), scales(n, 1)
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(4)).to(dtype).cuda() if with_c else None
    check(dg.int8_gemm_nt(a, sa, b, sb, c=c, out_dtype=dtype), a, sa, b, sb, c)


@pytest.mark.parametrize("m", [1, 12, 40, 70, 300])
def test_integers_are_exact(m):
    """Sums below 2^8 as BF16: every one an integer that BF16 holds; all 256 codes."""
    k, n = 256, 256
    a = torch.zeros(m, k, dtype=torch.int8, device="cuda")
    at = torch.arange(m, device="cuda") * 37 % k
    a[torch.arange(m, device="cuda"), at] = 1
    b = (torch.arange(n, device="cuda")[:, None] + torch.arange(k, device="cuda")).remainder(256).sub(128).to(torch.int8)
    one = torch.ones(max(m, n), device="cuda")
    got = dg.int8_gemm_nt(a, one[:m], b, one[:n])
    assert torch.equal(got.float(), b[:, at].t().float())
    got = dg.int8_gemm_nt(b, one[:n], a, one[:m])
    assert torch.equal(got.float(), b[:, at].float())


@pytest.mark.parametrize("m", [5, 64, 130])
def test_largest_sums(m):
    """All codes -128: K 2^14, past 2^24, where FP32 still holds every such sum."""
    k, n = 4096, 72
    a, b = torch.full((m, k), -128, dtype=torch.int8, device="cuda"), torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(m + n, device="cuda")
    got = dg.int8_gemm_nt(a, one[:m], b, one[:n])
    assert (got.float() == k * 2.0 ** 14).all()


@pytest.mark.parametrize("m,n,k", [(3, 40, 96), (50, 64, 256), (150, 200, 320)])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_strides_and_results_in_place(m, n, k, shift):
    wide = codes(m, k + 48)
    a, b = wide[:, 16:16 + k], codes(n, k + 16, 1)[:, :k]
    sa, sb = scales(m), scales(n, 1)
    room = torch.full((m, n + 24), 9.0, dtype=BF16, device="cuda")
    d = room[:, shift:shift + n]
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    assert dg.int8_gemm_nt(a, sa, b, sb, c=c, d=d) is d
    check(d, a, sa, b, sb, c)
    assert (room[:, :shift] == 9.0).all() and (room[:, shift + n:] == 9.0).all()
    d.copy_(c)
    dg.int8_gemm_nt(a, sa, b, sb, c=d, d=d)
    check(d, a, sa, b, sb, c)


def test_empty():
    a, b = codes(4, 32), codes(8, 32)
    assert dg.int8_gemm_nt(a[:0], scales(0), b, scales(8)).shape == (0, 8)
    assert dg.int8_gemm_nt(a, scales(4), b[:0], scales(0)).shape == (4, 0)
    q, s = dg.quantize_int8(torch.empty(0, 5, device="cuda"))
    assert q.shape == (0, 5) and s.shape == (0,)


@pytest.mark.parametrize("m", [7, 40, 500])
def test_bits_do_not_change(m):
    n, k = 1024, 2064
    a, b, sa, sb = codes(m, k), codes(n, k, 1), scales(m), scales(n, 1)
    want = dg.int8_gemm_nt(a, sa, b, sb).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dg.int8_gemm_nt(a, sa, b, sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        assert torch.equal(dg.int8_gemm_nt(a, sa, b, sb), want)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        got = dg.int8_gemm_nt(a, sa, b, sb, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    assert dg.get_device_error()[0] == 0


def test_fewer_sms():
    try:
        for n in (1, 9):
            dg.set_num_sms(n)
            for m in (5, 300):
                a, b, sa, sb = codes(m, 320), codes(700, 320, 1), scales(m), scales(700, 1)
                check(dg.int8_gemm_nt(a, sa, b, sb), a, sa, b, sb)
    finally:
        dg.set_num_sms(0)


# ---------------------------------------------------------------- the quantiser


def quantised(x):
    """The definition, in 64 bits: 127 x / amax is a quotient of a 31-bit number by a 24-bit one, so its rounding to 53
    bits neither makes nor hides a half."""
    top = x.double().abs().amax(1)
    q = torch.round(127 * x.double() / torch.where(top > 0, top, 1).unsqueeze(1))
    return q.to(torch.int8), top / 127


def check_codes(x, **kw):
    q, s = dg.quantize_int8(x, **kw)
    want, top = quantised(x)
    assert torch.equal(q, want)
    # one FP32 rounding (below 2^-126 half of FP32's smallest)
    assert ((s.double() - top).abs() <= top * 2.0 ** -24 + 2.0 ** -150).all()
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7168), (3, 8), (5, 100), (197, 1001), (2, 2048), (9, 2049), (4, 4096),
                                       (3, 8200), (2, 16384), (2, 16400), (3, 40001), (1000, 512), (64, 33)])
@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
def test_codes(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    check_codes((torch.randn(rows, cols, generator=g) * torch.exp2(torch.randn(rows, 1, generator=g))).to(dtype).cuda())


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
def test_halves_round_to_even(dtype):
    """Quotients that are half integers exactly, and their neighbours."""
    n = torch.arange(-127, 127, dtype=F32) + 0.5
    x = torch.cat([n, torch.tensor([127.0])]).to(dtype).cuda()
    rows = [x * 2.0 ** -3]
    if dtype is F32:
        rows += [torch.nextafter(x, torch.tensor(0.0, device="cuda")), torch.nextafter(x, torch.tensor(200.0, device="cuda"))]
        rows[1][-1] = rows[2][-1] = 127.0
    for r in rows:
        check_codes(r.unsqueeze(0).contiguous())
    g = torch.Generator().manual_seed(0)
    check_codes(torch.randint(-254, 255, (300, 256), generator=g).to(dtype).cuda())  # halves wherever amax is 254


@pytest.mark.parametrize("size", [1e-45, 1e-42, 1e-38, 1e-33, 1e-30, 1e30, 2.5e38])
def test_magnitudes(size):
    g = torch.Generator().manual_seed(1)
    x = torch.rand(7, 300, generator=g).mul(2).sub(1).cuda() * size
    check_codes(x)
    check_codes(x.to(BF16))


def test_rows_of_zeros_and_rows_that_are_not_finite():
    x = torch.randn(6, 200, generator=torch.Generator().manual_seed(2)).cuda()
    x[1] = 0
    x[2, 7], x[3, 199], x[4, 0] = float("nan"), float("inf"), float("-inf")
    for dtype in (F32, BF16, FP16):
        y = x.to(dtype)
        q, s = dg.quantize_int8(y)
        rest = [0, 1, 5]
        want, top = quantised(y[rest])
        assert torch.equal(q[rest], want) and s[1] == 0 and torch.isfinite(s[rest]).all()
        assert (q[2:5] == 0).all() and torch.isnan(s[2:5]).all()
    b, sb = dg.quantize_int8(torch.randn(16, 208, generator=torch.Generator().manual_seed(2)).cuda())
    q, s = dg.quantize_int8(torch.nn.functional.pad(x, (0, 8)))
    d = dg.int8_gemm_nt(q, s, b, sb)
    assert torch.isnan(d[2:5].float()).all() and torch.isfinite(d[rest].float()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows_and_given_results(dtype):
    wide = torch.randn(20, 333, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    for x in (wide[:, 1:300], wide[::3, :256], wide[:1]):
        q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(len(x), device="cuda")
        got = check_codes(x, out=(q, s))
        assert got[0] is q and got[1] is s


def test_quantised_layer():
    """Activations by token, weights by channel: the product of the real values, within both roundings' half steps."""
    m, n, k = 70, 136, 512
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(m, k, generator=g).to(BF16).cuda(), torch.randn(n, k, generator=g).cuda()
    (a, sa), (b, sb) = dg.quantize_int8(x), dg.quantize_int8(w)
    got = dg.int8_gemm_nt(a, sa, b, sb).double()
    want = x.double() @ w.double().t()
    sa, sb = sa.double()[:, None], sb.double()
    off = 0.5 * sa * w.double().abs().sum(1) + 0.5 * sb * x.double().abs().sum(1)[:, None] + 0.25 * k * sa * sb
    assert ((got - want).abs() <= off + (want.abs() + off) * 2.0 ** -7).all()
