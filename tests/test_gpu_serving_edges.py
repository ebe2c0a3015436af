"""Serving operators at the ends of what their documentation allows: widths,
offsets past 32 bits, operands given twice, results in place, calls at once on
two streams, waits that may run out."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import test_gpu_int8 as I
import test_gpu_moe_few_tokens as M

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
DG_ERR_DEVICE_TIMEOUT = 5


@pytest.mark.parametrize("t,d,f,e,k", [(64, 1152, 896, 1, 1), (64, 20480, 128, 2, 1), (3, 128, 16384, 3, 2), (20, 65536, 128, 2, 2),
                                       (2, 128, 65536, 2, 1), (32, 384, 384, 16, 16), (16, 128, 128, 512, 1)])
def test_moe_widths(t, d, f, e, k):
    w, x, r, c = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d), M.tokens(t, d, seed=5)
    M.check(dg.fp8_moe_few_tokens(x, r, *w, k, c=c), M.reference(x, r, w, k, c=c))


def test_moe_experts_behind_4_gb():
    """The last two of many experts give what they give alone."""
    d, f, many = 7168, 2048, 150
    w = M.weights(2, d, f)
    x = M.tokens(5, d)
    router = torch.zeros(many, d, device="cuda")
    router[-2:] = M.gate(2, d)
    bias = torch.zeros(many, device="cuda")
    bias[-2:] = 2.0
    large = [torch.zeros(many, *v.shape[1:], dtype=v.dtype, device="cuda") for v in w]
    for to, v in zip(large, w):
        to.view(torch.uint8 if v.element_size() == 1 else v.dtype)[-2:] = v.view(torch.uint8 if v.element_size() == 1 else v.dtype)
    assert large[0].numel() > 2 ** 32
    got = dg.fp8_moe_few_tokens(x, router, *large, 2, router_bias=bias, score="sigmoid", renormalize=False)
    assert (got.experts.sort(1)[0] == torch.tensor([many - 2, many - 1], device="cuda")).all()
    alone = dg.fp8_moe_few_tokens(x, M.gate(2, d), *w, 2, router_bias=bias[-2:].contiguous(), score="sigmoid", renormalize=False)
    assert torch.equal(got.y, alone.y) and torch.equal(got.weights, alone.weights)
    assert torch.equal(got.experts - (many - 2), alone.experts)
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("m,n,k", [(1300, 1001, 80), (1300, 1024, 80), (700, 2999, 144)])
@pytest.mark.parametrize("shift", [0, 1])
def test_tiles_in_place(m, n, k, shift):
    """Large enough for the tiled kernel, on and off 16-byte boundaries."""
    a, b, sa, sb = I.codes(m, k), I.codes(n, k, 1), I.scales(m), I.scales(n, 1)
    room = torch.full((m + 1, n + 24), 9.0, dtype=BF16, device="cuda")
    d = room[:m, shift:shift + n]
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    d.copy_(c)
    dg.int8_gemm_nt(a, sa, b, sb, c=d, d=d)
    I.check(d, a, sa, b, sb, c)
    assert (room[:, :shift] == 9.0).all() and (room[:, shift + n:] == 9.0).all() and (room[m] == 9.0).all()


@pytest.mark.parametrize("m", [1, 30, 100, 2000])
def test_one_operand_twice(m):
    a, s = I.codes(m, 272), I.scales(m)
    got = dg.int8_gemm_nt(a, s, a, s)
    I.check(got, a, s, a, s)


@pytest.mark.parametrize("m", [3, 40, 300])
def test_int8_offsets_past_32_bits(m):
    """Rows so far apart that the last ones lie behind 4 GB, of b and of the result (c in place)."""
    n, k = 320, 64
    step = (2 ** 32 // (n - 8) + 15) // 16 * 16
    b = torch.zeros(n * step, dtype=torch.int8, device="cuda").as_strided((n, k), (step, 1))
    b.copy_(I.codes(n, k, 1))
    assert (n - 1) * step > 2 ** 32
    a, sa, sb = I.codes(m, k), I.scales(m), I.scales(n, 1)
    I.check(dg.int8_gemm_nt(a, sa, b, sb), a, sa, b, sb)
    del b
    b = I.codes(n, k, 1)
    step = max(2 ** 31 // (m - 1), n) // 16 * 16 + 16
    d = torch.zeros(m * step, dtype=BF16, device="cuda").as_strided((m, n), (step, 1))
    assert (m - 1) * step > 2 ** 31
    c = torch.randn(m, n, generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    d.copy_(c)
    dg.int8_gemm_nt(a, sa, b, sb, c=d, d=d)
    I.check(d, a, sa, b, sb, c)


def test_quantiser_offsets_past_32_bits():
    rows, cols = 70000, 61600
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, cols, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    x[:-3] = 1.0
    assert x.numel() > 2 ** 32
    q, s = dg.quantize_int8(x)
    want, top = I.quantised(x[-3:])
    assert torch.equal(q[-3:], want)
    assert ((s[-3:].double() - top).abs() <= top * 2.0 ** -24).all()
    assert (q[:-3:997] == 127).all()


def test_two_calls_at_once():
    """Layers and products of different sizes on two streams, many in flight."""
    jobs = []
    for t, d, f, e, k in [(1, 1024, 512, 8, 2), (40, 512, 256, 6, 3)]:
        w, x, r = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d)
        jobs.append(lambda x=x, r=r, w=w, k=k: dg.fp8_moe_few_tokens(x, r, *w, k).y)
    for m, n, k in [(600, 1000, 1024), (64, 4096, 512)]:
        a, b, sa, sb = I.codes(m, k), I.codes(n, k, 1), I.scales(m), I.scales(n, 1)
        jobs.append(lambda a=a, b=b, sa=sa, sb=sb: dg.int8_gemm_nt(a, sa, b, sb))
    want = [j().clone() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(40):
        for s, shift in zip(streams, (0, 1)):
            with torch.cuda.stream(s):
                at = (i + shift) % len(jobs)
                got.append((at, jobs[at]()))
    torch.cuda.synchronize()
    for at, y in got:
        assert torch.equal(y, want[at])
    assert dg.get_device_error()[0] == 0


def test_waits_that_may_run_out():
    """With a limit of a microsecond waits of these kernels run out, or do not: the call ends by itself, says so, and the
    next one is right."""
    calls = []
    for t, d, f, e, k in [(1, 7168, 1024, 8, 4), (16, 1024, 512, 8, 2), (40, 512, 256, 6, 3)]:
        w, x, r = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d)
        calls.append(lambda x=x, r=r, w=w, k=k: dg.fp8_moe_few_tokens(x, r, *w, k).y)
    for m, n, k in [(2000, 2000, 1024), (64, 4096, 2048)]:
        a, b, sa, sb = I.codes(m, k), I.codes(n, k, 1), I.scales(m), I.scales(n, 1)
        calls.append(lambda a=a, b=b, sa=sa, sb=sb: dg.int8_gemm_nt(a, sa, b, sb))
    for call in calls:
        want = call().clone()
        assert dg.get_device_error()[0] == 0
        dg.set_wait_timeout_ns(1000)
        try:
            call()
            status = dg.get_device_error()[0]
        finally:
            dg.set_wait_timeout_ns(2_000_000_000)
        assert status in (0, DG_ERR_DEVICE_TIMEOUT)
        assert torch.equal(call(), want) and dg.get_device_error()[0] == 0


@pytest.mark.parametrize("dtype,digits", [(BF16, 8), (torch.float16, 11)])
@pytest.mark.parametrize("pad", [0, 1])
def test_codes_of_all_significands(dtype, digits, pad):
    """A row for each significand of its maximum, in it every significand at the nine binades that have codes; rows on
    16 bytes and off them."""
    half = 2 ** (digits - 1)
    s = torch.arange(half, 2 * half, dtype=torch.float64)
    values = torch.cat([s * 2.0 ** -k for k in range(1, 10)])
    rows = torch.cat([s[:, None], values.expand(half, -1), torch.zeros(half, 7 + pad, dtype=torch.float64)], 1)
    below = torch.where(s[None, :] <= s[:, None], s[None, :], 0.0)   # the maximum's own binade
    x = torch.cat([rows[:, :1 + len(values)], below, rows[:, 1 + len(values):]], 1) * 2.0 ** -4
    x = x * torch.where(torch.arange(x.shape[1]) % 3 == 2, -1.0, 1.0)
    y = x.to(dtype)
    assert torch.equal(y.double(), x) and x.shape[1] % 8 == (0 if pad == 0 else 1)
    I.check_codes(y.cuda())


def test_many_rows_of_the_quantiser():
    """More rows than CTAs run at once, at each number of warps a row takes."""
    g = torch.Generator().manual_seed(0)
    for rows, cols in [(9001, 24), (6000, 1032), (3001, 2056), (1300, 4104), (700, 8200), (400, 16400), (160, 33000)]:
        x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randn(rows, 1, generator=g))
        x[rows // 2, 3] = float("nan")
        x[7] = 0
        for dtype in (BF16, torch.float16, torch.float32):
            y = x.to(dtype).cuda()
            q, s = dg.quantize_int8(y)
            good = torch.arange(rows, device="cuda") != rows // 2
            want, top = I.quantised(y[good])
            assert torch.equal(q[good], want) and ((s[good].double() - top).abs() <= top * 2.0 ** -24).all()
            assert (q[~good] == 0).all() and torch.isnan(s[~good]).all()


def test_quantiser_on_fewer_sms():
    x = torch.randn(500, 1032, generator=torch.Generator().manual_seed(0)).to(BF16).cuda()
    try:
        for n in (1, 5):
            dg.set_num_sms(n)
            I.check_codes(x)
    finally:
        dg.set_num_sms(0)
