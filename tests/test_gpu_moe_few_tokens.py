"""A whole mixture-of-experts layer for a few tokens against the formula in 64
bits, with bounds from the roundings that it makes."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import block

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def weights(e, d, f, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    up = torch.randn(e, 2 * f, d, generator=g).cuda() * (size * d ** -0.5)
    down = torch.randn(e, d, f, generator=g).cuda() * f ** -0.5
    return dg.quantize_fp8(up, 128) + dg.quantize_fp8(down, 128)


def values(q, sf):
    return dg.dequantize_fp8(q, sf, torch.float32).double()


def reference(x, router, w, k, bias=None, score="softmax", renormalize=True, scale=1.0, activation="silu", c=None):
    """(y, experts, weights, how far y may be off) in 64 bits.

    Off by: BF16's half step of y; h as halves (half a step, 2^-11, of each h);
    FP32 sums, at most 2^-23 a step of at most 8 + columns / 128 + 8 steps; the
    activation's 2^-20 of h."""
    up, down = values(*w[:2]), values(*w[2:])
    f, d = up.shape[1] // 2, up.shape[2]
    xd = x.double()
    l = xd @ router.double().t()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    by = l if bias is None else s + bias.double()
    chosen = torch.sort(by, dim=1, descending=True, stable=True)[1][:, :k]
    ws = s.gather(1, chosen)
    ws = (ws / ws.sum(1, keepdim=True) if renormalize else ws) * scale
    y = torch.zeros_like(xd) if c is None else c.double()
    off = y.abs() * 2.0 ** -23
    up_step, down_step = (16 + d / 128) * 2.0 ** -23, (16 + f / 128 + k) * 2.0 ** -23
    for t in range(len(x)):
        for j in range(k):
            e = int(chosen[t, j])
            gu, size = up[e] @ xd[t], up[e].abs() @ xd[t].abs()
            g, u = gu[:f], gu[f:]
            if activation == "silu":
                a = g * torch.sigmoid(g)
            else:
                a = 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
            h = a * u
            dg_, du = size[:f] * up_step, size[f:] * up_step
            dh = 1.2 * dg_ * (u.abs() + du) + a.abs() * du + h.abs() * (2.0 ** -11 + 2.0 ** -20)
            wt = float(ws[t, j])
            y[t] += wt * (down[e] @ h)
            off[t] += abs(wt) * (down[e].abs() @ (dh + (h.abs() + dh) * down_step))
    return y, chosen, ws, off + y.abs() * 2.0 ** -8


def check(got, want):
    y, chosen, ws, off = want
    assert torch.equal(got.experts.long(), chosen)
    # expf, a sum and a quotient of FP32: a few steps of 2^-24
    assert ((got.weights.double() - ws).abs() <= ws.abs() * 2.0 ** -20).all()
    far = (got.y.double() - y).abs()
    assert (far <= off).all(), float((far / off).max())
    assert dg.get_device_error()[0] == 0


def tokens(t, d, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(t, d, generator=g) * torch.exp2(0.5 * torch.randn(1, d, generator=g))).to(BF16).cuda()


def gate(e, d, dtype=torch.float32, seed=2):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(e, d, generator=g) * d ** -0.5).to(dtype).cuda()


SIZES = [
    # t, d, f, e, k
    (1, 128, 128, 1, 1), (1, 256, 128, 4, 2), (2, 384, 640, 5, 3), (3, 1152, 384, 7, 2), (7, 128, 1024, 16, 8),
    (8, 512, 256, 2, 1), (9, 640, 128, 3, 2), (16, 1024, 512, 8, 2), (17, 256, 384, 6, 6), (33, 512, 512, 4, 2),
    (64, 256, 256, 3, 3), (64, 384, 128, 40, 8), (5, 128, 128, 512, 16), (64, 128, 256, 64, 16), (1, 7168, 2048, 9, 8),
]


@pytest.mark.parametrize("t,d,f,e,k", SIZES)
def test_sizes(t, d, f, e, k):
    w, x, r, c = weights(e, d, f), tokens(t, d), gate(e, d), tokens(t, d, seed=5)
    check(dg.fp8_moe_few_tokens(x, r, *w, k, c=c), reference(x, r, w, k, c=c))


@pytest.mark.parametrize("router", [torch.float32, BF16])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("renormalize,scale,activation", [(True, 1.0, "silu"), (False, 2.5, "gelu_tanh")])
def test_gates(router, score, bias, renormalize, scale, activation):
    t, d, f, e, k = 11, 640, 256, 24, 6
    w, x, r = weights(e, d, f), tokens(t, d), gate(e, d, router)
    b = 0.3 * torch.randn(e, generator=torch.Generator().manual_seed(3)).cuda() if bias else None
    kw = dict(score=score, renormalize=renormalize, scale=scale, activation=activation)
    check(dg.fp8_moe_few_tokens(x, r, *w, k, router_bias=b, **kw), reference(x, r, w, k, bias=b, **kw))


def test_ties_go_to_the_lowest_index():
    t, d, f, e, k = 4, 256, 128, 70, 5
    w, x, r = weights(e, d, f), tokens(t, d), gate(e, d)
    r[:] = r[0]
    got = dg.fp8_moe_few_tokens(x, r, *w, k)
    assert torch.equal(got.experts.cpu(), torch.arange(k, dtype=torch.int32).expand(t, k))
    check(got, reference(x, r, w, k))
    r[33:60] *= torch.where(x[0].float() @ r[0] > 0, 2.0, 0.5)  # a better set for token 0, itself equal
    check(dg.fp8_moe_few_tokens(x[:1], r, *w, k), reference(x[:1], r, w, k))


def test_near_scores_keep_their_order():
    """Scores that differ by less than FP32 sums can tell: the last column adds 2^-20 to some experts."""
    d, f, e, k = 1024, 128, 64, 8
    w, x, r = weights(e, d, f), tokens(3, d), gate(e, d)
    r[:] = r[0]
    x[:, -1] = 1.0
    better = torch.randperm(e, generator=torch.Generator().manual_seed(7))[:k]
    r[:, -1] = 0.0
    r[better.cuda(), -1] = 2.0 ** -20
    got = dg.fp8_moe_few_tokens(x, r, *w, k)
    assert torch.equal(got.experts[0].cpu().long(), better.sort()[0])
    check(got, reference(x, r, w, k))


@pytest.mark.parametrize("live", [0, 1, 5, 8])
def test_padded_batch(live):
    t, d, f, e, k = 8, 384, 256, 6, 2
    w, x, r, c = weights(e, d, f), tokens(t, d), gate(e, d), tokens(t, d, seed=5)
    x[live:] = float("nan")
    y = torch.full((t, d), 7.0, dtype=BF16, device="cuda")
    n = torch.tensor([live], dtype=torch.int32, device="cuda")
    got = dg.fp8_moe_few_tokens(x, r, *w, k, c=c, num_tokens=n, d=y)
    assert got.y is y
    assert (y[live:] == 7.0).all() and (got.experts[live:] == -1).all() and (got.weights[live:] == 0).all()
    if live:
        want = reference(x[:live], r, w, k, c=c[:live])
        check(dg.MoeOutput(y[:live], got.experts[:live], got.weights[:live]), want)


@pytest.mark.parametrize("bad,taken", [(-3, 0), (9, 4)])
def test_a_token_count_out_of_range_is_reported(bad, taken):
    t, d, f, e, k = 4, 128, 128, 3, 2
    w, x, r = weights(e, d, f), tokens(t, d), gate(e, d)
    y = torch.full((t, d), 7.0, dtype=BF16, device="cuda")
    n = torch.tensor([bad], dtype=torch.int32, device="cuda")
    got = dg.fp8_moe_few_tokens(x, r, *w, k, num_tokens=n, d=y)
    assert dg.get_device_error()[0] == 6
    assert (y[taken:] == 7.0).all() and (got.experts[taken:] == -1).all() and (got.experts[:taken] >= 0).all()


def test_strides_and_results_in_place():
    t, d, f, e, k = 6, 256, 128, 4, 2
    w, r = weights(e, d, f), gate(e, d)
    wide = torch.full((t, 3 * d + 8), 3.0, dtype=BF16, device="cuda")
    x, c, y = wide[:, :d], wide[:, d:2 * d], wide[:, 2 * d + 3:3 * d + 3]  # y on no boundary
    x.copy_(tokens(t, d))
    c.copy_(tokens(t, d, seed=5))
    want = reference(x, r, w, k, c=c)
    check(dg.fp8_moe_few_tokens(x, r, *w, k, c=c, d=y), want)
    assert (wide[:, 2 * d:2 * d + 3] == 3.0).all() and (wide[:, 3 * d + 3:] == 3.0).all()
    check(dg.fp8_moe_few_tokens(x, r, *w, k, c=c, d=c), want)
    plain = reference(x, r, w, k, c=x)
    check(dg.fp8_moe_few_tokens(x, r, *w, k, c=x, d=x), plain)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 30])
def test_magnitudes(size):
    """Scales of x and h follow the values: nothing overflows or vanishes on the way.
    (silu is about g / 2 for small g and g or 0 for large: h grows with the square.)"""
    t, d, f, e, k = 3, 512, 256, 4, 2
    w, r = weights(e, d, f), gate(e, d)
    x = (tokens(t, d).float() * size).to(BF16)
    r = r / size
    check(dg.fp8_moe_few_tokens(x, r, *w, k), reference(x, r, w, k))


def test_columns_of_very_different_size():
    """A loud column in each 128: the others keep their digits."""
    t, d, f, e, k = 3, 512, 128, 4, 2
    w, r, x = weights(e, d, f), gate(e, d), tokens(t, d)
    x[:, 5::128] *= 2.0 ** 14
    r[:, 5::128] = 0
    up = values(*w[:2])
    up[:, :, 5::128] = 0
    w = dg.quantize_fp8(up.float(), 128) + w[2:]
    check(dg.fp8_moe_few_tokens(x, r, *w, k), reference(x, r, w, k))


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_row(what):
    t, d, f, e, k = 5, 256, 128, 4, 2
    w, x, r = weights(e, d, f), tokens(t, d), gate(e, d)
    want = reference(x, r, w, k)
    x[2, 17] = what
    got = dg.fp8_moe_few_tokens(x, r, *w, k)
    assert not torch.isfinite(got.y[2].float()).any()
    chosen = got.experts[2].tolist()
    assert len(set(chosen)) == k and all(0 <= c < e for c in chosen)
    rest = [0, 1, 3, 4]
    check(dg.MoeOutput(got.y[rest], got.experts[rest], got.weights[rest]), [v[rest] for v in want])


def test_scores_that_are_no_numbers_come_last():
    t, d, f, e, k = 2, 128, 128, 40, 3
    w, x, r = weights(e, d, f), tokens(t, d), gate(e, d)
    best = dg.fp8_moe_few_tokens(x, r, *w, k).experts
    r[best[0].long()] = float("nan")
    r[37] = float("nan")
    got = dg.fp8_moe_few_tokens(x, r, *w, k, renormalize=True)
    good = [i for i in range(e) if not torch.isnan(r[i]).any()]
    want = reference(x, r[good], tuple(v[good].contiguous() for v in w), k)
    assert torch.equal(got.experts.long().cpu(), torch.tensor(good)[want[1].cpu()])


def test_empty_batch():
    w, r = weights(3, 128, 128), gate(3, 128)
    got = dg.fp8_moe_few_tokens(torch.empty(0, 128, dtype=BF16, device="cuda"), r, *w, 2)
    assert got.y.shape == (0, 128) and got.experts.shape == (0, 2)


def test_bits_do_not_change_between_calls_graphs_and_streams():
    t, d, f, e, k = 13, 1024, 512, 12, 4
    w, x, r, c = weights(e, d, f), tokens(t, d), gate(e, d), tokens(t, d, seed=5)
    call = lambda **kw: dg.fp8_moe_few_tokens(x, r, *w, k, c=c, **kw)  # noqa: E731
    want = [v.clone() for v in call()]
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))  # noqa: E731
    for _ in range(20):
        assert same(call())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert same(got)
    graphs = []
    for _ in range(2):  # two graphs of one pool, replayed in turn and at once on two streams
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for _ in range(5):
        for g, out in graphs:
            out.y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert same(out)
    other = torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1]) and same(graphs[1][1])
    assert dg.get_device_error()[0] == 0


def test_fewer_sms():
    t, d, f, e, k = 5, 512, 256, 6, 2
    w, x, r = weights(e, d, f), tokens(t, d), gate(e, d)
    want = reference(x, r, w, k)
    try:
        for n in (1, 7, 40):
            dg.set_num_sms(n)
            check(dg.fp8_moe_few_tokens(x, r, *w, k), want)
    finally:
        dg.set_num_sms(0)


def test_experts_of_the_block():
    """GatedExperts' whole layer: near what its masked form gives for the same choice (which rounds
    activations to 8 bits: 2^-4 of each at most, in the mean of many far less)."""
    t, d, f, e, k = 6, 512, 256, 4, 2
    g = torch.Generator().manual_seed(0)
    up, down = torch.randn(e, 2 * f, d, generator=g).cuda() * d ** -0.5, torch.randn(e, d, f, generator=g).cuda() * f ** -0.5
    net = block.GatedExperts(up, down)
    x, r = tokens(t, d), gate(e, d)
    got = net.few_tokens(x, r, k, c=x)
    check(got, reference(x, r, (net.up.q, net.up.sf, net.down.q, net.down.sf), k, c=x))
    rows = torch.zeros(e, 64, d, device="cuda")
    counts = [0] * e
    at = {}
    for i in range(t):
        for j in range(k):
            n = int(got.experts[i, j])
            rows[n, counts[n]] = x[i].float()
            at[i, j] = n, counts[n]
            counts[n] += 1
    q, sf = dg.quantize_fp8(rows, 1)
    y = net.decode(q, sf, torch.tensor(counts, dtype=torch.int32, device="cuda")).float()
    want = torch.stack([x[i].float() + sum(float(got.weights[i, j]) * y[at[i, j]] for j in range(k)) for i in range(t)])
    assert (got.y.float() - want).norm() <= 2.0 ** -4 * (want - x.float()).norm()
