"""Layer norm, forward and backward, against the formulas in FP64."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import _fp8ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-5
# rounding of the result's own type: half a unit in the last place
U = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# FP32 arithmetic: sums of n terms in trees and runs of at most 64, a handful
# of roundings each; 2^-20 leaves room for 16 roundings of 2^-24
ACC = 2.0 ** -20


def _inputs(rows, cols, dtype, seed, wdtype=torch.float32, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randn(1, cols, generator=g))
    x = (x + mean * torch.randn(rows, 1, generator=g)).to(dtype)
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(wdtype)
    b = (0.3 * torch.randn(cols, generator=g)).to(wdtype)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    return x, w, b, dy


def _forward64(x, w, b):
    x = x.double().numpy()
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + EPS)
    y = (x - mean) * rstd * w.double().numpy()
    return mean, rstd, y if b is None else y + b.double().numpy()


def _check_forward(r, x, w, b):
    mean, rstd, y = _forward64(x, w, b)
    X = np.abs(x.double().numpy())
    dm = ACC * X.mean(1, keepdims=True)  # the mean's error
    assert (np.abs(r.mean.double().cpu().numpy()[:, None] - mean) <= dm + 1e-40).all()
    assert (np.abs(r.rstd.double().cpu().numpy()[:, None] / rstd - 1) <= ACC + rstd * dm).all()
    wm = np.abs(w.double().numpy())
    slack = wm * rstd * (dm + ACC * np.abs(x.double().numpy() - mean)) * 2 + ACC * np.abs(y)
    if b is not None:
        slack = slack + ACC * np.abs(b.double().numpy())
    slack = slack + wm * np.abs(x.double().numpy() - mean) * rstd * rstd * dm
    if r.sf is None:
        err = np.abs(r.y.double().cpu().numpy() - y)
        tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0  # half of FP16's smallest subnormal
        assert (err <= U[x.dtype] * np.abs(y) + slack + tiny).all(), (err - U[x.dtype] * np.abs(y) - slack).max()
    else:
        rows, cols = x.shape
        R.check_codes(r.y.view(torch.uint8).cpu().numpy(),
                      np.repeat(R.unpack_rows(r.sf.cpu().numpy(), rows, cols), 128, 1), 1, y, slack, "y")
        assert not R.unused_bytes(r.sf.cpu().numpy(), rows, cols // 128).any()


SIZES = [(1, 1), (3, 7), (197, 1001), (5, 128), (64, 1024), (9, 2048), (33, 4104), (7, 7168), (2, 33000), (1, 70001)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, dtype):
    x, w, b, _ = _inputs(rows, cols, dtype, rows + cols)
    _check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS), x, w, b)
    _check_forward(dg.layer_norm(x.cuda(), w.cuda(), eps=EPS), x, w, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 384), (130, 1152), (6, 4224), (5, 7168), (2, 16384)])
def test_forward_to_8_bits(rows, cols, dtype):
    x, w, b, _ = _inputs(rows, cols, dtype, rows + cols)
    _check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, out_format="fp8"), x, w, b)


def test_rows_of_zeros_constants_and_a_large_mean():
    """var = 0: y is the bias; a mean 2^12 times the spread costs no more
    than the mean's own rounding."""
    x, w, b, _ = _inputs(8, 512, torch.float32, 1)
    x[0] = 0
    x[1] = 3.25
    x[2] += 4096.0
    r = dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    assert torch.equal(r.y[0].cpu(), b) and torch.equal(r.y[1].cpu(), b)
    _check_forward(r, x, w, b)
    z = dg.layer_norm(torch.zeros(4, 128, device="cuda"), torch.ones(128, device="cuda"), out_format="fp8")
    assert not z.y.view(torch.uint8).any()


def test_parameters_in_xs_type_strides_and_offsets():
    x, w, b, dy = _inputs(70, 520, torch.bfloat16, 2, wdtype=torch.bfloat16)
    _check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS), x, w, b)
    for left, right in ((8, 16), (3, 2)):  # a 16-byte aligned slice and an odd one
        wide = torch.full((70, left + 520 + right), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, left:left + 520] = x.cuda()
        view = wide[:, left:left + 520]
        r = dg.layer_norm(view, w.cuda(), b.cuda(), eps=EPS)
        _check_forward(r, x, w, b)
        widey = torch.zeros(70, 520 + left, dtype=torch.bfloat16, device="cuda")
        widey[:, left:] = dy.cuda()
        _check_backward(dg.layer_norm_backward(widey[:, left:], view, w.cuda(), r.mean, r.rstd), x, w, dy, r)


def _check_backward(got, x, w, dy, r):
    dx, dw, db = (t.double().cpu().numpy() for t in got)
    X, D, W = x.double().numpy(), dy.double().numpy(), w.double().numpy()
    mean, rstd = r.mean.double().cpu().numpy()[:, None], r.rstd.double().cpu().numpy()[:, None]
    xh = (X - mean) * rstd
    t = D * W
    c1, c2 = t.mean(1, keepdims=True), (t * xh).mean(1, keepdims=True)
    want = rstd * (t - c1 - xh * c2)
    # FP32: x - mean rounds at the size of both, the two means over the row's magnitudes
    exh = 2.0 ** -23 * (np.abs(X) + np.abs(mean)) * rstd
    slack = rstd * (ACC * (np.abs(t) + np.abs(t).mean(1, keepdims=True) + np.abs(xh) * np.abs(t * xh).mean(1, keepdims=True))
                    + exh * np.abs(c2) + np.abs(xh) * (np.abs(t) * exh).mean(1, keepdims=True))
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    err = np.abs(dx - want)
    assert (err <= U[x.dtype] * np.abs(want) + slack + tiny).all(), (err - slack).max()
    assert (np.abs(dw - (D * xh).sum(0)) <= ACC * np.abs(D * xh).sum(0) + (np.abs(D) * exh).sum(0) + 1e-40).all()
    assert (np.abs(db - D.sum(0)) <= ACC * np.abs(D).sum(0)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (197, 1001), (400, 128), (1000, 40), (9, 2048), (33, 4104),
                                       (700, 7168), (5, 9000), (3, 40001)])
def test_backward(rows, cols, dtype):
    x, w, b, dy = _inputs(rows, cols, dtype, 3 * rows + cols)
    r = dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    got = dg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), r.mean, r.rstd)
    assert got[0].dtype == dtype and got[1].dtype == got[2].dtype == torch.float32
    _check_backward(got, x, w, dy, r)


def test_backward_against_differences():
    """The loss sum(y * dy) along random directions of x, weight and bias, by
    central differences of the FP64 forward formula."""
    x, w, b, dy = _inputs(20, 300, torch.float32, 11)
    r = dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    dx, dw, db = (t.double().cpu() for t in dg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), r.mean, r.rstd))
    g = torch.Generator().manual_seed(12)
    loss = lambda x, w, b: float((torch.from_numpy(_forward64(x, w, b)[2]) * dy.double()).sum())  # noqa: E731
    h = 2.0 ** -12
    for p, grad in ((0, dx), (1, dw), (2, db)):
        args = [x.double(), w.double(), b.double()]
        v = torch.randn(args[p].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[p], down[p] = args[p] + h * v, args[p] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # h^2 third derivatives of a smooth function of order one per element, and FP32's own error
        bound = (h * h + 2.0 ** -18) * float((grad.abs() * v.abs()).sum()) + 1e-6
        assert abs(diff - float((grad * v).sum())) <= bound, (p, diff, float((grad * v).sum()))


def test_no_rows():
    w = torch.ones(16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    r = dg.layer_norm(x, w)
    assert r.y.shape == (0, 16)
    dx, dw, db = dg.layer_norm_backward(x, x, w, r.mean, r.rstd)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


def test_same_bits_every_time_and_on_a_side_stream():
    x, w, b, dy = (t.cuda() for t in _inputs(900, 1536, torch.bfloat16, 4))
    r = dg.layer_norm(x, w, b)
    a = dg.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        c = dg.layer_norm_backward(dy, x, w, r.mean, r.rstd, stream=s)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_refusals():
    x = torch.zeros(4, 200, device="cuda")
    w = torch.ones(200, device="cuda")
    with pytest.raises(ValueError):
        dg.layer_norm(x, w, out_format="fp8")      # 200 columns are no whole groups
    with pytest.raises(ValueError):
        dg.layer_norm(x, w, out_format="bf16")
    with pytest.raises(ValueError):
        dg.layer_norm(x, w[:100])
    with pytest.raises(TypeError):
        dg.layer_norm(x.double(), w)
    with pytest.raises(TypeError):
        dg.layer_norm(x, w.to(torch.float16))
    with pytest.raises(ValueError):
        dg.layer_norm(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(dg.DGError):
        dg.layer_norm(x, w, eps=-1.0)
    r = dg.layer_norm(x, w)
    with pytest.raises(ValueError):
        dg.layer_norm_backward(x[:2], x, w, r.mean, r.rstd)
    with pytest.raises(ValueError):
        dg.layer_norm_backward(x, x, w, r.mean[:2], r.rstd)
    with pytest.raises(TypeError):
        dg.layer_norm_backward(x.half(), x, w, r.mean, r.rstd)
    odd = torch.zeros(4, 130, device="cuda", dtype=torch.bfloat16)[:, 1:129]
    with pytest.raises(dg.DGError):                # 8-bit results need 16-byte aligned rows
        dg.layer_norm(odd, torch.ones(128, device="cuda"), out_format="fp8")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(40, 9), (700, 37), (513, 255), (300, 2047), (90, 2049), (60, 4414), (20, 7167)])
@pytest.mark.parametrize("left,right", [(0, 0), (1, 0), (3, 2), (2, 4)])
def test_rows_at_any_offset(rows, cols, dtype, left, right):
    """Views whose rows start at every kind of byte offset, between NaNs that
    must not be taken in; what lies around the results is not written."""
    x, w, b, dy = _inputs(rows, cols, dtype, rows + cols + left)
    def wide(t):
        big = torch.full((rows * (left + cols + right) + left + right + 8,), float("nan"), dtype=dtype, device="cuda")
        view = big[left:left + rows * (left + cols + right)].view(rows, -1)[:, :cols]
        view.copy_(t)
        return view
    xv, dv = wide(x), wide(dy)
    r = dg.layer_norm(xv, w.cuda(), b.cuda(), eps=EPS)
    _check_forward(r, x, w, b)
    _check_backward(dg.layer_norm_backward(dv, xv, w.cuda(), r.mean, r.rstd), x, w, dy, r)


# Enough rows that every SM works on several rounds of them, by each form of
# lanes (8, 16 and 32 values, rows of one and of several warps, whole or not).
MANY = [(9001, 40), (5001, 384), (4001, 1024), (2501, 2176), (1003, 7168)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", MANY + [(4002, 1001), (3001, 1514), (1100, 7001)])
def test_many_rows(rows, cols, dtype):
    x, w, b, dy = _inputs(rows, cols, dtype, rows + 7 * cols)
    r = dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    _check_forward(r, x, w, b)
    _check_backward(dg.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), r.mean, r.rstd), x, w, dy, r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(9001, 128)] + MANY[1:])
def test_many_rows_to_8_bits(rows, cols, dtype):
    x, w, b, _ = _inputs(rows, cols, dtype, rows + 5 * cols)
    _check_forward(dg.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=EPS, out_format="fp8"), x, w, b)


@pytest.mark.parametrize("rows,cols", [(4000, 1000), (4000, 1001), (1000, 7168)])
def test_rows_that_are_not_finite_stay_alone(rows, cols):
    """A row of NaN or with an infinity spoils its own results and no others."""
    x, w, b, dy = (t.cuda() for t in _inputs(rows, cols, torch.bfloat16, 21))
    bad = x.clone()
    rows_hit = list(range(5, rows, 97))
    for i in rows_hit:
        if i % 2:
            bad[i] = float("nan")
        else:
            bad[i, i % cols] = float("inf")
    fine = torch.ones(rows, dtype=torch.bool, device="cuda")
    fine[rows_hit] = False
    a, c = dg.layer_norm(x, w, b), dg.layer_norm(bad, w, b)
    assert torch.equal(a.y[fine], c.y[fine]) and torch.equal(a.mean[fine], c.mean[fine])
    assert torch.equal(a.rstd[fine], c.rstd[fine])
    assert not torch.isfinite(c.mean[~fine]).any()
    p = dg.layer_norm_backward(dy, x, w, a.mean, a.rstd)[0]
    q = dg.layer_norm_backward(dy, bad, w, c.mean, c.rstd)[0]
    assert torch.equal(p[fine], q[fine])
    if cols % 128 == 0:
        a, c = dg.layer_norm(x, w, b, out_format="fp8"), dg.layer_norm(bad, w, b, out_format="fp8")
        assert torch.equal(a.y.view(torch.uint8)[fine], c.y.view(torch.uint8)[fine])
        assert torch.equal(a.sf[:, :rows].t()[fine], c.sf[:, :rows].t()[fine])
