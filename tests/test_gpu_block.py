"""The feed-forward block end to end: forward and gradients, dense and as
experts, against FP64 on the FP32 weights and BF16 inputs."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
from moe_grouped_gemm_fp8_gb300 import block
import _fp8ref as R

pytestmark = pytest.mark.gpu

# Each product's operands are rounded to E4M3 (4 bits of significand): an
# independent relative error of at most 2^-4, about 2^-5.2 (2.7%) root mean
# square, per operand element.  A product averages such errors of its terms, so
# its own relative error is about 2.7% per operand rounded, and the few stages
# a result goes through (at most 6 roundings on the longest path, dW) add in
# squares: 2.7% sqrt(6) = 6.6%.  Twice that is allowed, in the 2-norm.
TOL = 0.13


def _rel(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def _d(t):
    return t.double().cpu().numpy()


def _reference(x, dy, up, down, w, b, activation, eps=1e-5):
    f = up.shape[0] // 2
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    xh = (x - mean) * rstd
    n = xh * w + b
    gu = n @ up.T
    g, u = gu[:, :f], gu[:, f:]
    h = R.act(g, activation) * u
    y = x + h @ down.T
    dh = dy @ down
    dgu = np.concatenate([dh * u * R.act_grad(g, activation), dh * R.act(g, activation)], 1)
    dn = dgu @ up
    t = dn * w
    dx = dy + rstd * (t - t.mean(1, keepdims=True) - xh * (t * xh).mean(1, keepdims=True))
    return y - x, dict(x=dx, up=dgu.T @ n, down=dy.T @ h, norm_weight=(dn * xh).sum(0), norm_bias=dn.sum(0))


@pytest.mark.parametrize("activation", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m,d,f", [(1, 256, 128), (77, 256, 384), (300, 512, 640)])
def test_block(m, d, f, activation):
    gen = torch.Generator().manual_seed(m + d)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    up, down = rand(2 * f, d) * d ** -0.5, rand(d, f) * f ** -0.5
    w, b = 1 + 0.1 * rand(d), 0.1 * rand(d)
    x, dy = rand(m, d).to(torch.bfloat16), rand(m, d).to(torch.bfloat16)
    net = block.GatedFeedForward(up.cuda(), down.cuda(), w.cuda(), b.cuda(), activation=activation)
    y, none = net.forward(x.cuda())
    y2, saved = net.forward(x.cuda(), training=True)
    assert none is None and torch.equal(y, y2)
    g = net.backward(dy.cuda(), saved)
    added, want = _reference(*(t.double().numpy() for t in (x, dy, up, down, w, b)), activation)
    assert _rel(_d(y) - x.double().numpy(), added) < TOL
    for name, value in want.items():
        assert _rel(_d(getattr(g, name)), value) < TOL, name
    assert dg.get_device_error()[0] == 0


def test_training_reduces_the_loss():
    losses = block.main(steps=24)
    assert losses[-1] < 0.7 * losses[0], losses


def test_experts():
    counts, d, f = [150, 0, 128, 33], 256, 384
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    up, down = rand(4, 2 * f, d) * d ** -0.5, rand(4, d, f) * f ** -0.5
    index, spans, ks = [], [], []
    for g, c in enumerate(counts):
        spans.append((g, len(index), c))
        index += [g] * c + [-1] * (-c % 128)
        ks.append(c + -c % 128)
    m = len(index)
    index = torch.tensor(index, dtype=torch.int32).cuda()
    x, dy = rand(m, d).cuda(), rand(m, d).to(torch.bfloat16).cuda()
    q, sf = dg.quantize_fp8(x, 1)
    dy[index < 0] = float("nan")
    net = block.GatedExperts(up.cuda(), down.cuda())
    y, kept = net.forward(q, sf, index, training=True)
    dx, d_up, d_down = net.backward(dy, q, sf, kept, index, torch.tensor(ks, dtype=torch.int32).cuda())
    for g, row, c in spans:
        if c == 0:
            assert not d_up[g].any() and not d_down[g].any()
            continue
        s = slice(row, row + c)
        xv, dyv, U, D = _d(x[s]), _d(dy[s]), _d(up[g]), _d(down[g])
        gu = xv @ U.T
        a, u = R.act(gu[:, :f], "silu"), gu[:, f:]
        dh = dyv @ D
        dgu = np.concatenate([dh * u * R.act_grad(gu[:, :f], "silu"), dh * a], 1)
        assert _rel(_d(y[s]), (a * u) @ D.T) < TOL
        assert _rel(_d(dx[s]), dgu @ U) < TOL
        assert _rel(_d(d_up[g]), dgu.T @ xv) < TOL
        assert _rel(_d(d_down[g]), dyv.T @ (a * u)) < TOL
    # the same tokens in the masked layout give the same rows
    cap = 256
    xm = torch.zeros(4, cap, d, device="cuda")
    for g, row, c in spans:
        xm[g, :c] = x[row:row + c]
    qm, sm = dg.quantize_fp8(xm, 1)
    ym = net.decode(qm, sm, torch.tensor(counts, dtype=torch.int32).cuda(), expected_m=64)
    for g, row, c in spans:
        assert _rel(_d(ym[g, :c]), _d(y[row:row + c])) < 1e-2 if c else True
    assert dg.get_device_error()[0] == 0
