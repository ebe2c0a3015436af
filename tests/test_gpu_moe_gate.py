"""Weights of the experts for logits far from 0, against the logistic function in 64 bits."""
import pytest
import torch

import moe_grouped_gemm_fp8_gb300 as dg
import test_gpu_moe_few_tokens as M

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# Steps u = 2^-24 of a weight: expf's 2 of FP32's last place are 4 u, the logit's low word 1; of 1 + exp(-|l|) 2 for
# expf (it is at most half of the sum) and 1; the quotient 1: 9. Of the sum of up to 16 as much and 5 additions; the
# last quotient and the scale 2: 25 in all, less than 2^-19. Below 2^-126 expf's 2, the low word's and the quotient's
# halves are of FP32's smallest, twice those divided by a sum of 1/2, and half of one again: less than 8.
STEP, SMALLEST = 2.0 ** -19, 2.0 ** -146


def check(x, r, w, k, **kw):
    got = dg.fp8_moe_few_tokens(x, r, *w, k, score="sigmoid", **{("router_bias" if n == "bias" else n): v for n, v in kw.items()})
    y, chosen, ws, off = M.reference(x, r, w, k, score="sigmoid", **kw)
    assert torch.equal(got.experts.long(), chosen)
    far = (got.weights.double() - ws).abs()
    assert (far <= ws * STEP + SMALLEST).all(), (got.weights, ws)
    # weights that vanish leave y at BF16's smallest
    assert ((got.y.double() - y).abs() <= off + 2.0 ** -133).all()
    assert dg.get_device_error()[0] == 0


@pytest.mark.parametrize("router", [F32, BF16])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("at", [60, -20, -30, -60, -80, -88, -90, -200, -300])
def test_logits_around(at, bias, renormalize, router):
    t, d, f, e, k = 3, 256, 128, 12, 4
    w, x, r = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d, router)
    x[:, 0], r[:, 0] = 1.0, at
    b = 0.1 * torch.randn(e, generator=torch.Generator().manual_seed(3)).cuda() if bias else None
    check(x, r, w, k, bias=b, renormalize=renormalize)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("best", [5.0, -0.5, -40.0, -85.0, -110.0])
def test_chosen_logits_far_apart(best, renormalize):
    """The choice by the bias takes logits up to hundreds below the largest of the chosen."""
    t, d, f, e, k = 9, 256, 128, 20, 16
    w, x, r = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d)
    x[:, 0] = 1.0
    r[:, 0] = best - torch.tensor([0, 0.25, 1, 4, 9, 16, 17, 30, 50, 70, 80, 86, 87, 88, 89, 100, 103, 110, 200, 400]).cuda()
    b = torch.linspace(3, 1, e).cuda()
    check(x, r, w, k, bias=b, renormalize=renormalize)


def test_one_chosen_expert_has_all_the_weight():
    t, d, f, e = 4, 256, 128, 6
    w, x, r = M.weights(e, d, f), M.tokens(t, d), M.gate(e, d)
    x[:, 0], r[:, 0] = 1.0, -500.0
    got = dg.fp8_moe_few_tokens(x, r, *w, 1, score="sigmoid")
    assert (got.weights == 1).all() and torch.isfinite(got.y.float()).all()


def test_infinite_logits():
    """+inf: the logistic function is 1; -inf: 0, and no number where it is divided by itself."""
    t, d, f, e, k = 2, 128, 128, 5, 3
    w, x = M.weights(e, d, f), torch.zeros(t, d, dtype=BF16, device="cuda")
    x[:, 0] = 1.0
    r = torch.zeros(e, d, device="cuda")
    inf = float("inf")
    for logits, weights in [([inf, 0.0, -inf, -inf, -inf], [1.0, 0.5, 0.0]), ([-1.0, -inf, -1.0, -inf, -inf], [None, None, 0.0]),
                            ([-inf] * 5, [0.0, 0.0, 0.0])]:
        r[:, 0] = torch.tensor(logits)
        got = dg.fp8_moe_few_tokens(x, r, *w, k, score="sigmoid", renormalize=False)
        for j, want in enumerate(weights):
            want = 1 / (1 + 2.718281828459045) if want is None else want
            assert ((got.weights[:, j].double() - want).abs() <= want * STEP).all()
        total = dg.fp8_moe_few_tokens(x, r, *w, k, score="sigmoid").weights
        if logits[0] == -inf:
            assert torch.isnan(total).all()
        else:
            assert ((total.double().sum(1) - 1).abs() <= 2.0 ** -18).all()
