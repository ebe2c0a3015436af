"""A pre-norm gated feed-forward block on this library's kernels, for training
and for serving, dense and as MoE experts:

    n = layer_norm(x),  h = act(n Wg^T) * (n Wu^T),  y = x + h Wd^T

Forward: the norm writes n as the first product's E4M3 operand, which is at the
same time the 8-bit checkpoint of n; the gated product writes h as the second
product's operand and, in training, keeps [g | u] in 8 bits; the second
product adds x as its C.  Backward: dh = dy Wd; the gated backward pass turns dh
and the checkpoint into the operands of dn = [dg | du] W and of the weights'
gradients, for which the saved n and dy are requantised over columns.

``python -m moe_grouped_gemm_fp8_gb300.block`` trains a small one on the GPU.
"""
from typing import NamedTuple, Optional

import torch

from .api import (fp8_gemm_nn, fp8_gemm_nt, k_grouped_fp8_gemm_tn_contiguous, m_grouped_fp8_gemm_nt_contiguous,
                  m_grouped_fp8_gemm_nt_masked, quantize_fp8)
from .feedforward import (fp8_gated_backward, fp8_gated_gemm_nt, layer_norm, layer_norm_backward,
                          m_grouped_fp8_gated_gemm_nt_contiguous, m_grouped_fp8_gated_gemm_nt_masked,
                          requantize_fp8_cols)
from .serving import MoeOutput, fp8_moe_few_tokens


class Weight(NamedTuple):
    """An FP32 weight's E4M3 codes with one scale per 128 x 128 block, as the
    NT products read it and (t, t_sf) transposed.  The dense backward products
    read q in place (MN-major) and need only t_sf."""
    q: torch.Tensor
    sf: torch.Tensor
    t: Optional[torch.Tensor]
    t_sf: torch.Tensor

    @staticmethod
    def of(w: torch.Tensor, keep_transposed: bool) -> "Weight":
        q, sf = quantize_fp8(w, 128)
        t, t_sf = quantize_fp8(w.transpose(-1, -2).contiguous(), 128)
        return Weight(q, sf, t if keep_transposed else None, t_sf)


class Saved(NamedTuple):
    """What a forward pass keeps for its backward pass."""
    x: torch.Tensor         # BF16 (the block's input; the norm's backward pass reads it)
    n: torch.Tensor         # the normed activation: E4M3 codes and packed scales
    n_sf: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    gu: torch.Tensor        # [g | u]: E4M3 codes and packed scales
    gu_sf: torch.Tensor


class Gradients(NamedTuple):
    x: torch.Tensor         # BF16
    up: torch.Tensor        # FP32 [2F, D] (experts: [G, 2F, D])
    down: torch.Tensor      # FP32 [D, F] (experts: [G, D, F])
    norm_weight: torch.Tensor
    norm_bias: torch.Tensor


class GatedFeedForward:
    """The dense block.  up: FP32 [2F, D] (gate rows, then up rows), down: FP32
    [D, F]; D and F multiples of 128.  The E4M3 weights are laid out once;
    after a change of the FP32 weights call ``load``."""

    def __init__(self, up: torch.Tensor, down: torch.Tensor, norm_weight: torch.Tensor, norm_bias: torch.Tensor,
                 activation: str = "silu", eps: float = 1e-5):
        self.norm_weight, self.norm_bias = norm_weight, norm_bias
        self.activation, self.eps = activation, eps
        self.load(up, down)

    def load(self, up: torch.Tensor, down: torch.Tensor) -> None:
        self.up = Weight.of(up, keep_transposed=False)
        self.down = Weight.of(down, keep_transposed=False)

    def forward(self, x: torch.Tensor, training: bool = False):
        """x BF16 [M, D] -> (y BF16 [M, D], Saved or None); any M, one token upwards."""
        n = layer_norm(x, self.norm_weight, self.norm_bias, eps=self.eps, out_format="fp8")
        r = fp8_gated_gemm_nt(n.y, n.sf, self.up.q, self.up.sf, activation=self.activation, out_format="fp8",
                              checkpoint=training)
        y = fp8_gemm_nt(r.h, r.h_sf, self.down.q, self.down.sf, c=x)
        return y, Saved(x, n.y, n.sf, n.mean, n.rstd, r.checkpoint, r.checkpoint_sf) if training else None

    def backward(self, dy: torch.Tensor, saved: Saved) -> Gradients:
        """dy BF16 [M, D] (contiguous) and a forward pass's Saved -> the gradients."""
        rows = torch.full((1,), (dy.shape[0] + 127) // 128 * 128, dtype=torch.int32, device=dy.device)
        d, d_sf = quantize_fp8(dy, 1)
        dh = fp8_gemm_nn(d, d_sf, self.down.q, self.down.t_sf)                    # dy [M, D] @ down [D, F]
        g = fp8_gated_backward(dh, saved.gu, saved.gu_sf, activation=self.activation)
        dn = fp8_gemm_nn(g.q, g.sf, self.up.q, self.up.t_sf)                      # [dg | du] [M, 2F] @ up [2F, D]
        n_cols, n_sf = requantize_fp8_cols(saved.n, saved.n_sf)
        d_cols, d_cols_sf = requantize_fp8_cols(d, d_sf)
        up = k_grouped_fp8_gemm_tn_contiguous(g.q_cols, g.sf_cols, n_cols, n_sf, rows)[0]
        down = k_grouped_fp8_gemm_tn_contiguous(d_cols, d_cols_sf, g.h_cols, g.h_sf_cols, rows)[0]
        dx, dw, db = layer_norm_backward(dn, saved.x, self.norm_weight, saved.mean, saved.rstd)
        return Gradients(dx.add_(dy), up, down, dw, db)


class GatedExperts:
    """The block's products as MoE experts, without norm and residual: up FP32
    [G, 2F, D], down FP32 [G, D, F].  Tokens come as E4M3 rows with packed
    scales (layer_norm or quantize_fp8), routed by the library's contiguous
    (training, prefill) or masked (decode) layout."""

    def __init__(self, up: torch.Tensor, down: torch.Tensor, activation: str = "silu"):
        self.activation = activation
        self.up = Weight.of(up, keep_transposed=True)
        self.down = Weight.of(down, keep_transposed=True)

    def forward(self, x: torch.Tensor, x_sf: torch.Tensor, m_indices: torch.Tensor, training: bool = False):
        """(y BF16 [m_sum, D], checkpoint or None); padding rows of y are not written."""
        r = m_grouped_fp8_gated_gemm_nt_contiguous(x, x_sf, self.up.q, self.up.sf, m_indices,
                                                   activation=self.activation, out_format="fp8", checkpoint=training)
        y = m_grouped_fp8_gemm_nt_contiguous(r.h, r.h_sf, self.down.q, self.down.sf, m_indices)
        return y, (r.checkpoint, r.checkpoint_sf) if training else None

    def decode(self, x: torch.Tensor, x_sf: torch.Tensor, masked_m: torch.Tensor, expected_m: int = 0) -> torch.Tensor:
        """The masked layout: x E4M3 [G, max_m, D] -> y BF16 [G, max_m, D]; rows past masked_m are not written."""
        r = m_grouped_fp8_gated_gemm_nt_masked(x, x_sf, self.up.q, self.up.sf, masked_m, expected_m=expected_m,
                                               activation=self.activation, out_format="fp8")
        return m_grouped_fp8_gemm_nt_masked(r.h, r.h_sf, self.down.q, self.down.sf, masked_m, expected_m=expected_m)

    def few_tokens(self, x: torch.Tensor, router: torch.Tensor, top_k: int, **options) -> MoeOutput:
        """The whole layer for up to 64 tokens, gate included: x BF16 [T, D], router
        [G, D]; options as fp8_moe_few_tokens takes them (c: the residual)."""
        return fp8_moe_few_tokens(x, router, self.up.q, self.up.sf, self.down.q, self.down.sf, top_k,
                                  activation=self.activation, **options)

    def backward(self, dy: torch.Tensor, x: torch.Tensor, x_sf: torch.Tensor, checkpoint, m_indices: torch.Tensor,
                 ks: torch.Tensor):
        """dy BF16 [m_sum, D] -> (dx BF16 [m_sum, D], d_up, d_down); ks int32 [G]:
        rows of each expert, padding included.  Padding rows of dy, x and the
        checkpoint may hold anything; those of dx are not written."""
        d, d_sf = quantize_fp8(dy, 1)
        dh = m_grouped_fp8_gemm_nt_contiguous(d, d_sf, self.down.t, self.down.t_sf, m_indices)
        g = fp8_gated_backward(dh, checkpoint[0], checkpoint[1], m_indices=m_indices, activation=self.activation)
        dx = m_grouped_fp8_gemm_nt_contiguous(g.q, g.sf, self.up.t, self.up.t_sf, m_indices)
        x_cols, x_cols_sf = requantize_fp8_cols(x, x_sf, m_indices=m_indices)
        d_cols, d_cols_sf = requantize_fp8_cols(d, d_sf, m_indices=m_indices)
        d_up = k_grouped_fp8_gemm_tn_contiguous(g.q_cols, g.sf_cols, x_cols, x_cols_sf, ks)
        d_down = k_grouped_fp8_gemm_tn_contiguous(d_cols, d_cols_sf, g.h_cols, g.h_sf_cols, ks)
        return dx, d_up, d_down


def main(steps: int = 40, m: int = 512, d: int = 256, f: int = 512, lr: float = 0.5) -> list:
    """Fits a block to another one's outputs by gradient descent; the losses."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    new = lambda: [rand(2 * f, d) * d ** -0.5, rand(d, f) * f ** -0.5]  # noqa: E731
    one, zero = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    target = GatedFeedForward(*new(), one, zero)
    up, down = new()
    w, b = one.clone(), zero.clone()
    block = GatedFeedForward(up, down, w, b)
    x = rand(m, d).to(torch.bfloat16)
    want, _ = target.forward(x)
    losses = []
    for _ in range(steps):
        y, saved = block.forward(x, training=True)
        diff = (y - want).float()
        losses.append(float(diff.square().mean()))
        g = block.backward((diff * (2.0 / m)).to(torch.bfloat16), saved)
        for p, dp in ((up, g.up), (down, g.down), (w, g.norm_weight), (b, g.norm_bias)):
            p.sub_(lr / 64 * dp)
        block.load(up, down)
    return losses


if __name__ == "__main__":
    for i, loss in enumerate(main()):
        if i % 8 == 0 or i == 39:
            print("step %2d  loss %.4f" % (i, loss))
