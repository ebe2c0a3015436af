"""Torch-facing wrappers of the serving operators: a whole mixture-of-experts
layer for a few tokens, and products of 8-bit integers with a scale per token
and channel.

Argument marshalling only, as in ``api``: every step of the computation runs
in libdg.so's kernels; there is no fallback.  With ``stream=`` a call runs as
under ``torch.cuda.stream(stream)``: its results and workspaces are that
stream's memory.
"""
import ctypes as C
import functools
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .api import FP8_DTYPES, _check, _need, _on_current_device, _under, sf_packed_shape
from .feedforward import _BF16, _DTYPES, _E4M3, _F32, _I32, _activation, _contiguous, _device, _handle, _p, _usual

SCORES = {"softmax": _lib.DG_SCORE_SOFTMAX, "sigmoid": _lib.DG_SCORE_SIGMOID}
_I8 = torch.int8
_OUT = {torch.bfloat16: _lib.DG_DTYPE_BF16, torch.float16: _lib.DG_DTYPE_FP16}


def _rows(t: torch.Tensor, name: str, shape, dtypes) -> int:
    """The row stride of a matrix of this shape with unit column stride, checked."""
    _need(t, name, dtypes, 2)
    if tuple(t.shape) != tuple(shape) or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("%s must be %s with unit column stride" % (name, tuple(shape)))
    if t.shape[0] < 2:
        return t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise ValueError("%s has rows that overlap" % name)
    return t.stride(0)


# ---------------------------------------------------------------- mixture of experts


class MoeOutput(NamedTuple):
    y: torch.Tensor        # BF16 [T, D]
    experts: torch.Tensor  # int32 [T, top_k], best first; -1 in rows that are no tokens
    weights: torch.Tensor  # FP32 [T, top_k]


@functools.lru_cache(maxsize=1024)
def _moe_workspace(tokens: int, d: int, f: int, experts: int, top_k: int) -> int:
    need = C.c_uint64(0)
    _check(_lib.lib().dg_fp8_moe_few_tokens_workspace_size(tokens, d, f, experts, top_k, C.byref(need)),
           "dg_fp8_moe_few_tokens_workspace_size")
    return need.value


def fp8_moe_few_tokens(x: torch.Tensor, router: torch.Tensor, up: torch.Tensor, up_sf: torch.Tensor,
                       down: torch.Tensor, down_sf: torch.Tensor, top_k: int,
                       router_bias: Optional[torch.Tensor] = None, score: str = "softmax", renormalize: bool = True,
                       scale: float = 1.0, activation: str = "silu", c: Optional[torch.Tensor] = None,
                       num_tokens: Optional[torch.Tensor] = None, d: Optional[torch.Tensor] = None,
                       stream=None) -> MoeOutput:
    """A whole mixture-of-experts layer for up to 64 tokens, gate included:
    y = c + sum over each token's top_k experts of weight act(x Wg^T) (x Wu^T) Wd^T.

    x BF16 [T, D]; router FP32 or BF16 [E, D] (logits x router^T); up E4M3
    [E, 2F, D] (gate rows, then up rows) and down E4M3 [E, D, F] with packed
    UE8M0 scales, as the grouped GEMMs take them; D and F multiples of 128.
    score "softmax" (over the experts) or "sigmoid"; the experts with the largest
    logits are chosen (with router_bias FP32 [E], "sigmoid" only: the largest
    score + bias), ties to the lowest index; their scores, divided by their
    sum with renormalize, times scale, are the weights.  Activations are not
    rounded to 8 bits.

    c: BF16 [T, D] to add (the residual).  num_tokens: int32 [1] on the device;
    rows past it are not computed and not written (a captured graph's padded
    batch).  d: a preallocated y; it may be x, or c with c's strides."""
    if stream is not None:
        return MoeOutput(*_under(stream, fp8_moe_few_tokens, x, router, up, up_sf, down, down_sf, top_k, router_bias,
                                 score, renormalize, scale, activation, c, num_tokens, d))
    act = _activation(activation)
    if score not in SCORES:
        raise ValueError("score %r not in %s" % (score, sorted(SCORES)))
    dev = _device()
    t, dim = x.shape if x.dim() == 2 else (0, 0)
    e, f2 = up.shape[:2] if up.dim() == 3 else (0, 0)
    f = f2 // 2
    ldx = ldc = ldy = dim
    kp, fp = (dim + 511) // 512, (f + 511) // 512
    usual = f2 % 2 == 0 and e and f and dim % 128 == 0 and f % 128 == 0 and _usual(x, _BF16, (t, dim), dev) and \
        router.dtype in (_F32, _BF16) and _usual(router, router.dtype, (e, dim), dev) and \
        _usual(up, _E4M3, (e, f2, dim), dev) and _usual(up_sf, _I32, (e, kp, f2), dev) and \
        _usual(down, _E4M3, (e, dim, f), dev) and _usual(down_sf, _I32, (e, fp, dim), dev) and \
        (router_bias is None or _usual(router_bias, _F32, (e,), dev)) and \
        (c is None or _usual(c, _BF16, (t, dim), dev)) and (num_tokens is None or _usual(num_tokens, _I32, (1,), dev)) and \
        (d is None or _usual(d, _BF16, (t, dim), dev))
    if not usual:
        _need(x, "x", (_BF16,), 2)
        _need(router, "router", (_F32, _BF16), 2)
        _need(up, "up", FP8_DTYPES, 3)
        _need(down, "down", FP8_DTYPES, 3)
        _need(up_sf, "up_sf", (_I32,), 3)
        _need(down_sf, "down_sf", (_I32,), 3)
        if f2 % 2 or tuple(up.shape) != (e, f2, dim) or tuple(down.shape) != (e, dim, f) or \
                tuple(router.shape) != (e, dim):
            raise ValueError("router %s, up %s and down %s do not belong to x %s: expected [E, D], [E, 2F, D], [E, D, F]"
                             % (tuple(router.shape), tuple(up.shape), tuple(down.shape), tuple(x.shape)))
        if dim % 128 or f % 128:
            raise ValueError("D and F must be multiples of 128, got %d and %d" % (dim, f))
        if tuple(up_sf.shape) != sf_packed_shape(f2, dim, e) or tuple(down_sf.shape) != sf_packed_shape(dim, f, e):
            raise ValueError("scale shapes %s / %s, expected %s / %s" % (
                tuple(up_sf.shape), tuple(down_sf.shape), sf_packed_shape(f2, dim, e), sf_packed_shape(dim, f, e)))
        if router_bias is not None:
            _need(router_bias, "router_bias", (_F32,), 1)
            if router_bias.numel() != e:
                raise ValueError("router_bias must be [%d]" % e)
        if num_tokens is not None:
            _need(num_tokens, "num_tokens", (_I32,), 1)
            if num_tokens.numel() != 1:
                raise ValueError("num_tokens must be [1]")
        _contiguous(router=router, up=up, up_sf=up_sf, down=down, down_sf=down_sf, router_bias=router_bias)
        ldx = _rows(x, "x", (t, dim), (_BF16,))
        if c is not None:
            ldc = _rows(c, "c", (t, dim), (_BF16,))
        if d is not None:
            ldy = _rows(d, "d", (t, dim), (_BF16,))
        _on_current_device(None, x, router, up, up_sf, down, down_sf, router_bias, c, num_tokens, d)
    if router_bias is not None and score != "sigmoid":
        raise ValueError("router_bias goes with score 'sigmoid'")
    if t > 64:
        raise ValueError("%d tokens: at most 64 (more go through the grouped layouts)" % t)
    need = _moe_workspace(t, dim, f, e, int(top_k))
    device = x.device
    y = torch.empty((t, dim), dtype=_BF16, device=device) if d is None else d
    experts = torch.empty((t, top_k), dtype=_I32, device=device)
    weights = torch.empty((t, top_k), dtype=_F32, device=device)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    rc = _lib.lib().dg_fp8_moe_few_tokens(
        x.data_ptr(), ldx, router.data_ptr(), _DTYPES[router.dtype], _p(router_bias), up.data_ptr(), up_sf.data_ptr(),
        down.data_ptr(), down_sf.data_ptr(), _p(c), ldc, _p(num_tokens), y.data_ptr(), ldy, experts.data_ptr(),
        weights.data_ptr(), ws.data_ptr(), need, t, dim, f, e, int(top_k), SCORES[score], 1 if renormalize else 0,
        float(scale), act, _handle(dev))
    if rc:
        _check(rc, "dg_fp8_moe_few_tokens")
    return MoeOutput(y, experts, weights)


# ---------------------------------------------------------------- 8-bit integers


def quantize_int8(x: torch.Tensor, out=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """FP32, BF16 or FP16 [rows, cols] -> (int8 codes [rows, cols], FP32 scales
    [rows]): scale = amax / 127 of the row, code = the integer nearest to
    127 x / amax, ties to even.  A row with an infinity or NaN has a NaN scale and
    codes 0.  The operands of int8_gemm_nt: activations by token, weights by
    channel.  out=(q, scales) writes into preallocated contiguous tensors."""
    if stream is not None:
        return _under(stream, quantize_int8, x, out)
    dev = _device()
    rows, cols = x.shape if x.dim() == 2 else (0, 0)
    ld = cols
    if cols < 1 or x.dtype not in _DTYPES or not _usual(x, x.dtype, (rows, cols), dev) or out is not None:
        _need(x, "x", tuple(_DTYPES), 2)
        if cols < 1:
            raise ValueError("x needs at least one column")
        ld = _rows(x, "x", (rows, cols), tuple(_DTYPES))
        _on_current_device(None, x, *(out or ()))
    if out is None:
        q = torch.empty((rows, cols), dtype=_I8, device=x.device)
        scales = torch.empty(rows, dtype=_F32, device=x.device)
    else:
        q, scales = out
        _need(q, "q", (_I8,), 2)
        _need(scales, "scales", (_F32,), 1)
        if tuple(q.shape) != (rows, cols) or scales.numel() != rows:
            raise ValueError("out must be [%d, %d] / [%d]" % (rows, cols, rows))
        _contiguous(q=q, scales=scales)
    rc = _lib.lib().dg_quantize_int8(x.data_ptr(), _DTYPES[x.dtype], q.data_ptr(), scales.data_ptr(), rows, cols, ld,
                                     _handle(dev))
    if rc:
        _check(rc, "dg_quantize_int8")
    return q, scales


def int8_gemm_nt(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                 d: Optional[torch.Tensor] = None, c: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """D = C + sa sb (A @ B.T): A int8 [M, K] with FP32 scales [M], B int8 [N, K]
    with FP32 scales [N] (quantize_int8's), K % 16 == 0, any M and N.

    out_dtype BF16 or FP16, also c's and d's; c may be d.  Products are exact,
    sums FP32: exact within 2^24, always up to K = 1024."""
    if stream is not None:
        return _under(stream, int8_gemm_nt, a, sa, b, sb, d, c, out_dtype)
    if out_dtype not in _OUT:
        raise TypeError("out_dtype %s is not bfloat16 or float16" % out_dtype)
    dev = _device()
    m, k = a.shape if a.dim() == 2 else (0, 0)
    n = b.shape[0] if b.dim() == 2 else 0
    lda = ldb = k
    ldc = ldd = n
    if not _usual(a, _I8, (m, k), dev) or not _usual(b, _I8, (n, k), dev) or not _usual(sa, _F32, (m,), dev) or \
            not _usual(sb, _F32, (n,), dev) or k < 1 or not (c is None or _usual(c, out_dtype, (m, n), dev)) or \
            not (d is None or _usual(d, out_dtype, (m, n), dev)):
        _need(a, "a", (_I8,), 2)
        _need(b, "b", (_I8,), 2)
        _need(sa, "sa", (_F32,), 1)
        _need(sb, "sb", (_F32,), 1)
        if b.shape[1] != k:
            raise ValueError("K mismatch: a %s, b %s" % (tuple(a.shape), tuple(b.shape)))
        if sa.numel() != m or sb.numel() != n:
            raise ValueError("scales must be [%d] and [%d], got %s and %s" % (m, n, tuple(sa.shape), tuple(sb.shape)))
        _contiguous(sa=sa, sb=sb)
        lda, ldb = _rows(a, "a", (m, k), (_I8,)), _rows(b, "b", (n, k), (_I8,))
        if c is not None:
            ldc = _rows(c, "c", (m, n), (out_dtype,))
        if d is not None:
            ldd = _rows(d, "d", (m, n), (out_dtype,))
        _on_current_device(None, a, sa, b, sb, c, d)
    if d is None:
        d = torch.empty((m, n), dtype=out_dtype, device=a.device)
    rc = _lib.lib().dg_int8_gemm_nt(a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), _p(c), d.data_ptr(), m, n,
                                    k, lda, ldb, ldc, ldd, _OUT[out_dtype], _handle(dev))
    if rc:
        _check(rc, "dg_int8_gemm_nt")
    return d
