"""Torch-facing wrappers of the operators around a feed-forward block's GEMMs:
8-bit activation checkpoints, the gated product's backward pass and layer norm.

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
from .api import (FP8_DTYPES, _check, _need, _on_current_device, _ptr, _raw_stream, _stream, _under, get_num_sms,
                  sf_packed_shape)

ACTIVATIONS = {"silu": _lib.DG_ACT_SILU, "gelu_tanh": _lib.DG_ACT_GELU_TANH}
_DTYPES = {torch.float32: _lib.DG_DTYPE_FP32, torch.bfloat16: _lib.DG_DTYPE_BF16,
           torch.float16: _lib.DG_DTYPE_FP16}


# Small calls are bound by this file: a tensor's attribute costs 0.1-0.2 us, an
# allocation 1-2 us.  So a call first asks only whether every argument is as it
# usually is (one expression a tensor); what is not goes through the full
# checks, which accept the unusual forms or say what is wrong.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_E4M3, _I32, _BF16, _F32 = torch.float8_e4m3fn, torch.int32, torch.bfloat16, torch.float32


def _usual(t, dtype, shape, dev) -> bool:
    """A contiguous tensor of this type and shape on the current device."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _sf(rows: int, cols: int):
    """sf_packed_shape(rows, cols) of a tensor without a group axis."""
    return (cols + 511) // 512, (rows + 3) // 4 * 4


def _handle(dev):
    """The current stream's; a call on an explicit one runs with that one current."""
    return _raw_stream(dev) if _raw_stream is not None else _stream(None)


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError("activation %r not in %s" % (name, sorted(ACTIVATIONS)))
    return ACTIVATIONS[name]


def _contiguous(**tensors) -> None:
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)


def _row_index(m_indices: Optional[torch.Tensor], rows: int) -> None:
    if m_indices is not None:
        _need(m_indices, "m_indices", (torch.int32,), 1)
        if m_indices.numel() != rows or not m_indices.is_contiguous():
            raise ValueError("m_indices must be contiguous [%d]" % rows)


# ---------------------------------------------------------------- 8-bit checkpoints


def dequantize_fp8(q: torch.Tensor, sf: torch.Tensor, dtype: torch.dtype = torch.bfloat16, out=None,
                   stream=None) -> torch.Tensor:
    """E4M3 codes [rows, cols] or [G, rows, cols] with packed 1x128 row-group
    scales -> the values they stand for, in BF16 or FP32."""
    if stream is not None:
        return _under(stream, dequantize_fp8, q, sf, dtype, out)
    if q.dim() not in (2, 3):
        raise ValueError("q must be [rows, cols] or [groups, rows, cols]")
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dtype %s is not float32 or bfloat16" % dtype)
    _need(q, "q", FP8_DTYPES, q.dim())
    _need(sf, "sf", (torch.int32,), q.dim())
    groups = q.shape[0] if q.dim() == 3 else 1
    rows, cols = q.shape[-2:]
    want = sf_packed_shape(rows, cols, groups if q.dim() == 3 else None)
    if tuple(sf.shape) != want:
        raise ValueError("scale shape %s, expected %s" % (tuple(sf.shape), want))
    _contiguous(q=q, sf=sf)
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    _need(out, "out", (dtype,), q.dim())
    if out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous %s" % (tuple(q.shape),))
    _on_current_device(None, q, sf, out)
    _check(_lib.lib().dg_dequantize_fp8(_ptr(q), _ptr(sf), _ptr(out), _DTYPES[dtype], groups, rows, cols,
                                        _stream(None)), "dg_dequantize_fp8")
    return out


def requantize_fp8_cols(q: torch.Tensor, sf: torch.Tensor, m_indices: Optional[torch.Tensor] = None,
                        out=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows saved in 8 bits as an operand of a weight gradient: E4M3 [rows,
    cols] with packed 1x128 row-group scales -> (E4M3 [align(rows, 128), cols],
    packed scales [ceil(rows/512), cols]) with one scale per 128 rows of each
    column, the layout of k_grouped_fp8_gemm_tn_contiguous's operands.

    m_indices: int32 [rows]; rows with a negative entry (padding of the
    contiguous layout) and rows past `rows` are zero in the result."""
    if stream is not None:
        return _under(stream, requantize_fp8_cols, q, sf, m_indices, out)
    dev = _device()
    rows, cols = q.shape if q.dim() == 2 else (0, 0)
    if out is not None or q.dim() != 2 or not _usual(q, _E4M3, q.shape, dev) or \
            not _usual(sf, _I32, _sf(rows, cols), dev) or \
            not (m_indices is None or _usual(m_indices, _I32, (rows,), dev)):
        _need(q, "q", FP8_DTYPES, 2)
        _need(sf, "sf", (torch.int32,), 2)
        if tuple(sf.shape) != sf_packed_shape(rows, cols):
            raise ValueError("scale shape %s, expected %s" % (tuple(sf.shape), sf_packed_shape(rows, cols)))
        _contiguous(q=q, sf=sf)
        _row_index(m_indices, rows)
        _on_current_device(None, q, sf, m_indices, *(out or ()))
    qc, sfc = _cols_out(out, (rows + 127) // 128 * 128, cols, q.device, "out")
    rc = _lib.lib().dg_requantize_fp8_cols(q.data_ptr(), sf.data_ptr(),
                                           None if m_indices is None else m_indices.data_ptr(), qc.data_ptr(),
                                           sfc.data_ptr(), rows, cols, _handle(dev))
    if rc:
        _check(rc, "dg_requantize_fp8_cols")
    return qc, sfc


def _codes_out(out, shape, sf_shape, device, name):
    """(codes, packed scales) to write: the caller's, checked, or new ones."""
    if out is None:
        return torch.empty(shape, dtype=_E4M3, device=device), torch.empty(sf_shape, dtype=_I32, device=device)
    q, sf = out
    _need(q, name + " codes", FP8_DTYPES, len(shape))
    _need(sf, name + " scales", (torch.int32,), len(sf_shape))
    if tuple(q.shape) != tuple(shape) or tuple(sf.shape) != tuple(sf_shape) or \
            not q.is_contiguous() or not sf.is_contiguous():
        raise ValueError("%s must be contiguous %s / %s" % (name, tuple(shape), tuple(sf_shape)))
    return q, sf


def _cols_out(out, rows128, cols, device, name):
    return _codes_out(out, (rows128, cols), _sf(cols, rows128), device, name)


# ---------------------------------------------------------------- gated product


class GatedOutput(NamedTuple):
    """Results of the gated products."""
    h: torch.Tensor                         # BF16, or E4M3 codes
    h_sf: Optional[torch.Tensor]            # packed 1x128 row-group scales of the codes, else None
    checkpoint: Optional[torch.Tensor]      # E4M3 codes of [g | u] with checkpoint=True, else None
    checkpoint_sf: Optional[torch.Tensor]   # their packed scales


def _gated_out(d, checkpoint, out_format, lead, f, device):
    """The tensors a gated product writes: rows `lead` + (m,), the caller's or new ones."""
    m = lead[-1]
    groups = lead[:-1]
    if out_format == "fp8":
        h, h_sf = _codes_out(d, lead + (f,), groups + _sf(m, f), device, "d")
    elif out_format == "bf16":
        h, h_sf = d, None
        if h is None:
            h = torch.empty(lead + (f,), dtype=_BF16, device=device)
        else:
            _need(h, "d", (_BF16,), len(lead) + 1)
            if tuple(h.shape) != lead + (f,) or h.stride(-1) != 1:
                raise ValueError("d must be %s with unit column stride" % (lead + (f,),))
    else:
        raise ValueError("out_format %r not in ('bf16', 'fp8')" % (out_format,))
    if (h_sf is not None or checkpoint) and f % 128:
        raise ValueError("8-bit results need F %% 128 == 0, got %d" % f)
    gu = gu_sf = None
    if checkpoint:
        gu, gu_sf = _codes_out(None if checkpoint is True else checkpoint, lead + (2 * f,),
                               groups + _sf(m, 2 * f), device, "checkpoint")
    return h, h_sf, gu, gu_sf


def _gated_operands(a, sfa, b, sfb, dev, lead_dims, b_dims):
    """(F, K) of a gated product's operands, checked; True when all are as
    usual (contiguous codes on the current device)."""
    k = a.shape[-1]
    n = b.shape[-2] if b.dim() == b_dims else 0
    if a.dim() == lead_dims + 1 and n % 2 == 0 and n and \
            _usual(a, _E4M3, a.shape, dev) and _usual(b, _E4M3, b.shape[:-1] + (k,), dev) and \
            _usual(sfa, _I32, tuple(a.shape[:-2]) + _sf(a.shape[-2], k), dev) and \
            _usual(sfb, _I32, tuple(b.shape[:-2]) + _sf(n, k), dev):
        return n // 2, k, True
    _need(a, "a", FP8_DTYPES, lead_dims + 1)
    _need(sfa, "sfa", (torch.int32,), lead_dims + 1)
    _need(b, "b", FP8_DTYPES, b_dims)
    _need(sfb, "sfb", (torch.int32,), b_dims)
    if b.shape[-1] != k or n % 2:
        raise ValueError("b must be [.., 2F, %d], got %s" % (k, tuple(b.shape)))
    ga = a.shape[0] if lead_dims == 2 else None
    gb = b.shape[0] if b_dims == 3 else None
    if tuple(sfa.shape) != sf_packed_shape(a.shape[-2], k, ga) or tuple(sfb.shape) != sf_packed_shape(n, k, gb):
        raise ValueError("scale shapes %s / %s, expected %s / %s" % (
            tuple(sfa.shape), tuple(sfb.shape), sf_packed_shape(a.shape[-2], k, ga), sf_packed_shape(n, k, gb)))
    _contiguous(sfa=sfa, sfb=sfb)
    if a.stride(-1) != 1 or b.stride(-1) != 1:
        raise ValueError("a and b need unit stride along K")
    return n // 2, k, False


def _p(t):
    return None if t is None else t.data_ptr()


def fp8_gated_gemm_nt(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor, d=None,
                      activation: str = "silu", out_format: str = "bf16", checkpoint=False,
                      stream=None) -> GatedOutput:
    """h = act(A Wg^T) * (A Wu^T) in one kernel: A [M, K] and B = [Wg; Wu]
    [2F, K] E4M3 with packed UE8M0 scales (as fp8_gemm_nt's).

    activation "silu" or "gelu_tanh".  out_format "bf16": h BF16 [M, F]
    (F % 8 == 0); "fp8": h as E4M3 codes with packed 1x128 row-group scales,
    the next GEMM's operand (F % 128 == 0).  checkpoint=True also keeps
    [g | u] in 8 bits for fp8_gated_backward (F % 128 == 0).  d, checkpoint:
    preallocated results (a BF16 tensor, or (codes, scales))."""
    if stream is not None:
        return _under(stream, fp8_gated_gemm_nt, a, sfa, b, sfb, d, activation, out_format, checkpoint)
    act = _activation(activation)
    dev = _device()
    f, k, usual = _gated_operands(a, sfa, b, sfb, dev, 1, 2)
    m = a.shape[0]
    h, h_sf, gu, gu_sf = _gated_out(d, checkpoint, out_format, (m,), f, a.device)
    lda = ldb = k
    ldh = f
    if not usual or d is not None or not isinstance(checkpoint, bool):
        _on_current_device(None, a, sfa, b, sfb, h, h_sf, gu, gu_sf)
        lda, ldb, ldh = a.stride(0) if m > 1 else k, b.stride(0), h.stride(0) if m > 1 else f
    rc = _lib.lib().dg_fp8_gated_gemm_nt(a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), h.data_ptr(),
                                         _p(h_sf), _p(gu), _p(gu_sf), m, f, k, lda, ldb, ldh, act,
                                         _handle(dev))
    if rc:
        _check(rc, "dg_fp8_gated_gemm_nt")
    return GatedOutput(h, h_sf, gu, gu_sf)


def m_grouped_fp8_gated_gemm_nt_contiguous(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                                           m_indices: torch.Tensor, d=None, activation: str = "silu",
                                           out_format: str = "bf16", checkpoint=False,
                                           stream=None) -> GatedOutput:
    """fp8_gated_gemm_nt for the experts of the contiguous layout: rows of A
    [m_sum, K] routed to B [G, 2F, K] by m_indices (-1 = padding: those rows
    of the results are left as they are)."""
    if stream is not None:
        return _under(stream, m_grouped_fp8_gated_gemm_nt_contiguous, a, sfa, b, sfb, m_indices, d, activation,
                      out_format, checkpoint)
    act = _activation(activation)
    dev = _device()
    f, k, usual = _gated_operands(a, sfa, b, sfb, dev, 1, 3)
    m = a.shape[0]
    usual = usual and _usual(m_indices, _I32, (m,), dev)
    if not usual:
        _need(m_indices, "m_indices", (torch.int32,), 1)
        _row_index(m_indices, m)
        _contiguous(a=a, b=b)
    h, h_sf, gu, gu_sf = _gated_out(d, checkpoint, out_format, (m,), f, a.device)
    if not usual or d is not None or not isinstance(checkpoint, bool):
        _contiguous(d=h)
        _on_current_device(None, a, sfa, b, sfb, m_indices, h, h_sf, gu, gu_sf)
    rc = _lib.lib().dg_m_grouped_fp8_gated_gemm_nt_contiguous(
        a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), h.data_ptr(), _p(h_sf), _p(gu), _p(gu_sf),
        m_indices.data_ptr(), m, f, k, b.shape[0], act, _handle(dev))
    if rc:
        _check(rc, "dg_m_grouped_fp8_gated_gemm_nt_contiguous")
    return GatedOutput(h, h_sf, gu, gu_sf)


def m_grouped_fp8_gated_gemm_nt_masked(a: torch.Tensor, sfa: torch.Tensor, b: torch.Tensor, sfb: torch.Tensor,
                                       masked_m: torch.Tensor, expected_m: int = 0, d=None,
                                       activation: str = "silu", out_format: str = "bf16",
                                       stream=None) -> GatedOutput:
    """fp8_gated_gemm_nt for the masked layout: A [G, max_m, K] x B [G, 2F, K];
    rows at or past masked_m[g] (read on the device) are left as they are.
    expected_m is taken as m_grouped_fp8_gemm_nt_masked takes it, and chooses
    nothing here: this form has one tile."""
    if stream is not None:
        return _under(stream, m_grouped_fp8_gated_gemm_nt_masked, a, sfa, b, sfb, masked_m, expected_m, d, activation,
                      out_format)
    act = _activation(activation)
    dev = _device()
    f, k, usual = _gated_operands(a, sfa, b, sfb, dev, 2, 3)
    g, max_m = a.shape[:2]
    if b.shape[0] != g:
        raise ValueError("shape mismatch")
    usual = usual and _usual(masked_m, _I32, (g,), dev)
    if not usual:
        _need(masked_m, "masked_m", (torch.int32,), 1)
        if masked_m.numel() != g:
            raise ValueError("shape mismatch")
        _contiguous(a=a, b=b, masked_m=masked_m)
    h, h_sf, _, _ = _gated_out(d, False, out_format, (g, max_m), f, a.device)
    if not usual or d is not None:
        _contiguous(d=h)
        _on_current_device(None, a, sfa, b, sfb, masked_m, h, h_sf)
    rc = _lib.lib().dg_m_grouped_fp8_gated_gemm_nt_masked(
        a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), h.data_ptr(), _p(h_sf), masked_m.data_ptr(), g,
        max_m, f, k, int(expected_m), act, _handle(dev))
    if rc:
        _check(rc, "dg_m_grouped_fp8_gated_gemm_nt_masked")
    return GatedOutput(h, h_sf, None, None)


class GatedGradients(NamedTuple):
    """fp8_gated_backward's results, E4M3 codes and packed scales each."""
    q: torch.Tensor          # [dg | du] [M, 2F], 1x128 row groups: dX = q @ W (fp8_gemm_nn)
    sf: torch.Tensor
    q_cols: torch.Tensor     # [dg | du] [align(M, 128), 2F], 128 rows of a column: dW = q_cols^T X
    sf_cols: torch.Tensor
    h_cols: torch.Tensor     # act(g) u [align(M, 128), F], the same grouping: dW_down = dY^T h_cols
    h_sf_cols: torch.Tensor


def fp8_gated_backward(dh: torch.Tensor, gu: torch.Tensor, gu_sf: torch.Tensor,
                       m_indices: Optional[torch.Tensor] = None, activation: str = "silu",
                       stream=None) -> GatedGradients:
    """Backward pass of h = act(g) * u from the 8-bit checkpoint of [g | u]:
    dg = dh u act'(g) and du = dh act(g), with h recomputed, as the E4M3
    operands of the gradient products.

    dh BF16 [M, F] (unit column stride); gu E4M3 [M, 2F] with packed 1x128
    row-group scales gu_sf (what the gated product keeps with
    checkpoint=True); F % 128 == 0.  m_indices: int32 [M]; rows with a
    negative entry count as zero, whatever dh and gu hold there."""
    if stream is not None:
        return _under(stream, fp8_gated_backward, dh, gu, gu_sf, m_indices, activation)
    act = _activation(activation)
    dev = _device()
    m, f = dh.shape if dh.dim() == 2 else (0, 0)
    ld = f
    if dh.dim() != 2 or not _usual(dh, _BF16, dh.shape, dev) or \
            not _usual(gu, _E4M3, (m, 2 * f), dev) or not _usual(gu_sf, _I32, _sf(m, 2 * f), dev) or \
            not (m_indices is None or _usual(m_indices, _I32, (m,), dev)):
        _need(dh, "dh", (torch.bfloat16,), 2)
        _need(gu, "gu", FP8_DTYPES, 2)
        _need(gu_sf, "gu_sf", (torch.int32,), 2)
        if tuple(gu.shape) != (m, 2 * f):
            raise ValueError("gu %s, expected %s" % (tuple(gu.shape), (m, 2 * f)))
        if tuple(gu_sf.shape) != sf_packed_shape(m, 2 * f):
            raise ValueError("scale shape %s, expected %s" % (tuple(gu_sf.shape), sf_packed_shape(m, 2 * f)))
        if dh.stride(1) != 1:
            raise ValueError("dh needs unit column stride")
        _contiguous(gu=gu, gu_sf=gu_sf)
        _row_index(m_indices, m)
        _on_current_device(None, dh, gu, gu_sf, m_indices)
        ld = dh.stride(0) if m > 1 else f
    device = dh.device
    m128 = (m + 127) // 128 * 128
    q, sf = _codes_out(None, (m, 2 * f), _sf(m, 2 * f), device, "q")
    qc, sfc = _cols_out(None, m128, 2 * f, device, "q_cols")
    hc, hsfc = _cols_out(None, m128, f, device, "h_cols")
    rc = _lib.lib().dg_fp8_gated_backward(dh.data_ptr(), ld, gu.data_ptr(), gu_sf.data_ptr(), _p(m_indices),
                                          q.data_ptr(), sf.data_ptr(), qc.data_ptr(), sfc.data_ptr(), hc.data_ptr(),
                                          hsfc.data_ptr(), m, f, act, _handle(dev))
    if rc:
        _check(rc, "dg_fp8_gated_backward")
    return GatedGradients(q, sf, qc, sfc, hc, hsfc)


# ---------------------------------------------------------------- layer norm


class LayerNormOutput(NamedTuple):
    y: torch.Tensor                # x's type, or E4M3 codes
    sf: Optional[torch.Tensor]     # packed 1x128 row-group scales of the codes, else None
    mean: torch.Tensor             # FP32 [rows], for the backward pass
    rstd: torch.Tensor


def _norm_args(x, weight, bias):
    _need(x, "x", tuple(_DTYPES), 2)
    cols = x.shape[1]
    if cols < 1:
        raise ValueError("x needs at least one column")
    if x.stride(1) != 1 and cols > 1:
        raise ValueError("x needs unit column stride")
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _need(t, name, (torch.float32, x.dtype), 1)
            if t.numel() != cols or not t.is_contiguous():
                raise ValueError("%s must be contiguous [%d]" % (name, cols))
    if bias is not None and bias.dtype != weight.dtype:
        raise TypeError("weight and bias must have one dtype")


def _row_stride(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
               out_format: str = "same", stream=None) -> LayerNormOutput:
    """y = (x - mean) * rstd * weight + bias over the last axis of [rows, cols].

    x FP32, BF16 or FP16 (unit column stride), weight and bias FP32 or x's
    type.  out_format "same": y in x's type; "fp8": y as E4M3 codes with
    packed 1x128 row-group scales (cols % 128 == 0), the operand of the FP8
    GEMMs and at the same time the 8-bit checkpoint of the normed activation."""
    if stream is not None:
        return _under(stream, layer_norm, x, weight, bias, eps, out_format)
    dev = _device()
    rows, cols = x.shape if x.dim() == 2 else (0, 0)
    ld = cols
    if cols < 1 or x.dtype not in _DTYPES or not _usual(x, x.dtype, x.shape, dev) or \
            not _usual(weight, _F32, (cols,), dev) or not (bias is None or _usual(bias, _F32, (cols,), dev)):
        _norm_args(x, weight, bias)
        _on_current_device(None, x, weight, bias)
        ld = _row_stride(x)
    sf = None
    device = x.device
    if out_format == "same":
        y = torch.empty((rows, cols), dtype=x.dtype, device=device)
    elif out_format == "fp8":
        if cols % 128:
            raise ValueError("out_format 'fp8' needs cols %% 128 == 0, got %d" % cols)
        y, sf = _codes_out(None, (rows, cols), _sf(rows, cols), device, "y")
    else:
        raise ValueError("out_format %r not in ('same', 'fp8')" % (out_format,))
    mean = torch.empty(rows, dtype=_F32, device=device)
    rstd = torch.empty(rows, dtype=_F32, device=device)
    rc = _lib.lib().dg_layer_norm(x.data_ptr(), _DTYPES[x.dtype], weight.data_ptr(), _p(bias), _DTYPES[weight.dtype],
                                  y.data_ptr(), _p(sf), mean.data_ptr(), rstd.data_ptr(), rows, cols, ld, float(eps),
                                  _handle(dev))
    if rc:
        _check(rc, "dg_layer_norm")
    return LayerNormOutput(y, sf, mean, rstd)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dx, dweight, dbias) of layer_norm: dx in x's type, the parameters'
    gradients in FP32 (summed in a fixed order)."""
    if stream is not None:
        return _under(stream, layer_norm_backward, dy, x, weight, mean, rstd)
    dev = _device()
    rows, cols = x.shape if x.dim() == 2 else (0, 0)
    ldx = ldy = cols
    if cols < 1 or x.dtype not in _DTYPES or not _usual(x, x.dtype, x.shape, dev) or \
            not _usual(dy, x.dtype, x.shape, dev) or not _usual(weight, _F32, (cols,), dev) or \
            not _usual(mean, _F32, (rows,), dev) or not _usual(rstd, _F32, (rows,), dev):
        _norm_args(x, weight, None)
        _need(dy, "dy", (x.dtype,), 2)
        _need(mean, "mean", (torch.float32,), 1)
        _need(rstd, "rstd", (torch.float32,), 1)
        if dy.shape != x.shape or (dy.stride(1) != 1 and cols > 1):
            raise ValueError("dy must be %s with unit column stride" % (tuple(x.shape),))
        if mean.numel() != rows or rstd.numel() != rows:
            raise ValueError("mean and rstd must be [%d]" % rows)
        _contiguous(mean=mean, rstd=rstd)
        _on_current_device(None, dy, x, weight, mean, rstd)
        ldx, ldy = _row_stride(x), _row_stride(dy)
    device = x.device
    dx = torch.empty((rows, cols), dtype=x.dtype, device=device)
    dw = torch.empty(cols, dtype=_F32, device=device)
    db = torch.empty(cols, dtype=_F32, device=device)
    need = _backward_workspace(cols, get_num_sms())
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    rc = _lib.lib().dg_layer_norm_backward(dy.data_ptr(), x.data_ptr(), _DTYPES[x.dtype], weight.data_ptr(),
                                           _DTYPES[weight.dtype], mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
                                           dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need, rows, cols, ldy, ldx,
                                           _handle(dev))
    if rc:
        _check(rc, "dg_layer_norm_backward")
    return dx, dw, db


@functools.lru_cache(maxsize=256)
def _backward_workspace(cols: int, num_sms: int) -> int:
    need = C.c_uint64(0)
    _check(_lib.lib().dg_layer_norm_backward_workspace_size(cols, num_sms, C.byref(need)),
           "dg_layer_norm_backward_workspace_size")
    return need.value
