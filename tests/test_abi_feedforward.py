"""CPU-only checks of the feed-forward entry points: bad arguments are refused
on the host, before anything is enqueued (the pointers are never read)."""
import ctypes as C

import pytest
import torch

from moe_grouped_gemm_fp8_gb300 import _lib, feedforward

DG_OK, INVALID, ALIGN, TOO_LARGE = 0, 1, 2, 7
P, ODD = C.c_void_p(0x1000), C.c_void_p(0x1008)


@pytest.fixture(scope="module")
def L():
    from moe_grouped_gemm_fp8_gb300 import build
    build.build()
    return _lib.lib()


def test_checkpoint_checks(L):
    save, restore, use = L.dg_quantize_fp8_bf16, L.dg_dequantize_fp8, L.dg_requantize_fp8_cols
    assert save(P, P, P, 1, 4, 100, None) == ALIGN
    assert save(P, P, P, 1, -4, 128, None) == INVALID
    assert save(None, P, P, 1, 4, 128, None) == INVALID
    assert save(ODD, P, P, 1, 4, 128, None) == ALIGN
    assert save(P, P, P, 0, 4, 128, None) == DG_OK
    assert save(P, P, P, 1, 1 << 31, 128, None) == TOO_LARGE
    assert restore(P, P, P, 2, 1, 4, 128, None) == INVALID          # FP16
    assert restore(P, P, P, 0, 1, 4, 130, None) == ALIGN
    assert restore(P, P, None, 1, 1, 4, 128, None) == INVALID
    assert restore(P, P, P, 1, 1, 0, 128, None) == DG_OK
    assert use(P, P, None, P, P, 4, 100, None) == ALIGN
    assert use(P, P, C.c_void_p(0x1002), P, P, 4, 128, None) == ALIGN
    assert use(P, P, None, None, P, 4, 128, None) == INVALID
    assert use(P, P, None, P, P, 0, 128, None) == DG_OK
    assert use(P, P, None, P, P, 1 << 31, 128, None) == TOO_LARGE


def _gated(L, **kw):
    a = dict(a=P, sfa=P, b=P, sfb=P, h=P, h_sf=None, gu=None, gu_sf=None, m=200, f=256, k=512, lda=512, ldb=512, ldh=256,
             act=0)
    a.update(kw)
    return L.dg_fp8_gated_gemm_nt(a["a"], a["sfa"], a["b"], a["sfb"], a["h"], a["h_sf"], a["gu"], a["gu_sf"], a["m"],
                                  a["f"], a["k"], a["lda"], a["ldb"], a["ldh"], a["act"], None)


def test_gated_checks(L):
    assert _gated(L, k=100) == ALIGN
    assert _gated(L, k=0) == INVALID
    assert _gated(L, f=100, ldh=104) == ALIGN                  # F % 8
    assert _gated(L, f=136, ldh=136, h_sf=P) == ALIGN          # 8-bit results: F % 128
    assert _gated(L, f=136, ldh=136, gu=P, gu_sf=P) == ALIGN
    assert _gated(L, gu=P) == INVALID                          # a checkpoint without its scales
    assert _gated(L, h_sf=P, ldh=264) == INVALID               # 8-bit results are contiguous
    assert _gated(L, ldh=248) == INVALID
    assert _gated(L, ldh=260) == ALIGN
    assert _gated(L, lda=520) == ALIGN
    assert _gated(L, lda=256) == INVALID
    assert _gated(L, act=2) == INVALID
    assert _gated(L, b=None) == INVALID
    assert _gated(L, h=ODD) == ALIGN
    assert _gated(L, m=-1) == INVALID
    assert _gated(L, m=0) == DG_OK
    assert _gated(L, f=0, ldh=0) == DG_OK
    assert _gated(L, m=1 << 31) == TOO_LARGE
    cont, masked = L.dg_m_grouped_fp8_gated_gemm_nt_contiguous, L.dg_m_grouped_fp8_gated_gemm_nt_masked
    assert cont(P, P, P, P, P, None, None, None, P, 130, 256, 512, 4, 0, None) == ALIGN     # m_sum % 128
    assert cont(P, P, P, P, P, None, None, None, None, 128, 256, 512, 4, 0, None) == INVALID
    assert cont(P, P, P, P, P, None, None, None, P, 128, 256, 512, 0, 0, None) == DG_OK
    assert masked(P, P, P, P, P, None, P, 513, 64, 256, 512, 0, 0, None) == TOO_LARGE
    assert masked(P, P, P, P, P, None, None, 4, 64, 256, 512, 0, 0, None) == INVALID
    assert masked(P, P, P, P, P, None, P, 4, 64, 256, 512, -1, 0, None) == INVALID
    assert masked(P, P, P, P, P, None, P, 4, 0, 256, 512, 0, 0, None) == DG_OK


def test_gated_backward_checks(L):
    def call(**kw):
        a = dict(dh=P, ld=256, gu=P, gu_sf=P, idx=None, q=P, sf=P, qc=P, sfc=P, hc=P, hsf=P, m=100, f=256, act=0)
        a.update(kw)
        return L.dg_fp8_gated_backward(*a.values(), None)
    assert call(f=200, ld=200) == ALIGN
    assert call(ld=128) == INVALID
    assert call(ld=258) == ALIGN
    assert call(dh=C.c_void_p(0x1004)) == ALIGN
    assert call(dh=None) == INVALID
    assert call(hsf=None) == INVALID
    assert call(qc=ODD) == ALIGN
    assert call(act=7) == INVALID
    assert call(m=0) == DG_OK
    assert call(m=1 << 31) == TOO_LARGE


def test_layer_norm_checks(L):
    def fwd(**kw):
        a = dict(x=P, dt=1, w=P, b=P, wdt=0, y=P, sf=None, mean=P, rstd=P, rows=4, cols=256, ldx=256, eps=1e-5)
        a.update(kw)
        return L.dg_layer_norm(*a.values(), None)
    assert fwd(dt=3) == INVALID
    assert fwd(wdt=2) == INVALID                    # FP16 parameters with BF16 rows
    assert fwd(cols=0) == INVALID
    assert fwd(ldx=100) == INVALID
    assert fwd(eps=-1.0) == INVALID
    assert fwd(eps=float("nan")) == INVALID
    assert fwd(x=None) == INVALID
    assert fwd(x=C.c_void_p(0x1001)) == ALIGN
    assert fwd(rows=0) == DG_OK
    assert fwd(sf=P, cols=200) == ALIGN             # 8-bit results: whole groups of 128 columns
    assert fwd(sf=P, x=ODD) == ALIGN
    assert fwd(sf=P, ldx=260) == ALIGN
    assert fwd(sf=P, cols=32896, ldx=32896) == TOO_LARGE

    def bwd(**kw):
        a = dict(dy=P, x=P, dt=1, w=P, wdt=0, mean=P, rstd=P, dx=P, dw=P, db=P, ws=P, nb=1 << 40, rows=4, cols=256,
                 lddy=256, ldx=256)
        a.update(kw)
        return L.dg_layer_norm_backward(*a.values(), None)
    assert bwd(dt=5) == INVALID
    assert bwd(ws=None) == INVALID
    assert bwd(dy=None) == INVALID
    assert bwd(lddy=128) == INVALID
    assert bwd(dw=C.c_void_p(0x1002)) == ALIGN
    out = C.c_uint64(0)
    assert L.dg_layer_norm_backward_workspace_size(0, 152, C.byref(out)) == INVALID
    assert L.dg_layer_norm_backward_workspace_size(256, 0, C.byref(out)) == INVALID
    assert L.dg_layer_norm_backward_workspace_size(256, 152, None) == INVALID
    assert L.dg_layer_norm_backward_workspace_size(256, 152, C.byref(out)) == DG_OK
    assert out.value >= 2 * 256 * 4 * 152


def test_binding_refuses_host_tensors_and_wrong_types():
    codes = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    words = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        feedforward.dequantize_fp8(codes, words, dtype=torch.float16)
    with pytest.raises(ValueError):
        feedforward.dequantize_fp8(codes, words)            # not on a CUDA device
    with pytest.raises(TypeError):
        feedforward.dequantize_fp8(codes.float(), words)
    with pytest.raises(ValueError):
        feedforward._activation("relu")
    with pytest.raises(ValueError):
        feedforward._gated_out(None, False, "fp8", (4,), 200, torch.device("cpu"))
    with pytest.raises(ValueError):
        feedforward._gated_out(None, True, "bf16", (4,), 200, torch.device("cpu"))
    with pytest.raises(ValueError):
        feedforward._codes_out((codes, words), (4, 128), (1, 4), torch.device("cpu"), "d")
