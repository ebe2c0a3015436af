"""CPU-only checks of the serving entry points: bad arguments are refused on the
host, before anything is enqueued (the pointers are never read)."""
import ctypes as C

import pytest

from moe_grouped_gemm_fp8_gb300 import _lib

DG_OK, INVALID, ALIGN, TOO_LARGE = 0, 1, 2, 7
P, ODD8, ODD2, ODD1 = C.c_void_p(0x1000), C.c_void_p(0x1008), C.c_void_p(0x1002), C.c_void_p(0x1001)


@pytest.fixture(scope="module")
def L():
    from moe_grouped_gemm_fp8_gb300 import build
    build.build()
    return _lib.lib()


def size(L, t=4, d=256, f=128, e=8, k=2):
    need = C.c_uint64(0)
    return L.dg_fp8_moe_few_tokens_workspace_size(t, d, f, e, k, C.byref(need)), need.value


def moe(L, **kw):
    a = dict(x=P, ldx=256, router=P, router_dtype=0, bias=None, up=P, up_sf=P, down=P, down_sf=P, c=None, ldc=0, n=None,
             y=P, ldy=256, experts=P, weights=P, ws=P, bytes=1 << 40, tokens=4, d=256, f=128, e=8, k=2, score=0, renorm=1,
             scale=1.0, act=0)
    a.update(kw)
    return L.dg_fp8_moe_few_tokens(*a.values(), None)


def test_moe_checks(L):
    assert moe(L, d=200, ldx=200, ldy=200) == ALIGN
    assert moe(L, f=100) == ALIGN
    assert moe(L, tokens=-1) == INVALID
    assert moe(L, tokens=65) == TOO_LARGE
    assert moe(L, k=0) == INVALID
    assert moe(L, k=9) == INVALID                    # more than the experts
    assert moe(L, e=600, k=17) == TOO_LARGE
    assert moe(L, e=513) == TOO_LARGE
    assert moe(L, d=65536 + 128, ldx=1 << 20, ldy=1 << 20) == TOO_LARGE
    assert moe(L, e=0) == INVALID
    assert moe(L, d=0) == INVALID
    assert moe(L, router_dtype=2) == INVALID
    assert moe(L, score=2) == INVALID
    assert moe(L, act=2) == INVALID
    assert moe(L, bias=P) == INVALID                 # a bias goes with the logistic score
    assert moe(L, bias=ODD2, score=1) == ALIGN
    assert moe(L, ldx=255) == INVALID
    assert moe(L, ldx=260) == ALIGN
    assert moe(L, ldy=255) == INVALID
    assert moe(L, c=P, ldc=255) == INVALID
    for name in ("x", "router", "up", "up_sf", "down", "down_sf", "y", "experts", "weights", "ws"):
        assert moe(L, **{name: None}) == INVALID, name
    for name in ("x", "router", "up", "up_sf", "down", "down_sf", "ws"):
        assert moe(L, **{name: ODD8}) == ALIGN, name
    for name in ("experts", "weights", "n"):
        assert moe(L, **{name: ODD2}) == ALIGN, name
    assert moe(L, y=ODD1) == ALIGN
    assert moe(L, tokens=0) == DG_OK
    assert moe(L, bytes=size(L)[1] - 1) == INVALID   # a workspace that is too small


def test_moe_workspace_size(L):
    st, small = size(L)
    assert st == DG_OK and small > 0
    assert size(L, t=64)[1] > small
    assert size(L, t=65)[0] == TOO_LARGE
    assert size(L, d=100)[0] == ALIGN
    assert size(L, t=0)[0] == DG_OK
    assert L.dg_fp8_moe_few_tokens_workspace_size(4, 256, 128, 8, 2, None) == INVALID


def int8(L, **kw):
    a = dict(a=P, sa=P, b=P, sb=P, c=None, d=P, m=100, n=50, k=64, lda=64, ldb=64, ldc=0, ldd=50, out=1)
    a.update(kw)
    return L.dg_int8_gemm_nt(*a.values(), None)


def test_int8_checks(L):
    assert int8(L, k=0) == INVALID
    assert int8(L, k=72, lda=80, ldb=80) == ALIGN
    assert int8(L, m=-1) == INVALID
    assert int8(L, out=0) == INVALID                 # FP32
    assert int8(L, lda=48) == INVALID
    assert int8(L, ldb=72) == ALIGN
    assert int8(L, ldd=49) == INVALID
    assert int8(L, c=P, ldc=49) == INVALID
    assert int8(L, c=P, ldc=60) == INVALID           # in place with another stride
    for name in ("a", "sa", "b", "sb", "d"):
        assert int8(L, **{name: None}) == INVALID, name
    assert int8(L, a=ODD8) == ALIGN and int8(L, b=ODD8) == ALIGN
    assert int8(L, sa=ODD2) == ALIGN and int8(L, d=ODD1) == ALIGN and int8(L, c=ODD1, ldc=50) == ALIGN
    assert int8(L, m=0) == DG_OK and int8(L, n=0, ldd=0) == DG_OK
    assert int8(L, m=1 << 31) == TOO_LARGE
    assert int8(L, m=1 << 29, n=1 << 29, ldd=1 << 29) == TOO_LARGE


def test_quantise_checks(L):
    def call(x=P, dtype=1, q=P, s=P, rows=4, cols=10, ld=10):
        return L.dg_quantize_int8(x, dtype, q, s, rows, cols, ld, None)
    assert call(cols=0, ld=0) == INVALID
    assert call(rows=-1) == INVALID
    assert call(ld=9) == INVALID
    assert call(dtype=3) == INVALID
    assert call(x=None) == INVALID and call(q=None) == INVALID and call(s=None) == INVALID
    assert call(x=ODD1) == ALIGN and call(x=ODD2, dtype=0) == ALIGN and call(s=ODD2) == ALIGN
    assert call(rows=0) == DG_OK
    assert call(rows=1 << 31) == TOO_LARGE
