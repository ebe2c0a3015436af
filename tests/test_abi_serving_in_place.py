"""CPU-only checks: results in place of an operand with other strides are refused on the host."""
import pytest

from test_abi_serving import ALIGN, INVALID, L, ODD2, P, moe  # noqa: F401  (L: a fixture)


@pytest.mark.parametrize("ldc,ldy", [(256, 264), (512, 256)])
def test_moe_residual_in_place_keeps_its_stride(L, ldc, ldy):  # noqa: F811
    # (an address off its boundary ends those that pass: nothing is launched)
    call = lambda **kw: moe(L, c=P, experts=ODD2, **kw)  # noqa: E731
    assert call(ldc=ldc, ldy=ldy) == INVALID
    assert call(ldc=ldc, ldy=ldc) == ALIGN
    assert call(ldc=ldc, ldy=ldy, tokens=1) == ALIGN
    assert moe(L, c=ODD2, ldc=ldc, ldy=ldy, experts=ODD2) == ALIGN
