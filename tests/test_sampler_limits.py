"""The sampler's documented limits on sizes together: the first size past each is refused, the last
within it is not (a missing operand is what such a call is refused for)."""
import pytest

from tests.test_abi import EINVAL, ERANGE, lib  # noqa: F401  (the library fixture)
from tests.test_sampler_refusals import GEMM, GOOD_GEMM, GOOD_MOE, GOOD_QUANT, MOE, QUANT, call


@pytest.mark.parametrize("t,cols,code", [(2 ** 23 - 1, 8192, EINVAL), (2 ** 23, 8192, ERANGE), (2 ** 24 - 1, 7 * 512, EINVAL),
                                         (2 ** 24 - 1, 7 * 512 + 8, ERANGE), (4095, 2 ** 24, EINVAL), (4096, 2 ** 24, ERANGE)])
def test_pieces_of_the_quantiser(lib, t, cols, code):  # noqa: F811
    assert (t * (-(-cols // 512)) >= 2 ** 27 - 8) == (code == ERANGE)
    assert call(lib, "fp8_group_quant", QUANT, GOOD_QUANT, dict(t=t, n=cols, ldx=2 * cols, x=None)) == code


@pytest.mark.parametrize("m,n,code", [(2 ** 18, 2 ** 18, ERANGE), (2 ** 18 - 64, 2 ** 18, EINVAL), (2 ** 18, 2 ** 18 - 128, EINVAL),
                                      (64 * (2 ** 23 - 1), 1, ERANGE), (2 ** 24 - 1, 32 * 128, ERANGE), (2 ** 24 - 1, 31 * 128, EINVAL)])
def test_tiles_of_a_product(lib, m, n, code):  # noqa: F811
    assert (-(-m // 64) * -(-n // 128) >= 2 ** 23 or m >= 2 ** 24) == (code == ERANGE)
    assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, dict(m=m, n=n, ldy=n, x=None)) == code


def test_more_choices_than_experts(lib):  # noqa: F811
    assert call(lib, "pulse_moe_forward", MOE, GOOD_MOE, dict(e=3, k=4)) == EINVAL
