"""A workspace made for a number of tokens serves every smaller one."""
import random

import pytest

from tests.test_abi import ERANGE, EWORKSPACE, lib  # noqa: F401  (the library fixture)
from tests.test_sampler_refusals import GEMM, GOOD_GEMM, I32, I64, call

TOKENS = sorted({*range(1, 300), *range(300, 2100, 37), *(2 ** i + d for i in range(1, 18) for d in (-1, 0, 1))} - {0})


def sizes(rng):
    """Widths of projections, and any others."""
    yield from [(7168, 5120), (5120, 27648), (55296, 5120), (28672, 4096), (4096, 28672), (512, 27648), (16, 16), (128, 1 << 20)]
    for _ in range(60):
        yield 16 * int(2 ** rng.uniform(0, 11)), 16 * int(2 ** rng.uniform(0, 11))


@pytest.mark.parametrize("form", [0, 1])
def test_products(lib, form):  # noqa: F811
    size = lib.fp8_block_gemm_ws_bytes
    size.argtypes, size.restype = [I64, I64, I64, I32], I64
    for n, k in sizes(random.Random(form)):
        had = 0
        for m in TOKENS:
            need = size(m, n, k, form)
            if need == ERANGE:  # (2^23 tiles of 64 x 128: nor is a product of more rows taken)
                assert (m + 63) // 64 * (((k if form else n) + 127) // 128) >= 2 ** 23
                break
            assert need >= had, (m, n, k)
            had = need


def test_a_product_takes_a_larger_ones_workspace(lib):  # noqa: F811
    """What is refused for want of a workspace is refused below its own size, which no larger m's is."""
    size = lib.fp8_block_gemm_ws_bytes
    size.argtypes, size.restype = [I64, I64, I64, I32], I64
    for m, n, k in [(96, 7168, 5120), (1024, 55296, 5120), (4096, 55296, 5120)]:
        bad = dict(m=m, n=n, k=k, ldy=n)
        assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, bad | dict(ws=None)) == EWORKSPACE
        assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, bad | dict(wsb=size(m, n, k, 0) - 1)) == EWORKSPACE
        assert size(8192, n, k, 0) >= size(m, n, k, 0) > 0


def test_norm_and_experts(lib):  # noqa: F811
    norm, moe = lib.pulse_rms_norm_ws_bytes, lib.pulse_moe_ws_bytes
    norm.argtypes, norm.restype, moe.argtypes, moe.restype = [I64] * 2, I64, [I64] * 5, I64
    for cols in (8, 2048, 2056, 16384):
        need = [norm(t, cols) for t in TOKENS]
        assert need == sorted(need)
    for hidden, inter, experts, top_k in ((16, 16, 1, 1), (7168, 2048, 384, 8), (4096, 14336, 16, 2)):
        need = [moe(t, hidden, inter, experts, top_k) for t in range(1, 1025)]
        assert need == sorted(need) and need[0] > 0
