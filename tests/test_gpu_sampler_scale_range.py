"""Scales whose product lies at the ends of float32's normal range: sums that float32 holds exactly."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref
from tests.test_gpu_sampler_gemm import multiply, pytestmark  # noqa: F401


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("m", [1, 12, 40, 300])
@pytest.mark.parametrize("sx,sw,x,w", [
    (2.0 ** 100, 2.0 ** 27, 0x01, 0x01),    # 2^127 times products of 2^-18
    (2.0 ** 119, 2.0 ** 8, 0x08, 0x01),     # the largest scale of a BF16 group
    (2.0 ** -104, 2.0 ** -22, 0x78, 0x78),  # 2^-126 times products of 2^16, from about the smallest scale on
    (2.0 ** -60, 2.0 ** -66, 0x38, 0x38)])  # ... of 1
def test_ends_of_the_range(m, form, sx, sw, x, w):
    n, k = (130, 400) if form == "nt" else (400, 144)
    inner = 400
    g = np.random.default_rng(m)
    xs = (g.integers(0, 2, (m, inner)) * x).astype(np.uint8)
    ws = (g.integers(0, 2, (n, k)) * w).astype(np.uint8)
    fx, fw = np.full((m, ref.groups(inner)), sx, np.float32), np.full((ref.groups(n), ref.groups(k)), sw, np.float32)
    y, _ = ref.gemm(xs, fx, ws, fw, form)
    # each is a power of two times a whole number below 401: rounded once
    got = multiply(xs, fx, ws, fw, form)
    np.testing.assert_array_equal(got, torch.from_numpy(y).to(torch.bfloat16).double().numpy())
    assert np.isfinite(got).all() and (got != 0).any()


def test_the_largest_group_of_bf16():
    """Rows of the largest BF16 values through the quantiser and a unit matrix."""
    x = torch.full((20, 256), 3.3895e38, device="cuda").to(torch.bfloat16)
    x[::2, ::2] *= -0.5
    codes, scales = torch.empty((20, 256), dtype=torch.uint8, device="cuda"), torch.empty((20, 2), device="cuda")
    pulse.fp8_group_quant(x, codes, scales)
    unit, one = torch.zeros((256, 256), dtype=torch.uint8, device="cuda"), torch.ones((2, 2), device="cuda")
    unit.fill_diagonal_(0x38)
    y = torch.empty_like(x)
    pulse.fp8_block_gemm(codes, scales, unit, one, y, pulse.fp8_gemm_workspace(20, 256, 256))
    assert torch.equal(y, x)  # 448 and -224 times the scale
