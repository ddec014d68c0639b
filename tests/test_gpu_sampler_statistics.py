"""The norm's statistics and sums are float32 throughout: bounds by the depth of its own sums, which
are short, and rows whose statistics float32 holds exactly."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref
from tests.test_gpu_sampler_norm import f64, rows

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = ref.HALF_F32
# a lane adds up at most 64 squares or products, six steps join a wave's lanes, at most 15 more its waves
DEPTH = 64 + 6 + 15
# dweight: a workgroup's rows (256 workgroups at least), then at most 8 parts, six steps and what is added to
WGS = 256

SHAPES = [(1, 8), (3, 136), (1, 5120), (5, 1000), (2, 8200), (2, 16384), (1030, 2056), (1024, 6152), (1100, 8192), (1024, 16384),
          (4099, 4096), (700, 512)]


def rstd_error():
    """A sum, the mean and eps under the root, which halves them; root and quotient."""
    return (0.5 * (DEPTH + 2) + 2) * U


@pytest.mark.parametrize("t,n", SHAPES)
def test_rstd(t, n):
    x, w = rows(t, n, 0.7, 21), (1 + rows(1, n, 0.1, 22)[0]).contiguous()
    y, rstd = torch.empty_like(x), torch.empty(t, device="cuda")
    pulse.pulse_rms_norm(x, w, eps=EPS, y=y, rstd=rstd)
    want, want_rstd = ref.rms_norm(f64(x), f64(w), EPS)
    np.testing.assert_allclose(f64(rstd), want_rstd, rtol=1.02 * rstd_error())
    np.testing.assert_allclose(f64(y), want, rtol=1.02 * (rstd_error() + 2 * U + ref.HALF_BF16), atol=0)


@pytest.mark.parametrize("t", [1, 3, 1024])
@pytest.mark.parametrize("n", [8, 128, 1024, 16384])
def test_rows_of_exact_statistics(t, n):
    """Columns of 2^j and 2^(j + 1) in turn: the mean of the squares is 2.5 * 4^j, and eps is nothing beside it."""
    j = torch.arange(t, device="cuda") % 41 - 20
    x = torch.pow(2.0, j[:, None] + torch.arange(n, device="cuda")[None] % 2).to(torch.bfloat16)
    x[:, 1::4] *= -1
    rstd, y = torch.empty(t, device="cuda"), torch.empty_like(x)
    pulse.pulse_rms_norm(x, torch.ones(n, dtype=torch.bfloat16, device="cuda"), eps=1e-30, y=y, rstd=rstd)
    want = 2.0 ** -f64(j) / np.sqrt(2.5)
    np.testing.assert_allclose(f64(rstd), want, rtol=1.02 * 2 * U, atol=0)  # root and quotient


@pytest.mark.parametrize("t,n", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_gradients(t, n, residual):
    """dx and dweight of the rstd that the forward pass left, with every operand and dx in strides of their own."""
    s, w = rows(t, n, 1.5, 23, pad=8), (1 + rows(1, n, 0.1, 24)[0]).contiguous()
    dy, dres = rows(t, n, 1e-2, 25, pad=16), rows(t, n, 1e-2, 26, pad=24) if residual else None
    whole = torch.full((t, n + 32), -77.0, dtype=torch.bfloat16, device="cuda")
    dx, dw, rstd = whole[:, :n], torch.full((n,), 3.0, device="cuda"), torch.empty(t, device="cuda")
    pulse.pulse_rms_norm(s, w, eps=EPS, y=torch.empty((t, n), dtype=torch.bfloat16, device="cuda"), rstd=rstd)
    pulse.pulse_rms_norm_backward(s, w, rstd, dy, dx, dw, pulse.rms_norm_workspace(t, n), dres=dres)
    assert (whole[:, n:] == -77).all()
    a, b, d, r = f64(s), f64(w), f64(dy), f64(rstd)[:, None]
    hat = a * r
    mean = (d * b * hat).mean(axis=1, keepdims=True)
    want = r * (d * b - hat * mean) + (0 if dres is None else f64(dres))
    # the mean: two roundings of a product, the sum, the quotient
    mean_error = np.abs(d * b * hat).mean(axis=1, keepdims=True) * (DEPTH + 3) * U
    # dy w: one, the difference, the factor; hat * mean one more
    room = r * (np.abs(d * b) * 3 * U + np.abs(hat * mean) * 4 * U + np.abs(hat) * mean_error) + np.abs(want) * U
    room = 1.02 * (room + (np.abs(want) + room) * ref.HALF_BF16)
    assert (np.abs(f64(dx) - want) <= room + 1e-35).all()
    # hat, the sums' depth
    room = np.abs(d * hat).sum(axis=0) * (1 + -(-t // min(t, WGS)) + 8 + 6) * U * 1.02
    assert (np.abs(f64(dw) - (d * hat).sum(axis=0)) <= room + 1e-35).all()
    before, first = dw.clone(), dx.clone()
    # over dres, or dy, in its stride
    over = dy if dres is None else dres
    pulse.pulse_rms_norm_backward(s, w, rstd, dy, over, dw, pulse.rms_norm_workspace(t, n), dres=dres, accumulate=True)
    assert torch.equal(over, first) and torch.equal(dw, before + before)
