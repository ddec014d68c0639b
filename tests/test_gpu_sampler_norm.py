"""The norm with its quantised output, its gradients, and the group quantiser against
float64 and against the documented float32 arithmetic."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


def rows(t, n, std=1.0, seed=0, pad=0):
    """BF16 rows on the GPU, with a row stride of n + pad."""
    g = torch.Generator().manual_seed(seed * 7919 + t * 31 + n)
    x = (torch.randn((t, n + pad), generator=g) * std).to(torch.bfloat16).cuda()
    return x[:, :n]


def f64(t):
    return t.detach().cpu().double().numpy()


def quant_buffers(t, n):
    """Codes and scales whose rows behind the last must stay as they are."""
    codes = torch.full((t + 1, n), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((t + 1, ref.groups(n)), 7.0, device="cuda")
    return codes, scales


def untouched(codes, scales):
    assert (codes[-1] == 0xAB).all() and (scales[-1] == 7.0).all()


SHAPES = [(1, 8), (1, 128), (3, 136), (1, 5120), (2, 520), (5, 1000), (7, 4096), (2, 8192), (3, 8200), (2, 16384),
          (1030, 2056), (1025, 264), (1024, 6152), (1100, 8192), (1027, 12296), (1024, 16384), (1500, 4096)]


@pytest.mark.parametrize("t,n", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(t, n, residual):
    x, w = rows(t, n, 0.7, 1, pad=16), (1 + rows(1, n, 0.1, 2)[0]).contiguous()
    r = rows(t, n, 1.5, 3, pad=8) if residual else None
    y, rstd = rows(t, n, 1.0, 4, pad=24), torch.empty(t, device="cuda")
    codes, scales = quant_buffers(t, n)
    behind = None if r is None else r.as_strided((t, n + 8), (n + 8, 1))[:, n:].clone()
    s = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
    pulse.pulse_rms_norm(x, w, eps=EPS, residual=r, y=y, codes=codes[:t], scales=scales[:t], rstd=rstd)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(r, s)  # one float32 addition, rounded: bit for bit
        assert torch.equal(r.as_strided((t, n + 8), (n + 8, 1))[:, n:], behind)
    want, want_rstd = ref.rms_norm(f64(s), f64(w), EPS)
    rel = ref.rstd_error(n) + 2 * ref.HALF_F32
    np.testing.assert_allclose(f64(rstd), want_rstd, rtol=ref.rstd_error(n))
    np.testing.assert_allclose(f64(y), want, rtol=1.02 * (rel + ref.HALF_BF16), atol=0)
    ref.check_codes(codes[:t].cpu().numpy(), scales[:t].cpu().numpy(), want, rel)
    untouched(codes, scales)


def test_norm_outputs_agree():
    """y alone, codes alone and both together are the same."""
    t, n = 37, 1408
    x, w = rows(t, n), (1 + rows(1, n, 0.1, 2)[0]).contiguous()
    y = [torch.empty((t, n), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c = [torch.empty((t, n), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.empty((t, 11), device="cuda") for _ in range(2)]
    pulse.pulse_rms_norm(x, w, y=y[0])
    pulse.pulse_rms_norm(x, w, codes=c[0], scales=s[0])
    pulse.pulse_rms_norm(x, w, y=y[1], codes=c[1].view(torch.float8_e4m3fn), scales=s[1])
    assert torch.equal(y[0], y[1]) and torch.equal(c[0], c[1]) and torch.equal(s[0], s[1])


def test_norm_edges():
    """Rows of zeros, of the smallest values, with Inf and with NaN."""
    n = 256
    x = torch.zeros((5, n), dtype=torch.bfloat16, device="cuda")
    x[1, 3] = 2.0 ** -133
    x[2, 130] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 1e18
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y, codes, scales = torch.empty_like(x), torch.empty((5, n), dtype=torch.uint8, device="cuda"), torch.empty((5, 2), device="cuda")
    pulse.pulse_rms_norm(x, w, eps=EPS, y=y, codes=codes, scales=scales)
    y, s = y.float().cpu(), scales.cpu()
    assert (y[0] == 0).all() and (codes[0] == 0).all() and (s[0] == 1).all()
    assert y[1, 3] == 0 or abs(y[1, 3] / (2.0 ** -133 * 1e3) - 1) < 0.02
    assert (codes[1] == 0).all() and (s[1] == 1).all()
    # Inf: rstd 0, so 0 everywhere and Inf * 0 in its place
    assert torch.isnan(y[2, 130]) and (y[2, :128] == 0).all()
    assert torch.isnan(y[3]).all()
    for r in (2, 3):  # what a group with a NaN stands for is no number
        g = 1
        assert not np.isfinite(ref.E4M3[codes[r, 128:].cpu().numpy()] * s[r, g].item()).any()
    assert ((y[4] - 1).abs() < 0.01).all()


@pytest.mark.parametrize("t,n", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_backward(t, n, residual):
    s, w = rows(t, n, 1.5, 5, pad=8), (1 + rows(1, n, 0.1, 2)[0]).contiguous()
    dy = rows(t, n, 1e-2, 6, pad=16)
    dres = rows(t, n, 1e-2, 7) if residual else None
    dx, dw = torch.empty((t, n), dtype=torch.bfloat16, device="cuda"), torch.full((n,), 3.0, device="cuda")
    rstd = torch.empty(t, device="cuda")
    pulse.pulse_rms_norm(s, w, eps=EPS, y=torch.empty_like(dx), rstd=rstd)
    ws = pulse.rms_norm_workspace(t, n)
    pulse.pulse_rms_norm_backward(s, w, rstd, dy, dx, dw, ws, dres=dres)
    a, b, d = f64(s), f64(w), f64(dy)
    want, want_dw = ref.rms_norm_backward(a, b, d, EPS, None if dres is None else f64(dres))
    hat = a / np.sqrt((a * a).mean(axis=1, keepdims=True) + EPS)
    r = 1 / np.sqrt((a * a).mean(axis=1, keepdims=True) + EPS)
    rel = ref.rstd_error(n)
    # the mean: n products of two roundings and a sum; then three roundings of the difference
    mean = (np.abs(d * b * hat)).mean(axis=1, keepdims=True) * ((n + 8) * ref.HALF_F32 + rel)
    bound = np.abs(want) * (ref.HALF_BF16 + 2 * ref.HALF_F32)
    bound = bound + r * (np.abs(d * b) + np.abs(hat) * np.abs((d * b * hat).mean(axis=1, keepdims=True))) * (6 * ref.HALF_F32 + 2 * rel)
    bound = 1.02 * (bound + r * np.abs(hat) * mean) + 1e-30
    assert (np.abs(f64(dx) - want) <= bound).all()
    bound_dw = 1.02 * np.abs(d * hat).sum(axis=0) * ((t + 4) * ref.HALF_F32 + rel) + 1e-30
    assert (np.abs(f64(dw) - want_dw) <= bound_dw).all()
    # accumulated on top; dx written over dy, and not wanted at all
    before = dw.clone()
    over = dy.contiguous().clone()
    pulse.pulse_rms_norm_backward(s, w, rstd, over, over, dw, ws, dres=dres, accumulate=True)
    assert torch.equal(over, dx)
    assert torch.equal(dw, before + before)
    pulse.pulse_rms_norm_backward(s, w, rstd, dy, None, dw, ws)
    assert torch.equal(dw, before)


def test_norm_backward_against_differences():
    """dx and dweight against central differences of the float64 formula."""
    t, n = 2, 24
    g = np.random.default_rng(3)
    s, w, dy = ref.bf16(g.normal(0, 1, (t, n))), ref.bf16(1 + g.normal(0, 0.2, n)), ref.bf16(g.normal(0, 1, (t, n)))
    to = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()  # noqa: E731
    rstd, dx = torch.empty(t, device="cuda"), torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(n, device="cuda")
    pulse.pulse_rms_norm(to(s), to(w), eps=EPS, y=torch.empty_like(dx), rstd=rstd)
    pulse.pulse_rms_norm_backward(to(s), to(w), rstd, to(dy), dx, dw, pulse.rms_norm_workspace(t, n))
    loss = lambda a, b: (ref.rms_norm(a, b, EPS)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for i in range(t):
        for j in range(n):
            e = np.zeros((t, n))
            e[i, j] = h
            d = (loss(s + e, w) - loss(s - e, w)) / (2 * h)
            assert abs(f64(dx)[i, j] - d) <= ref.HALF_BF16 * abs(d) + 1e-5
    for j in range(n):
        e = np.zeros(n)
        e[j] = h
        assert abs(f64(dw)[j] - (loss(s, w + e) - loss(s, w - e)) / (2 * h)) <= 1e-5


@pytest.mark.parametrize("t,n", [(1, 8), (1, 128), (3, 200), (1, 27648), (5, 1408), (37, 512), (129, 1032), (9, 4104),
                                 (260, 648)])
def test_group_quant_is_the_documented_arithmetic(t, n):
    """BF16 inputs: codes and scales bit for bit."""
    x = rows(t, n, 1e-2, 11, pad=8)
    x[0, :8] = torch.tensor([0.0, -0.0, 2.0 ** -133, 1.0, -448.0, 3e38, -3e38, 2.0 ** -60], dtype=torch.bfloat16)
    if t > 2:
        x[1] = 0
        x[2] = x[2] * 2.0 ** -90  # groups above and below the smallest amax
        x[2, ::2] = 0
    codes, scales = quant_buffers(t, n)
    pulse.fp8_group_quant(x, codes[:t], scales[:t])
    want, want_s = ref.quantise(x.float().cpu().numpy())
    np.testing.assert_array_equal(scales[:t].cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    np.testing.assert_array_equal(codes[:t].cpu().numpy(), want)
    untouched(codes, scales)


def test_group_quant_all_magnitudes():
    """Every positive BF16 value as a group's largest, with random values below it."""
    top = np.arange(1, 0x7F80, dtype=np.uint16)
    g = np.random.default_rng(5)
    x = (g.random((top.size, 128)) * top[:, None]).astype(np.uint16) | (g.integers(0, 2, (top.size, 128)).astype(np.uint16) << 15)
    x[:, 77] = top
    t = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    codes, scales = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.empty((top.size, 1), device="cuda")
    pulse.fp8_group_quant(t, codes, scales)
    want, want_s = ref.quantise(t.float().cpu().numpy())
    np.testing.assert_array_equal(scales.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    np.testing.assert_array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("t,n", [(1, 8), (3, 136), (96, 27648), (17, 1408), (129, 1032)])
def test_glu_quant(t, n):
    x = rows(t, 2 * n, 1.5, 13, pad=16)
    x[0, :8] = torch.tensor([80.0, -80.0, 1e4, -1e4, 0.0, -0.0, 100.0, -100.0], dtype=torch.bfloat16)
    codes, scales = quant_buffers(t, n)
    pulse.fp8_group_quant(x, codes[:t], scales[:t], glu=True)
    v = f64(x)
    want = ref.silu(v[:, :n]) * v[:, n:]
    # product, 1 + e, reciprocal (one step), its product and the exponential (one step and two roundings)
    ref.check_codes(codes[:t].cpu().numpy(), scales[:t].cpu().numpy(), want, 9 * ref.HALF_F32)
    untouched(codes, scales)


def test_glu_edges():
    """Gates where the formula has no number, and where it is zero or the gate itself."""
    x = torch.ones((4, 256), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0], x[3, :128] = float("inf"), float("-inf"), float("nan"), -3e38
    codes, scales = torch.empty((4, 128), dtype=torch.uint8, device="cuda"), torch.empty((4, 1), device="cuda")
    pulse.fp8_group_quant(x, codes, scales, glu=True)
    s = scales.cpu().numpy()[:, 0]
    assert np.isinf(s[0]) and np.isnan(s[1]) and np.isnan(s[2])
    # -3e38 / (1 + inf) is -0
    assert s[3] == 1 and ((codes[3].cpu().numpy() & 0x7F) == 0).all()


def test_empty_batches():
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    c, s = torch.empty((0, 256), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), device="cuda")
    w, dw = torch.ones(256, dtype=torch.bfloat16, device="cuda"), torch.full((256,), 2.0, device="cuda")
    pulse.pulse_rms_norm(e, w, codes=c, scales=s)
    pulse.fp8_group_quant(e, c, s)
    r = torch.empty(0, device="cuda")
    pulse.pulse_rms_norm_backward(e, w, r, e, e.clone(), dw, pulse.rms_norm_workspace(0, 256), accumulate=True)
    assert (dw == 2).all()
    pulse.pulse_rms_norm_backward(e, w, r, e, e.clone(), dw, pulse.rms_norm_workspace(0, 256))
    assert (dw == 0).all()
