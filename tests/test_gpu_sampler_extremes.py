"""The sampler's calls at the largest sizes that they take, one at a time."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref
from tests.test_gpu_sampler_moe import check, forward, layer

pytestmark = pytest.mark.gpu

MOST = 2 ** 24 - 1  # rows
SIDE = 2 ** 22      # of a product's weights


def whole(shape, seed):
    """-8 ... 8 in E4M3."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-8, 9, shape, device="cuda", generator=gen, dtype=torch.int8).to(torch.bfloat16)


def codes(t):
    return t.to(torch.float8_e4m3fn).view(torch.uint8)


def test_rows_of_the_norm():
    n = 8
    x, w = whole((MOST, n), 1), torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(MOST, device="cuda")
    c, s = torch.empty((MOST, n), dtype=torch.uint8, device="cuda"), torch.empty((MOST, 1), device="cuda")
    pulse.pulse_rms_norm(x, w, y=y, codes=c, scales=s, rstd=rstd)
    want = torch.rsqrt(x.double().square().mean(1) + 1e-6)
    # eight squares, mean, eps, root, quotient
    assert ((rstd.double() / want - 1).abs() <= 1.02 * 10 * ref.HALF_F32).all()
    hat = x.double() * want[:, None]
    assert ((y.double() - hat).abs() <= hat.abs() * 1.02 * (ref.HALF_BF16 + 12 * ref.HALF_F32)).all()
    live = hat.abs().amax(1) > 0
    assert ((s[:, 0].double() * 448 / hat.abs().amax(1) - 1).abs()[live] <= 1.02 * 13 * ref.HALF_F32).all()
    assert (c.view(torch.float8_e4m3fn).float().abs().amax(1)[live] == 448).all() and ((c[~live] & 0x7F) == 0).all()
    dx, dw = torch.empty_like(x), torch.empty(n, device="cuda")
    pulse.pulse_rms_norm_backward(x, w, rstd, x, dx, dw, pulse.rms_norm_workspace(MOST, n))
    r = rstd.double()[:, None]
    want = (x.double().square() * r).sum(0)
    # each of 512 workgroups adds up 2^15 rows, then their parts
    assert ((dw.double() / want - 1).abs() <= 1.02 * (2 ** 15 + 20) * ref.HALF_F32).all()
    a = x.double() * r
    mean = (x.double() * a).mean(1, keepdim=True)
    bound = r * (x.double().abs() * 3 + a.abs() * mean * 4 + a.abs() * mean * 12) * ref.HALF_F32
    want = r * (x.double() - a * mean)
    assert ((dx.double() - want).abs() <= 1.02 * (bound + (want.abs() + bound) * ref.HALF_BF16) + 1e-35).all()


@pytest.mark.parametrize("t,cols", [(MOST, 8), (1, 2 ** 24), (4095, 8200)])
def test_the_quantiser(t, cols):
    x = whole((t, cols), 2)
    x[:, ::128] = 7  # every group's largest is 7 or 8: scales of 1/64 and 8/448
    c, s = torch.empty((t, cols), dtype=torch.uint8, device="cuda"), torch.empty((t, ref.groups(cols)), device="cuda")
    pulse.fp8_group_quant(x, c, s)
    for at in range(0, t, 2 ** 20):
        rows = x[at:at + 2 ** 20].float()
        amax = torch.nn.functional.pad(rows, (0, -cols % 128)).view(rows.shape[0], -1, 128).abs().amax(2)
        # (7 / 448 is 2^-6, 8 / 448 rounded once, as numpy's)
        want = torch.where(amax == 8, float(np.float32(8) / np.float32(448)), 2.0 ** -6)
        assert torch.equal(s[at:at + 2 ** 20], want)
        full = want.repeat_interleave(128, 1)[:, :cols].double()
        q = rows.double() / full
        half = torch.pow(2.0, torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 4)
        err = (c[at:at + 2 ** 20].view(torch.float8_e4m3fn).double() - q).abs()
        assert (err <= half + q.abs() * 2 * ref.HALF_F32).all()


def product(m, n, k, form):
    """Whole numbers: sparse along the contraction, so that float32 holds every sum."""
    inner, out = (k, n) if form == "nt" else (n, k)
    x, w = whole((m, inner), 3), whole((n, k), 4)
    if inner > 4096:
        keep = torch.zeros(inner, dtype=torch.bool, device="cuda")
        keep[torch.randint(0, inner, (900,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))] = True
        keep[-1] = keep[0] = True
        x.mul_(keep)
    one = lambda a, b: torch.ones((a, b), device="cuda")  # noqa: E731
    y = torch.full((m + 1, out), -77.0, dtype=torch.bfloat16, device="cuda")
    pulse.fp8_block_gemm(codes(x), one(m, ref.groups(inner)), codes(w), one(ref.groups(n), ref.groups(k)), y[:m],
                         pulse.fp8_gemm_workspace(m, n, k, form), form=form)
    assert (y[m] == -77).all()
    for at in range(0, m, 2 ** 20):
        rows = x[at:at + 2 ** 20].float()
        want = rows @ (w.float().t() if form == "nt" else w.float())  # exact in float32
        assert torch.equal(y[at:min(m, at + 2 ** 20)], want.to(torch.bfloat16))


@pytest.mark.parametrize("m,n,k,form", [(1, 16, SIDE, "nt"), (9, 40, SIDE, "nt"), (20, 16, SIDE, "nt"), (300, 130, SIDE, "nt"), (1, SIDE, 16, "nt"),
                                        (20, SIDE, 16, "nt"), (1, SIDE, 16, "nn"), (40, SIDE, 144, "nn"), (1, 16, SIDE, "nn"), (20, 16, SIDE, "nn"),
                                        (MOST, 16, 16, "nt"), (MOST, 16, 16, "nn")])
def test_products(m, n, k, form):
    product(m, n, k, form)


def test_rows_of_the_router():
    logits = whole((MOST, 3), 6).float()
    ids, w = torch.empty((MOST, 2), dtype=torch.int32, device="cuda"), torch.empty((MOST, 2), device="cuda")
    pulse.pulse_moe_route(logits, ids, w)
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids, order.indices[:, :2].int())
    want = torch.softmax(order.values[:, :2].double(), 1)
    assert ((w.double() / want - 1).abs() <= 1.02 * (8 + 2 * 16) * ref.HALF_F32).all()


@pytest.mark.parametrize("t", [1, 2, 3, 24])
@pytest.mark.parametrize("h,i", [(65536, 16), (16, 65536)])
def test_widths_of_the_experts(t, h, i):
    args = layer(t, h, i, 2, 1, 21)
    check(forward(*args, pad=8), *ref.moe(*args))


@pytest.mark.parametrize("t,e,k", [(1024, 1024, 8), (1024, 64, 8), (256, 40, 32), (1024, 8, 8), (1024, 1024, 1)])
def test_pairs_of_the_experts(t, e, k):
    args = layer(t, 144, 48, e, k, 22)
    check(forward(*args), *ref.moe(*args))


def test_a_stride_of_2_20():
    args = list(layer(3, 272, 144, 4, 2, 23))
    clean = forward(*args)
    wide = torch.zeros((3, 2 ** 20), dtype=torch.bfloat16, device="cuda")
    wide[:, :272] = torch.from_numpy(args[0]).cuda()
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    y, st = torch.empty((3, 272), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pulse.pulse_moe_forward(wide[:, :272], *map(dev, args[1:]), y, st, pulse.moe_workspace(3, 272, 144, 4, 2))
    np.testing.assert_array_equal(y.double().cpu().numpy(), clean)


@pytest.mark.parametrize("h,i", [(65536, 16), (16, 65536)])
def test_all_pairs_at_the_widest(h, i):
    """1024 tokens with 8 of 16 experts: the first and the last tokens' results are those of them alone."""
    t, e, k = 1024, 16, 8
    args = list(layer(8, h, i, e, k, 24))
    g = np.random.default_rng(25)
    args[0] = ref.bf16(g.standard_normal((t, h), dtype=np.float32))
    args[1] = np.stack([g.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    args[2] = g.uniform(0.1, 1, (t, k)).astype(np.float32)
    got = forward(*args)
    for rows in (slice(0, 4), slice(t - 4, t)):
        some = [a[rows] for a in args[:3]] + args[3:]
        alone = forward(*some)
        np.testing.assert_array_equal(got[rows], alone)
        check(alone, *ref.moe(*some))
