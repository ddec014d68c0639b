"""Pins of the sampler's float64 reference: worked values, torch's own operators and
gradients, and the E4M3 of the codec's oracle."""
import numpy as np
import torch

import oracle
from tests import sampler_ref as ref


def test_e4m3_table_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.isnan(ref.E4M3), np.isnan(want))
    fine = ~np.isnan(want)
    np.testing.assert_array_equal(ref.E4M3[fine], want[fine])


def test_quantise_is_the_block_quantisers_rule():
    """Rows in groups of 128: what the oracle gives for a matrix of one such row each."""
    g = np.random.default_rng(1)
    x = ref.bf16(g.normal(0, 2, (5, 300)))
    codes, scales = ref.quantise(x)
    for r in range(5):
        bits = oracle.cast_bf16(x[r].astype(np.float32)).reshape(1, -1)
        # 300 columns are no multiple of 8: padded with zeros, which change no maximum
        c, s = oracle.fp8_block_quant([np.pad(bits, ((0, 0), (0, 4)))])
        np.testing.assert_array_equal(codes[r], np.asarray(c).reshape(-1)[:300])
        np.testing.assert_array_equal(scales[r], np.asarray(s).reshape(-1))


def test_quantise_below_its_smallest_maximum():
    x = np.zeros((3, 128), dtype=np.float32)
    x[0, 0], x[1, 0], x[2, 0] = 2.0 ** -96, np.nextafter(np.float32(2.0 ** -96), np.float32(0)), -0.0
    codes, scales = ref.quantise(x)
    assert codes[0, 0] == 0x7E and scales[0, 0] == np.float32(2.0 ** -96) / np.float32(448)
    assert (codes[1] == 0).all() and scales[1, 0] == 1
    assert codes[2, 0] == 0x80 and scales[2, 0] == 1


def test_norm_and_its_gradients_are_autograds():
    g = torch.Generator().manual_seed(2)
    s = torch.randn(4, 24, dtype=torch.float64, generator=g, requires_grad=True)
    w = torch.randn(24, dtype=torch.float64, generator=g, requires_grad=True)
    dy, dres = torch.randn(4, 24, dtype=torch.float64, generator=g), torch.randn(4, 24, dtype=torch.float64, generator=g)
    y = s * torch.rsqrt((s * s).mean(dim=1, keepdim=True) + 1e-6) * w
    ((y * dy).sum() + (s * dres).sum()).backward()
    want, _ = ref.rms_norm(s.detach().numpy(), w.detach().numpy(), 1e-6)
    np.testing.assert_allclose(want, y.detach().numpy(), rtol=1e-12)
    dx, dw = ref.rms_norm_backward(s.detach().numpy(), w.detach().numpy(), dy.numpy(), 1e-6, dres.numpy())
    np.testing.assert_allclose(dx, s.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-10)


def test_gemm_is_the_product_of_the_values():
    g = np.random.default_rng(3)
    n, k = 200, 304
    x, dy, w = g.integers(0, 127, (3, k)).astype(np.uint8), g.integers(0, 127, (3, n)).astype(np.uint8), g.integers(0, 127, (n, k)).astype(np.uint8)
    sx, sd, sw = (g.uniform(0.5, 2, s).astype(np.float32) for s in ((3, 3), (3, 2), (2, 3)))
    y, e = ref.gemm(x, sx, w, sw, "nt")
    np.testing.assert_allclose(y, ref.row_values(x, sx) @ ref.block_values(w, sw).T, rtol=1e-12)
    dx, e2 = ref.gemm(dy, sd, w, sw, "nn")
    np.testing.assert_allclose(dx, ref.row_values(dy, sd) @ ref.block_values(w, sw), rtol=1e-12)
    assert (e > 0).all() and (e2 > 0).all()


def test_moe_is_torchs():
    g = np.random.default_rng(4)
    t, h, i, e, k = 3, 32, 16, 4, 2
    up, down = g.integers(0, 100, (e, 2 * i, h)).astype(np.uint8), g.integers(0, 100, (e, h, i)).astype(np.uint8)
    su, sd = np.full((e, 1, 1), 0.01, np.float32), np.full((e, 1, 1), 0.02, np.float32)
    x, ids, p = g.normal(0, 1, (t, h)), np.array([[0, 3], [3, -1], [2, 2]]), g.uniform(0, 1, (t, k)).astype(np.float32)
    y, _ = ref.moe(x, ids, p, up, su, down, sd)
    want = np.zeros((t, h))
    for a in range(t):
        for j in range(k):
            if ids[a, j] >= 0:
                both = torch.from_numpy(ref.block_values(up[ids[a, j]], su[ids[a, j]])) @ torch.from_numpy(x[a])
                hid = torch.nn.functional.silu(both[:i]) * both[i:]
                want[a] += p[a, j] * (ref.block_values(down[ids[a, j]], sd[ids[a, j]]) @ hid.numpy())
    np.testing.assert_allclose(y, want, rtol=1e-10)


def test_route_is_a_stable_sort_and_a_softmax():
    g = np.random.default_rng(5)
    logits = np.round(g.normal(0, 2, (40, 30))).astype(np.float32)
    ids, w = ref.route(logits, 6)
    order = torch.sort(torch.from_numpy(logits), dim=1, descending=True, stable=True)
    np.testing.assert_array_equal(ids, order.indices[:, :6].numpy())
    np.testing.assert_allclose(w, torch.softmax(order.values[:, :6].double(), 1).numpy(), rtol=1e-12)
    _, w = ref.route(logits, 6, over_all=True, scale=2.0)
    np.testing.assert_allclose(w, 2 * torch.softmax(torch.from_numpy(logits).double(), 1).gather(1, order.indices[:, :6]).numpy(), rtol=1e-12)


def test_route_edges():
    inf, nan = np.inf, np.nan
    logits = np.array([[-inf, 1, -inf], [-inf] * 3, [0, nan, 5]], dtype=np.float32)
    ids, w = ref.route(logits, 2)
    np.testing.assert_array_equal(ids, [[1, -1], [-1, -1], [1, 2]])
    np.testing.assert_array_equal(w[:2], [[1, 0], [0, 0]])
    assert np.isnan(w[2]).all()
