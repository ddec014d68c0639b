"""A layer of an FP8 sampler behind the receiver's pass, its operators one after the other:
each against float64 on what the one before it left, and the gradients' formulas."""
import numpy as np
import pytest
import torch

from examples import fp8_layer as ex
from tests import sampler_ref as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().cpu().double().numpy()


def near(got, y, e):
    """Within the bound of the sums and one rounding to BF16."""
    bad = np.abs(got - y) > 1.02 * (e + (np.abs(y) + e) * ref.HALF_BF16) + 1e-30
    assert not bad.any(), (int(bad.sum()), np.abs(got - y).max())


def cpu(*ts):
    return [t.cpu().numpy() for t in ts]


@pytest.mark.parametrize("tokens", [1, 2, 20, 77, 300])
def test_layer_and_gradients(tokens):
    view, layer, x, front, before, after, dy = ex.run(tokens)
    assert int(view.status.item()) == 0
    up, su, down, sd = cpu(view.up, view.up_scales, view.down, view.down_scales)
    # the codes are those of the patched weights: half a step of E4M3, and the quotient's own rounding
    gate_up = f64(view.bf16[ex.HIDDEN:ex.HIDDEN + 2 * ex.INTER * ex.HIDDEN]).reshape(2 * ex.INTER, ex.HIDDEN)
    s = ref.block_scales(su, up.shape)
    assert (np.abs(ref.E4M3[up] - gate_up / s) <= np.maximum(np.abs(gate_up / s) * ref.HALF_E4M3, 2.0 ** -10) * 1.001).all()

    # forward: norm, products, activation, norm
    want, rstd = ref.rms_norm(f64(before), f64(view.norm), ex.EPS)
    xc, xs = cpu(layer.x, layer.x_scales)
    ref.check_codes(xc, xs, want, ref.rstd_error(ex.HIDDEN) + 2 * ref.HALF_F32)
    near(f64(layer.both), *ref.gemm(xc, xs, up, su, "nt"))
    both = f64(layer.both)
    h = ref.silu(both[:, :ex.INTER]) * both[:, ex.INTER:]
    hc, hs = cpu(layer.h, layer.h_scales)
    ref.check_codes(hc, hs, h, 9 * ref.HALF_F32)
    near(f64(layer.out), *ref.gemm(hc, hs, down, sd, "nt"))
    assert torch.equal(after, (layer.out.float() + before.float()).to(torch.bfloat16))
    last, _ = ref.rms_norm(f64(after), f64(view.last_norm), ex.EPS)
    np.testing.assert_allclose(f64(layer.last), last, rtol=1.02 * (ref.rstd_error(ex.HIDDEN) + 2 * ref.HALF_F32 + ref.HALF_BF16))
    # the experts
    ids, shares = ref.route(layer.logits.cpu().numpy(), ex.TOP_K)
    np.testing.assert_array_equal(layer.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(f64(layer.shares), shares, rtol=1e-5)
    near(f64(layer.mixed), *ref.moe(f64(layer.last), ids, layer.shares.cpu().numpy(), *cpu(
        view.experts_up, view.experts_up_scales, view.experts_down, view.experts_down_scales)))

    # gradients, step by step
    dyc, dys = cpu(layer.dy, layer.dy_scales)
    want_c, want_s = ref.quantise(dy.float().cpu().numpy())
    np.testing.assert_array_equal(dyc, want_c)
    np.testing.assert_array_equal(dys, want_s)
    near(f64(layer.dh), *ref.gemm(dyc, dys, down, sd, "nn"))
    dbc, dbs = cpu(layer.dboth, layer.dboth_scales)
    want_c, _ = ref.quantise(layer.dgate_up.float().cpu().numpy())
    np.testing.assert_array_equal(dbc, want_c)
    near(f64(layer.dnorm), *ref.gemm(dbc, dbs, up, su, "nn"))
    a, w, d = f64(before), f64(view.norm), f64(layer.dnorm)
    dx, dw = ref.rms_norm_backward(a, w, d, ex.EPS, f64(dy))
    hat, n = a * rstd[:, None], ex.HIDDEN
    room = rstd[:, None] * (np.abs(d * w) + np.abs(hat) * np.abs(d * w * hat).mean(axis=1, keepdims=True)) * (n + 20) * ref.HALF_F32
    assert (np.abs(f64(layer.dx) - dx) <= 1.02 * (room + np.abs(dx) * ref.HALF_BF16)).all()
    room = np.abs(d * hat).sum(axis=0) * (tokens + n) * ref.HALF_F32
    assert (np.abs(f64(layer.dweight) - dw) <= room + 1e-30).all()


def test_the_gradients_formula_against_differences():
    """The float64 gradient that the example's steps follow, of norm, [gate; up], activation, down
    and the residual, against differences of the float64 layer."""
    g = np.random.default_rng(2)
    t, n, i = 2, 12, 8
    x, w, up, down = g.normal(0, 1, (t, n)), 1 + g.normal(0, 0.1, n), g.normal(0, 0.3, (2 * i, n)), g.normal(0, 0.3, (n, i))
    dy = g.normal(0, 1, (t, n))

    def layer(x, w):
        both = ref.rms_norm(x, w, ex.EPS)[0] @ up.T
        return x + (ref.silu(both[:, :i]) * both[:, i:]) @ down.T

    both = ref.rms_norm(x, w, ex.EPS)[0] @ up.T
    gate, u, s = both[:, :i], both[:, i:], 1 / (1 + np.exp(-both[:, :i]))
    d = dy @ down
    dboth = np.concatenate([d * u * s * (1 + gate * (1 - s)), d * gate * s], axis=1)
    dx, dw = ref.rms_norm_backward(x, w, dboth @ up, ex.EPS, dy)
    step = 1e-6
    for k in range(t * n):
        e = np.zeros(t * n)
        e[k] = step
        diff = ((layer(x + e.reshape(t, n), w) - layer(x - e.reshape(t, n), w)) * dy).sum() / (2 * step)
        assert abs(dx.ravel()[k] - diff) < 1e-6
    for k in range(n):
        e = np.zeros(n)
        e[k] = step
        assert abs(dw[k] - ((layer(x, w + e) - layer(x, w - e)) * dy).sum() / (2 * step)) < 1e-6
