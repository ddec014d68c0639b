"""The router's choice and the expert layer for a few tokens against float64."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref
from tests.test_gpu_sampler_gemm import codes_like

pytestmark = pytest.mark.gpu


def choose(logits, top_k, **kw):
    t = logits.shape[0]
    ids = torch.full((t + 1, top_k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((t + 1, top_k), 99.0, device="cuda")
    pulse.pulse_moe_route(torch.from_numpy(logits).cuda(), ids[:t], w[:t], **kw)
    assert (ids[t] == 99).all() and (w[t] == 99).all()
    return ids[:t].cpu().numpy(), w[:t].cpu().numpy()


@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 384, 8), (7, 8, 2), (61, 60, 4), (5, 129, 32), (130, 1000, 6), (33, 1024, 1), (4, 40, 32)])
@pytest.mark.parametrize("over_all", [False, True])
def test_route(t, e, k, over_all):
    g = np.random.default_rng(t + e)
    logits = g.normal(0, 2, (t, e)).astype(np.float32)
    logits[::3] = np.round(logits[::3])  # many equal ones
    if t > 4 and e > 4:
        logits[1, 2], logits[2] = -np.inf, -np.inf
        logits[3, 1:] = -np.inf
    ids, w = choose(logits, k, over_all=over_all, scale=2.5)
    want, want_w = ref.route(logits, k, over_all, 2.5)
    np.testing.assert_array_equal(ids, want)
    # exponentials (of differences, one step), a sum of at most e of them, quotient and product
    np.testing.assert_allclose(w, want_w, rtol=(e + 8 + 2 * 16) * ref.HALF_F32, atol=1e-30)


def test_route_takes_nan_and_infinity():
    logits = np.zeros((4, 70), dtype=np.float32)
    logits[0, 66] = np.nan
    logits[1, 3] = np.inf
    logits[2, 5], logits[2, 6] = 3e38, -3e38
    logits[3] = -3.4e38
    ids, w = choose(logits, 3)
    want, _ = ref.route(logits, 3)
    np.testing.assert_array_equal(ids, want)
    assert np.isnan(w[0]).all() and np.isnan(w[1, 0])
    np.testing.assert_array_equal(w[2], [1, 0, 0])
    np.testing.assert_allclose(w[3], [1 / 3] * 3, rtol=1e-6)


def layer(t, h, i, e, k, seed=0):
    g = np.random.default_rng(seed + t + h + i + e)
    up, down = codes_like((e, 2 * i, h), g), codes_like((e, h, i), g)
    su = (g.uniform(0.5, 2, (e, ref.groups(2 * i), ref.groups(h))) / 60 / np.sqrt(h)).astype(np.float32)
    sd = (g.uniform(0.5, 2, (e, ref.groups(h), ref.groups(i))) / 60 / np.sqrt(i)).astype(np.float32)
    x = ref.bf16(g.normal(0, 1, (t, h)))
    ids = np.stack([g.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    weights = g.uniform(0.1, 1, (t, k)).astype(np.float32)
    return x, ids, weights, up, su, down, sd


def forward(x, ids, weights, up, su, down, sd, pad=0, ws=None, status=0):
    t, h = x.shape
    e, _, i = down.shape
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    xs = torch.zeros((t, h + pad), dtype=torch.bfloat16, device="cuda")
    xs[:, :h] = torch.from_numpy(x).cuda()
    y = torch.full((t + 1, h + pad), -77.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = pulse.moe_workspace(t, h, i, e, ids.shape[1]) if ws is None else ws
    ws.fill_(255)
    pulse.pulse_moe_forward(xs[:, :h], dev(ids), dev(weights), dev(up), dev(su), dev(down), dev(sd), y[:t, :h], st, ws)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    assert (y[t] == -77).all() and (y[:, h:] == -77).all()
    return y[:t, :h].double().cpu().numpy()


def check(got, y, e):
    bad = np.abs(got - y) > 1.02 * (e + (np.abs(y) + e) * ref.HALF_BF16) + 1e-30
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(got - y).max())


SHAPES = [(1, 16, 16, 1, 1), (1, 256, 128, 4, 2), (1, 272, 144, 8, 3), (2, 1040, 208, 6, 2), (1, 4112, 272, 12, 8), (2, 528, 4112, 3, 2),
          (3, 256, 256, 5, 2), (5, 400, 80, 9, 4), (17, 272, 144, 4, 2), (40, 304, 176, 6, 3), (33, 512, 64, 1, 1), (64, 256, 336, 3, 2),
          (100, 144, 48, 4, 4), (130, 128, 128, 2, 1), (9, 784, 528, 200, 8)]


@pytest.mark.parametrize("t,h,i,e,k", SHAPES)
def test_layer(t, h, i, e, k):
    args = layer(t, h, i, e, k)
    check(forward(*args, pad=(0, 8, 24)[t % 3]), *ref.moe(*args))


@pytest.mark.parametrize("t", [1, 2, 6, 40])
def test_places_without_an_expert(t):
    """-1 is left out, a token without any has zeros; the same expert twice counts twice."""
    args = list(layer(t, 272, 144, 4, 3, 5))
    ids = args[1]
    ids[0] = [2, 2, 2]
    if t > 1:
        ids[1] = -1
    if t > 2:
        ids[2] = [-1, 3, -1]
    got = forward(*args)
    check(got, *ref.moe(*args))
    if t > 1:
        assert (got[1] == 0).all()


@pytest.mark.parametrize("t", [1, 5])
def test_no_expert_at_all(t):
    args = list(layer(t, 272, 144, 4, 2, 6))
    args[1][:] = -1
    assert (forward(*args) == 0).all()


@pytest.mark.parametrize("t", [1, 2, 20])
def test_bad_ids_are_reported_and_left_out(t):
    args = list(layer(t, 272, 144, 4, 2, 7))
    args[1][0] = [4, 1]
    got = forward(*args, status=pulse.PULSE_DS_BADINDEX)
    check(got, *ref.moe(*args))
    args[1][0] = [-5, 2 ** 31 - 1]
    got = forward(*args, status=pulse.PULSE_DS_BADINDEX)
    assert (got[0] == 0).all()


@pytest.mark.parametrize("t", [1, 24])
def test_repeats_bit_for_bit(t):
    args = layer(t, 512, 272, 6, 3, 8)
    np.testing.assert_array_equal(forward(*args), forward(*args))


@pytest.mark.parametrize("t", [1, 3, 24])
def test_an_unused_experts_nan_stays_out(t):
    """Codes of experts that no token has are not multiplied with anything."""
    args = list(layer(t, 272, 144, 5, 2, 9))
    args[1][args[1] == 3] = 0
    clean = forward(*args)
    args[3][3], args[5][3], args[4][3], args[6][3] = 0x7F, 0x7F, np.nan, np.nan
    np.testing.assert_array_equal(forward(*args), clean)


def test_infinite_input_reaches_its_token_only():
    args = list(layer(6, 272, 144, 4, 2, 10))
    clean = forward(*args)
    args[0][2, 270] = np.inf
    got = forward(*args)
    assert not np.isfinite(got[2]).any()
    keep = np.arange(6) != 2
    np.testing.assert_array_equal(got[keep], clean[keep])


def test_no_tokens():
    args = list(layer(2, 64, 32, 3, 2))
    for a in range(3):
        args[a] = args[a][:0]
    assert forward(*args).shape == (0, 64)


@pytest.mark.parametrize("t,e,k", [(1, 40, 32), (2, 40, 32), (2, 3, 3), (3, 33, 32), (100, 50, 1), (70, 300, 2), (300, 5, 2), (1000, 3, 2)])
def test_crowded_experts(t, e, k):
    """Nearly all tokens at one expert: many items of it, and most experts without any."""
    args = list(layer(t, 144, 48, e, k, 11))
    g = np.random.default_rng(t)
    args[1][g.random(args[1].shape) < 0.9] = min(7, e - 1)
    check(forward(*args), *ref.moe(*args))


def test_routed_tokens_end_to_end():
    """The router's choice fed on: an expert with -inf is left out, a token with nothing but -inf has zeros."""
    t, e, k = 50, 12, 3
    g = np.random.default_rng(3)
    logits = g.normal(0, 1, (t, e)).astype(np.float32)
    logits[:, 4], logits[10], logits[11, 2:] = -np.inf, -np.inf, -np.inf
    ids, w = choose(logits, k)
    args = list(layer(t, 272, 144, e, k, 12))
    args[1], args[2] = ids, w
    got = forward(*args)
    check(got, *ref.moe(*args))
    assert (ids != 4).all() and (ids[10] == -1).all() and (got[10] == 0).all() and (ids[11] == [*np.argsort(-logits[11, :2]), -1]).all()


def test_codes_past_31_bits():
    """Experts whose codes begin past 2^31: the last expert's results are those of it alone."""
    h, i, e = 4096, 1024, 520  # up: 4.4e9 codes, down 2.2e9
    args = list(layer(3, h, i, 1, 1, 13))
    x, _, weights, up, su, down, sd = args
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    alone = forward(*args)
    big_up, big_down = (torch.zeros((e, *a.shape[1:]), dtype=torch.uint8, device="cuda") for a in (up, down))
    big_su, big_sd = (torch.ones((e, *a.shape[1:]), device="cuda") for a in (su, sd))
    for b, a in ((big_up, up), (big_down, down), (big_su, su), (big_sd, sd)):
        b[e - 1] = dev(a[0])
    for t in (1, 3):
        ids = torch.full((t, 1), e - 1, dtype=torch.int32, device="cuda")
        y, st = torch.empty((t, h), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        pulse.pulse_moe_forward(dev(x[:t]).to(torch.bfloat16), ids, dev(weights[:t]), big_up, big_su, big_down, big_sd, y, st,
                                pulse.moe_workspace(t, h, i, e, 1))
        got = y.double().cpu().numpy()
        # (one token's sums are made in another order than three's)
        check(got, *ref.moe(x[:t], np.zeros((t, 1), dtype=int), weights[:t], up, su, down, sd))
        if t == 3:
            np.testing.assert_array_equal(got, alone)
