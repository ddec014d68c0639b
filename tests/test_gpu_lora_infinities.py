"""Where infinities are in y, dx, dA and dB, and what h above the largest BF16 gives."""
import numpy as np
import pytest

from tests import lora_ref as ref
from tests.lora_exact import bf16_round, spread_ids
from tests.test_gpu_lora_precision import run

pytestmark = pytest.mark.gpu


def kinds(v):
    """Finite, +inf, -inf or NaN, of every value."""
    return np.where(np.isnan(v), 3, np.where(np.isposinf(v), 1, np.where(np.isneginf(v), 2, 0)))


@pytest.mark.parametrize("where", ["x", "dy", "a", "b", "scale", "all"])
@pytest.mark.parametrize("t,k,n,r,s", [(1, 72, 136, 24, 1), (65, 520, 1032, 40, 2), (100, 264, 136, 16, 30), (2, 14344, 136, 128, 1),
                                       (1500, 136, 264, 128, 3), (4200, 64, 8200, 24, 300)])
def test_infinities_are_where_the_formula_has_them(where, t, k, n, r, s):
    """Also where h has few bits and the parts below the first are zero: an infinity times
    such a part would be NaN.  All sums are exact in float32, so none is zero in one
    computation and not in the other."""
    rng = np.random.default_rng(t + r)
    ids = spread_ids(t, s)
    draw = lambda *shape: rng.choice([-1.0, 1.0], shape) * 2.0 ** rng.integers(-3, 3, shape)  # noqa: E731
    x, a, b, y, dy, dx = draw(t, k), draw(s, r, k), draw(s, r, n), draw(t, n), draw(t, n), draw(t, k)
    sc = np.ones(s)
    sparse = rng.random(a.shape) < 1 - 2.0 / k  # a few products in a sum: many h of few bits
    a[sparse] = 2.0 ** -12 if where in ("x", "all") else 0.0
    for name, v in (("x", x), ("dy", dy), ("a", a), ("b", b)):
        if where in (name, "all"):
            for at in rng.integers(0, v.size, 2):
                v.reshape(-1)[at] = rng.choice([np.inf, -np.inf])
    if where == "scale":
        sc[s // 2] = np.inf
    with np.errstate(all="ignore"):
        yw, _ = ref.forward(x, a, b, sc, ids, y)
        dxw, daw, dbw, _ = ref.backward(x, dy, a, b, sc, ids, dx)
    for name, got, want in zip(("y", "dx", "da", "db"), run(x, a, b, sc, ids, y, dy, dx), (yw, dxw, daw, dbw)):
        assert np.array_equal(kinds(got), kinds(want)), name
    got = run(x, a, b, sc, ids, y)[0]
    assert np.array_equal(kinds(got), kinds(yw))


@pytest.mark.parametrize("t,k,n,r,s", [(1, 72, 136, 24, 1), (300, 264, 1032, 40, 7), (4200, 64, 8200, 16, 3)])
def test_h_above_the_largest_bf16_stays_finite(t, k, n, r, s):
    """h = 1.0019 times the largest BF16 is a float32 number, and so are its products with
    a quarter: y, dx, dA and dB are finite, within the roundings of their own types."""
    ids = spread_ids(t, s)
    most, sc = float(bf16_round(np.float64(3.3895313892515355e38))), np.full(s, np.float32(1.0019))
    h = most * float(sc[0])
    one = lambda *shape: np.eye(1, int(np.prod(shape[1:])), 0).repeat(shape[0], 0).reshape(shape)  # noqa: E731
    # x and dy: 1 in the first column; A and B: the largest BF16 at rank 0, column 0, 1/4 at column 1 of rank 0
    x, dy, a, b = one(t, k), one(t, n), np.zeros((s, r, k)), np.zeros((s, r, n))
    a[:, 0, 0] = b[:, 0, 0] = most
    a[:, 0, 1] = b[:, 0, 1] = 0.25
    first = np.zeros(t, bool)  # a single token of each adapter counts in the sums
    first[[np.flatnonzero(ids == i)[0] for i in set(ids.tolist()) - {-1}]] = True
    x[~first], dy[~first] = 0, 0
    x[first, 1], dy[first, 1] = 0.5, 0.5
    h2 = h + float(sc[0]) * 0.125  # absorbed: the same number in any type here
    assert np.float32(h2) == np.float32(h)
    y, dx, da, db = run(x, a, b, sc, ids, np.zeros((t, n)), dy, np.zeros((t, k)))
    for rows, grad in ((y, db), (dx, da)):
        assert np.all(np.abs(rows[first, 1] - h * 0.25) <= h * 0.25 * (2.0 ** -8 + 2.0 ** -16 + 2.0 ** -20))
        assert not rows[~first].any()
        for i in sorted(set(ids.tolist()) - {-1}):
            assert abs(grad[i, 0, 1] - h * 0.5) <= h * 0.5 * 2.0 ** -22 and abs(grad[i, 0, 0] - h) <= h * 2.0 ** -22
