"""The router's choice at every number of logits that a lane may hold, and one to either side."""
import numpy as np
import pytest

from tests import sampler_ref as ref
from tests.test_gpu_sampler_moe import choose, pytestmark  # noqa: F401

SIZES = sorted({min(1024, max(1, 64 * i + d)) for i in range(17) for d in (-1, 0, 1)})


@pytest.mark.parametrize("over_all", [False, True])
@pytest.mark.parametrize("e", SIZES)
def test_route(e, over_all):
    """The largest logits at both ends, and equal ones across the lanes."""
    g = np.random.default_rng(e)
    logits = np.round(g.normal(0, 2, (9, e))).astype(np.float32)
    logits[0, -1], logits[1, 0], logits[2] = 50, 50, 1
    logits[3, :-1] = -np.inf
    k = min(6, e)
    ids, w = choose(logits, k, over_all=over_all)
    want, want_w = ref.route(logits, k, over_all)
    np.testing.assert_array_equal(ids, want)
    np.testing.assert_allclose(w, want_w, rtol=(e + 8 + 2 * 52) * ref.HALF_F32, atol=1e-30)
