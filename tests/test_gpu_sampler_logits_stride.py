"""The router's choice from logits in a row stride of their own."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,e,k,pad", [(1, 384, 8, 3), (7, 60, 4, 5), (130, 1000, 6, 24), (33, 129, 2, 1), (5, 200, 32, 7)])
@pytest.mark.parametrize("over_all", [False, True])
def test_a_choice_from_logits_in_a_stride(t, e, k, pad, over_all):
    """Rows of a wider matrix, as a projection with other outputs behind the router's leaves them."""
    g = np.random.default_rng(t)
    logits = g.normal(0, 2, (t, e)).astype(np.float32)
    wide = torch.full((t, e + pad), float("inf"), device="cuda")
    wide[:, :e] = torch.from_numpy(logits).cuda()
    ids, w = torch.empty((t, k), dtype=torch.int32, device="cuda"), torch.empty((t, k), device="cuda")
    pulse.pulse_moe_route(wide[:, :e], ids, w, over_all=over_all)
    want, want_w = ref.route(logits, k, over_all)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    np.testing.assert_allclose(w.cpu().numpy(), want_w, rtol=(e + 8 + 2 * 16) * ref.HALF_F32, atol=1e-30)
