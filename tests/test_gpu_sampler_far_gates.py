"""silu(gate) * up between gates of -60 and -104, where e^-gate nears and passes float32's range
and a large up brings the product back: the quantiser and the expert layer against float64."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref

pytestmark = pytest.mark.gpu

GATES = np.arange(-60.0, -104.5, -0.5)  # in BF16 as they are


def far_error(gate):
    """Relative: the roundings that silu has everywhere, and half a step of float32's subnormal numbers."""
    return 9 * ref.HALF_F32 + 2.0 ** -150 / np.abs(ref.silu(gate))


def test_quantised_rows():
    """A gate a row with ups from 1e37 to 3e38; ordinary gates and ups in the group beside them."""
    g = np.random.default_rng(1)
    n = GATES.size
    up = ref.bf16(10.0 ** g.uniform(37, 38.47, (n, 128)) * g.choice([-1, 1], (n, 128)))
    near, near_up = ref.bf16(g.normal(0, 1.5, (n, 128))), ref.bf16(g.normal(0, 1.5, (n, 128)))
    x = np.concatenate([np.repeat(GATES[:, None], 128, axis=1), near, up, near_up], axis=1)
    codes, scales = torch.empty((n, 256), dtype=torch.uint8, device="cuda"), torch.empty((n, 2), device="cuda")
    pulse.fp8_group_quant(torch.from_numpy(x).to(torch.bfloat16).cuda(), codes, scales, glu=True)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    for r, gate in enumerate(GATES):
        ref.check_codes(codes[r:r + 1, :128], scales[r:r + 1, :1], ref.silu(gate) * up[r:r + 1], far_error(gate))
    ref.check_codes(codes[:, 128:], scales[:, 1:], ref.silu(near) * near_up, 9 * ref.HALF_F32)


@pytest.mark.parametrize("t", [1, 2, 3, 20])
def test_experts(t):
    """One product in each sum, so that gate and up are exact: gate -72, -80, -88 and -96, up 448 * 2^118."""
    n = 16
    gates = -np.array([72.0, 80.0, 88.0, 96.0] * 4)
    code = lambda v: torch.from_numpy(np.asarray(v)).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    up = np.zeros((1, 2 * n, n))
    up[0, np.arange(n), 0], up[0, n:, 1] = gates, 448
    x = np.zeros((t, n))
    x[:, 0], x[:, 1] = 1, 2.0 ** 118
    y = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    status, one = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones((1, 1, 1), device="cuda")
    pulse.pulse_moe_forward(torch.from_numpy(x).to(torch.bfloat16).cuda(), torch.zeros((t, 1), dtype=torch.int32, device="cuda"),
                            torch.ones((t, 1), device="cuda"), code(up).cuda(), one, code(np.eye(n)[None]).cuda(), one, y, status,
                            pulse.moe_workspace(t, n, n, 1, 1))
    assert int(status.item()) == 0
    want = ref.silu(gates) * 448 * 2.0 ** 118
    # silu's error, what two BF16 leave out, and y's rounding
    room = np.abs(want) * (far_error(gates) + 2.0 ** -16 + ref.HALF_BF16) * 1.02
    assert (np.abs(y.double().cpu().numpy() - want[None]) <= room[None]).all()
