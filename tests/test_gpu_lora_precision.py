"""What the roundings of h and dh may not lose, on data whose results are exact, at every
size where another kernel takes over."""
import numpy as np
import pytest
import torch

from tests.lora_exact import spread_ids, whole_rows

try:
    import sparse_delta_codec_amd as pulse
except ImportError:
    if torch.cuda.is_available():
        raise
    pulse = None

from tests.gpu_util import host, zeros  # noqa: E402


def cuda16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def run(x, a, b, sc, ids, y, dy=None, dx=None):
    """Forward, and with dy backward too: (y, dx, da, db)."""
    (t, k), (s, r, n) = x.shape, b.shape
    X, A, B, Y, SC = cuda16(x), cuda16(a), cuda16(b), cuda16(y), torch.from_numpy(np.asarray(sc, np.float32)).cuda()
    plan, st = pulse.LoraPlan(t, s), zeros(1, torch.int32)
    pulse.pulse_lora_plan(plan, torch.from_numpy(ids.astype(np.int32)).cuda(), st)
    train = dy is not None
    ws = pulse.lora_workspace(t, k, n, r, s, train=train)
    ws.fill_(255)
    if not train:
        pulse.pulse_lora_forward(X, A, B, SC, plan, Y, ws)
        torch.cuda.synchronize()
        return f64(Y), None, None, None
    h, DY, DX = pulse.lora_hidden(t, r, s), cuda16(dy), cuda16(dx)
    h.fill_(255)
    da, db = torch.full((s, r, k), 9.0, device="cuda"), torch.full((s, r, n), 9.0, device="cuda")
    pulse.pulse_lora_forward(X, A, B, SC, plan, Y, ws, h=h)
    pulse.pulse_lora_backward(X, DY, A, B, SC, plan, h, DX, da, db, ws)
    torch.cuda.synchronize()
    assert int(host(st)[0]) == 0
    return f64(Y), f64(DX), f64(da), f64(db)


# one launch; the long axis in parts; two launches; 32 places a workgroup; rows past the last-level cache
ROWS = [(1, 64, 136, 8, 1), (5, 40, 24, 24, 3), (64, 512, 520, 16, 1), (250, 520, 2048, 104, 4), (3, 8200, 40, 32, 2),
        (2, 14344, 136, 128, 1), (40, 4104, 264, 40, 6), (70, 5128, 7176, 32, 60), (300, 264, 1032, 80, 7),
        (777, 200, 4104, 128, 3), (8300, 136, 72, 40, 7), (9000, 520, 40, 112, 60), (65_600, 16, 1032, 48, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,k,n,r,s", ROWS)
def test_y_takes_sixteen_bits_of_h(t, k, n, r, s):
    """y0 cancels what BF16 holds of the sum; the rest is whole numbers, exact in every step."""
    ids = spread_ids(t, s)
    x, a, b, y, want = whole_rows(t, k, n, r, s, ids)
    assert np.array_equal(run(x, a, b, np.ones(s), ids, y)[0], want)


# dh from one launch with dx; from shrink; from the pass that reads dy once
DROWS = [(1, 64, 136, 8, 1), (65, 136, 520, 24, 2), (300, 264, 1032, 40, 7), (1500, 136, 264, 128, 3), (64, 40, 72, 104, 64),
         (3000, 520, 200, 16, 1), (4200, 64, 8200, 16, 3), (8200, 72, 4104, 24, 40), (2100, 136, 16_392, 32, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,k,n,r,s", DROWS)
def test_dx_takes_sixteen_bits_of_dh(t, k, n, r, s):
    ids = spread_ids(t, s)
    dy, b, a, dx, want = whole_rows(t, n, k, r, s, ids)
    assert np.array_equal(run(np.ones((t, k)), a, b, np.ones(s), ids, np.zeros((t, n)), dy, dx)[1], want)
