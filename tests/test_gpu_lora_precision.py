"""What the roundings of h and dh may not lose, on data whose results are exact, at every
size where another kernel takes over."""
import numpy as np
import pytest
import torch

from tests.lora_exact import bf16_round, spread_ids, whole_rows, whole_sums

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


SUMS = [(1, 64, 136, 8, 1), (900, 264, 520, 24, 3), (300, 72, 136, 128, 2), (1500, 136, 264, 96, 3), (5, 40, 24, 8, 65),
        (3000, 520, 200, 16, 1), (4200, 64, 8200, 16, 1), (4200, 64, 8200, 32, 900), (33_000, 40, 1032, 8, 700)]


@pytest.mark.parametrize("t,k,n,r,s", SUMS)
@pytest.mark.parametrize("drop", [1, 2])
def test_the_sums_data_needs_all_three_parts(t, k, n, r, s, drop):
    """On the CPU: without the second or the third part of h the sums are others."""
    ids = spread_ids(t, s)
    for cols in (k, n):
        z, u, _, _, want = whole_sums(t, cols, n if cols == k else k, r, s, ids)
        top = bf16_round(u)
        mid = bf16_round(u - top)
        low = bf16_round(u - top - mid)
        assert np.array_equal(top + mid + low, u)
        less = top + (0 if drop == 1 else mid) + (0 if drop == 2 else low)
        got = np.zeros(want.shape)
        for i in range(s):
            rows = np.flatnonzero(ids == i)
            got[i] = less[rows].T @ z[rows]
        assert not np.array_equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("t,k,n,r,s", SUMS)
def test_weight_gradients_take_all_bits_of_h_and_dh(t, k, n, r, s):
    """Each column of z belongs to one token of an adapter, so a sum is one product: exact."""
    ids = spread_ids(t, s)
    dy, _, x, a, db = whole_sums(t, n, k, r, s, ids)
    got = run(x, a, np.ones((s, r, n)), np.ones(s), ids, np.zeros((t, n)), dy, np.zeros((t, k)))
    assert np.array_equal(got[3], db)
    x, _, dy, b, da = whole_sums(t, k, n, r, s, ids)
    got = run(x, np.ones((s, r, k)), b, np.ones(s), ids, np.zeros((t, n)), dy, np.zeros((t, k)))
    assert np.array_equal(got[2], da)
