"""Low-rank adapters on the GPU at the sizes where another kernel takes over: the
long axis in parts, one launch for h and y, 32 places a workgroup, dy read once for
two products, rows past the last-level cache; and what infinities may reach."""
import numpy as np
import pytest
import torch

from tests import lora_ref as ref

pytestmark = pytest.mark.gpu

try:
    import sparse_delta_codec_amd as pulse
except ImportError:
    if torch.cuda.is_available():
        raise
    pulse = None

from tests.gpu_util import host, zeros  # noqa: E402
from tests.test_gpu_lora import Batch, f64  # noqa: E402


@pytest.mark.parametrize("t,k,n,r,s", [
    (3, 8200, 40, 32, 2), (2, 14344, 136, 128, 1), (40, 4104, 264, 64, 6), (1, 24584, 24, 8, 1),   # the long axis in parts
    (1, 64, 16392, 16, 3), (64, 1032, 2056, 64, 2), (250, 520, 2048, 104, 4), (4000, 72, 520, 16, 4),  # one launch
    (70, 5128, 7176, 32, 60), (5, 136, 20488, 128, 5),                                              # two launches
    (8300, 136, 72, 40, 7), (8200, 264, 136, 64, 2), (9000, 520, 40, 112, 60), (8200, 72, 72, 128, 3)])  # 32 places
def test_forward_paths(t, k, n, r, s):
    c = Batch(t, k, n, r, s, seed=t + r, pad=8 * (t % 3), none=0.0 if t < 4 else 0.15)
    c.gpu_plan()
    ws = pulse.lora_workspace(t, k, n, r, s)
    ws.fill_(255)  # a workspace may hold anything
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, c.Y, ws)
    torch.cuda.synchronize()
    c.check_forward()


@pytest.mark.parametrize("t,k,n,r,s", [
    (4200, 64, 8200, 16, 3), (8200, 72, 4104, 24, 40), (33_000, 40, 1032, 8, 700), (2100, 136, 16_392, 32, 1),  # dy once
    (300, 264, 136, 16, 2), (64, 40, 72, 104, 64), (380, 72, 264, 40, 1), (5, 40, 24, 8, 65),  # one chunk or a few
    (700, 136, 2056, 128, 2), (600, 264, 72, 56, 3), (2200, 520, 136, 88, 5)])                 # rank groups
def test_backward_paths(t, k, n, r, s):
    c = Batch(t, k, n, r, s, seed=t + r, pad=8 * (t % 3))
    c.gpu_plan()
    ws, h = pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s)
    ws.fill_(255)
    h.fill_(255)
    da, db = torch.full(c.A.shape, 9.0, device="cuda"), torch.full(c.B.shape, 9.0, device="cuda")
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, c.Y, ws, h=h)
    pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, c.DX, da, db, ws)
    torch.cuda.synchronize()
    hid, eh = c.check_forward()
    c.check_backward(da, db, hid, eh)
    for s_ in sorted(set(range(s)) - set(c.ids.tolist()))[:8]:
        assert not da[s_].any() and not db[s_].any()
    da.fill_(0.25)
    db.fill_(0.25)
    pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, None, da, db, ws, accumulate=True)
    torch.cuda.synchronize()
    c.check_backward(da, db, hid, eh, add=0.25, dx=False)


@pytest.mark.parametrize("t,k,n,r,s", [(900, 264, 520, 24, 3), (300, 72, 136, 128, 2), (4200, 64, 8200, 16, 1)])
def test_weight_gradients_have_float32_precision(t, k, n, r, s):
    """h and dh enter dA and dB as float32: besides their own error, each of the three
    parts' products and sums rounds once, (3 tokens + 4) half steps of float32, and no
    rounding of h to BF16 is in it."""
    c = Batch(t, k, n, r, s, seed=7, none=0.0)
    c.gpu_plan()
    ws, h = pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s)
    da, db = torch.zeros(c.A.shape, device="cuda"), torch.zeros(c.B.shape, device="cuda")
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, c.Y, ws, h=h)
    pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, None, da, db, ws)
    torch.cuda.synchronize()
    x, a, b, dy = f64(c.x), f64(c.a), f64(c.b), f64(c.dy)
    _, daw, dbw, dh = ref.backward(x, dy, a, b, c.sc, c.ids, f64(c.dx))
    _, hid = ref.forward(x, a, b, c.sc, c.ids, f64(c.y))
    eh, edh = ref.hidden_error(x, a, c.sc, c.ids), ref.hidden_error(dy, b, c.sc, c.ids)
    for got, want, u, eu, z in ((da, daw, dh, edh, x), (db, dbw, hid, eh, dy)):
        for i in range(s):
            rows = np.flatnonzero(c.ids == i)
            bound = (np.abs(u[rows]) * (3 * rows.size + 4) * ref.HALF_F32 + eu[rows]).T @ np.abs(z[rows])
            assert np.all(np.abs(f64(got[i]) - want[i]) <= 1.02 * bound + 1e-30)


def test_rows_past_the_last_level_cache():
    """128 MB of y and more, against torch in 64 bits on the device, in slices."""
    t, k, n, r, s = 65_600, 16, 1032, 8, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    x, y = (torch.empty(t, c, device="cuda").normal_(generator=g).bfloat16() for c in (k, n))
    a, b = (torch.empty(s, r, c, device="cuda").normal_(0.0, 0.1, generator=g).bfloat16() for c in (k, n))
    sc = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    ids = torch.randint(-1, s, (t,), device="cuda", generator=g, dtype=torch.int32)
    before, plan, st = y.clone(), pulse.LoraPlan(t, s), zeros(1, torch.int32)
    pulse.pulse_lora_plan(plan, ids, st)
    pulse.pulse_lora_forward(x, a, b, sc, plan, y, pulse.lora_workspace(t, k, n, r, s))
    torch.cuda.synchronize()
    assert int(host(st)[0]) == 0
    for i in range(-1, s):
        rows = (ids == i).nonzero()[:, 0]
        if i < 0:
            assert torch.equal(y[rows], before[rows])
            continue
        h = float(sc[i]) * torch.mm(x[rows].double(), a[i].double().t())
        eh = float(sc[i]) * torch.mm(x[rows].double().abs(), a[i].double().abs().t()) * (k + 2) * ref.HALF_F32
        want = before[rows].double() + torch.mm(h, b[i].double())
        part = h.abs() * (ref.HALF_BF16 + (r + 2) * ref.HALF_F32) + eh
        bound = 1.02 * (torch.mm(part, b[i].double().abs()) + want.abs() * (ref.HALF_BF16 + (r + 2) * ref.HALF_F32)) + 1e-30
        assert bool(((y[rows].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("t,k,n,r,s", [(130, 64, 72, 16, 3), (65, 520, 1032, 40, 2), (4200, 64, 8200, 24, 3)])
def test_an_infinity_in_one_adapter_stays_where_the_formula_puts_it(t, k, n, r, s):
    """A rank of adapter 1 holds an infinity in A: the other adapters are what they are
    without it, and so are the other ranks of adapter 1's dB, also where places of a
    tile are empty (an empty place times an infinity would be NaN)."""
    c = Batch(t, k, n, r, s, seed=5)
    outs = []
    for bad in (False, True):
        a = c.A.clone()
        if bad:
            a[1, 3, 5] = float("inf")
        y, dx = c.Y.clone(), c.DX.clone()
        plan, st = pulse.LoraPlan(t, s), zeros(1, torch.int32)
        ws, h = pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s)
        da, db = torch.zeros(c.A.shape, device="cuda"), torch.zeros(c.B.shape, device="cuda")
        pulse.pulse_lora_plan(plan, c.IDS, st)
        pulse.pulse_lora_forward(c.X, a, c.B, c.SC, plan, y, ws, h=h)
        pulse.pulse_lora_backward(c.X, c.DY, a, c.B, c.SC, plan, h, dx, da, db, ws)
        torch.cuda.synchronize()
        outs.append((y, dx, da, db))
    (y0, dx0, da0, db0), (y1, dx1, da1, db1) = outs
    other = c.IDS != 1
    assert torch.equal(y0[other], y1[other]) and torch.equal(dx0[other], dx1[other])
    assert torch.equal(da0, da1)  # dA does not depend on A
    rest = [i for i in range(s) if i != 1]
    ranks = [i for i in range(r) if i != 3]
    assert torch.equal(db0[rest], db1[rest]) and torch.equal(db0[1][ranks], db1[1][ranks])
    assert not bool(torch.isfinite(db1[1, 3]).any())


@pytest.mark.parametrize("t,s,shape", [(1, 1, "one"), (1000, 3, "runs"), (5000, 1024, "random"), (513, 2, "none"),
                                       (40_000, 600, "random"), (20_000, 1, "one"), (100, 700, "random")])
def test_plan_lists_the_places_in_use(t, s, shape):
    rng = np.random.default_rng(t)
    ids = {"one": np.zeros(t), "runs": np.repeat([2, -1, 0, 2], t // 4), "none": np.full(t, -1),
           "random": rng.integers(-1, s, t)}[shape].astype(np.int32)
    plan, st = pulse.LoraPlan(t, s), zeros(1, torch.int32)
    plan.buffer.fill_(7)
    pulse.pulse_lora_plan(plan, torch.from_numpy(ids).cuda(), st)
    torch.cuda.synchronize()
    assert int(host(st)[0]) == 0
    w = plan.buffer.cpu().numpy().view(np.int32)
    mt, mg = min(t, (t + 63) // 64 + s), min(t, (t + 15) // 16 + s)
    r4 = lambda n: (n + 3) // 4 * 4  # noqa: E731
    first = w[16 + 2 * r4(mt):][:s + 1]
    group = w[16 + 2 * r4(mt) + r4(s + 1) + mt * 64:][:mg]
    want = [(first[a] * 4 + i) for a in range(s) for i in range((int((ids == a).sum()) + 15) // 16)]
    assert np.array_equal(group[:len(want)], want) and np.all(group[len(want):] == -1)
    assert first[s] == w[0] == sum((int((ids == a).sum()) + 63) // 64 for a in range(s))


def test_one_row_of_any_stride():
    """A single token's rows may be cut from wider ones of any length."""
    c = Batch(1, 64, 40, 16, 2, ids=[1], seed=2)
    c.gpu_plan()
    x, y = torch.zeros(2, 1001, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 333, dtype=torch.bfloat16, device="cuda")
    x[:1, :64], y[:1, :40] = c.X, c.Y
    c.Y = y[:1, :40]
    pulse.pulse_lora_forward(x[:1, :64], c.A, c.B, c.SC, c.plan, c.Y, pulse.lora_workspace(1, 64, 40, 16, 2))
    torch.cuda.synchronize()
    c.check_forward()
    assert not y[0, 40:].any() and not y[1].any()
