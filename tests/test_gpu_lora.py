"""Low-rank adapters on the GPU (pulse_lora_plan, pulse_lora_forward,
pulse_lora_backward) against the float64 reference, within the bounds that the
documented roundings give (tests/lora_ref.py)."""
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


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(t, pad):
    """t as a view of rows that are pad elements longer, and the whole buffer; the gap holds 7."""
    whole = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype)
    whole[:, :t.shape[1]] = t
    whole = whole.cuda()
    return whole[:, :t.shape[1]], whole


class Batch:
    def __init__(self, t, k, n, r, s, ids=None, seed=0, pad=0, none=0.15):
        rng = np.random.default_rng(seed)
        if ids is None:
            ids = rng.integers(0, s, t)
            ids[rng.random(t) < none] = -1
        self.t, self.k, self.n, self.r, self.s, self.ids = t, k, n, r, s, np.asarray(ids, np.int32)
        self.x = bf16(rng.standard_normal((t, k)))
        self.y = bf16(rng.standard_normal((t, n)))
        self.dy = bf16(rng.standard_normal((t, n)) * 1e-2)
        self.dx = bf16(rng.standard_normal((t, k)) * 1e-2)
        self.a = bf16(rng.standard_normal((s, r, k)) * k ** -0.5)
        self.b = bf16(rng.standard_normal((s, r, n)) * 0.05)
        self.sc = rng.uniform(0.25, 2.0, s).astype(np.float32)
        self.A, self.B, self.SC = self.a.cuda(), self.b.cuda(), torch.from_numpy(self.sc).cuda()
        self.IDS = torch.from_numpy(self.ids).cuda()
        (self.X, _), (self.Y, self.Yw) = strided(self.x, pad), strided(self.y, pad)
        (self.DY, _), (self.DX, self.DXw) = strided(self.dy, pad), strided(self.dx, pad)
        self.pad = pad

    def gpu_plan(self, plan=None):
        self.plan = pulse.LoraPlan(self.t, self.s) if plan is None else plan
        st = zeros(1, torch.int32)
        pulse.pulse_lora_plan(self.plan, self.IDS, st)
        torch.cuda.synchronize()
        assert int(host(st)[0]) == 0

    def check_rows(self, got, whole, before, want, bound):
        """The result within its bound; rows without an adapter and the gaps untouched."""
        err = np.abs(f64(got) - want)
        assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())
        rest = torch.from_numpy(self.ids < 0)
        assert torch.equal(got.cpu()[rest].view(torch.int16), before[rest].view(torch.int16))
        if self.pad:
            assert bool((whole[:, before.shape[1]:] == 7).all())

    def check_forward(self):
        x, a, b = f64(self.x), f64(self.a), f64(self.b)
        want, h = ref.forward(x, a, b, self.sc, self.ids, f64(self.y))
        eh = ref.hidden_error(x, a, self.sc, self.ids)
        self.check_rows(self.Y, self.Yw, self.y, want, ref.row_bound(want, h, eh, b, self.ids))
        return h, eh

    def check_backward(self, da, db, h, eh, add=0.0, dx=True):
        x, a, b, dy = f64(self.x), f64(self.a), f64(self.b), f64(self.dy)
        dxw, daw, dbw, dh = ref.backward(x, dy, a, b, self.sc, self.ids, f64(self.dx))
        edh = ref.hidden_error(dy, b, self.sc, self.ids)
        if dx:
            self.check_rows(self.DX, self.DXw, self.dx, dxw, ref.row_bound(dxw, dh, edh, a, self.ids))
        for got, want, u, eu, z in ((da, daw, dh, edh, x), (db, dbw, h, eh, dy)):
            bound = ref.grad_bound(u, eu, z, self.ids, want.shape) + abs(add) * 2 * ref.HALF_F32
            err = np.abs(f64(got) - add - want)
            assert np.all(err <= bound), float((err / bound).max())


FORWARD = [(1, 8, 8, 8, 1), (1, 4096, 1000, 16, 8), (5, 40, 24, 8, 3), (64, 512, 520, 16, 1), (65, 136, 4104, 24, 2),
           (96, 1024, 2048, 32, 64), (300, 264, 1032, 40, 7), (1000, 768, 640, 64, 5), (777, 200, 4104, 128, 3),
           (130, 1160, 136, 80, 1), (700, 72, 88, 16, 1000), (4100, 512, 5000, 8, 2), (33, 4104, 96, 96, 4),
           (257, 128, 136, 112, 2), (2100, 96, 4200, 48, 4)]


@pytest.mark.parametrize("t,k,n,r,s", FORWARD)
def test_forward(t, k, n, r, s):
    c = Batch(t, k, n, r, s, seed=t + r, pad=8 * (t % 3), none=0.0 if t == 1 else 0.15)
    c.gpu_plan()
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, c.Y, pulse.lora_workspace(t, k, n, r, s))
    torch.cuda.synchronize()
    c.check_forward()


BACKWARD = [(1, 8, 8, 8, 1), (3, 1024, 40, 16, 2), (64, 264, 136, 8, 1), (65, 136, 520, 24, 2), (100, 512, 96, 64, 30),
            (300, 264, 1032, 40, 7), (1013, 448, 1000, 24, 5), (1500, 136, 264, 128, 3), (3000, 520, 200, 16, 1),
            (600, 72, 88, 32, 900), (900, 256, 128, 96, 2), (5000, 64, 72, 56, 3)]


@pytest.mark.parametrize("t,k,n,r,s", BACKWARD)
def test_forward_and_backward(t, k, n, r, s):
    c = Batch(t, k, n, r, s, seed=t + r, pad=8 * (t % 3), none=0.0 if t == 1 else 0.15)
    c.gpu_plan()
    ws, h = pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s)
    da, db = torch.full(c.A.shape, 9.0, device="cuda"), torch.full(c.B.shape, 9.0, device="cuda")
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, c.Y, ws, h=h)
    pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, c.DX, da, db, ws)
    torch.cuda.synchronize()
    c.check_backward(da, db, *c.check_forward())
    # adapters without a token: zero, and the workspace serves again, added to what is there
    for s_ in set(range(s)) - set(c.ids.tolist()):
        assert not da[s_].any() and not db[s_].any()
    da.fill_(0.5)
    db.fill_(0.5)
    pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, None, da, db, ws, accumulate=True)
    torch.cuda.synchronize()
    h_, eh = ref.forward(f64(c.x), f64(c.a), f64(c.b), c.sc, c.ids, f64(c.y))[1], ref.hidden_error(f64(c.x), f64(c.a), c.sc, c.ids)
    c.check_backward(da, db, h_, eh, add=0.5, dx=False)


@pytest.mark.parametrize("t,s,shape", [(1, 1, "one"), (64, 1, "one"), (1000, 3, "runs"), (5000, 1024, "random"),
                                       (513, 2, "none"), (20_000, 37, "random"), (200, 200, "each")])
def test_plan_is_a_stable_sort(t, s, shape):
    rng = np.random.default_rng(t)
    ids = {"one": np.zeros(t), "runs": np.repeat([2, -1, 0, 2], t // 4), "none": np.full(t, -1), "each": rng.permutation(t),
           "random": rng.integers(-1, s, t)}[shape].astype(np.int32)
    plan, st = pulse.LoraPlan(t, s), zeros(1, torch.int32)
    pulse.pulse_lora_plan(plan, torch.from_numpy(ids).cuda(), st)
    torch.cuda.synchronize()
    assert int(host(st)[0]) == 0
    w = plan.buffer.cpu().numpy().view(np.int32)
    mt = min(t, (t + 63) // 64 + s)
    r4 = lambda n: (n + 3) // 4 * 4  # noqa: E731
    slot, count = w[16:16 + mt], w[16 + r4(mt):16 + r4(mt) + mt]
    order = w[16 + 2 * r4(mt) + r4(s + 1):][:mt * 64].reshape(mt, 64)
    at = 0
    for a in range(s):
        mine = np.flatnonzero(ids == a)
        for i in range(0, mine.size, 64):
            part = mine[i:i + 64]
            assert slot[at] == a and count[at] == part.size
            assert np.array_equal(order[at, :part.size], part) and np.all(order[at, part.size:] == -1)
            at += 1
    assert w[0] == at and np.all(slot[at:] == -1)


def test_ids_out_of_range_are_flagged_and_have_no_adapter():
    ids = np.array([0, 5, -1, 1, -7, 2 ** 30, 1], np.int32)
    c = Batch(7, 64, 32, 16, 2, ids=ids, seed=3)
    plan, st = pulse.LoraPlan(7, 2), zeros(1, torch.int32)
    pulse.pulse_lora_plan(plan, c.IDS, st)
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, plan, c.Y, pulse.lora_workspace(7, 64, 32, 16, 2))
    torch.cuda.synchronize()
    assert int(host(st)[0]) == pulse.PULSE_DS_BADINDEX
    c.ids = np.where((ids >= 0) & (ids < 2), ids, -1)
    c.check_forward()


@pytest.mark.parametrize("ids", [np.full(70, -1), np.where(np.arange(70) % 2, 1, -1)])
def test_rows_without_an_adapter_may_hold_anything(ids):
    """NaN and infinities in their x, dy and y reach nothing; a NaN in one adapter's
    token stays with that adapter."""
    c = Batch(70, 64, 72, 16, 3, ids=ids.astype(np.int32), seed=4)
    rest = torch.from_numpy(c.ids < 0)
    for host_t, dev_t in ((c.x, c.X), (c.dy, c.DY), (c.y, c.Y), (c.dx, c.DX)):
        host_t[rest] = float("nan")
        host_t[rest, ::2] = float("inf")
        dev_t.copy_(host_t)
    c.gpu_plan()
    ws, h = pulse.lora_workspace(70, 64, 72, 16, 3, train=True), pulse.lora_hidden(70, 16, 3)
    da, db = torch.full(c.A.shape, 9.0, device="cuda"), torch.full(c.B.shape, 9.0, device="cuda")
    pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, c.Y, ws, h=h)
    pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, c.DX, da, db, ws)
    torch.cuda.synchronize()
    for host_t, dev_t in ((c.y, c.Y), (c.dx, c.DX)):
        assert torch.equal(dev_t.cpu()[rest].view(torch.int16), host_t[rest].view(torch.int16))
        assert bool(torch.isfinite(dev_t.cpu()[~rest]).all())
    assert bool(torch.isfinite(da).all()) and bool(torch.isfinite(db).all())
    assert not da[0].any() and not db[2].any()


def test_one_workspace_and_plan_for_batches_of_any_size():
    """Batches of changing size and ranks of changing layers on one plan buffer and
    one workspace, sized for the largest: the counters are zero after every call."""
    plan, ws = pulse.LoraPlan(3000, 20), pulse.lora_workspace(3000, 2048, 1024, 64, 20, train=True)
    for i, (t, k, n, r) in enumerate([(3, 2048, 64, 16), (3000, 128, 1024, 64), (40, 1536, 512, 8), (1, 2048, 1024, 64),
                                      (500, 2048, 96, 32), (0, 64, 64, 16), (17, 2048, 1024, 64)]):
        c = Batch(t, k, n, r, 20, seed=50 + i)
        c.gpu_plan(plan)
        h = pulse.lora_hidden(t, r, 20)
        da, db = torch.full(c.A.shape, 9.0, device="cuda"), torch.full(c.B.shape, 9.0, device="cuda")
        pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, plan, c.Y, ws, h=h)
        pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, plan, h, c.DX, da, db, ws)
        torch.cuda.synchronize()
        c.check_backward(da, db, *c.check_forward())


def test_results_do_not_change_from_run_to_run():
    c = Batch(1200, 1024, 520, 32, 6, seed=9)
    c.gpu_plan()
    ws, h = pulse.lora_workspace(1200, 1024, 520, 32, 6, train=True), pulse.lora_hidden(1200, 32, 6)
    first = None
    for _ in range(4):
        y, dx = c.Y.clone(), c.DX.clone()
        da, db = torch.zeros(c.A.shape, device="cuda"), torch.zeros(c.B.shape, device="cuda")
        pulse.pulse_lora_forward(c.X, c.A, c.B, c.SC, c.plan, y, ws, h=h)
        pulse.pulse_lora_backward(c.X, c.DY, c.A, c.B, c.SC, c.plan, h, dx, da, db, ws)
        torch.cuda.synchronize()
        now = (y, dx, da, db)
        first = now if first is None else first
        assert all(torch.equal(p, q) for p, q in zip(first, now))


def test_a_replayed_graph_on_another_stream():
    """Plan, forward and backward captured once and replayed with new inputs,
    eager work between the replays, against the eager calls."""
    t, k, n, r, s = 150, 256, 264, 16, 4
    c = Batch(t, k, n, r, s, seed=11)
    plan, st = pulse.LoraPlan(t, s), zeros(1, torch.int32)
    ws, h = pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s)
    da, db = torch.zeros(c.A.shape, device="cuda"), torch.zeros(c.B.shape, device="cuda")

    def step(plan, ws, h, x, y, dy, dx, da, db, ids):
        pulse.pulse_lora_plan(plan, ids, st)
        pulse.pulse_lora_forward(x, c.A, c.B, c.SC, plan, y, ws, h=h)
        pulse.pulse_lora_backward(x, dy, c.A, c.B, c.SC, plan, h, dx, da, db, ws)

    X, Y, DY, DX = (v.contiguous() for v in (c.X, c.Y, c.DY, c.DX))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(plan, ws, h, X, Y, DY, DX, da, db, c.IDS)
    side = torch.cuda.Stream()
    for i in range(4):
        d = Batch(t, k, n, r, s, seed=20 + i)
        for dst, src in ((X, d.X), (Y, d.Y), (DY, d.DY), (DX, d.DX), (c.IDS, d.IDS)):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        da2, db2 = torch.zeros_like(da), torch.zeros_like(db)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(pulse.LoraPlan(t, s), pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s), d.X,
                 d.Y, d.DY, d.DX, da2, db2, d.IDS)
            side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(Y, d.Y) and torch.equal(DX, d.DX) and torch.equal(da, da2) and torch.equal(db, db2)
    assert int(host(st)[0]) == 0


def test_binding_refuses_wrong_shapes():
    c = Batch(10, 64, 32, 16, 2, seed=1)
    c.gpu_plan()
    ws = pulse.lora_workspace(10, 64, 32, 16, 2)
    args = [c.X, c.A, c.B, c.SC, c.plan, c.Y, ws]
    for i, bad in ((0, c.X[:9]), (0, c.X.float()), (0, c.X.t()), (0, c.x), (1, c.A[:1]), (2, c.B[:, :8]), (3, c.SC[:1]),
                   (5, c.Y[:, :24]), (1, c.A.transpose(1, 2))):
        with pytest.raises(ValueError):
            pulse.pulse_lora_forward(*(args[:i] + [bad] + args[i + 1:]))
    with pytest.raises(RuntimeError):
        pulse.pulse_lora_forward(*args[:6], ws[:64])
    with pytest.raises(ValueError):
        pulse.pulse_lora_plan(c.plan, torch.zeros(11, dtype=torch.int32, device="cuda"), zeros(1, torch.int32))
    with pytest.raises(RuntimeError):
        pulse.LoraPlan(10, 2000)
