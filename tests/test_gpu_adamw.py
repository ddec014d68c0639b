"""The trainer's step on the GPU (pulse_grad_norm, pulse_adamw_step) against the
CPU reference: every output bit for bit (the reference's own distance from the
float64 formula is pinned in test_oracle_adamw.py), the norm against a sum in
64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import adamw_ref as ref

pytestmark = pytest.mark.gpu

try:
    import sparse_delta_codec_amd as pulse
except ImportError:
    if torch.cuda.is_available():
        raise
    pulse = None

from tests.gpu_util import dev, host, zeros  # noqa: E402

BETAS, EPS = (0.9, 0.999), 1e-8


class Case:
    """A list of tensors on the host and on the GPU."""

    def __init__(self, sizes, seed, grad="float32", bits=32, view=True, mag=1e-3):
        rng = np.random.default_rng(seed)
        self.bits, self.p, self.g, self.m, self.v, self.ms, self.vs = bits, [], [], [], [], [], []
        for i, n in enumerate(sizes):
            k = mag * 10.0 ** (i % 3)
            self.p.append((rng.standard_normal(n) * 0.02).astype(np.float32))
            g = (rng.standard_normal(n) * k).astype(np.float32)
            if grad == "bfloat16":
                g = ref.bf16_value(ref.bf16_bits(g))
            self.g.append(g)
            m = (rng.standard_normal(n) * 0.3 * k).astype(np.float32)
            v = ((rng.standard_normal(n) * k) ** 2).astype(np.float32)
            if bits == 8:
                r = ref.random_bits(n, i, 99)
                m, ms = ref.encode8(m, r & 0xFFFFF, False)
                v, vs = ref.encode8(np.sqrt(v), r >> np.uint64(12), True)
                self.ms.append(ms)
                self.vs.append(vs)
            self.m.append(m)
            self.v.append(v)
        self.b = [ref.bf16_bits(p) for p in self.p]
        self.wd = [0.1 if i % 2 else 0.0 for i in range(len(sizes))]
        self.mult = [1.0 if i % 3 else 0.5 for i in range(len(sizes))]
        D = {k: [dev(x) for x in getattr(self, k)] for k in ("p", "m", "v", "b", "ms", "vs")}
        D["g"] = [dev(g) if grad == "float32" else dev(g).to(torch.bfloat16) for g in self.g]
        self.D = D
        scales = dict(m_scale=D["ms"], v_scale=D["vs"]) if bits == 8 else {}
        self.table = pulse.AdamWTable(D["p"], D["g"], D["m"], D["v"], b=D["b"] if view else None, lr_mult=self.mult,
                                      weight_decay=self.wd, **scales)
        self.ws = pulse.workspace(pulse.PULSE_OP_ADAMW, self.table.ntiles)
        self.st = zeros(1, torch.int32)

    def step_host(self, step, lr, scale=1.0, seed=0):
        c = ref.constants(lr, BETAS, EPS, step)
        for i in range(len(self.p)):
            kw = dict(scale=scale, lr_mult=self.mult[i], wd=self.wd[i])
            if self.bits == 8:
                (self.p[i], self.m[i], self.v[i], self.ms[i],
                 self.vs[i]) = ref.step8(self.p[i], self.g[i], self.m[i], self.v[i], self.ms[i], self.vs[i], c, i, seed,
                                         **kw)
            else:
                self.p[i], self.m[i], self.v[i] = ref.step32(self.p[i], self.g[i], self.m[i], self.v[i], c, **kw)
            self.b[i] = ref.bf16_bits(self.p[i])

    def step_gpu(self, step, lr, seed=0, **kw):
        pulse.pulse_adamw_step(self.table, step, lr, betas=BETAS, eps=EPS, seed=seed, d_status=self.st, ws=self.ws, **kw)

    def check(self, view=True):
        torch.cuda.synchronize()
        assert int(host(self.st)[0]) == 0
        for i in range(len(self.p)):
            assert np.array_equal(host(self.D["p"][i], np.uint32), self.p[i].view(np.uint32)), ("p", i)
            for k in ("m", "v"):
                want = getattr(self, k)[i]
                assert np.array_equal(host(self.D[k][i]).view(np.uint8), want.view(np.uint8)), (k, i)
            if self.bits == 8:
                for k in ("ms", "vs"):
                    assert np.array_equal(host(self.D[k][i], np.uint32), getattr(self, k)[i].view(np.uint32)), (k, i)
            if view:
                assert np.array_equal(host(self.D["b"][i], np.uint16), self.b[i]), ("b", i)


SIZES = [1, 3, 255, 256, 257, 1023, 4096, 4097, 16384, 16385, 40001, 2]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["float32", "bfloat16"])
def test_steps_match_the_reference(bits, grad):
    c = Case(SIZES, 1, grad, bits)
    scale = dev(np.array([0.625], np.float32))
    for step in (1, 2, 3):
        c.step_host(step, 1e-3, scale=0.625, seed=step)
        c.step_gpu(step, 1e-3, seed=step, d_scale=scale)
        c.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_whole_tile_lists_and_no_view(bits):
    """1024 tiles and more: a workgroup takes a whole tile."""
    sizes = [1024 * 16384 - 5000, 70_001]
    c = Case(sizes, 2, "bfloat16", bits, view=False)
    assert c.table.ntiles >= 1024
    c.step_host(10, 3e-6, seed=5)
    c.step_gpu(10, 3e-6, seed=5)
    c.check(view=False)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [SIZES, [1024 * 16384 + 3, 513]])
def test_patch_is_the_views_changes(bits, sizes):
    c = Case(sizes, 3, "float32", bits)
    before = [b.copy() for b in c.b]
    total = sum(sizes)
    idx, val = zeros(total, torch.int32), zeros(total, torch.int16)
    offs = zeros(len(sizes) + 1, torch.int64)
    for step in (1, 2):
        c.step_host(step, 1e-5, seed=step)
        c.step_gpu(step, 1e-5, seed=step, patch_idx=idx, patch_val=val, seg_offsets=offs)
        c.check()
        want = [np.flatnonzero(a != b) for a, b in zip(before, c.b)]
        assert np.array_equal(host(offs), np.cumsum([0] + [w.size for w in want]))
        n = sum(w.size for w in want)
        assert 0 < n < total
        assert np.array_equal(host(idx)[:n], np.concatenate(want))
        assert np.array_equal(host(val, np.uint16)[:n], np.concatenate([b[w] for b, w in zip(c.b, want)]))
        before = [b.copy() for b in c.b]


def test_patch_capacity_and_the_receivers_side():
    c = Case([30_000, 77], 4)
    old = [b.copy() for b in c.b]
    c.step_host(1, 1e-3)
    idx, val, offs = zeros(100, torch.int32), zeros(100, torch.int16), zeros(3, torch.int64)
    c.step_gpu(1, 1e-3, patch_idx=idx, patch_val=val, seg_offsets=offs)
    torch.cuda.synchronize()
    assert int(host(c.st)[0]) == pulse.PULSE_DS_CAPACITY
    want = [np.flatnonzero(a != b) for a, b in zip(old, c.b)]
    assert host(offs)[2] == sum(w.size for w in want) > 100
    assert np.array_equal(host(idx)[:100], want[0][:100])
    c.st.zero_()
    # the next step's patch, with room, brings a copy of the view up to date
    copies = [dev(b) for b in c.b]
    c.step_host(2, 1e-3)
    idx, val = zeros(30_077, torch.int32), zeros(30_077, torch.int16)
    c.step_gpu(2, 1e-3, patch_idx=idx, patch_val=val, seg_offsets=offs)
    pulse.pulse_apply_patch_segments(pulse.ViewTable(copies), idx, val, offs, c.st)
    c.check()
    for t, b in zip(copies, c.b):
        assert np.array_equal(host(t, np.uint16), b)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [math.nan, math.inf])
def test_a_scale_that_is_not_finite_skips_the_step(bits, scale):
    c = Case([5000, 300], 5, "float32", bits)
    idx, val, offs = zeros(5300, torch.int32), zeros(5300, torch.int16), zeros(3, torch.int64)
    offs.fill_(7)
    c.step_gpu(1, 1e-3, d_scale=dev(np.array([scale], np.float32)), patch_idx=idx, patch_val=val, seg_offsets=offs)
    c.check()
    assert not host(offs).any()
    c.step_gpu(1, 1e-3, d_scale=dev(np.array([scale], np.float32)))
    c.check()


def test_extreme_blocks_in_8_bits():
    """Zero gradients and states, a block of values below 2^-96, one element far
    above its block, and a block that ends after one element."""
    c = Case([256 * 4 + 1], 6, "float32", 8)
    g = c.g[0]
    g[:256] = 0
    g[256:512] = 1e-33
    g[512] = 1e4
    c.ms[0][:2] = 0
    c.vs[0][:2] = 0
    c.D["g"][0].copy_(dev(g))
    c.D["ms"][0].copy_(dev(c.ms[0]))
    c.D["vs"][0].copy_(dev(c.vs[0]))
    for step in (1, 2):
        c.step_host(step, 1e-3, seed=step)
        c.step_gpu(step, 1e-3, seed=step)
        c.check()
    assert c.ms[0][0] == 0 and c.vs[0][1] == 0 and np.all(np.isfinite(c.p[0]))


def test_a_broken_table_entry_is_flagged_and_nothing_of_it_written():
    c = Case([3000, 3000], 7)
    tab = c.table.segs.cpu()
    tab[1, 2] += 4  # m of tensor 1 no longer 16-byte aligned
    c.table.segs = tab.cuda()
    p1, b1 = c.p[1].copy(), c.b[1].copy()
    c.step_host(1, 1e-3)
    c.step_gpu(1, 1e-3)
    torch.cuda.synchronize()
    assert int(host(c.st)[0]) == pulse.PULSE_DS_BADSEGMENT
    assert np.array_equal(host(c.D["p"][0]), c.p[0])
    assert np.array_equal(host(c.D["p"][1]), p1) and np.array_equal(host(c.D["b"][1], np.uint16), b1)


def test_binding_checks_sizes():
    t = zeros(512, torch.float32)
    with pytest.raises(ValueError):
        pulse.AdamWTable([t], [t[:500]], [t], [t])
    with pytest.raises(ValueError):
        pulse.AdamWTable([t[1:]], [t], [t], [t])
    u = zeros(512, torch.uint8)
    with pytest.raises(ValueError):
        pulse.AdamWTable([t], [t], [u], [u], m_scale=[t[:1]], v_scale=[t[:2]])
    with pytest.raises(ValueError):
        pulse.AdamWTable([t], [t], [t], [t], lr_mult=[1.0, 2.0])
    table = pulse.AdamWTable([t], [t], [t], [t])
    with pytest.raises(ValueError):
        pulse.pulse_adamw_step(table, 1, 1e-3, d_status=zeros(1, torch.int32), patch_idx=zeros(4, torch.int32),
                               patch_val=zeros(4, torch.int16), seg_offsets=zeros(2, torch.int64))
    with pytest.raises(RuntimeError):
        pulse.pulse_adamw_step(table, 0, 1e-3, d_status=zeros(1, torch.int32))


# ---- the norm -----------------------------------------------------------------------
def norm_of(tensors, ws=None, **kw):
    table = pulse.GradTable(tensors)
    ws = pulse.workspace(pulse.PULSE_OP_GRAD_NORM, table.ntiles) if ws is None else ws
    out = zeros(2, torch.float32)
    pulse.pulse_grad_norm(table, out, ws, **kw)
    torch.cuda.synchronize()
    return host(out), ws


@pytest.mark.parametrize("grad", ["float32", "bfloat16"])
@pytest.mark.parametrize("sizes", [[1], [3, 16384, 16385, 1, 255], [7] * 50, [1024 * 16384 + 7, 5]])
def test_norm_and_clip_factor(grad, sizes):
    """Both results are float64 values rounded once: half a float32 step, 2^-24,
    and a little for the order of the float64 sums."""
    rng = np.random.default_rng(8)
    g = [(rng.standard_normal(n) * 0.01 * (i + 1)).astype(np.float32) for i, n in enumerate(sizes)]
    if grad == "bfloat16":
        g = [ref.bf16_value(ref.bf16_bits(x)) for x in g]
    D = [dev(x).to(getattr(torch, grad)) for x in g]
    want = math.sqrt(math.fsum(float((x.astype(np.float64) ** 2).sum()) for x in g))
    ws = None
    for mul, most in ((1.0, math.inf), (0.25, want * 0.1), (1.0, want * 10)):
        out, ws = norm_of(D, ws, grad_mul=mul, max_norm=most)
        n = want * mul
        assert abs(out[1] - n) <= n * 2.0 ** -23.9
        s = mul * min(1.0, most / (n + 1e-6))
        assert abs(out[0] - s) <= s * 2.0 ** -23.9


def test_norm_of_extremes():
    out, ws = norm_of([dev(np.zeros(1000, np.float32))], max_norm=1.0)
    assert out[1] == 0 and out[0] == 1
    for mag in (1e25, 1e-30):
        out, ws = norm_of([dev(np.full(10_000, mag, np.float32))], ws)
        n = float(np.float32(mag)) * 100
        assert abs(out[1] - n) <= n * 2.0 ** -23.9 and out[0] == 1
    for bad in (math.nan, math.inf, -math.inf):
        x = np.ones(40_000, np.float32)
        x[33_333] = bad
        out, ws = norm_of([dev(x)], ws, max_norm=1.0)
        assert np.isnan(out[0]) and not np.isfinite(out[1])
    out, ws = norm_of([dev(np.full(64, 2.0, np.float32))], ws, max_norm=4.0)
    assert out[1] == 16 and abs(out[0] - 0.25) <= 0.25 * 2.0 ** -22


def test_norm_is_the_same_on_every_run():
    g = dev((np.random.default_rng(9).standard_normal(3_000_000)).astype(np.float32))
    first, ws = norm_of([g])
    for _ in range(5):
        again, ws = norm_of([g], ws)
        assert np.array_equal(first.view(np.uint32), again.view(np.uint32))


def test_clip_and_step_in_a_replayed_graph():
    """Norm, step and patch captured once on a side stream and replayed, with
    eager work between the replays, against the same eager steps."""
    a, b = Case([50_000, 333], 10, "bfloat16", 8), Case([50_000, 333], 10, "bfloat16", 8)
    outs = []
    for c in (a, b):
        table = pulse.GradTable(c.D["g"])
        o = dict(s=zeros(2, torch.float32), idx=zeros(50_333, torch.int32), val=zeros(50_333, torch.int16),
                 offs=zeros(3, torch.int64), ws=pulse.workspace(pulse.PULSE_OP_GRAD_NORM, table.ntiles), table=table)
        outs.append(o)

    def step(c, o):
        pulse.pulse_grad_norm(o["table"], o["s"], o["ws"], max_norm=0.5)
        c.step_gpu(5, 1e-4, seed=3, d_scale=o["s"], patch_idx=o["idx"], patch_val=o["val"], seg_offsets=o["offs"])

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, outs[0])
    for _ in range(4):
        graph.replay()
        step(b, outs[1])
        torch.cuda.synchronize()
        assert int(host(a.st)[0]) == 0 and int(host(b.st)[0]) == 0
        for k in ("p", "m", "v", "b", "ms", "vs"):
            for x, y in zip(a.D[k], b.D[k]):
                assert torch.equal(x, y), k
        n = int(host(outs[0]["offs"])[2])
        assert n == int(host(outs[1]["offs"])[2]) > 0
        assert torch.equal(outs[0]["s"], outs[1]["s"]) and torch.equal(outs[0]["idx"][:n], outs[1]["idx"][:n])


@pytest.mark.parametrize("bits", [32, 8])
def test_patch_of_a_long_list_on_a_used_workspace(bits):
    """More pieces than the patch kernel has workgroups, tensors of every length
    between, and a workspace that holds anything: the patch lists exactly the elements
    whose view changed, in order, tensor by tensor."""
    sizes = [1, 2, 3, 1023, 1025, 16384, 16383, 5] * 20 + [2080 * 16384 + 13, 7]
    g = torch.Generator(device="cuda").manual_seed(4)
    total = sum(sizes)
    p = [torch.empty(n, device="cuda").normal_(0.0, 0.02, generator=g) for n in sizes]
    grads = [torch.empty(n, device="cuda").normal_(0.0, 1e-3, generator=g) for n in sizes]
    b = [x.bfloat16() for x in p]
    before = [x.clone() for x in b]
    dtype = torch.uint8 if bits == 8 else torch.float32
    m, v = ([torch.zeros(n, dtype=dtype, device="cuda") for n in sizes] for _ in "mv")
    scales = {}
    if bits == 8:
        scales = {k: [torch.zeros((n + 255) // 256, device="cuda") for n in sizes] for k in ("m_scale", "v_scale")}
    table, st = pulse.AdamWTable(p, grads, m, v, b=b, **scales), zeros(1, torch.int32)
    ws = pulse.workspace(pulse.PULSE_OP_ADAMW, table.ntiles)
    ws.fill_(255)
    idx, val = zeros(total, torch.int32), zeros(total, torch.bfloat16)
    offs = torch.full((len(sizes) + 1,), -1, dtype=torch.int64, device="cuda")
    pulse.pulse_adamw_step(table, 1, 1e-5, seed=1, d_status=st, ws=ws, patch_idx=idx, patch_val=val, seg_offsets=offs)
    torch.cuda.synchronize()
    assert int(host(st)[0]) == 0
    want = [(x.view(torch.int16) != y.view(torch.int16)).nonzero()[:, 0] for x, y in zip(before, b)]
    counts = torch.tensor([0] + [w.numel() for w in want]).cumsum(0)
    assert torch.equal(offs.cpu(), counts) and 0 < int(counts[-1]) < total
    n = int(counts[-1])
    assert torch.equal(idx[:n].long(), torch.cat(want))
    assert torch.equal(val[:n].view(torch.int16), torch.cat([x[w].view(torch.int16) for x, w in zip(b, want)]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", ["float32", "bfloat16"])
@pytest.mark.parametrize("tiles", [63, 64, 130])
def test_patch_around_the_sizes_of_a_piece(bits, grad, tiles):
    """Lists of just under and over the lengths at which a tile is cut otherwise."""
    sizes = [300, 257, 16384 * 2 + 1, 16384 * (tiles - 6), 255]
    c = Case(sizes, tiles, grad, bits)
    assert c.table.ntiles == tiles
    before, total = [b.copy() for b in c.b], sum(sizes)
    idx, val = zeros(total, torch.int32), zeros(total, torch.int16)
    offs = zeros(len(sizes) + 1, torch.int64)
    c.step_host(3, 1e-5, seed=9)
    c.step_gpu(3, 1e-5, seed=9, patch_idx=idx, patch_val=val, seg_offsets=offs)
    c.check()
    want = [np.flatnonzero(a != b) for a, b in zip(before, c.b)]
    assert np.array_equal(host(offs), np.cumsum([0] + [w.size for w in want]))
    n = sum(w.size for w in want)
    assert 0 < n < total and np.array_equal(host(idx)[:n], np.concatenate(want))
    assert np.array_equal(host(val, np.uint16)[:n], np.concatenate([b[w] for b, w in zip(c.b, want)]))
