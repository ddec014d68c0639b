"""The sampler's calls captured into graphs, on streams of their own, and beside each other."""
import pytest
import torch

import sparse_delta_codec_amd as pulse
from examples import fp8_layer as ex

pytestmark = pytest.mark.gpu


def rand_codes(shape, gen):
    return (torch.randn(shape, device="cuda", generator=gen) * 60).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


class Chain:
    """Every call of the layer, forward and back, on fixed buffers."""

    def __init__(self, t, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.view = ex.View(self.gen)
        self.view.update(*ex.patch(self.gen, self.view.bf16.numel()))
        self.layer = ex.Layer(self.view, t)
        self.x, self.stream = (torch.zeros(t, ex.HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in "ab")
        self.dy = torch.zeros(t, ex.HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.refill()

    def refill(self):
        for b in (self.x, self.stream, self.dy):
            b.copy_(torch.randn(b.shape, device="cuda", generator=self.gen))
        self.layer.logits.copy_(torch.randn(self.layer.logits.shape, device="cuda", generator=self.gen))

    def go(self, stream=None):
        v, l = self.view, self.layer
        s = dict(stream=stream)
        pulse.pulse_rms_norm(self.x, v.norm, ex.EPS, codes=l.x, scales=l.x_scales, rstd=l.rstd, **s)
        pulse.fp8_block_gemm(l.x, l.x_scales, v.up, v.up_scales, l.both, l.ws[0], **s)
        pulse.fp8_group_quant(l.both, l.h, l.h_scales, glu=True, **s)
        pulse.fp8_block_gemm(l.h, l.h_scales, v.down, v.down_scales, l.out, l.ws[1], **s)
        pulse.pulse_rms_norm(l.out, v.last_norm, ex.EPS, y=l.last, **s)
        pulse.pulse_moe_route(l.logits, l.ids, l.shares, **s)
        pulse.pulse_moe_forward(l.last, l.ids, l.shares, v.experts_up, v.experts_up_scales, v.experts_down,
                                v.experts_down_scales, l.mixed, v.status, l.ws[2], **s)
        pulse.fp8_group_quant(self.dy, l.dy, l.dy_scales, **s)
        pulse.fp8_block_gemm(l.dy, l.dy_scales, v.down, v.down_scales, l.dh, l.back_ws[0], form="nn", **s)
        pulse.pulse_rms_norm_backward(self.x, v.norm, l.rstd, self.dy, l.dx, l.dweight, l.back_ws[2], dres=self.dy, **s)

    def outputs(self):
        l = self.layer
        return [t.clone() for t in (l.x, l.x_scales, l.both, l.h, l.h_scales, l.out, l.last, l.ids, l.shares, l.mixed, l.dy,
                                    l.dh, l.dx, l.dweight)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [1, 2, 9, 40, 200])
def test_replays_of_a_captured_chain(t):
    """Every replay on new inputs gives what the eager calls give, with eager work between replays."""
    c = Chain(t, 3)
    c.go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.go()
    for _ in range(4):
        c.refill()
        graph.replay()
        got = c.outputs()
        torch.cuda.synchronize()
        for ws in (*c.layer.ws, *c.layer.back_ws):
            ws.fill_(255)
        for o in (c.layer.both, c.layer.out, c.layer.mixed, c.layer.dx):
            o.fill_(-1)
        c.go()
        assert same(got, c.outputs())
    assert int(c.view.status.item()) == 0


def test_two_captured_chains_share_their_workspaces():
    """In order on one stream: each replay leaves its own results."""
    a, b = Chain(30, 4), Chain(30, 5)
    b.layer.ws, b.layer.back_ws = a.layer.ws, a.layer.back_ws
    graphs = []
    for c in (a, b):
        c.go()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.go()
        graphs.append(g)
    want = []
    for c in (a, b):
        c.go()
        want.append(c.outputs())
    for _ in range(3):
        for c, g in zip((a, b), graphs):
            g.replay()
        assert same(a.outputs(), want[0]) and same(b.outputs(), want[1])


def test_chains_on_two_streams_at_once():
    """Streams and workspaces of their own; the current stream waits for nothing but events."""
    chains = [Chain(60, 6), Chain(60, 7)]
    want = []
    for c in chains:
        c.go()
        want.append(c.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(5):
        for c, s in zip(chains, streams):
            c.go(stream=s)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for c, w in zip(chains, want):
        assert same(c.outputs(), w)


def test_the_current_stream_is_used():
    """Within torch's stream context, calls without a stream go there."""
    c = Chain(10, 8)
    c.go()
    want = c.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.go()
        got = c.outputs()
    torch.cuda.current_stream().wait_stream(s)
    assert same(got, want)


def test_refusals_of_the_binding():
    t, n = 4, 256
    x = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    c, s = torch.zeros(t, n, dtype=torch.uint8, device="cuda"), torch.zeros(t, 2, device="cuda")
    bad = [lambda: pulse.pulse_rms_norm(x.cpu(), w, codes=c, scales=s), lambda: pulse.pulse_rms_norm(x, w.cpu(), codes=c, scales=s),
           lambda: pulse.pulse_rms_norm(x.float(), w, codes=c, scales=s), lambda: pulse.pulse_rms_norm(x, w[:-8], codes=c, scales=s),
           lambda: pulse.pulse_rms_norm(x, w, codes=c[:2], scales=s), lambda: pulse.pulse_rms_norm(x, w, codes=c, scales=s[:, :1]),
           lambda: pulse.pulse_rms_norm(x.t(), w[:t], codes=c.t(), scales=s), lambda: pulse.pulse_rms_norm(x, w, codes=c.float(), scales=s),
           lambda: pulse.fp8_group_quant(x, c, s, glu=True), lambda: pulse.fp8_group_quant(x[0], c, s),
           lambda: pulse.fp8_group_quant(x, c, s.double()), lambda: pulse.fp8_group_quant(x, c.cpu(), s)]
    wq, ws = torch.zeros(128, n, dtype=torch.uint8, device="cuda"), torch.ones(1, 2, device="cuda")
    y = torch.zeros(t, 128, dtype=torch.bfloat16, device="cuda")
    bad += [lambda: pulse.fp8_block_gemm(c, s, wq, ws, y[:, :64]), lambda: pulse.fp8_block_gemm(c[:, :128], s, wq, ws, y),
            lambda: pulse.fp8_block_gemm(c, s[:, :1], wq, ws, y), lambda: pulse.fp8_block_gemm(c, s, wq, ws[:, :1], y),
            lambda: pulse.fp8_block_gemm(c, s, wq, ws, y.t().contiguous().t()), lambda: pulse.fp8_block_gemm(c, s, wq.cpu(), ws, y),
            lambda: pulse.fp8_block_gemm(c[:, :128].contiguous(), s[:, :1].contiguous(), wq, ws, x, form="nn", bias=w),
            lambda: pulse.fp8_block_gemm(c, s, wq, ws, y, bias=w)]
    lg, ids, p = torch.zeros(t, 8, device="cuda"), torch.zeros(t, 2, dtype=torch.int32, device="cuda"), torch.zeros(t, 2, device="cuda")
    bad += [lambda: pulse.pulse_moe_route(lg.half(), ids, p), lambda: pulse.pulse_moe_route(lg, ids.long(), p),
            lambda: pulse.pulse_moe_route(lg, ids, p[:, :1]), lambda: pulse.pulse_moe_route(lg.t(), ids, p)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pulse.pulse_rms_norm(x, w), lambda: pulse.pulse_rms_norm(x, w, codes=c),
                 lambda: pulse.pulse_rms_norm(x, w, eps=0.0, codes=c, scales=s),
                 lambda: pulse.pulse_rms_norm(x[:, :12], w[:12], codes=c[:, :12].contiguous(), scales=s[:, :1].contiguous())):
        with pytest.raises(RuntimeError):
            call()
