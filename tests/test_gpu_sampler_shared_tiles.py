"""Products whose tiles share the contraction, in two launches through the caller's workspace:
captured and replayed, two captured ones on one workspace, and two at once on streams of their own."""
import pytest
import torch

import sparse_delta_codec_amd as pulse

pytestmark = pytest.mark.gpu

# n, k, form: few tiles and a contraction of 12 and more steps, the layers of an adapter's trainer among them
PRODUCTS = [(640, 5120, "nt"), (512, 1536, "nt"), (1536, 512, "nn")]


class Products:
    """Rows quantised, and each product of them, on fixed buffers."""

    def __init__(self, t, seed, products=PRODUCTS):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.calls = []
        for n, k, form in products:
            inner, out = (k, n) if form == "nt" else (n, k)
            blocks = lambda v: (v + 127) // 128  # noqa: E731
            codes = (torch.randn((n, k), device="cuda", generator=self.gen) * 60).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.calls.append(dict(rows=torch.zeros((t, inner), dtype=torch.bfloat16, device="cuda"),
                                   x=torch.zeros((t, inner), dtype=torch.uint8, device="cuda"), x_scales=torch.zeros((t, blocks(inner)), device="cuda"),
                                   w=codes, w_scales=torch.rand((blocks(n), blocks(k)), device="cuda", generator=self.gen) + 0.5,
                                   y=torch.zeros((t, out), dtype=torch.bfloat16, device="cuda"),
                                   ws=pulse.fp8_gemm_workspace(t, n, k, form), form=form))
        self.refill()
        # these do share: without a workspace they are refused
        for c in self.calls:
            with pytest.raises(RuntimeError):
                pulse.fp8_block_gemm(c["x"], c["x_scales"], c["w"], c["w_scales"], c["y"], form=c["form"])

    def refill(self):
        for c in self.calls:
            c["rows"].copy_(torch.randn(c["rows"].shape, device="cuda", generator=self.gen))

    def go(self, stream=None):
        for c in self.calls:
            pulse.fp8_group_quant(c["rows"], c["x"], c["x_scales"], stream=stream)
            pulse.fp8_block_gemm(c["x"], c["x_scales"], c["w"], c["w_scales"], c["y"], c["ws"], form=c["form"], stream=stream)

    def spoil(self):
        for c in self.calls:
            c["ws"].fill_(255)
            c["y"].fill_(-1)

    def outputs(self):
        return [c["y"].clone() for c in self.calls]

    def captured(self):
        self.go()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.go()
        return graph


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("t", [20, 60, 200])
def test_replays(t):
    """Every replay on new inputs gives what the eager calls give, with eager work between replays."""
    p = Products(t, 1)
    graph = p.captured()
    for _ in range(4):
        p.refill()
        p.spoil()
        graph.replay()
        got = p.outputs()
        torch.cuda.synchronize()
        p.spoil()
        p.go()
        assert same(got, p.outputs())


@pytest.mark.parametrize("t", [1, 9])
def test_replays_of_the_gradients_form(t):
    """A few rows: the form nn alone goes through the workspace."""
    p = Products(t, 2, PRODUCTS[2:])
    graph = p.captured()
    for _ in range(3):
        p.refill()
        p.spoil()
        graph.replay()
        got = p.outputs()
        p.spoil()
        p.go()
        assert same(got, p.outputs())


def test_two_graphs_on_one_workspace():
    """In order on one stream, all products through one buffer."""
    a, b = Products(60, 3), Products(24, 4)
    one = max((c["ws"] for c in a.calls), key=lambda ws: ws.numel())
    for c in (*a.calls, *b.calls):
        c["ws"] = one
    graphs = [p.captured() for p in (a, b)]
    want = []
    for p in (a, b):
        p.go()
        want.append(p.outputs())
    for _ in range(3):
        a.spoil(), b.spoil()
        for g in graphs:
            g.replay()
        assert same(a.outputs(), want[0]) and same(b.outputs(), want[1])


def test_two_streams_at_once():
    """Streams and workspaces of their own; the current stream waits for nothing but events."""
    ps = [Products(60, 5), Products(60, 6)]
    want = []
    for p in ps:
        p.go()
        want.append(p.outputs())
        p.spoil()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(8):
        for p, s in zip(ps, streams):
            p.go(stream=s)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for p, w in zip(ps, want):
        assert same(p.outputs(), w)


def test_a_context_stream():
    """Within torch's stream context, both launches go to its stream."""
    p = Products(40, 7)
    p.go()
    want = p.outputs()
    p.spoil()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.go()
        got = p.outputs()
    torch.cuda.current_stream().wait_stream(s)
    assert same(got, want)
