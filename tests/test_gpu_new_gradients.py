"""Gradients that lie elsewhere in every step, as autograd makes them after
zero_grad(set_to_none=True): the tables follow with set_gradients."""
import pytest
import torch

pytestmark = pytest.mark.gpu

try:
    import sparse_delta_codec_amd as pulse
except ImportError:
    if torch.cuda.is_available():
        raise
    pulse = None

SIZES = [5, 16385, 300]


def lists(dtype):
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = [torch.empty(n, device="cuda").normal_(generator=gen) for n in SIZES]
    return p, *([torch.zeros(n, device="cuda") for n in SIZES] for _ in "mv"), [torch.zeros(n, dtype=dtype, device="cuda") for n in SIZES]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("side", [False, True])
def test_steps_follow_gradients_that_move(dtype, side):
    """Against tables made anew in every step; the old gradients hold NaN by then, and work is
    queued in front."""
    (p, m, v, g), (q, mq, vq, _) = lists(dtype), lists(dtype)
    table, norms = pulse.AdamWTable(p, g, m, v), pulse.GradTable(g)
    ws, st = pulse.workspace(pulse.PULSE_OP_GRAD_NORM, norms.ntiles), torch.zeros(1, dtype=torch.int32, device="cuda")
    clip, clip2 = torch.zeros(2, device="cuda"), torch.zeros(2, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    for step in range(1, 6):
        old, g = g, [torch.empty(n, device="cuda").normal_(generator=gen).to(dtype) for n in SIZES]
        for t in old:
            t.fill_(float("nan"))
        if side:
            stream.wait_stream(torch.cuda.current_stream())
        table.set_gradients(g, stream=stream)
        norms.set_gradients(g, stream=stream)
        pulse.pulse_grad_norm(norms, clip, ws, max_norm=1.0, stream=stream)
        pulse.pulse_adamw_step(table, step, 1e-3, d_scale=clip, d_status=st, stream=stream)
        if side:
            torch.cuda.current_stream().wait_stream(stream)
        pulse.pulse_grad_norm(pulse.GradTable(g), clip2, ws, max_norm=1.0)
        pulse.pulse_adamw_step(pulse.AdamWTable(q, g, mq, vq), step, 1e-3, d_scale=clip2, d_status=st)
        assert torch.equal(clip, clip2)
    torch.cuda.synchronize()
    assert int(st) == 0
    for a, b in zip(p + m + v, q + mq + vq):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


def test_set_gradients_refuses_others():
    p, m, v, g = lists(torch.float32)
    table, norms = pulse.AdamWTable(p, g, m, v), pulse.GradTable(g)
    before = table.segs.clone(), norms.segs.clone()
    wide = [torch.zeros(n + 4, device="cuda") for n in SIZES]
    for t in (table, norms):
        for bad in ([], g[:2], [x.bfloat16() for x in g], [x.cpu() for x in g], [wide[0][1:6]] + g[1:], [g[0][:4]] + g[1:],
                    [g[0], g[1], None], g + g):
            with pytest.raises(ValueError):
                t.set_gradients(bad)
    assert torch.equal(table.segs, before[0]) and torch.equal(norms.segs, before[1])


def test_set_gradients_refuses_a_capture():
    """The same gradients are fine there, for nothing is written; others are refused, and the
    table stays as it was."""
    p, m, v, g = lists(torch.float32)
    table, x = pulse.AdamWTable(p, g, m, v), torch.zeros(4, device="cuda")
    before = table.segs.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        table.set_gradients(g)
        with pytest.raises(RuntimeError):
            table.set_gradients(v)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(table.segs, before) and bool((x == 1).all())
    table.set_gradients(v)
    torch.cuda.synchronize()
    assert table.segs[:, 1].tolist() == [t.data_ptr() for t in v]
