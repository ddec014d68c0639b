"""What weight decay takes from the masters over many steps, at the learning rates of RL
post-training, where 1 - lr * decay lies between the float32 numbers next to 1."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

try:
    import sparse_delta_codec_amd as pulse
except ImportError:
    if torch.cuda.is_available():
        raise
    pulse = None


def masters(steps, lr, wd, bits, n):
    """The masters after steps with gradients of their own in each step."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    p = torch.empty(n, device="cuda").normal_(0.0, 0.02, generator=gen)
    start = p.double().clone()
    g = torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32, device="cuda") for _ in "mv")
    scales = {}
    if bits == 8:
        scales = {k: [torch.zeros(-(-n // 256), device="cuda")] for k in ("m_scale", "v_scale")}
    table = pulse.AdamWTable([p], [g], [m], [v], weight_decay=wd, **scales)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(1, steps + 1):
        g.normal_(0.0, 1e-3, generator=gen)
        pulse.pulse_adamw_step(table, step, lr, d_status=st, seed=step)
    assert int(st) == 0
    return start, p.double()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,wd", [(2e-6, 0.01), (3e-6, 0.01), (1e-6, 0.1), (1e-7, 0.1)])
def test_small_decays_add_up(bits, lr, wd):
    """Against the same steps without decay: the masters shrink by steps * lr * wd of
    themselves, measured along the start's.  A step rounds each run's masters by half a step
    of float32 at most, 2^-24 |p|, to either side as the updates make it (a standard
    deviation of 2^-24 |p| / sqrt(3)); weighted with p, two runs of n normal masters come to
    2^-24 sqrt(2 steps / n).  The updates, 2 lr each at most and not along p, change what
    is decayed by a standard deviation of 2 steps lr / (0.02 sqrt(n)) of it.  Six of each are
    allowed, the second order of the decay, and 2^-22 for the constants."""
    steps, n = 400, 1 << 18
    (p0, plain), (_, less) = masters(steps, lr, 0.0, bits, n), masters(steps, lr, wd, bits, n)
    got = float((p0 * (plain - less)).sum() / (p0 * p0).sum())
    want = steps * lr * wd
    noise = 6 * 2.0 ** -24 * np.sqrt(2 * steps / n)
    assert abs(got - want) <= noise + want * (12 * steps * lr / (0.02 * np.sqrt(n)) + want + 2.0 ** -22)


@pytest.mark.parametrize("lr,wd", [(2e-6, 0.01), (1e-3, 0.1), (1e-3, 0.0)])
def test_extreme_masters(lr, wd):
    """Infinite, NaN, zero and largest masters with and without a step of the gradient."""
    values = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 3.4e38, -3.4e38, 1.0], device="cuda")
    p = values.repeat(2).contiguous()
    g = torch.cat([torch.zeros(8, device="cuda"), torch.full((8,), 1e-3, device="cuda")])
    m, v = torch.zeros(16, device="cuda"), torch.zeros(16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pulse.pulse_adamw_step(pulse.AdamWTable([p], [g], [m], [v], weight_decay=wd), 1, lr, d_status=st)
    got = p.cpu()
    for half in (got[:8], got[8:]):
        assert torch.equal(half[:2], values[:2].cpu()) and bool(torch.isnan(half[2]))
        assert bool(torch.isfinite(half[3:]).all())
    assert not got[3:5].any()  # zero masters without a gradient stay zero
