"""The trainer's step and the adapters past 2^31: a tensor of the most elements there are,
and matrices of more."""
import pytest
import torch

pytestmark = pytest.mark.gpu

try:
    import sparse_delta_codec_amd as pulse
except ImportError:
    if torch.cuda.is_available():
        raise
    pulse = None


@pytest.mark.parametrize("bits", [32, 8])
def test_the_longest_tensor(bits):
    """2^31 - 1 elements, after a short tensor, gradients in a few places: those change and
    are the patch, and the norm is theirs."""
    n = (1 << 31) - 1
    at = torch.tensor([0, 1 << 20, (1 << 30) - 1, 1 << 30, n - 16385, n - 2, n - 1], device="cuda")
    p, b = torch.ones(n, device="cuda"), torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[at] = 2.0
    short = [torch.ones(5, device="cuda"), torch.zeros(5, dtype=torch.bfloat16, device="cuda")]
    m, v = ([torch.zeros(s, dtype=torch.uint8 if bits == 8 else torch.float32, device="cuda") for s in (5, n)] for _ in "mv")
    scales = {}
    if bits == 8:
        scales = {k: [torch.zeros(-(-s // 256), device="cuda") for s in (5, n)] for k in ("m_scale", "v_scale")}
    views = [torch.ones(5, dtype=torch.bfloat16, device="cuda"), b]
    table = pulse.AdamWTable([short[0], p], [short[1], g], m, v, b=views, **scales)
    norms = pulse.GradTable([short[1], g])
    clip, st = torch.zeros(2, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    idx, val = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    offs = torch.zeros(3, dtype=torch.int64, device="cuda")
    pulse.pulse_grad_norm(norms, clip, pulse.workspace(pulse.PULSE_OP_GRAD_NORM, norms.ntiles))
    pulse.pulse_adamw_step(table, 1, 0.25, d_scale=clip, d_status=st, ws=pulse.workspace(pulse.PULSE_OP_ADAMW, table.ntiles),
                           patch_idx=idx, patch_val=val, seg_offsets=offs)
    torch.cuda.synchronize()
    assert int(st) == 0 and offs.tolist() == [0, 0, 7]
    assert clip.tolist()[0] == 1.0 and abs(clip.tolist()[1] - 28 ** 0.5) < 1e-6
    assert torch.equal(idx[:7].long(), at) and bool((val[:7] == 0.75).all()) and not idx[7:].any()
    assert bool(((p[at] - 0.75).abs() < 1e-6).all()) and bool((b[at] == 0.75).all()) and bool((views[0] == 1).all())
    p[at], b[at] = 1.0, 1.0
    for part in range(0, n, 1 << 28):
        assert bool((p[part:part + (1 << 28)] == 1).all()) and bool((b[part:part + (1 << 28)] == 1).all())


def test_rows_past_two_to_the_thirty_one_elements():
    """66,000 rows of 32,776: forward and backward of one rank, whole numbers, every element."""
    t, k, n, r, s = 66_000, 16, 32_776, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(-1, s, (t,), device="cuda", generator=gen, dtype=torch.int32)
    x = torch.randint(-3, 4, (t, k), device="cuda", generator=gen).bfloat16()
    a, b = torch.zeros(s, r, k, device="cuda"), torch.zeros(s, r, n, device="cuda")
    a[:, 3, 5] = 1
    b[:, 3] = torch.randint(-3, 4, (s, n), device="cuda", generator=gen).float()
    y, dy = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    dy[:, 7], dy[:, n - 1] = 1, 2
    dx = torch.zeros(t, k, dtype=torch.bfloat16, device="cuda")
    da, db = torch.full((s, r, k), 9.0, device="cuda"), torch.full((s, r, n), 9.0, device="cuda")
    plan, st = pulse.LoraPlan(t, s), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, h = pulse.lora_workspace(t, k, n, r, s, train=True), pulse.lora_hidden(t, r, s)
    a16, b16, sc = a.bfloat16(), b.bfloat16(), torch.ones(s, device="cuda")
    pulse.pulse_lora_plan(plan, ids, st)
    pulse.pulse_lora_forward(x, a16, b16, sc, plan, y, ws, h=h)
    pulse.pulse_lora_backward(x, dy, a16, b16, sc, plan, h, dx, da, db, ws)
    torch.cuda.synchronize()
    assert int(st) == 0
    mine = ids.clamp(min=0).long()
    hid = x[:, 5].float() * (ids >= 0)
    for part in range(0, t, 4096):
        rows = slice(part, part + 4096)
        assert torch.equal(y[rows].float(), hid[rows, None] * b[mine[rows], 3])
    dh = (b[mine, 3, 7] + 2 * b[mine, 3, n - 1]) * (ids >= 0)
    want = torch.zeros(t, k, device="cuda")
    want[:, 5] = dh
    assert torch.equal(dx.float(), want)
    for i in range(s):
        rows = ids == i
        wa, wb = torch.zeros(r, k, device="cuda"), torch.zeros(r, n, device="cuda")
        wb[3, 7], wb[3, n - 1] = hid[rows].sum(), 2 * hid[rows].sum()
        wa[3] = (dh[rows, None].double() * x[rows].double()).sum(0).float()
        for q in range(r):  # dh of the other ranks is zero: their rows of B are
            assert torch.equal(da[i, q], wa[q])
        assert torch.equal(db[i], wb)
