"""CPU pins of the tests' own AdamW reference (tests/adamw_ref.py) and of the
trainer calls' refusals, which return before anything is enqueued."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import adamw_ref as ref
from tests.test_abi import EINVAL, ERANGE, EWORKSPACE, lib  # noqa: F401  (the library fixture)

V, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


def inputs(n, seed, mag=1e-3):
    rng = np.random.default_rng(seed)
    p = (rng.standard_normal(n) * 0.02).astype(np.float32)
    g = (rng.standard_normal(n) * mag).astype(np.float32)
    m = (rng.standard_normal(n) * 0.3 * mag).astype(np.float32)
    v = ((rng.standard_normal(n) * mag) ** 2).astype(np.float32)
    return p, g, m, v


def test_float32_reference_follows_the_formula():
    """Against float64: m' and v' carry three roundings of their parts (one
    half step, 2^-24, each); p' two of p and, on the update, about eight."""
    p, g, m, v = inputs(50_000, 1)
    for step in (1, 7, 1000):
        c = ref.constants(3e-6, (0.9, 0.999), 1e-8, step)
        got = ref.step32(p, g, m, v, c, scale=0.5, lr_mult=0.5, wd=0.1)
        want = ref.step64(p, g, m, v, 3e-6, (0.9, 0.999), 1e-8, step, scale=0.5, lr_mult=0.5, wd=0.1)
        h = 2.0 ** -24
        size = np.abs(m) * 0.9 + np.abs(g) * 0.05
        assert np.all(np.abs(got[1] - want[1]) <= 4 * h * size + 1e-45)
        assert np.all(np.abs(got[2] - want[2]) <= 6 * h * want[2] + 1e-45)
        upd = np.abs(want[0] - p * (1 - 1.5e-7))
        rough = size / np.sqrt(want[2] + 1e-30) * 1.5e-6 / (1 - 0.9 ** step)
        assert np.all(np.abs(got[0] - want[0]) <= 3 * h * np.abs(p) + 16 * h * (upd + rough))


def test_reference_equals_torch_adamw():
    p, g, m, v = inputs(4096, 2)
    t = torch.nn.Parameter(torch.from_numpy(p.copy()).double())
    opt = torch.optim.AdamW([t], lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    q, mm, vv = p.astype(np.float64), np.zeros(p.size), np.zeros(p.size)
    for step in range(1, 4):
        t.grad = torch.from_numpy(g * step).double()
        opt.step()
        q, mm, vv = ref.step64(q, g * step, mm, vv, 1e-3, (0.9, 0.95), 1e-8, step, wd=0.1)
    assert np.allclose(t.detach().numpy(), q, rtol=1e-12, atol=0)


def test_codes_decode_as_torch_e4m3():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=-1), np.nan_to_num(ref.E4M3.astype(np.float32), nan=-1))


def test_random_rounding_is_between_neighbours_and_unbiased():
    """Every code is one of the two neighbours of its value, exact values stay,
    and over many seeds the mean of the decoded values is the value: the mean
    of k roundings of spacing d is off by at most 6 d / (2 sqrt(k)) (six
    standard deviations of a Bernoulli draw)."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal(256) * np.exp(rng.standard_normal(256) * 2)).astype(np.float32)
    x[0], x[1], x[2] = 448.0, 1.75, 0.0
    x[3:] = np.clip(x[3:], -448, 448)
    grid = np.array(sorted(set(ref.E4M3[np.isfinite(ref.E4M3)])))
    lo = grid[np.clip(np.searchsorted(grid, x, side="right") - 1, 0, grid.size - 2)]
    hi = grid[np.minimum(np.searchsorted(grid, x, side="right"), grid.size - 1)]
    k = 400
    total = np.zeros(256)
    for seed in range(k):
        code, scale = ref.encode8(x, ref.random_bits(256, 5, seed) & 0xFFFFF, False)
        assert scale[0] == 1.0
        d = ref.E4M3[code]
        assert np.all((d == lo) | (d == hi)) and d[0] == 448 and d[1] == 1.75 and d[2] == 0
        total += d
    assert np.all(np.abs(total / k - x) <= 3 * (hi - lo) / math.sqrt(k) + 1e-6)


def test_random_bits_are_spread():
    """Each of the 32 bits is set in half of 2^16 elements, within six standard
    deviations (6 * 128), and two tensors or seeds share none of their order."""
    a, b, c = ref.random_bits(1 << 16, 0, 0), ref.random_bits(1 << 16, 1, 0), ref.random_bits(1 << 16, 0, 1)
    for bit in range(32):
        for x in (a, b, c, a ^ b, a ^ c, a[1:] ^ a[:-1]):
            assert abs(int(((x >> np.uint64(bit)) & np.uint64(1)).sum()) - x.size // 2) <= 6 * 128


def test_small_values_keep_a_code_and_tiny_blocks_are_zero():
    x = np.zeros(300, np.float32)
    x[0], x[1] = 1.0, 1e-30
    x[256:] = 2.0 ** -100
    code, scale = ref.encode8(x, np.zeros(300, np.uint64), True)
    assert code[0] == 126 and code[1] == 1 and code[2] == 0
    assert scale[1] == 0 and not code[256:].any()


# ---- the calls' refusals ----------------------------------------------------------
class Params(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", I64), ("seed", ctypes.c_uint32), ("grad_bf16", I32),
                ("state_bits", I32), ("reserved", I32)]


def good():
    return dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0, grad_bf16=0, state_bits=32, reserved=0)


@pytest.mark.parametrize("bad", [dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                                 dict(beta2=1.0), dict(beta2=math.nan), dict(eps=0.0), dict(eps=math.inf), dict(step=0),
                                 dict(grad_bf16=2), dict(state_bits=16), dict(reserved=1)])
def test_adamw_refuses_bad_parameters(lib, bad):  # noqa: F811
    f = lib.pulse_adamw_step
    f.argtypes = [V, I32, V, I64, V, V, V, V, I64, V, V, V, ctypes.c_size_t, V]
    al = V(0x10000)
    q = Params(**(good() | bad))
    assert f(al, 1, al, 1, ctypes.byref(q), None, None, None, 0, None, al, None, 0, None) == EINVAL


def test_adamw_refuses_bad_arguments(lib):  # noqa: F811
    f = lib.pulse_adamw_step
    f.argtypes = [V, I32, V, I64, V, V, V, V, I64, V, V, V, ctypes.c_size_t, V]
    al, q = V(0x10000), Params(**good())
    p = ctypes.byref(q)
    assert f(None, 1, al, 1, p, None, None, None, 0, None, al, None, 0, None) == EINVAL
    assert f(al, 1, None, 1, p, None, None, None, 0, None, al, None, 0, None) == EINVAL
    assert f(al, 1, al, 1, None, None, None, None, 0, None, al, None, 0, None) == EINVAL
    assert f(al, 1, al, 1, p, None, None, None, 0, None, None, None, 0, None) == EINVAL       # no status
    assert f(al, 0, al, 1, p, None, None, None, 0, None, al, None, 0, None) == EINVAL
    assert f(al, 3, al, 2, p, None, None, None, 0, None, al, None, 0, None) == EINVAL         # fewer tiles than tensors
    assert f(al, 1, al, 1, p, None, al, None, 0, None, al, al, 1 << 20, None) == EINVAL       # partial patch
    assert f(al, 1, al, 1, p, None, al, al, -1, al, al, al, 1 << 20, None) == EINVAL
    assert f(al, 1, al, 1 << 33, p, None, None, None, 0, None, al, None, 0, None) == ERANGE
    assert f(al, 1, al, 100, p, None, al, al, 10, al, al, al, 256 + 8 * 399, None) == EWORKSPACE
    assert f(al, 1, al, 100, p, None, al, al, 10, al, al, None, 1 << 20, None) == EWORKSPACE


def test_grad_norm_refuses_bad_arguments(lib):  # noqa: F811
    f = lib.pulse_grad_norm
    f.argtypes = [V, I32, V, I64, I32, ctypes.c_double, ctypes.c_double, V, V, ctypes.c_size_t, V]
    al, ws = V(0x10000), lib.pulse_workspace_bytes(11, 5, 0)
    assert f(None, 1, al, 1, 0, 1.0, 1.0, al, al, ws, None) == EINVAL
    assert f(al, 1, al, 1, 0, 1.0, 1.0, None, al, ws, None) == EINVAL
    assert f(al, 1, al, 1, 2, 1.0, 1.0, al, al, ws, None) == EINVAL
    for mul, most in ((0.0, 1.0), (-1.0, 1.0), (math.inf, 1.0), (math.nan, 1.0), (1.0, 0.0), (1.0, math.nan)):
        assert f(al, 1, al, 1, 0, mul, most, al, al, ws, None) == EINVAL
    assert f(al, 2, al, 1, 0, 1.0, 1.0, al, al, ws, None) == EINVAL
    assert f(al, 1, al, 1 << 33, 0, 1.0, 1.0, al, al, ws, None) == ERANGE
    assert f(al, 1, al, 1, 0, 1.0, 1.0, al, al, ws - 1, None) == EWORKSPACE
    assert f(al, 1, al, 1, 0, 1.0, 1.0, al, None, ws, None) == EWORKSPACE


def test_binding_refuses_host_tensors_and_uneven_lists():
    import sparse_delta_codec_amd as pulse

    t = torch.zeros(16)
    with pytest.raises(ValueError):
        pulse.GradTable([])
    with pytest.raises(ValueError):
        pulse.GradTable([t])
    with pytest.raises(ValueError):
        pulse.AdamWTable([t], [t], [t], [t, t])
    with pytest.raises(ValueError):
        pulse.AdamWTable([t], [t], [t], [t], m_scale=[t])
    with pytest.raises(ValueError):
        pulse.AdamWTable([t], [t], [t], [t])


def test_adamw_refuses_an_unaligned_workspace(lib):  # noqa: F811
    from tests.test_abi import EALIGN

    f = lib.pulse_adamw_step
    f.argtypes = [V, I32, V, I64, V, V, V, V, I64, V, V, V, ctypes.c_size_t, V]
    al, p = V(0x10000), ctypes.byref(Params(**good()))
    assert f(al, 1, al, 1, p, None, al, al, 10, al, al, V(0x10008), 1 << 20, None) == EALIGN
