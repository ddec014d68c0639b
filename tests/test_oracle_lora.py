"""CPU pins of the tests' own adapter reference (tests/lora_ref.py): the gradients
against differences and against torch's, and the adapter calls' refusals, which
return before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

from tests import lora_ref as ref
from tests.test_abi import EALIGN, EINVAL, ERANGE, EWORKSPACE, lib  # noqa: F401  (the library fixture)

V, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


def small(seed=0):
    rng = np.random.default_rng(seed)
    t, k, n, r, s = 9, 5, 7, 3, 4
    ids = np.array([0, 2, -1, 2, 0, 1, 2, -1, 0])
    return (rng.standard_normal((t, k)), rng.standard_normal((s, r, k)), rng.standard_normal((s, r, n)),
            rng.uniform(0.5, 2, s), ids, rng.standard_normal((t, n)), rng.standard_normal((t, n)))


def test_gradients_against_differences():
    """d/dp of <dy, y> by central differences, step 1e-5: y is linear in x and in
    each of A and B alone, so the difference is exact up to rounding, 1e-9."""
    x, a, b, sc, ids, y, dy = small()
    dx, da, db, _ = ref.backward(x, dy, a, b, sc, ids, np.zeros(x.shape))
    for arr, grad in ((x, dx), (a, da), (b, db)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + 1e-5
            up = (dy * ref.forward(x, a, b, sc, ids, y)[0]).sum()
            arr[i] = keep - 1e-5
            down = (dy * ref.forward(x, a, b, sc, ids, y)[0]).sum()
            arr[i] = keep
            assert abs((up - down) / 2e-5 - grad[i]) <= 1e-8 * (1 + abs(grad[i]))


def test_gradients_against_torch():
    x, a, b, sc, ids, y, dy = small(1)
    tx, ta, tb = (torch.from_numpy(v).requires_grad_() for v in (x, a, b))
    out = [torch.from_numpy(y[t]) + (0 if i < 0 else sc[i] * (tb[i].t() @ (ta[i] @ tx[t]))) for t, i in enumerate(ids)]
    torch.stack(out).backward(torch.from_numpy(dy))
    dx, da, db, _ = ref.backward(x, dy, a, b, sc, ids, np.zeros(x.shape))
    assert np.allclose(ref.forward(x, a, b, sc, ids, y)[0], torch.stack(out).detach().numpy(), rtol=1e-13)
    for g, w in ((tx.grad, dx), (ta.grad, da), (tb.grad, db)):
        assert np.allclose(g.numpy(), w, rtol=1e-12, atol=1e-13)


# ---- the calls' refusals and sizes --------------------------------------------------
def calls(lib):  # noqa: F811
    for f in (lib.pulse_lora_plan_bytes, lib.pulse_lora_hidden_bytes, lib.pulse_lora_ws_bytes):
        f.restype = I64
    lib.pulse_lora_plan_bytes.argtypes = [I64, I32]
    lib.pulse_lora_hidden_bytes.argtypes = [I64, I64, I32]
    lib.pulse_lora_ws_bytes.argtypes = [I64, I64, I64, I64, I32, I32]
    lib.pulse_lora_plan.argtypes = [V, I64, I32, V, I64, V, V]
    lib.pulse_lora_forward.argtypes = [V, I64, V, V, V, V, I64, I64, I64, I64, I64, I32, V, I64, V, I64, V,
                                       ctypes.c_size_t, V]
    lib.pulse_lora_backward.argtypes = [V, I64, V, I64, V, V, V, V, I64, I64, I64, I64, I64, I32, V, I64, V, I64, V, V,
                                        I32, V, ctypes.c_size_t, V]
    return lib


SIZES = [(dict(rank=4), EINVAL), (dict(rank=12), EINVAL), (dict(rank=136), ERANGE), (dict(k=12), EINVAL),
         (dict(k=0), EINVAL), (dict(n=7), EINVAL), (dict(n_adapters=0), EINVAL), (dict(n_adapters=1025), ERANGE),
         (dict(n_tokens=-1), EINVAL), (dict(n_tokens=1 << 25), ERANGE), (dict(k=1 << 25), ERANGE)]
POINTERS = ["x", "a", "b", "scales", "plan", "y", "ws"]


@pytest.mark.parametrize("bad,code", SIZES + [({p: None}, EINVAL if p != "ws" else EWORKSPACE) for p in POINTERS] + [
    ({p: 0x10008}, EALIGN) for p in POINTERS if p != "scales"] + [
    (dict(h=0x10008), EALIGN), (dict(ldx=56), EINVAL), (dict(ldx=68), EINVAL), (dict(ldy=24), EINVAL),
    (dict(plan_bytes=100), EWORKSPACE), (dict(ws_bytes=100), EWORKSPACE), (dict(h=0x10000, h_bytes=8), EWORKSPACE)])
def test_forward_refuses(lib, bad, code):  # noqa: F811
    calls(lib)
    c = dict(x=0x10000, ldx=64, a=0x10000, b=0x10000, scales=0x10000, plan=0x10000, plan_bytes=1 << 30, n_tokens=10,
             k=64, n=32, rank=16, n_adapters=4, y=0x10000, ldy=32, h=None, h_bytes=0, ws=0x10000, ws_bytes=1 << 30) | bad
    assert lib.pulse_lora_forward(*c.values(), None) == code


@pytest.mark.parametrize("bad,code", SIZES + [({p: None}, EINVAL if p != "ws" else EWORKSPACE)
                                              for p in ("x", "dy", "a", "b", "scales", "plan", "h", "da", "db", "ws")] + [
    ({p: 0x10008}, EALIGN) for p in ("x", "dy", "a", "b", "plan", "h", "dx", "da", "db", "ws")] + [
    (dict(lddy=24), EINVAL), (dict(lddx=60), EINVAL), (dict(accumulate=2), EINVAL), (dict(h_bytes=8), EWORKSPACE),
    (dict(ws_bytes=100), EWORKSPACE)])
def test_backward_refuses(lib, bad, code):  # noqa: F811
    calls(lib)
    c = dict(x=0x10000, ldx=64, dy=0x10000, lddy=32, a=0x10000, b=0x10000, scales=0x10000, plan=0x10000,
             plan_bytes=1 << 30, n_tokens=10, k=64, n=32, rank=16, n_adapters=4, h=0x10000, h_bytes=1 << 30, dx=0x10000,
             lddx=64, da=0x10000, db=0x10000, accumulate=0, ws=0x10000, ws_bytes=1 << 30) | bad
    assert lib.pulse_lora_backward(*c.values(), None) == code


def test_plan_refuses_and_empty_batches_enqueue_nothing(lib):  # noqa: F811
    calls(lib)
    al, big = 0x10000, 1 << 30
    assert lib.pulse_lora_plan(None, 3, 4, al, big, al, None) == EINVAL
    assert lib.pulse_lora_plan(al, 3, 4, None, big, al, None) == EINVAL
    assert lib.pulse_lora_plan(al, 3, 4, al, big, None, None) == EINVAL
    assert lib.pulse_lora_plan(al, 3, 4, 0x10004, big, al, None) == EALIGN
    assert lib.pulse_lora_plan(al, 3, 1025, al, big, al, None) == ERANGE
    assert lib.pulse_lora_plan(al, 3, 4, al, lib.pulse_lora_plan_bytes(3, 4) - 1, al, None) == EWORKSPACE
    assert lib.pulse_lora_plan(None, 0, 4, al, big, al, None) == 0
    assert lib.pulse_lora_forward(None, 0, al, al, al, al, big, 0, 64, 32, 16, 4, None, 0, None, 0, al, big, None) == 0
    assert lib.pulse_lora_backward(None, 0, None, 0, al, al, al, al, big, 0, 64, 32, 16, 4, None, 0, None, 0, al, al, 1,
                                   al, big, None) == 0


def test_sizes_serve_every_smaller_batch(lib):  # noqa: F811
    calls(lib)
    assert lib.pulse_lora_ws_bytes(10, 64, 32, 12, 4, 0) == EINVAL and lib.pulse_lora_ws_bytes(10, 64, 32, 16, 4, 2) == EINVAL
    assert lib.pulse_lora_hidden_bytes(10, 256, 4) == ERANGE and lib.pulse_lora_plan_bytes(10, 0) == EINVAL
    for k, n, r, s in ((64, 32, 8, 1), (4096, 14336, 16, 1), (5120, 27648, 64, 8), (1024, 1024, 128, 1000)):
        last = (0, 0, 0, 0)
        for t in (0, 1, 2, 15, 16, 17, 63, 64, 65, 100, 500, 1000, 1023, 1024, 4000, 8192, 16384, 16385, 100_000):
            now = (lib.pulse_lora_plan_bytes(t, s), lib.pulse_lora_hidden_bytes(t, r, s),
                   lib.pulse_lora_ws_bytes(t, k, n, r, s, 0), lib.pulse_lora_ws_bytes(t, k, n, r, s, 1))
            assert all(a >= b >= 0 for a, b in zip(now, last)), t
            last = now
