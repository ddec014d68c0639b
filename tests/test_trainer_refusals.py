"""Values of the trainer's calls that are refused because of what they are in float32;
the calls return before anything is enqueued."""
import ctypes

import pytest

from tests.test_abi import EALIGN, EINVAL, lib  # noqa: F401  (the library fixture)
from tests.test_oracle_adamw import I32, I64, Params, V, good


@pytest.mark.parametrize("bad", [dict(eps=1e-50), dict(eps=7e-46), dict(eps=1e39), dict(lr=1e39), dict(lr=3.5e38),
                                 dict(beta1=1 - 1e-9), dict(beta2=1 - 1e-9),
                                 dict(lr=-1e-50), dict(beta1=-1e-50)])
def test_adamw_refuses_what_float32_does_not_hold(lib, bad):  # noqa: F811
    """eps that is zero there (0 / 0 where gradient and states are zero), a rate or eps that is
    infinite, a beta that is one (states that never decay); and below zero in either type."""
    f = lib.pulse_adamw_step
    f.argtypes = [V, I32, V, I64, V, V, V, V, I64, V, V, V, ctypes.c_size_t, V]
    al, q = V(0x10000), Params(**(good() | bad))
    assert f(al, 1, al, 1, ctypes.byref(q), None, None, None, 0, None, al, None, 0, None) == EINVAL


def test_grad_norm_refuses_an_unaligned_workspace(lib):  # noqa: F811
    """It holds float64 partial sums and a counter."""
    f = lib.pulse_grad_norm
    f.argtypes = [V, I32, V, I64, I32, ctypes.c_double, ctypes.c_double, V, V, ctypes.c_size_t, V]
    al = V(0x10000)
    for off in (1, 2, 4):
        assert f(al, 1, al, 1, 0, 1.0, 1.0, al, V(0x10000 + off), 1 << 20, None) == EALIGN
