"""Arguments that the sampler's calls refuse; they return before anything is enqueued."""
import ctypes

import pytest

import sparse_delta_codec_amd as pulse
from tests.test_abi import EALIGN, EINVAL, ERANGE, EWORKSPACE, lib  # noqa: F401  (the library fixture)

V, I64, I32, F64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_size_t
A = 0x10000  # an aligned address that no call gets to
NAN, INF = float("nan"), float("inf")


def call(lib, name, types, good, bad):  # noqa: F811
    f = getattr(lib, name)
    f.argtypes = types
    f.restype = ctypes.c_int
    return f(*(good | bad).values(), None)


NORM = [V, I64, V, F64, V, I64, V, I64, V, V, V, I64, I64, V]
GOOD_NORM = dict(x=A, ldx=256, w=A, eps=1e-6, res=A, ldr=256, y=A, ldy=256, codes=A, scales=A, rstd=A, t=4, n=256)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None, codes=None, scales=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(codes=None), EINVAL), (dict(n=0), EINVAL), (dict(n=12), EINVAL), (dict(n=-8), EINVAL), (dict(n=16392), ERANGE),
    (dict(t=-1), EINVAL), (dict(t=2 ** 24 + 1), ERANGE), (dict(eps=0), EINVAL), (dict(eps=-1e-6), EINVAL), (dict(eps=NAN), EINVAL),
    (dict(eps=INF), EINVAL), (dict(eps=1e-50), EINVAL), (dict(eps=1e39), EINVAL), (dict(ldx=248), EINVAL), (dict(ldx=260), EINVAL),
    (dict(ldr=248), EINVAL), (dict(ldy=257), EINVAL), (dict(x=A + 2), EALIGN), (dict(w=A + 8), EALIGN), (dict(res=A + 8), EALIGN),
    (dict(y=A + 2), EALIGN), (dict(codes=A + 8), EALIGN)])
def test_norm(lib, bad, code):  # noqa: F811
    assert call(lib, "pulse_rms_norm", NORM, GOOD_NORM, bad) == code


BACK = [V, I64, V, V, V, I64, V, I64, V, I64, V, I32, I64, I64, V, SZ, V]
GOOD_BACK = dict(s=A, lds=256, w=A, rstd=A, dy=A, lddy=256, dres=A, lddr=256, dx=A, lddx=256, dw=A, acc=0, t=4, n=256, ws=A,
                 wsb=4 * 256 * 4)


@pytest.mark.parametrize("bad,code", [
    (dict(s=None), EINVAL), (dict(w=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dy=None), EINVAL), (dict(dw=None), EINVAL),
    (dict(acc=2), EINVAL), (dict(acc=-1), EINVAL), (dict(lds=255), EINVAL), (dict(lddy=8), EINVAL), (dict(lddr=252), EINVAL),
    (dict(lddx=260), EINVAL), (dict(n=20), EINVAL), (dict(n=16392), ERANGE), (dict(t=-2), EINVAL), (dict(ws=None), EWORKSPACE),
    (dict(wsb=4095), EWORKSPACE), (dict(ws=A + 8), EALIGN), (dict(dw=A + 4), EALIGN), (dict(dx=A + 2), EALIGN),
    (dict(dres=A + 2), EALIGN), (dict(dy=A + 2), EALIGN), (dict(s=A + 2), EALIGN), (dict(w=A + 2), EALIGN)])
def test_norm_backward(lib, bad, code):  # noqa: F811
    assert call(lib, "pulse_rms_norm_backward", BACK, GOOD_BACK, bad) == code


QUANT = [V, I64, I64, I64, I32, V, V, V]
GOOD_QUANT = dict(x=A, ldx=512, t=4, n=256, glu=1, codes=A, scales=A)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(glu=2), EINVAL), (dict(n=4), EINVAL),
    (dict(n=0), EINVAL), (dict(ldx=504), EINVAL), (dict(ldx=516), EINVAL), (dict(t=-1), EINVAL), (dict(n=2 ** 24 + 8), ERANGE),
    (dict(t=2 ** 24 + 1), ERANGE), (dict(t=2 ** 24, n=2 ** 24, ldx=2 ** 25), ERANGE), (dict(x=A + 8), EALIGN), (dict(codes=A + 8), EALIGN)])
def test_group_quant(lib, bad, code):  # noqa: F811
    assert call(lib, "fp8_group_quant", QUANT, GOOD_QUANT, bad) == code


GEMM = [V, V, V, V, V, I32, I64, I64, I64, V, I64, V, SZ, V]
GOOD_GEMM = dict(x=A, sx=A, w=A, sw=A, bias=A, form=0, m=4, n=256, k=5120, y=A, ldy=256, ws=A, wsb=1 << 40)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), EINVAL), (dict(sx=None), EINVAL), (dict(w=None), EINVAL), (dict(sw=None), EINVAL), (dict(y=None), EINVAL),
    (dict(form=2), EINVAL), (dict(form=-1), EINVAL), (dict(k=24), EINVAL), (dict(k=0), EINVAL), (dict(n=0), EINVAL), (dict(m=-1), EINVAL),
    (dict(form=1, n=257, ldy=5120), EINVAL), (dict(form=1), EINVAL), (dict(ldy=255), EINVAL), (dict(k=2 ** 22 + 16), ERANGE),
    (dict(n=2 ** 22 + 1, ldy=2 ** 23), ERANGE), (dict(m=2 ** 24 + 1), ERANGE), (dict(m=2 ** 24, n=2 ** 22, ldy=2 ** 22), ERANGE),
    (dict(x=A + 8), EALIGN), (dict(w=A + 4), EALIGN), (dict(y=A + 2), EALIGN), (dict(ws=A + 8), EALIGN)])
def test_gemm(lib, bad, code):  # noqa: F811
    assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, bad) == code


def test_gemm_workspace(lib):  # noqa: F811
    """A call that shares the contraction refuses less than it asks for; sizes that are refused have no size."""
    size = lib.fp8_block_gemm_ws_bytes
    size.argtypes, size.restype = [I64, I64, I64, I32], I64
    need = size(96, 512, 27648, 0)
    assert need > 0
    bad = dict(m=96, n=512, k=27648, ldy=512)
    assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, bad | dict(ws=None)) == EWORKSPACE
    assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, bad | dict(wsb=need - 1)) == EWORKSPACE
    assert size(0, 512, 27648, 0) == 0
    assert size(96, 512, 27640, 0) == EINVAL and size(96, 2 ** 22 + 1, 256, 0) == ERANGE and size(1, 10, 16, 1) == EINVAL


ROUTE = [V, I64, I64, I64, I64, I32, F64, V, V, V]
GOOD_ROUTE = dict(logits=A, ld=60, t=4, e=60, k=4, over=0, scale=1.0, ids=A, w=A)


@pytest.mark.parametrize("bad,code", [
    (dict(logits=None), EINVAL), (dict(ids=None), EINVAL), (dict(w=None), EINVAL), (dict(ld=59), EINVAL), (dict(k=0), EINVAL),
    (dict(k=61), EINVAL), (dict(e=0), EINVAL), (dict(over=2), EINVAL), (dict(scale=NAN), EINVAL), (dict(scale=1e39), EINVAL),
    (dict(t=-1), EINVAL), (dict(t=2 ** 24 + 1), ERANGE), (dict(e=1025, ld=1025), ERANGE), (dict(k=33), ERANGE)])
def test_route(lib, bad, code):  # noqa: F811
    assert call(lib, "pulse_moe_route", ROUTE, GOOD_ROUTE, bad) == code


MOE = [V, I64, V, V, V, V, V, V, I64, I64, I64, I64, I64, V, I64, V, V, SZ, V]
GOOD_MOE = dict(x=A, ldx=256, ids=A, w=A, up=A, su=A, down=A, sd=A, t=4, h=256, i=128, e=8, k=2, y=A, ldy=256, status=A, ws=A,
                wsb=1 << 40)


@pytest.mark.parametrize("bad,code", [
    *((dict([(n, None)]), EINVAL) for n in ("x", "ids", "w", "up", "su", "down", "sd", "y", "status")),
    (dict(h=8), EINVAL), (dict(h=264, ldx=264, ldy=264), EINVAL), (dict(i=0), EINVAL), (dict(i=24), EINVAL), (dict(e=0), EINVAL),
    (dict(k=0), EINVAL), (dict(k=9), EINVAL), (dict(t=-1), EINVAL), (dict(ldx=248), EINVAL), (dict(ldx=260), EINVAL),
    (dict(ldy=255), EINVAL), (dict(t=1025), ERANGE), (dict(h=65552, ldx=65552, ldy=65552), ERANGE), (dict(i=65552), ERANGE),
    (dict(e=1025), ERANGE), (dict(e=64, k=33), ERANGE), (dict(t=1024, e=64, k=9), ERANGE), (dict(ldx=2 ** 20 + 8), ERANGE),
    (dict(x=A + 8), EALIGN), (dict(up=A + 8), EALIGN), (dict(down=A + 8), EALIGN), (dict(y=A + 8), EALIGN), (dict(ws=A + 8), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(wsb=100), EWORKSPACE)])
def test_moe(lib, bad, code):  # noqa: F811
    assert call(lib, "pulse_moe_forward", MOE, GOOD_MOE, bad) == code


@pytest.mark.parametrize("name,types,good,bad", [
    ("pulse_rms_norm", NORM, GOOD_NORM, dict(t=2 ** 24)), ("pulse_rms_norm_backward", BACK, GOOD_BACK, dict(t=2 ** 24, wsb=1 << 40)),
    ("fp8_group_quant", QUANT, GOOD_QUANT, dict(t=2 ** 24)),
    ("fp8_group_quant", QUANT, GOOD_QUANT, dict(t=2 ** 23, n=32 * 512, ldx=2 ** 15)),
    ("fp8_block_gemm", GEMM, GOOD_GEMM, dict(m=2 ** 24)), ("pulse_moe_route", ROUTE, GOOD_ROUTE, dict(t=2 ** 24)),
    ("fp8_block_gemm", GEMM, GOOD_GEMM, dict(m=2 ** 20, n=2 ** 16, k=16, ldy=2 ** 16))])
def test_launches_that_count_past_32_bits(lib, name, types, good, bad):  # noqa: F811
    """2^24 workgroups of 256 threads, 2^23 of 512."""
    assert call(lib, name, types, good, bad) == ERANGE


def test_unknown_form():
    with pytest.raises(ValueError, match="expected one of"):
        pulse.fp8_gemm_workspace(4, 256, 256, "tn", device="cpu")


def test_nothing_to_do(lib):  # noqa: F811
    """No tokens: nothing is read, written or launched."""
    none = dict(x=None, y=None, codes=None, scales=None, res=None, rstd=None)
    assert call(lib, "pulse_rms_norm", NORM, GOOD_NORM, none | dict(t=0)) == 0
    assert call(lib, "fp8_group_quant", QUANT, GOOD_QUANT, dict(t=0, x=None, codes=None, scales=None)) == 0
    assert call(lib, "fp8_block_gemm", GEMM, GOOD_GEMM, dict(m=0, x=None, y=None, ws=None, wsb=0)) == 0
    assert call(lib, "pulse_moe_route", ROUTE, GOOD_ROUTE, dict(t=0, logits=None, ids=None, w=None)) == 0
    assert call(lib, "pulse_moe_forward", MOE, GOOD_MOE, dict(t=0, x=None, ids=None, w=None, y=None, ws=None, wsb=0)) == 0


def test_sizes(lib):  # noqa: F811
    for f, types, args, want in [("pulse_rms_norm_ws_bytes", [I64, I64], (-1, 256), EINVAL), ("pulse_rms_norm_ws_bytes", [I64, I64], (1, 20), EINVAL),
                                 ("pulse_rms_norm_ws_bytes", [I64, I64], (1, 16392), ERANGE),
                                 ("pulse_moe_ws_bytes", [I64] * 5, (1, 256, 128, 8, 9), EINVAL),
                                 ("pulse_moe_ws_bytes", [I64] * 5, (1025, 256, 128, 8, 2), ERANGE)]:
        g = getattr(lib, f)
        g.argtypes, g.restype = types, I64
        assert g(*args) == want
