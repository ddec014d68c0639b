"""Products of quantised rows with weights in 128 x 128 blocks against float64."""
import numpy as np
import pytest
import torch

import sparse_delta_codec_amd as pulse
from tests import sampler_ref as ref

pytestmark = pytest.mark.gpu


def codes_like(shape, g, std=60.0):
    z = np.clip(g.normal(0, std, shape), -448, 448).astype(np.float32)
    return torch.from_numpy(z).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def problem(m, n, k, form, seed=0):
    g = np.random.default_rng(seed + m * 7 + n * 3 + k)
    inner = k if form == "nt" else n
    x, w = codes_like((m, inner), g), codes_like((n, k), g)
    sx = g.uniform(0.5, 2.0, (m, ref.groups(inner))).astype(np.float32)
    sw = (g.uniform(0.5, 2.0, (ref.groups(n), ref.groups(k))) * 1e-3).astype(np.float32)
    return x, sx, w, sw


def multiply(x, sx, w, sw, form, bias=None, pad=0, ws=None):
    m, (n, k) = x.shape[0], w.shape
    out = n if form == "nt" else k
    y = torch.full((m + 1, out + pad), -77.0, dtype=torch.bfloat16, device="cuda")
    ws = pulse.fp8_gemm_workspace(m, n, k, form) if ws is None else ws
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    b = None if bias is None else torch.from_numpy(bias).to(torch.bfloat16).cuda()
    pulse.fp8_block_gemm(dev(x), dev(sx), dev(w), dev(sw), y[:m, :out], ws, bias=b, form=form)
    torch.cuda.synchronize()
    assert (y[m] == -77).all() and (y[:, out:] == -77).all()  # what is not the result stays
    return y[:m, :out].double().cpu().numpy()


def check(got, y, e):
    bad = np.abs(got - y) > 1.02 * (e + (np.abs(y) + e) * ref.HALF_BF16) + 1e-30
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(got - y).max())


# one token to many, odd rows and columns, contractions that end inside a step, each variant's edges
NT = [(1, 1, 16), (1, 16, 128), (1, 130, 144), (1, 512, 4096), (2, 257, 1040), (3, 100, 272), (5, 640, 2000), (7, 1000, 5120),
      (16, 128, 256), (17, 300, 640), (31, 77, 1936), (33, 136, 4096), (48, 256, 1264), (64, 384, 1024), (65, 129, 400), (96, 513, 2560),
      (128, 128, 128), (129, 255, 272), (200, 700, 1552), (257, 300, 528), (640, 1001, 336), (1030, 2050, 400), (300, 3500, 656), (4100, 2050, 272), (2049, 4100, 128),
      (1, 7168, 1040), (8, 5136, 2064), (9, 5136, 2064), (16, 4112, 1040), (12, 300, 5136), (1, 128, 27200), (16, 130, 9232), (100, 128, 9232)]
NN = [(1, 16, 16), (1, 128, 128), (1, 144, 272), (2, 1040, 256), (5, 640, 2000), (16, 272, 144), (33, 4096, 136 + 8), (64, 1024, 384),
      (65, 400, 144), (100, 2560, 528), (129, 272, 256), (257, 528, 304), (640, 336, 1008), (1030, 400, 2064), (300, 656, 3504), (4100, 272, 2064), (2049, 128, 4112),
      (1, 27200, 128), (20, 9232, 144)]


@pytest.mark.parametrize("m,n,k", NT)
def test_projection(m, n, k):
    x, sx, w, sw = problem(m, n, k, "nt")
    bias = ref.bf16(np.random.default_rng(1).normal(0, 3, n)) if (m + n) % 2 else None
    y, e = ref.gemm(x, sx, w, sw, "nt", bias)
    check(multiply(x, sx, w, sw, "nt", bias, pad=(0, 3, 8)[n % 3]), y, e)


@pytest.mark.parametrize("m,n,k", NN)
def test_input_gradient(m, n, k):
    x, sx, w, sw = problem(m, n, k, "nn")
    y, e = ref.gemm(x, sx, w, sw, "nn")
    check(multiply(x, sx, w, sw, "nn", pad=(0, 5, 8)[m % 3]), y, e)


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("m", [1, 20, 100, 300])
def test_every_place_of_a_tile(form, m):
    """Whole numbers that the sums hold exactly: every row, column and step in its own place."""
    n, k = (384, 640) if form == "nt" else (640, 384)
    g = np.random.default_rng(9)
    inner = 640
    small = torch.arange(-8, 9).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    x, w = small[g.integers(0, 17, (m, inner))], small[g.integers(0, 17, (n, k))]
    sx = (2.0 ** g.integers(-1, 2, (m, 5))).astype(np.float32)
    sw = (2.0 ** g.integers(-1, 2, (ref.groups(n), ref.groups(k)))).astype(np.float32)
    y, _ = ref.gemm(x, sx, w, sw, form)
    np.testing.assert_array_equal(multiply(x, sx, w, sw, form), ref.bf16(y))


def test_gradient_is_the_projections():
    """dx of the sum of dy * (x w^T), against differences: the product is linear, so dy w is exact."""
    n, k = 128, 256
    _, _, w, sw = problem(1, n, k, "nt", 4)
    small = torch.arange(-8, 9).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    dy = small[np.random.default_rng(2).integers(0, 17, (3, n))]
    one = np.ones((3, 1), dtype=np.float32)
    dx = multiply(dy, one, w, sw, "nn")
    # rows of the unit matrix through the projection give w's columns
    unit = np.zeros((k, k), dtype=np.uint8)
    unit[np.arange(k), np.arange(k)] = 0x38  # 1.0
    wt = multiply(unit, np.ones((k, 2), dtype=np.float32), w, sw, "nt")  # [k, n], each rounded to BF16
    want = ref.E4M3[dy] @ wt.T
    room = np.abs(ref.E4M3[dy]) @ np.abs(wt.T) * (ref.HALF_BF16 + 7 * ref.CUT + 40 * ref.HALF_F32)
    assert (np.abs(dx - want) <= 1.02 * (room + np.abs(want) * ref.HALF_BF16)).all()


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("m", [1, 40, 300])
def test_nan_codes_reach_their_rows_and_columns_only(form, m):
    """A NaN in a row of x makes that row of y NaN, one in a weight that column, also where the
    contraction ends inside a step."""
    n, k = (144, 272) if form == "nt" else (272, 144)
    x, sx, w, sw = problem(m, n, k, form, 6)
    if form == "nt":
        w[5, 256], w[9, 271] = 0x7F, 0xFF
    else:
        w[256, 5], w[271, 9] = 0x7F, 0xFF
    if m > 1:
        x[m - 1, 270] = 0x7F
    got = multiply(x, sx, w, sw, form)
    want = np.zeros(got.shape, dtype=bool)
    want[:, [5, 9]] = True
    if m > 1:
        want[m - 1] = True
    np.testing.assert_array_equal(np.isnan(got), want)


def test_scales_of_zero_groups_and_infinity():
    """A scale of Inf or NaN reaches its row; other rows keep their results."""
    x, sx, w, sw = problem(40, 130, 400, "nt", 8)
    sx[3, 1], sx[17, 3] = np.inf, np.nan
    clean = sx.copy()
    clean[3, 1] = clean[17, 3] = 1
    got = multiply(x, sx, w, sw, "nt")
    y, e = ref.gemm(x, clean, w, sw, "nt")
    keep = np.ones(40, dtype=bool)
    keep[[3, 17]] = False
    check(got[keep], y[keep], e[keep])
    assert not np.isfinite(got[3]).any() and np.isnan(got[17]).all()


@pytest.mark.parametrize("m", [1, 24, 64, 300])
def test_repeats_bit_for_bit(m):
    """The same call gives the same bits, whatever the workspace held."""
    x, sx, w, sw = problem(m, 640, 5120, "nt", 3)
    ws = pulse.fp8_gemm_workspace(m, 640, 5120)
    a = multiply(x, sx, w, sw, "nt", ws=ws)
    ws.fill_(255)
    b = multiply(x, sx, w, sw, "nt", ws=ws)
    np.testing.assert_array_equal(a, b)


def test_no_tokens():
    x, sx, w, sw = problem(3, 128, 128, "nt")
    assert multiply(x[:0], sx[:0], w, sw, "nt").shape == (0, 128)


# rows, columns of y and contraction that make each size of tile, alone, shared, both at once, and
# one row of tiles: 256 x 256, 128 x 256, 128 x 128 and 64 x 128
TILES = [(900, 8208, 144), (2000, 8208, 528), (900, 5136, 8208), (4100, 1000 + 8, 144), (1500, 1008, 8208), (2000, 8208, 144),
         (250, 8208, 8208), (250, 8208, 144), (1500, 512, 4112), (70, 4112, 8208), (4100, 4112, 144), (70, 256, 144), (70, 8208, 144),
         (250, 8208, 4112), (4099, 4112, 1040), (4099, 8208, 528), (40, 16400, 4112), (40, 33040, 144), (70, 33040, 4112),
         (70, 16400, 144), (70, 16400, 4112), (40, 33040, 1040), (40, 144, 144), (40, 16400, 144), (900, 16400, 528), (130, 33040, 4112),
         (130, 16400, 4112), (120, 16400, 4112), (70, 144, 4112), (20, 144, 1040), (70, 2064, 4112)]


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("m,j,c", TILES)
def test_each_tile_holds_whole_numbers(m, j, c, form):
    """Whole numbers up to 8 by 8 that the sums hold exactly, over every row and column."""
    n, k = (j, c) if form == "nt" else (c, j)
    gen = torch.Generator(device="cuda").manual_seed(m + j + c)
    whole = lambda *s: torch.randint(-8, 9, s, device="cuda", generator=gen).float()  # noqa: E731
    power = lambda *s: torch.pow(2.0, torch.randint(-1, 2, s, device="cuda", generator=gen).float())  # noqa: E731
    x, w = whole(m, c), whole(n, k)
    sx, sw = power(m, ref.groups(c)), power(ref.groups(n), ref.groups(k))
    y = torch.full((m + 1, j), -77.0, dtype=torch.bfloat16, device="cuda")
    codes = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    ws = pulse.fp8_gemm_workspace(m, n, k, form)
    ws.fill_(255)
    pulse.fp8_block_gemm(codes(x), sx, codes(w), sw, y[:m], ws, form=form)
    wide = lambda s, d, size: s.repeat_interleave(128, d).narrow(d, 0, size)  # noqa: E731
    xv = (x * wide(sx, 1, c)).double()
    wv = (w * wide(wide(sw, 0, n), 1, k)).double()
    want = xv @ (wv.t() if form == "nt" else wv)
    assert torch.equal(y[:m], want.to(torch.bfloat16))
    assert (y[m] == -77).all()


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("m,j,c", [(900, 8208, 144), (2000, 2064, 1040), (1500, 1008, 8208), (70, 4112, 8208), (250, 1040, 4112)])
def test_tiles_of_any_values(m, j, c, form):
    """Some rows of larger products against float64."""
    n, k = (j, c) if form == "nt" else (c, j)
    x, sx, w, sw = problem(m, n, k, form, 12)
    rows = np.unique(np.r_[0, 1, 15, 16, 63, 64, m - 2, m - 1, np.random.default_rng(m).integers(0, m, 24)])
    y, e = ref.gemm(x[rows], sx[rows], w, sw, form)
    check(multiply(x, sx, w, sw, form)[rows], y, e)


def test_offsets_past_31_bits():
    """Weights and output of more than 2^31 elements: the last rows and columns are right."""
    n, k, m = 1 << 17, 16400, 16
    w = torch.zeros((n, k), dtype=torch.uint8, device="cuda")  # 2.15e9 codes
    sw = torch.ones((ref.groups(n), ref.groups(k)), device="cuda")
    w[n - 1, k - 1], w[n - 1, 0], w[n - 130, k - 200], w[0, 5] = 0x38, 0x40, 0x38, 0x38  # 1, 2, 1, 1
    x = torch.zeros((m, k), dtype=torch.uint8, device="cuda")
    x[:, k - 1], x[:, 0], x[3, k - 200], x[:, 5] = 0x38, 0x40, 0x44, 0x38
    sx = torch.ones((m, ref.groups(k)), device="cuda")
    for rows in (m, 40):
        xs, ss = (x, sx) if rows == m else (torch.cat([x, x, x])[:rows].contiguous(), torch.ones((rows, ref.groups(k)), device="cuda"))
        y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
        pulse.fp8_block_gemm(xs, ss, w, sw, y, pulse.fp8_gemm_workspace(rows, n, k))
        assert (y[:, n - 1] == 5).all() and (y[:, 0] == 1).all() and y[3, n - 130] == 3 and y[2, n - 130] == 0
        assert int((y != 0).sum()) == 2 * rows + sum(r % m == 3 for r in range(rows))
    # nn: a contraction over those rows
    dy = torch.zeros((8, n), dtype=torch.uint8, device="cuda")
    dy[:, n - 1], dy[2, 0] = 0x38, 0x38
    dx = torch.empty((8, k), dtype=torch.bfloat16, device="cuda")
    pulse.fp8_block_gemm(dy, torch.ones((8, ref.groups(n)), device="cuda"), w, sw, dx, pulse.fp8_gemm_workspace(8, n, k, "nn"), form="nn")
    assert (dx[:, k - 1] == 1).all() and (dx[:, 0] == 2).all() and dx[2, 5] == 1 and int((dx != 0).sum()) == 17
