"""Plain float64 implementations of the sampler's operators for the tests, with the
bounds of what the library's documented roundings may change.  No code is shared
with the library."""
import numpy as np
import torch

HALF_BF16 = 2.0 ** -8   # half a step, relative
HALF_F32 = 2.0 ** -24
HALF_E4M3 = 2.0 ** -4
GROUP = 128
TOP = 448.0
TINY = 2.0 ** -96

E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)]
                + [np.nan])
E4M3 = np.concatenate([E4M3, -E4M3])


def bf16(x):
    """x rounded to BF16, as float64."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def groups(cols):
    return -(-cols // GROUP)


def per_group(scales, cols):
    """[rows, groups] scales as [rows, cols]."""
    return np.repeat(scales, GROUP, axis=-1)[..., :cols]


def quantise(x):
    """Codes and scales of float32 rows by the documented float32 arithmetic."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    t, c = x.shape
    scales = np.ones((t, groups(c)), dtype=np.float32)
    q = np.zeros_like(x)
    for g in range(groups(c)):
        part = x[:, g * GROUP:(g + 1) * GROUP]
        amax = np.abs(part).max(axis=1)
        scales[:, g] = np.where(amax >= np.float32(TINY), amax / np.float32(TOP), np.float32(1))
        q[:, g * GROUP:(g + 1) * GROUP] = part / scales[:, g:g + 1]
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scales


def block_scales(scales, shape):
    s = np.repeat(np.repeat(scales.astype(np.float64), GROUP, axis=-1), GROUP, axis=-2)
    return s[..., :shape[-2], :shape[-1]]


def row_values(codes, scales):
    return E4M3[codes] * per_group(scales.astype(np.float64), codes.shape[-1])


def block_values(codes, scales):
    return E4M3[codes] * block_scales(scales, codes.shape)


def check_codes(codes, scales, x, rel):
    """Codes and scales of rows whose float32 values lie within `rel` of x: the scale has
    that error and its division's, a code half a step of its value (of the smallest step below
    2^-6) and the error of its quotient."""
    want = np.zeros(scales.shape)
    for g in range(scales.shape[1]):
        want[:, g] = np.abs(x[:, g * GROUP:(g + 1) * GROUP]).max(axis=1) / TOP
    want = np.where(want * TOP < TINY, 1.0, want)
    np.testing.assert_allclose(scales, want, rtol=1.02 * (rel + HALF_F32), atol=0)
    s = per_group(scales.astype(np.float64), x.shape[1])
    q = x / s
    # half a step: 2^-4 of the value's power of two, 2^-10 below 2^-6
    half = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6))) - 4), 2.0 ** -10)
    err = np.abs(E4M3[codes] - q)
    assert (err <= half + 2.04 * np.abs(q) * (rel + 2 * HALF_F32) + 1e-12).all(), err.max()


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def rms_norm(s, w, eps):
    """(y, rstd)."""
    rstd = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s * rstd * w, rstd[:, 0]


def rstd_error(n):
    """Relative: a sum of n squares (n roundings at most), the mean, eps, root and quotient."""
    return (0.5 * (n + 4) + 3) * HALF_F32


def rms_norm_backward(s, w, dy, eps, dres=None):
    """(dx, dweight)."""
    n = s.shape[1]
    rstd = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    g = dy * w
    dx = rstd * g - s * rstd ** 3 * (g * s).sum(axis=1, keepdims=True) / n
    return dx if dres is None else dx + dres, (dy * s * rstd).sum(axis=0)


# The matrix instruction for 8-bit values adds up eight neighbouring products, each cut to a
# multiple of this part of the largest one's power of two (beside 2^16, a product of 2^3 counts
# and one of 2^2 does not, on the GPU); the sum of the eight lacks up to seven such parts.
CUT = 2.0 ** -13


def eights(v, axis):
    """The largest magnitude of each eight along the axis, which is a step of 16 such or shorter."""
    v = np.moveaxis(np.abs(v), axis, -1)
    return np.moveaxis(v.reshape(*v.shape[:-1], -1, 8).max(axis=-1), -1, axis)


def gemm(x, sx, w, sw, form, bias=None):
    """(y, bound of the error before y is rounded)."""
    xv, wv = E4M3[x], E4M3[w]
    if form == "nt":
        wv, sw = wv.T, sw.T
    m, inner = x.shape
    y, e, cut = (np.zeros((m, wv.shape[1])) for _ in range(3))
    blocks = groups(inner)
    for b in range(blocks):
        span = slice(b * GROUP, (b + 1) * GROUP)
        f = sx[:, b:b + 1].astype(np.float64) * np.repeat(sw[b].astype(np.float64), GROUP)[None, :wv.shape[1]]
        y += f * (xv[:, span] @ wv[span])
        e += np.abs(f) * (np.abs(xv[:, span]) @ np.abs(wv[span]))
        cut += np.abs(f) * (eights(xv[:, span], 1) @ eights(wv[span], 0)) * 7 * CUT
    if bias is not None:
        y = y + bias
    # cut products, float32 sums of a block (16 groups of eight) and of the blocks
    return y, cut + e * (16 + blocks + 4) * HALF_F32 + np.abs(y) * 2 * HALF_F32


def moe(x, ids, weights, up, su, down, sd):
    """(y, bound of the error before y is rounded)."""
    t, hidden = x.shape
    y, e = np.zeros((t, hidden)), np.zeros((t, hidden))
    inter = down.shape[2]
    for i in range(t):
        for j in range(ids.shape[1]):
            k = ids[i, j]
            if not 0 <= k < up.shape[0]:
                continue
            wu, wd = block_values(up[k], su[k]), block_values(down[k], sd[k])
            both, mag = wu @ x[i], np.abs(wu) @ np.abs(x[i])
            err = mag * (hidden + 4) * HALF_F32          # float32 sums
            g, u = both[:inter], both[inter:]
            h = silu(g) * u
            # silu' is at most 1.1; its own float32 error a few roundings
            eh = 1.1 * err[:inter] * np.abs(u) + np.abs(silu(g)) * err[inter:] + 1.1 * err[:inter] * err[inter:]
            eh += np.abs(h) * (8 * HALF_F32 + 2.0 ** -16)
            p = float(weights[i, j])
            y[i] += p * (wd @ h)
            e[i] += abs(p) * (np.abs(wd) @ eh + np.abs(wd) @ np.abs(h) * (2 * inter + 4 + ids.shape[1]) * HALF_F32)
    return y, 1.02 * e


def route(logits, top_k, over_all=False, scale=1.0):
    """(ids, weights): NaN above all, -inf not chosen, equal logits by the lowest index."""
    t, n = logits.shape
    ids, weights = np.full((t, top_k), -1, dtype=np.int32), np.zeros((t, top_k))
    for i in range(t):
        v = logits[i].astype(np.float64)
        order = sorted(range(n), key=lambda e: (not np.isnan(v[e]), -v[e] if not np.isnan(v[e]) else 0, e))
        chosen = [e for e in order[:top_k] if v[e] != -np.inf]
        ids[i, :len(chosen)] = chosen
        if not chosen:
            continue
        with np.errstate(invalid="ignore"):
            part = np.exp(v[chosen] - v[chosen[0]])
            total = np.exp(v - v[chosen[0]]).sum() if over_all else part.sum()
            weights[i, :len(chosen)] = part / total * scale
    return ids, weights
