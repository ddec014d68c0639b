"""Plain float64 implementation of the low-rank adapters for the tests, with the
bounds of what the library's documented roundings may change.  No code is
shared with the library."""
import numpy as np

HALF_BF16 = 2.0 ** -8   # half a step, relative
HALF_F32 = 2.0 ** -24


def forward(x, a, b, scales, ids, y):
    """(y', h): y' = y + B^T h, h = scale A x, zero for tokens without an adapter."""
    y, h = y.copy(), np.zeros((x.shape[0], a.shape[1]))
    for s in set(ids.tolist()) - {-1}:
        t = np.flatnonzero(ids == s)
        h[t] = scales[s] * (x[t] @ a[s].T)
        y[t] += h[t] @ b[s]
    return y, h


def backward(x, dy, a, b, scales, ids, dx):
    """(dx', da, db, dh)."""
    dx, da, db = dx.copy(), np.zeros(a.shape), np.zeros(b.shape)
    dh = np.zeros((x.shape[0], a.shape[1]))
    for s in set(ids.tolist()) - {-1}:
        t = np.flatnonzero(ids == s)
        h = scales[s] * (x[t] @ a[s].T)
        dh[t] = scales[s] * (dy[t] @ b[s].T)
        dx[t] += dh[t] @ a[s]
        da[s] = dh[t].T @ x[t]
        db[s] = h.T @ dy[t]
    return dx, da, db, dh


def hidden_error(x, a, scales, ids):
    """What float32 sums of K products and the scale may change in h: (K + 2) roundings."""
    e = np.zeros((x.shape[0], a.shape[1]))
    for s in set(ids.tolist()) - {-1}:
        t = np.flatnonzero(ids == s)
        e[t] = abs(scales[s]) * (np.abs(x[t]) @ np.abs(a[s]).T) * (x.shape[1] + 2) * HALF_F32
    return e


def row_bound(out, h, eh, w, ids):
    """For y or dx: one rounding of the result, one of h to BF16, h's own error and
    the R + 2 float32 roundings of the sum; 1.02 for the roundings' products."""
    bound = HALF_BF16 * np.abs(out)
    for s in set(ids.tolist()) - {-1}:
        t = np.flatnonzero(ids == s)
        part = np.abs(h[t]) * (HALF_BF16 + (h.shape[1] + 2) * HALF_F32) + eh[t]
        bound[t] += part @ np.abs(w[s])
        bound[t] += np.abs(out[t]) * (h.shape[1] + 2) * HALF_F32
    return 1.02 * bound + 1e-30


def grad_bound(u, eu, z, ids, shape):
    """For da or db: u enters with 2^-16 of itself, its own error, and the sum's
    float32 roundings, one per product (two of them a token)."""
    bound = np.zeros(shape)
    for s in set(ids.tolist()) - {-1}:
        t = np.flatnonzero(ids == s)
        part = np.abs(u[t]) * (2.0 ** -16 + (2 * t.size + 4) * HALF_F32) + eu[t]
        bound[s] = part.T @ np.abs(z[t])
    return 1.02 * bound + 1e-30
