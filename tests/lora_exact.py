"""Adapter inputs whose results are whole numbers, exact in float32 and in the type they
go out in, and that need the bits of h that one BF16 has not."""
import numpy as np


def bf16_round(v):
    """Nearest BF16, ties to even, of float32 values (finite), as float64."""
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32).astype(np.float64)


def spread_ids(t, s):
    """Adapters in turn, and no adapter for some tokens (not for the first of an adapter)."""
    ids = np.arange(t) * 7 % s if s % 7 else np.arange(t) % s
    ids[np.arange(t) % 11 == 10] = -1
    if t >= 11 * s:
        ids[:s] = np.arange(s)
    return ids


def whole_rows(t, k, n, r, s, ids, seed=0):
    """(x [t, k], a [s, r, k], b [s, r, n], y [t, n], y + B^T A x).  h are whole numbers below
    2^16, a column of y takes two of them, and y is minus their sum's nearest BF16, so that
    the result is the rest: at most 2^8, and not zero in most places."""
    rng = np.random.default_rng(seed)
    x = rng.integers(-127, 128, (t, k)).astype(np.float64)
    a = np.zeros((s, r, k))
    for i in range(3):
        at = rng.integers(0, k, (s, r, 1))
        np.put_along_axis(a, at, rng.integers(64, 128, (s, r, 1)).astype(np.float64), 2)
    b = np.zeros((s, r, n))
    cols = np.arange(n)
    b[:, cols % r, cols] = rng.choice([-1.0, 1.0], (s, n))
    b[:, (cols + 3) % r, cols] += rng.choice([-1.0, 1.0], (s, n)) if r > 3 else 0
    y, want = np.zeros((t, n)), np.zeros((t, n))
    for i in set(ids.tolist()) - {-1}:
        rows = np.flatnonzero(ids == i)
        h = x[rows] @ a[i].T
        add = h @ b[i]
        y[rows] = -bf16_round(add)
        want[rows] = add + y[rows]
    live = np.abs(want[ids >= 0])
    assert live.max() <= 256 and (live > 0).mean() > 0.5
    return x, a, b, y, want


def whole_sums(t, cols, k, r, s, ids, seed=1):
    """(z [t, cols], u [t, r], x [t, k], a [s, r, k], sum of u z^T per adapter): u = A x are
    whole numbers of up to 24 bits, and a column of z is not zero for one token of an adapter."""
    rng = np.random.default_rng(seed)
    x = rng.integers(1, 128, (t, k)).astype(np.float64)
    a = np.zeros((s, r, k))
    a[:, :, 0] = rng.integers(64, 128, (s, r)) * 512.0
    a[:, :, 1] = rng.integers(64, 128, (s, r))
    z, u, want = np.zeros((t, cols)), np.zeros((t, r)), np.zeros((s, r, cols))
    for i in set(ids.tolist()) - {-1}:
        rows = np.flatnonzero(ids == i)
        u[rows] = x[rows] @ a[i].T
        mine = rows[:cols]
        at = rng.permutation(cols)[:mine.size]
        z[mine, at] = rng.choice([-1.0, 1.0], mine.size)
        want[i] = u[rows].T @ z[rows]
    assert np.abs(u).max() < 2 ** 24
    return z, u, x, a, want
