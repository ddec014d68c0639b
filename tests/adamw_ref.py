"""Plain implementations of the trainer's step for the tests, on the CPU.

step32 / step8 follow the documented order of float32 operations, each rounded
once, so the library's results equal theirs bit for bit; step64 is the formula
in float64.  No code is shared with the library."""
import numpy as np

BLOCK = 256
F = np.float32


def bf16_bits(x):
    """float32 -> BF16 bits, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32)


def e4m3_table():
    """The 256 values of OCP E4M3 by code (NaN for 0x7F and 0xFF)."""
    v = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        a = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = -a if c & 128 else a
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = e4m3_table()


def mix(x):
    x = np.asarray(x, np.uint64) & 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(n, tensor, seed):
    key = mix((seed + (tensor + 1) * 0x9E3779B1) & 0xFFFFFFFF)
    return mix((np.arange(n, dtype=np.uint64) + key) & 0xFFFFFFFF)


def constants(lr, betas, eps, step):
    b1, b2 = betas
    return dict(lr=F(lr), b1=F(b1), omb1=F(1.0 - b1), b2=F(b2), omb2=F(1.0 - b2), eps=F(eps),
                inv_bc1=F(1.0 / (1.0 - b1 ** step)), inv_sqrt_bc2=F(1.0 / np.sqrt(1.0 - b2 ** step)))


def moments32(p, g, m, v, c, scale, lr_mult, wd):
    """(p', m', v', sqrt(v')) in float32."""
    with np.errstate(all="ignore"):
        lr = c["lr"] * F(lr_mult)
        decay, size = F(1) - lr * F(wd), lr * c["inv_bc1"]
        g = g.astype(np.float32) * F(scale)
        m = m * c["b1"] + g * c["omb1"]
        v = v * c["b2"] + (g * g) * c["omb2"]
        u = np.sqrt(v)
        upd = m / (u * c["inv_sqrt_bc2"] + c["eps"])
        return p * decay - upd * size, m, v, u


def encode8(x, rnd20, floor):
    """E4M3 codes and scales of x in blocks of 256, rounded by the 20 bits given."""
    n = x.size
    pad = -n % BLOCK
    b = np.concatenate([x, np.zeros(pad, np.float32)]).reshape(-1, BLOCK)
    r = np.concatenate([rnd20, np.zeros(pad, np.uint64)]).reshape(-1, BLOCK).astype(np.uint32)
    amax = np.abs(b).max(1)
    live = amax >= F(2.0 ** -96)
    with np.errstate(all="ignore"):
        scale = np.where(live, amax / F(448), F(0)).astype(np.float32)
        inv = np.where(live, F(448) / amax, F(0)).astype(np.float32)
        y = np.abs(b) * inv[:, None]
    small = y < F(2.0 ** -6)
    t = np.where(small, y + F(2.0 ** -6), y).astype(np.float32)
    code = ((t.view(np.uint32) + r) >> 20) - np.where(small, 968, 960).astype(np.uint32)
    code = np.minimum(code, 126)
    if floor:
        code = np.where((code == 0) & (b > 0) & live[:, None], 1, code)
    code = code | np.where(np.signbit(b), 128, 0)
    return code.reshape(-1)[:n].astype(np.uint8), scale


def decode8(code, scale):
    return E4M3[code].astype(np.float32) * np.repeat(scale, BLOCK)[:code.size]


def step32(p, g, m, v, c, scale=1.0, lr_mult=1.0, wd=0.0):
    p, m, v, _ = moments32(p, g, m, v, c, scale, lr_mult, wd)
    return p, m, v


def step8(p, g, m, v, ms, vs, c, tensor, seed, scale=1.0, lr_mult=1.0, wd=0.0):
    """(p', m codes, v codes, m scales, v scales)."""
    u = decode8(v, vs)
    p, m, _, u = moments32(p, g, decode8(m, ms), u * u, c, scale, lr_mult, wd)
    r = random_bits(p.size, tensor, seed)
    mc, ms = encode8(m, r & 0xFFFFF, False)
    vc, vs = encode8(u, r >> np.uint64(12), True)
    return p, mc, vc, ms, vs


def step64(p, g, m, v, lr, betas, eps, step, scale=1.0, lr_mult=1.0, wd=0.0):
    """The formula in float64."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    b1, b2 = betas
    g = g * scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    lr = lr * lr_mult
    upd = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - lr * upd, m, v
