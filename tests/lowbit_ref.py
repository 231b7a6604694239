"""Plain references of the low-bit training operators (numpy, no torch, no libzs)."""
from __future__ import annotations

import numpy as np

BLOCK, GROUP = 256, 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def philox(c, key, rounds):
    """Philox4x32 (Salmon et al. 2011) on uint32 counter words c[0..3]."""
    c = [np.asarray(x, dtype=np.uint64) for x in c]
    k0, k1 = int(key) & 0xFFFFFFFF, int(key) >> 32
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return [x.astype(np.uint32) for x in c]


def random16(numel, tensor, step, seed):
    """(for exp_avg, for the root of exp_avg_sq): 16 bits an element."""
    q = np.arange(-(-numel // 4), dtype=np.uint64)
    one = np.ones_like(q)
    w = np.stack(philox([q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), one * np.uint64(tensor),
                         one * np.uint64(step & 0xFFFFFFFF)], seed, 7), 1).ravel()[:numel]
    return w & 0xFFFF, w >> 16


def e4m3_values():
    """The 256 codes' values (0x7F and 0xFF: NaN)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-x if c & 0x80 else x)
    return v


E4M3 = e4m3_values()


def spacing(y):
    """Distance of neighbouring e4m3 values at |y|."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return 2.0 ** (e - 3)


def adam64(p, m, v, g, hp, step, coef):
    """The update in 64 bits, on the hyper-parameters that the library works with (float32)."""
    f = lambda x: float(np.float32(x))  # noqa: E731
    lr, b1, b2, eps, wd = (f(hp[k]) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    bc1, bc2 = (1 - b1 ** step, 1 - b2 ** step) if hp.get("bias_correction", 1) else (1.0, 1.0)
    p, m, v, g = (np.asarray(x, dtype=np.float64) for x in (p, m, v, g))
    g = g * coef
    if hp.get("adamw", 1):
        p = p - lr * wd * p
    else:
        g = g + wd * p
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return p - lr * (m / bc1) / (np.sqrt(v / bc2) + eps), m, v


def blocks(x):
    """x as rows of BLOCK, zero past its end."""
    return np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK)


def state_scales(x):
    """2^(floor(log2 max) - 7) a block of the finite values, at least 2^-126."""
    top = np.where(np.isfinite(blocks(x)), np.abs(blocks(x)), 0).max(1)
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.floor(np.log2(np.maximum(top, 1e-320))), -np.inf)
    return 2.0 ** (np.maximum(e, -119.0) - 7)


def mx4(x):
    """(codes [R, Kp], scale bytes [R, Kp / 32]) of a float matrix along its rows, in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    r, k = x.shape
    x = np.pad(x, ((0, 0), (0, -k % GROUP))).reshape(r, -1, GROUP)
    bad = ~np.isfinite(x).all(2)
    top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(x), x, 0)).max(2))
    _, e = np.frexp(top)
    normal = top >= 2.0 ** -126
    byte = np.where(bad, 255, np.where(normal, np.maximum(e - 1 - 2 + 127, 0), 0))
    y = np.where(bad[..., None], 0.0, np.where(np.isfinite(x), x, 0.0) * 2.0 ** (127.0 - byte[..., None]))
    a = np.abs(y)
    grid = E2M1[:8]
    low = np.clip(np.searchsorted(grid, a, side="right") - 1, 0, 7)
    high = np.minimum(low + 1, 7)
    d0, d1 = a - grid[low], grid[high] - a
    code = np.where((d1 < d0) | ((d1 == d0) & (high % 2 == 0)), high, low)
    code = code + 8 * np.signbit(y)
    return code.reshape(r, -1).astype(np.uint8), byte.astype(np.uint8)


def mx4_values(code, byte):
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return (E2M1[code].reshape(*byte.shape, GROUP) * s[..., None]).reshape(code.shape)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(b):
    return np.stack([b & 15, b >> 4], 2).reshape(b.shape[0], -1)


def tile_scales(byte):
    """Scale bytes [R, G] in the library's order."""
    r, g = byte.shape
    out = np.zeros((-(-r // 128), 2 * -(-g // 8), 512), dtype=np.uint8)
    rows, groups = np.meshgrid(np.arange(r), np.arange(g), indexing="ij")
    out[rows // 128, groups // 4, rows % 32 * 16 + rows % 128 // 32 * 4 + groups % 4] = byte
    return out.ravel()
