"""The 4-bit KV cache in numpy: packing and unpacking, head norms and rotary
positions, attention; written from the formulas in include/qk.h."""
import numpy as np


def unpack(q4, dm):
    """(q, d, m) of packed rows, the last two per group: uint8 [..., D / 2], fp16 [..., D / 32, 2]."""
    q = np.stack([q4 & 15, q4 >> 4], -1).reshape(*q4.shape[:-1], -1)
    return q, dm[..., 0].astype(np.float64), dm[..., 1].astype(np.float64)


def values(q4, dm):
    """fp16(d q + m): exact in 64 bits, then one rounding."""
    q, d, m = unpack(q4, dm)
    with np.errstate(over="ignore", invalid="ignore"):
        return (q * np.repeat(d, 32, -1) + np.repeat(m, 32, -1)).astype(np.float16)


def exact(q4, dm):
    """d q + m in 64 bits."""
    q, d, m = unpack(q4, dm)
    with np.errstate(invalid="ignore"):
        return q * np.repeat(d, 32, -1) + np.repeat(m, 32, -1)


def pack(x):
    """Packed rows of fp32 values [..., D], in fp32 as the library defines them."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    m = b.min(-1).astype(np.float16)
    m32 = m.astype(np.float32)
    d = (np.maximum(b.max(-1) - m32, np.float32(0)) / np.float32(15)).astype(np.float16)
    d32 = d.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d32 > 0, np.clip(np.rint((b - m32[..., None]) / d32), 0, 15), 0).astype(np.uint8)
    q = q.reshape(*x.shape)
    return (q[..., 0::2] | (q[..., 1::2] << 4)), np.stack([d, m], -1)


def random_cache(rng, Hkv, L, D=128):
    q4 = rng.integers(0, 256, (Hkv, L, D // 2), dtype=np.uint8)
    d = 0.2 + 0.15 * rng.random((Hkv, L, D // 32))
    m = -7.5 * d + 0.3 * rng.standard_normal(d.shape)
    return q4, np.stack([d, m], -1).astype(np.float16)


def head_norm(x, gamma, eps):
    x = x.astype(np.float64)
    if gamma is None:
        return x
    return x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * gamma.astype(np.float64)


def rotate(x, angle, n_rot, half, mag):
    """64-bit rotation of x [M][heads][D] by angle [M][n_rot / 2]."""
    y = x.copy()
    a = y[..., : n_rot // 2].copy() if half else y[..., 0:n_rot:2].copy()
    b = y[..., n_rot // 2: n_rot].copy() if half else y[..., 1:n_rot:2].copy()
    c, s = mag * np.cos(angle)[:, None], mag * np.sin(angle)[:, None]
    ra, rb = a * c - b * s, b * c + a * s
    if half:
        y[..., : n_rot // 2], y[..., n_rot // 2: n_rot] = ra, rb
    else:
        y[..., 0:n_rot:2], y[..., 1:n_rot:2] = ra, rb
    return y


def seen(p, window, sinks):
    j = np.arange(p + 1)
    return j[(j > p - window) | (j < sinks)]


def attention(q, k, v, H, Hkv, pos0, window, sinks, scale, rows=None):
    """64-bit attention of fp16 q [M][H][128] over rows k, v [Hkv][L][128]."""
    rows = np.arange(q.shape[0]) if rows is None else rows
    out = np.zeros((len(rows), H, q.shape[2]))
    G = H // Hkv
    for n, i in enumerate(rows):
        j = seen(pos0 + i, window, sinks)
        if not len(j):
            continue
        for g in range(Hkv):
            z = q[i, g * G:(g + 1) * G].astype(np.float64) @ k[g, j].astype(np.float64).T * scale
            e = np.exp(z - z.max(1, keepdims=True))
            out[n, g * G:(g + 1) * G] = e / e.sum(1, keepdims=True) @ v[g, j].astype(np.float64)
    return out
