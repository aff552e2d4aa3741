"""Plain float64 forms of the map operators, for the tests.

Arrays are [B, C, P] (P pixels) in float64; nothing here uses the package.
"""
import numpy as np

PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)


def philox4x32(counter, key, rounds=10):
    """Four words from counter words c0..c3 (arrays of unsigned numbers) and a key of two numbers."""
    u = np.uint64
    c = [np.asarray(w, dtype=u) for w in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        p0, p1 = c[0] * u(PHILOX_M[0]), c[2] * u(PHILOX_M[1])
        c = [(p1 >> u(32)) ^ c[1] ^ u(k0), p1 & u(0xFFFFFFFF), (p0 >> u(32)) ^ c[3] ^ u(k1), p0 & u(0xFFFFFFFF)]
        k0, k1 = (k0 + PHILOX_W[0]) & 0xFFFFFFFF, (k1 + PHILOX_W[1]) & 0xFFFFFFFF
    return c


def keep_mask(B, C, P, p, mode, seed, offset):
    """Truth values [B, C, P]: what stays."""
    n = {"element": B * P, "channel": B, "sample": B}[mode]
    quads = 1 if mode == "sample" else -(-C // 4)
    row = np.arange(n, dtype=np.uint64)[:, None] + np.zeros((1, quads), np.uint64)
    quad = np.arange(quads, dtype=np.uint64)[None, :] + np.zeros((n, 1), np.uint64)
    words = philox4x32((quad, row & np.uint64(0xFFFFFFFF), row >> np.uint64(32),
                        np.full_like(row, offset & 0xFFFFFFFF)), (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    u = np.stack(words, axis=-1).reshape(n, 4 * quads)
    keep = u >= np.uint64(int(np.floor(p * 2.0 ** 32)))
    if mode == "sample":
        return np.broadcast_to(keep[:, :1, None], (B, C, P))
    if mode == "channel":
        return np.broadcast_to(keep[:, :C, None], (B, C, P))
    return keep[:, :C].reshape(B, P, C).transpose(0, 2, 1)


def grown(p):
    """The factor of what stays, a float32 number."""
    return float(np.float32(1.0 / (1.0 - p)))


def join(x, residual, keep, p):
    v = x if keep is None else np.where(keep, x * grown(p), 0.0)
    return v if residual is None else residual + v


def norm(h, w, eps):
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h * r * w[None, :, None], r


def norm_grad(h, w, eps, dy, dh):
    """d (the gradient of h) and dweight."""
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    g = dy * w[None, :, None]
    d = r * (g - h * r * r * (g * h).mean(axis=1, keepdims=True))
    return (d if dh is None else d + dh), (dy * h * r).sum(axis=(0, 2))


def group_max(v, group):
    """max |v| of each group of channels: [B, groups, P]."""
    return np.concatenate([np.abs(v[:, k:k + group]).max(axis=1, keepdims=True)
                           for k in range(0, v.shape[1], group)], axis=1)
