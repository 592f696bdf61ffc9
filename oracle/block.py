"""The operators around the expert layer (oracle; test infrastructure only):
dropout from a counter-based generator and the root-mean-square norm of a
residual stream with its gradient, and low-rank adapters with theirs.

Plain definitions in float64, as include/moe_block.h states them. The generator
is exact integer arithmetic, pinned by its authors' known answers; the gradient
by central differences of the forward function (tests/test_oracle_block.py).
"""

import numpy as np

from .quant import mx_quantize_e4m3

_LOW = 0xFFFFFFFF


def philox4x32(counter, key, rounds=10):
    """Philox 4x32 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
    3", 2011): counter int [..., 4] and key [2] of 32-bit words -> uint64 words
    [..., 4]."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    low, half = np.uint64(_LOW), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k0), b & low, (a >> half) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return np.stack(c, axis=-1)


def dropout_threshold(p):
    """round(p * 65536) of p as a float, ties to even."""
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def dropout_keep(rows, n, p, seed, offset):
    """The kept elements [rows, n] (n a multiple of 8); seed and offset as
    unsigned 64-bit numbers."""
    i = np.arange(rows * n // 8, dtype=np.uint64)
    counter = np.stack([i & np.uint64(_LOW), i >> np.uint64(32), np.full_like(i, offset & _LOW),
                        np.full_like(i, offset >> 32)], axis=-1)
    w = philox4x32(counter, (seed & _LOW, seed >> 32))
    halves = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=-1)
    return halves.reshape(rows, n) >= np.uint64(dropout_threshold(p))


def dropout(x, p, seed=0, offset=0):
    x = np.asarray(x, dtype=np.float64)
    t = dropout_threshold(p)
    if t == 0:
        return x
    keep = dropout_keep(*x.shape, p, seed, offset)
    return np.where(keep, x * (65536 / (65536 - t) if t < 65536 else 0.0), 0.0)


def rmsnorm(v, weight, eps):
    v = np.asarray(v, dtype=np.float64)
    return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def quantize_per_token(u):
    """(E4M3 values as float64, scale per row): the nearest E4M3 number to u /
    scale, ties to even."""
    u = np.asarray(u, dtype=np.float64)
    s = np.maximum(np.abs(u).max(axis=1) / 448, 2.0 ** -126)
    r = u / s[:, None]
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -6))) - 3)
    return np.clip(np.rint(r / step) * step, -448, 448), s


def quantize_mxfp8(u):
    """(codes, scale bytes) of the MXFP8 rule."""
    return mx_quantize_e4m3(np.asarray(u, dtype=np.float64))


def rmsnorm_backward(dy, v, weight, eps, dsum=None):
    """(gradient of v, of the weight) for the gradient dy of rmsnorm(v) and dsum of v itself."""
    dy, v, w = (np.asarray(t, dtype=np.float64) for t in (dy, v, weight))
    s = 1 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    g = dy * w
    d = s * (g - v * s * s * (g * v).mean(axis=1, keepdims=True))
    return d if dsum is None else d + np.asarray(dsum, dtype=np.float64), (dy * v * s).sum(axis=0)


def lora(c, x, a, b, ids, scale=None, row_div=1):
    """(C with the adapters' products added, h): ids [S] the slots' groups;
    slots outside [0, G) keep their rows, their h is 0."""
    c, x, a, b = (np.asarray(t, dtype=np.float64) for t in (c, x, a, b))
    out, h = c.copy(), np.zeros((len(ids), a.shape[1]))
    for s, g in enumerate(ids):
        if 0 <= g < a.shape[0]:
            h[s] = a[g] @ x[s // row_div]
            out[s] += (1.0 if scale is None else float(scale[g])) * (b[g] @ h[s])
    return out, h


def lora_backward(dy, x, a, b, ids, h, scale=None, row_div=1):
    """(the adapters' part of dx by slot, da, db)."""
    dy, x, a, b, h = (np.asarray(t, dtype=np.float64) for t in (dy, x, a, b, h))
    dx, da, db = np.zeros((len(ids), x.shape[1])), np.zeros(a.shape), np.zeros(b.shape)
    for s, g in enumerate(ids):
        if 0 <= g < a.shape[0]:
            w = 1.0 if scale is None else float(scale[g])
            dh = w * (b[g].T @ dy[s])
            dx[s] = a[g].T @ dh
            da[g] += np.outer(dh, x[s // row_div])
            db[g] += w * np.outer(dy[s], h[s])
    return dx, da, db
