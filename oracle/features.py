"""fp64 oracle of the feature operators (norm, dropout, 8-bit rows, scoring,
softmax loss) in plain numpy, from their definitions.  Test infrastructure
only; it shares no code with the HIP path."""

from __future__ import annotations

import numpy as np


def philox4x32(ctr, key, rounds=10):
    """The four output words (uint64 arrays below 2^32) of Philox 4x32 at four counter words and two key words."""
    c = [np.asarray(x, dtype=np.uint64) for x in ctr]
    k0, k1 = int(key[0]), int(key[1])
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & low, (a >> sh) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) % 2**32, (k1 + 0xBB67AE85) % 2**32
    return c


def drop_factor(rows, cols, p, seed, offset):
    """rows x cols: 0 where an element is dropped, the kept elements' factor elsewhere."""
    thr = int(np.rint(p * 65536))
    if thr == 0:
        return np.ones((rows, cols))
    if thr == 65536:
        return np.zeros((rows, cols))
    per = -(-cols // 8)
    i = np.arange(rows * per, dtype=np.uint64)
    o = offset % 2**64
    w = philox4x32([i % np.uint64(2**32), i >> np.uint64(32), np.full_like(i, o % 2**32), np.full_like(i, o >> 32)],
                   [seed % 2**32, (seed >> 32) % 2**32])
    half = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], 1)
    f = np.where(half >= thr, 65536.0 / (65536 - thr), 0.0)
    return f.reshape(rows, 8 * per)[:, :cols]


def _masked(x, f):
    return np.where(f > 0, x * np.where(f > 0, f, 1.0), 0.0) if np.isfinite(x).all() else \
        np.where(f > 0, np.where(f > 0, x, 0.0) * f, 0.0)


def oracle_dropout(x, p, seed, offset, residual=None):
    y = _masked(np.asarray(x, np.float64), drop_factor(*x.shape, p, seed, offset))
    return y if residual is None else y + np.asarray(residual, np.float64)


def oracle_add_norm(x, gamma, residual, eps, p, seed, offset):
    v = oracle_dropout(x, p, seed, offset, residual)
    rstd = 1.0 / np.sqrt((v * v).mean(1) + eps)
    return {"sum": v, "rstd": rstd, "y": v * rstd[:, None] * gamma}


def oracle_add_norm_bwd(dy, v, gamma, rstd, dsum, p, seed, offset):
    xh, g = v * rstd[:, None], dy * gamma
    ds = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    if dsum is not None:
        ds = ds + dsum
    return {"dres": ds, "dx": _masked(ds, drop_factor(*dy.shape, p, seed, offset)), "dgamma": (dy * xh).sum(0)}


def oracle_score(hq, hs, Wq, ws):
    return (hq @ Wq.T) * hs[:, None] * ws


def oracle_softmax(h, W, rowptr, col, scale):
    """row_loss, lse, loss, dW, dh and D = softmax - target (B x L) in fp64."""
    B, L = h.shape[0], W.shape[0]
    D, row_loss, lse, dh = np.zeros((B, L)), np.zeros(B), np.zeros(B), np.zeros(h.shape)
    live = [b for b in range(B) if rowptr[b + 1] > rowptr[b]]
    for b in live:
        z = W @ h[b]
        y = np.unique(col[rowptr[b]:rowptr[b + 1]])
        top = z.max()
        lse[b] = top + np.log(np.exp(z - top).sum())
        row_loss[b] = lse[b] - z[y].mean()
        D[b] = np.exp(z - lse[b])
        D[b, y] -= 1.0 / y.size
    hl = h[live] if live else np.zeros((0, h.shape[1]))
    dW = scale * (D[live].T @ hl)
    if live:
        dh[live] = scale * (D[live] @ W)
    return {"row_loss": row_loss, "lse": lse, "loss": scale * row_loss.sum(), "dW": dW, "dh": dh, "D": D}
