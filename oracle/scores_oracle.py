"""fp64 CPU oracle of the token scores and of the embedding with dropout.

TEST INFRASTRUCTURE ONLY, like :mod:`oracle.vpce_oracle`: plain numpy restated
from the definitions, sharing no code with the CUDA library.

Token scores of a row of logits z at temperature T: x = z / T,
logp_k = x_k - logsumexp(x); the entropy is -sum p logp over columns with
p > 0; the alternatives are the columns sorted by (logit descending, NaN
first, column ascending).  Their gradient is written as the Jacobians of the
three outputs applied to the upstream gradients, column by column.

Dropout bits: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random
numbers: as easy as 1, 2, 3", SC 2011), whose published known-answer vectors
pin :func:`philox4x32_10`.
"""
from __future__ import annotations

import numpy as np

__all__ = ["token_scores", "token_scores_backward", "philox4x32_10", "keep_mask", "drop_threshold",
           "embedding_dropout_forward", "embedding_dropout_backward"]


def token_scores(z, y, top: int = 0, temperature: float = 1.0, ignore_index: int = -100):
    """``z`` [s, V] fp64, ``y`` [s] or None -> dict of logp, entropy, top_ids,
    top_logp, stats [s, 4] (largest z, ln sum exp((z - largest) / T), entropy,
    0) and bad (a target outside [0, V))."""
    z = np.asarray(z, dtype=np.float64)
    s, V = z.shape
    out = dict(logp=np.zeros(s), entropy=np.zeros(s), stats=np.zeros((s, 4)),
               top_ids=np.full((s, top), -1, dtype=np.int64), top_logp=np.zeros((s, top)), bad=False)
    for r in range(s):
        if y is not None and y[r] == ignore_index:
            continue
        m = np.nan if np.isnan(z[r]).any() else z[r].max()
        order = np.lexsort((np.arange(V), -np.where(np.isnan(z[r]), 0.0, z[r]), ~np.isnan(z[r])))[:top]
        out["top_ids"][r] = order
        if np.isfinite(m):
            u = (z[r] - m) / temperature
            log_s = np.log(np.exp(u).sum())
            lp = u - log_s
            some = np.exp(lp) > 0
            ent = -(np.exp(lp[some]) * lp[some]).sum()
        else:
            log_s = ent = np.nan
            lp = np.full(V, np.nan)
        out["entropy"][r] = ent
        out["stats"][r] = (m, log_s, ent, 0.0)
        out["top_logp"][r] = lp[order]
        if y is not None:
            if 0 <= y[r] < V:
                out["logp"][r] = lp[y[r]]
            else:
                out["logp"][r] = np.nan
                out["bad"] = True
    return out


def token_scores_backward(z, y, g_logp=None, g_entropy=None, top_ids=None, g_top=None, temperature: float = 1.0,
                          ignore_index: int = -100):
    """d(sum g_logp logp + g_entropy entropy + g_top top_logp) / dz, [s, V]."""
    z = np.asarray(z, dtype=np.float64)
    s, V = z.shape
    d = np.zeros((s, V))
    for r in range(s):
        if y is not None and y[r] == ignore_index:
            continue
        bad = g_logp is not None and not 0 <= y[r] < V
        if bad or np.isnan(z[r]).any() or not np.isfinite(z[r].max()):
            d[r] = np.nan
            continue
        u = (z[r] - z[r].max()) / temperature
        p = np.exp(u) / np.exp(u).sum()
        lp = u - np.log(np.exp(u).sum())
        if g_logp is not None:            # d logp_y / dx = onehot(y) - p
            d[r] -= g_logp[r] * p
            d[r, y[r]] += g_logp[r]
        if g_entropy is not None:         # d H / dx_k = -p_k (ln p_k + H)
            some = p > 0
            ent = -(p[some] * lp[some]).sum()
            d[r, some] -= g_entropy[r] * p[some] * (lp[some] + ent)
        if g_top is not None:
            for c, g in zip(top_ids[r], g_top[r]):
                if 0 <= c < V:
                    d[r] -= g * p
                    d[r, c] += g
        d[r] /= temperature
    return d


def philox4x32_10(counter, key):
    """Ten rounds on uint32 arrays: ``counter`` of 4 and ``key`` of 2."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [np.asarray(v, dtype=np.uint64) for v in key]
    low = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ k[0], b & low, (a >> sh) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def drop_threshold(p: float) -> int:
    return min(65535, int(np.floor(float(np.float32(p)) * 65536 + 0.5)))


def keep_mask(seed: int, offset: int, s: int, h: int, p: float):
    """Boolean [s, h]: the elements dropout keeps."""
    nb = (h + 7) // 8
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    cols, rows = np.meshgrid(np.arange(nb), np.arange(s))
    words = philox4x32_10((cols, rows, np.full_like(cols, offset & 0xFFFFFFFF), np.full_like(cols, offset >> 32)),
                          (seed & 0xFFFFFFFF, seed >> 32))
    halves = [w >> np.uint64(16 * i) & np.uint64(0xFFFF) for w in words for i in (0, 1)]
    return np.stack(halves, axis=2).reshape(s, nb * 8)[:, :h] >= drop_threshold(p)


def _factor(s, h, scale, p, seed, offset):
    drop = drop_threshold(p)
    if drop == 0:
        return np.full((s, h), float(scale))
    return np.where(keep_mask(seed, offset, s, h, p), scale * 65536.0 / (65536 - drop), 0.0)


def embedding_dropout_forward(table, ids, scale=1.0, p=0.0, seed=0, offset=0, padding_id=None):
    """``table`` [V, h] fp64 -> (out [s, h] fp64, bad)."""
    ids = np.asarray(ids, dtype=np.int64)
    V, h = table.shape
    f = _factor(ids.size, h, scale, p, seed, offset)
    out = np.zeros((ids.size, h))
    inside = (ids >= 0) & (ids < V)
    pad = np.zeros(ids.size, dtype=bool) if padding_id is None else ids == padding_id
    live = inside & ~pad
    out[live] = np.where(f[live] != 0, table[ids[live]] * f[live], 0.0)
    return out, bool(np.any(~inside & ~pad))


def embedding_dropout_backward(grad, ids, V, scale=1.0, p=0.0, seed=0, offset=0, padding_id=None):
    """``grad`` [s, h] fp64 -> (table gradient [V, h], sum of the terms'
    magnitudes [V, h], rows per id [V])."""
    ids = np.asarray(ids, dtype=np.int64)
    s, h = grad.shape
    f = _factor(s, h, scale, p, seed, offset)
    live = (ids >= 0) & (ids < V)
    if padding_id is not None:
        live &= ids != padding_id
    terms = np.where(f[live] != 0, grad[live] * f[live], 0.0)
    d, mag = np.zeros((V, h)), np.zeros((V, h))
    np.add.at(d, ids[live], terms)
    np.add.at(mag, ids[live], np.abs(terms))
    return d, mag, np.bincount(ids[live], minlength=V)
