"""fp64 definitions of the root-mean-square norm with residual (its output as
it is or in e4m3 with scales, and its gradient), the gradient norm and the
AdamW step with states in 32 bits or in 8.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

from oracle.scores_oracle import philox4x32_10

TINY = 2.0 ** -126
BLOCK = 256


def e4m3_grid():
    """The 127 finite non-negative values in the order of their codes."""
    low = [k * 2.0 ** -9 for k in range(8)]
    return np.array((low + [(8 + k) * 2.0 ** (e - 10) for e in range(1, 16) for k in range(8)])[:127])


def rmsnorm(x, weight, residual=None, eps=1e-6):
    """(out, sum, rstd) of fp64 rows."""
    r = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((r * r).mean(axis=1) + eps)
    return r * rstd[:, None] * weight, r, rstd


def group_scales(out, group=0):
    """Scale of each group of columns [s, groups], and of each element."""
    s, h = out.shape
    g = group or h
    edges = list(range(0, h, g))
    scale = np.maximum(np.maximum.reduceat(np.abs(out), edges, axis=1) / 448.0, TINY)
    return scale, np.repeat(scale, g, axis=1)[:, :h]


def nearest_e4m3(a):
    """Nearest finite e4m3 value of |a| <= 448 (ties: either), and the distance
    of |a| to the nearest midpoint between two values."""
    grid = e4m3_grid()
    mids = (grid[1:] + grid[:-1]) / 2
    at = np.searchsorted(mids, np.abs(a))
    near = np.minimum(np.abs(np.abs(a) - mids[np.minimum(at, 125)]), np.abs(np.abs(a) - mids[np.maximum(at - 1, 0)]))
    return np.copysign(grid[at], a), near


def rmsnorm_backward(dy, r, weight, rstd, dres=None):
    """(dr, dweight) and the sums of their terms' magnitudes."""
    n = r * rstd[:, None]
    wdy = dy * weight
    dot, mag = (wdy * n).mean(axis=1), np.abs(wdy * n).mean(axis=1)
    dr = rstd[:, None] * (wdy - n * dot[:, None])
    dr_mag = rstd[:, None] * (np.abs(wdy) + np.abs(n) * mag[:, None])
    if dres is not None:
        dr, dr_mag = dr + dres, dr_mag + np.abs(dres)
    return dr, (dy * n).sum(axis=0), dr_mag, np.abs(dy * n).sum(axis=0)


def grad_norm(grads, max_norm=np.inf):
    with np.errstate(all="ignore"):
        norm = float(np.sqrt(sum((np.asarray(g, np.float64) ** 2).sum() for g in grads)))
    if not np.isfinite(norm):
        return norm, 0.0
    return norm, 1.0 if norm <= max_norm else max_norm / norm


def adamw(p, g, m, v, step, lr, b1, b2, eps, wd, scale=1.0):
    """(p, m, v) after the step."""
    g = g * scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    u = m / (1 - b1 ** step) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - lr * u, m, v


def random_halves(n, tensor, seed, offset):
    """The 16 random bits of elements 0 .. n of the tensor at a position."""
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    k = np.arange((n + 7) // 8)
    words = philox4x32_10((k & 0xFFFFFFFF, np.full_like(k, tensor), np.full_like(k, offset & 0xFFFFFFFF),
                           np.full_like(k, offset >> 32)), (seed & 0xFFFFFFFF, seed >> 32))
    halves = [w >> np.uint64(16 * i) & np.uint64(0xFFFF) for w in words for i in (0, 1)]
    return np.stack(halves, axis=1).reshape(-1)[:n].astype(np.int64)


def block_scales(x):
    """Scale of each block of 256 elements, and of each element."""
    edges = list(range(0, x.size, BLOCK))
    scale = np.maximum(np.maximum.reduceat(np.abs(x), edges) / 448.0, TINY)
    return scale, np.repeat(scale, BLOCK)[:x.size]


def stochastic_codes(x, scale, u, squares):
    """Values of the e4m3 codes that ``x`` (>= 0 with ``squares``) takes under
    its elements' scales, and how far, in units of 2^-16, each random number
    was from the border between the two codes (around the circle)."""
    grid = np.append(e4m3_grid(), 480.0)
    a = np.minimum(np.abs(x) / scale, 448.0)
    at = np.searchsorted(grid[:127], a, side="right") - 1
    lo, hi = grid[at], grid[at + 1]
    part = (a * a - lo * lo) / (hi * hi - lo * lo) if squares else (a - lo) / (hi - lo)
    up = (u + 0.5) / 65536 < part
    c = np.where(up & (at < 126), hi, lo)
    if squares:
        c = np.where((x > 0) & (c == 0), grid[1], c)
    far = np.abs((u + 0.5) - part * 65536)
    return np.copysign(c, x), np.minimum(far, 65536 - far)
