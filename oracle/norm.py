"""Dropout and the row norms between message layers (oracle, float64; test
infrastructure).

Dropout by Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
numbers: as easy as 1, 2, 3", SC 2011): unit u = column // group of row r has
the 16-bit draw (u % 8) of the block with counter (u // 8, r, offset low,
offset high) and key seed; it is kept where the draw is at least
t = floor(65536 p + 1/2) and then multiplied by 65536 / (65536 - t).

The norm of features [N, C, (l_max+1)^2], each degree by itself:
  s = residual + factor * x
  l = 0:  mu = mean_c s,  q_0 = (mean_c (s - mu)^2 + eps)^-1/2,  h = (s - mu) q_0
  l > 0:  q_l = (mean_{c,m} s^2 + eps)^-1/2,                     h = s q_l
  y = h w[l,c]  (+ b[c] for l = 0)
With l_max = 0 it is the layer norm of rows of C values.  Pinned by the
generator's published vectors, finite differences, rotations and
loops over single rows (tests/test_oracle_norm.py).
"""
import numpy as np

_MASK = np.uint64(0xFFFFFFFF)
_HALF = np.uint64(32)


def philox(counter, key):
    """Four words (uint64 arrays below 2^32) of Philox4x32-10 of counter (4 arrays) and key (2 integers)."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        lo = c[0] * np.uint64(0xD2511F53)
        hi = c[2] * np.uint64(0xCD9E8D57)
        c = [(hi >> _HALF) ^ c[1] ^ np.uint64(k[0]), hi & _MASK, (lo >> _HALF) ^ c[3] ^ np.uint64(k[1]), lo & _MASK]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_factor(rows, cols, p, seed, offset=0, group=1, first_row=0):
    """[rows, cols] factors of the dropout: 0 or 65536 / (65536 - t)."""
    t = int(np.floor(65536.0 * p + 0.5))
    if p == 0.0 or t == 0:
        return np.ones((rows, cols))
    units = cols // group
    u, r = np.meshgrid(np.arange(units, dtype=np.uint64), np.arange(first_row, first_row + rows, dtype=np.uint64))
    off = np.full_like(u, offset)
    words = np.stack(philox((u // np.uint64(8), r, off & _MASK, off >> _HALF), (seed & 0xFFFFFFFF, seed >> 32)))
    word = np.take_along_axis(words, ((u % np.uint64(8)) // np.uint64(2)).astype(np.int64)[None], 0)[0]
    draw = (word >> (np.uint64(16) * (u % np.uint64(2)))) & np.uint64(0xFFFF)
    scale = 65536.0 / (65536 - t) if t < 65536 else 0.0
    return np.repeat(np.where(draw >= np.uint64(t), scale, 0.0), group, axis=1)


def apply_drop(x, factor):
    """factor * x, where a factor of 0 gives 0 for any x."""
    return np.where(factor == 0.0, 0.0, np.where(factor == 0.0, 0.0, x) * factor)


def degrees(l_max):
    return np.concatenate([np.full(2 * l + 1, l) for l in range(l_max + 1)])


def _blocks(l_max):
    return [slice(l * l, (l + 1) ** 2) for l in range(l_max + 1)]


def forward(x, w=None, b=None, eps=1e-5, residual=None, factor=None):
    """x [N, C, K] (or rows [N, C]) -> dict(s, y, stats), in float64."""
    rows = x.ndim == 2
    x = np.asarray(x, np.float64)
    s = x if factor is None else apply_drop(x, factor.reshape(x.shape))
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    v = s[:, :, None] if rows else s
    N, C, K = v.shape
    l_max = int(round(np.sqrt(K))) - 1
    mu = v[:, :, 0].mean(axis=1)
    d = v.copy()
    d[:, :, 0] -= mu[:, None]
    q = np.stack([1.0 / np.sqrt((d[:, :, k] ** 2).mean(axis=(1, 2)) + eps) for k in _blocks(l_max)], axis=1)
    y = d * q[:, degrees(l_max)][:, None, :]
    if w is not None:
        y = y * np.asarray(w, np.float64).reshape(l_max + 1, C)[degrees(l_max)].T
    if b is not None:
        y[:, :, 0] += np.asarray(b, np.float64)
    return dict(s=s, y=y[:, :, 0] if rows else y, stats=np.concatenate([mu[:, None], q], axis=1))


def backward(g, s, stats, w=None, grad_s=None, factor=None):
    """Gradients dict(r, x, w, b) of the norm at the sum s with the statistics given, in float64."""
    rows = s.ndim == 2
    cube = (lambda a: np.asarray(a, np.float64)[:, :, None]) if rows else (lambda a: np.asarray(a, np.float64))
    g3, s3, stats = cube(g), cube(s), np.asarray(stats, np.float64)
    N, C, K = s3.shape
    l_max = int(round(np.sqrt(K))) - 1
    deg = degrees(l_max)
    d = s3.copy()
    d[:, :, 0] -= stats[:, :1]
    q = stats[:, 1:]
    h = d * q[:, deg][:, None, :]
    a = g3 if w is None else g3 * np.asarray(w, np.float64).reshape(l_max + 1, C)[deg].T
    r = np.empty_like(a)
    for l, k in enumerate(_blocks(l_max)):
        m = (a[:, :, k] * h[:, :, k]).mean(axis=(1, 2))[:, None, None]
        r[:, :, k] = a[:, :, k] - h[:, :, k] * m
    r[:, :, 0] -= a[:, :, 0].mean(axis=1)[:, None]
    r *= q[:, deg][:, None, :]
    if grad_s is not None:
        r = r + cube(grad_s)
    gh = (g3 * h).sum(axis=0)
    dw = np.stack([gh[:, k].sum(axis=1) for k in _blocks(l_max)])
    x = r if factor is None else apply_drop(r, factor.reshape(r.shape))
    flat = (lambda t: t[:, :, 0]) if rows else (lambda t: t)
    return dict(r=flat(r), x=flat(x), w=dw[0] if rows else dw, b=g3[:, :, 0].sum(axis=0))
