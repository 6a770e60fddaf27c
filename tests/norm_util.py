"""Inputs and error bounds for the tests of the norms and of dropout.

The bounds are worst cases of the fp32 arithmetic, element by element, from
u = 2^-24 (the unit roundoff) and the number of additions behind each sum.
They hold for any order of the sums whose longest chain has at most `chain`
additions; a bf16 result adds half a unit in its last place, 2^-9 relative
(taken as 2^-8, which covers the rounding of an already rounded value).
"""
import numpy as np

from oracle import norm

U = 2.0 ** -24


def chain(n):
    """Additions on the longest path of a sum over n values of a row: a thread's own values, then a tree."""
    return 24 + -(-n // 128)


def _cube(a, K):
    a = np.asarray(a, np.float64)
    return a[:, :, None] if a.ndim == 2 else a


def _by_degree(v, l_max):
    """The mean of v [N, C, K] over each degree's values, spread over its components again."""
    out = np.empty_like(v)
    for l in range(l_max + 1):
        k = slice(l * l, (l + 1) ** 2)
        out[:, :, k] = v[:, :, k].mean(axis=(1, 2))[:, None, None]
    return out


def forward_bounds(x, w, b, eps, residual, factor, bf16):
    """Oracle's forward result and a bound on the error of each of s, y and stats."""
    want = norm.forward(x, w, b, eps, residual, factor)
    s, y = _cube(want["s"], 0), _cube(want["y"], 0)
    N, C, K = s.shape
    l_max = int(round(np.sqrt(K))) - 1
    deg, n = norm.degrees(l_max), chain(C * K)
    mu, q = want["stats"][:, 0], want["stats"][:, 1:][:, deg][:, None, :]
    ds = 2 * U * np.abs(s) + (3 * U * np.abs(norm.apply_drop(np.asarray(x, np.float64), factor.reshape(x.shape))).reshape(s.shape)
                              if factor is not None else 0.0)
    dmu = (n + 2) * U * np.abs(s[:, :, 0]).mean(1) + ds[:, :, 0].mean(1)
    d, dd = s.copy(), ds.copy()
    d[:, :, 0] -= mu[:, None]
    dd[:, :, 0] += dmu[:, None] + U * np.abs(d[:, :, 0])
    v = 1.0 / q ** 2 - eps
    dv = 2 * _by_degree(np.abs(d) * dd, l_max) + _by_degree(dd ** 2, l_max) + (n + 4) * U * np.maximum(v, 0)
    dq = 0.5 * q ** 3 * (dv + 2 * U * (v + eps)) + 4 * U * q
    ww = np.ones(K) if w is None else np.abs(np.asarray(w, np.float64).reshape(l_max + 1, C))[deg].T
    dy = (dd * q + np.abs(d) * dq + dd * dq + 3 * U * np.abs(d) * q) * ww + 2 * U * np.abs(y)
    if b is not None:
        dy[:, :, 0] += 2 * U * np.abs(np.asarray(b, np.float64))
    dstats = np.concatenate([dmu[:, None], np.stack([dq[:, :, l * l].max(axis=1) for l in range(l_max + 1)], 1)], 1)
    half = 2.0 ** -8 if bf16 else 0.0
    tiny = 1e-37
    return want, dict(s=(ds + half * np.abs(s) + tiny).reshape(want["s"].shape),
                      y=(dy + half * np.abs(y) + tiny).reshape(want["y"].shape), stats=dstats + U * np.abs(want["stats"]) + tiny)


def backward_bounds(g, s, stats, w, grad_s, factor, bf16):
    """Oracle's gradients (for the statistics given) and a bound on the error of each."""
    want = norm.backward(g, s, stats, w, grad_s, factor)
    g3, s3 = _cube(g, 0), _cube(s, 0)
    N, C, K = s3.shape
    l_max = int(round(np.sqrt(K))) - 1
    deg, n = norm.degrees(l_max), chain(C * K)
    stats = np.asarray(stats, np.float64)
    q = stats[:, 1:][:, deg][:, None, :]
    d = s3.copy()
    d[:, :, 0] -= stats[:, :1]
    h = np.abs(d * q)
    dh = 2 * U * h
    ww = np.ones(K) if w is None else np.abs(np.asarray(w, np.float64).reshape(l_max + 1, C))[deg].T
    a = np.abs(g3) * ww
    mah = _by_degree(a * h, l_max)  # the means of the absolute values bound those of the values
    dmah = (n + 4) * U * mah + _by_degree(a * dh, l_max)
    dr = q * (4 * U * a + h * dmah + dh * mah + 3 * U * h * mah)
    dr[:, :, 0] += q[:, :, 0] * (n + 4) * U * a[:, :, 0].mean(1)[:, None]
    r = np.abs(_cube(want["r"], 0))
    dr += 4 * U * r + (4 * U * np.abs(_cube(grad_s, 0)) if grad_s is not None else 0.0)
    dx = dr + 2 * U * r
    if factor is not None:
        dx = dx * factor.reshape(dx.shape) + 2 * U * np.abs(_cube(want["x"], 0))
    rows_chain = 64 + K + -(-N // 64)
    gh = (np.abs(g3) * (dh + rows_chain * U * h)).sum(0)
    dw = np.stack([gh[:, l * l:(l + 1) ** 2].sum(1) for l in range(l_max + 1)])
    db = rows_chain * U * np.abs(g3[:, :, 0]).sum(0)
    half = 2.0 ** -8 if bf16 else 0.0
    tiny = 1e-37
    return want, dict(r=(dr + half * r).reshape(want["r"].shape) + tiny,
                      x=(dx + half * np.abs(_cube(want["x"], 0))).reshape(want["x"].shape) + tiny,
                      w=dw.reshape(want["w"].shape) + tiny, b=db + tiny)


def worst(got, want, bound):
    """The largest error in units of its bound (at most 1 when the bounds hold)."""
    err = np.abs(np.asarray(got, np.float64) - want)
    return float((err / bound).max()) if err.size else 0.0
