"""Attention over a receiver's edges, and what stands in front of it (oracle, float64; test infrastructure).

head_norm: each head x [D] of queries and keys becomes u = x w / sqrt(mean(x^2) + eps), and its pairs (u[2p], u[2p+1]),
read as complex numbers, are multiplied by exp(i theta[p]), theta[p] = sum_a pos[a] freq[p, a].
edge_bias: table[number of borders that are at most |vec|].
edge_attention (E2Former-V2 section 2.2: node-centric softmax over the neighbours): for each receiver and head
  s[e] = scale q.k[src e] + bias[e],  m = max s,  z = sum exp(s - m),  out = sum exp(s - m) / z v[src e]
over the edges whose score is not -inf; zeros, and zeros as (m, z), where no edge is left.
Receivers are taken one after the other.  Pinned by finite differences, closed forms and rotations
(tests/test_oracle_attention.py).
"""
import numpy as np


def _turned(u, theta):
    if theta is None:
        return u
    c = (u[..., 0::2] + 1j * u[..., 1::2]) * np.exp(1j * theta)[:, None, :]
    return np.stack([c.real, c.imag], -1).reshape(u.shape)


def angles(pos, freq):
    return None if pos is None else np.asarray(pos, np.float64) @ np.asarray(freq, np.float64).T


def head_norm(x, w=None, eps=1e-6, theta=None):
    """x [N, H, D] -> (y, rstd [N, H])."""
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x ** 2).mean(-1) + eps)
    return _turned(x * r[..., None] * (1.0 if w is None else np.asarray(w, np.float64)), theta), r


def head_norm_backward(g, x, rstd, w=None, theta=None, freq=None):
    """(dx, dw, dpos) for the reciprocal deviations given."""
    g, x, r = (np.asarray(a, np.float64) for a in (g, x, rstd))
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    b = _turned(g, None if theta is None else -theta)
    h = x * r[..., None]
    a, u = b * w, h * w
    dx = r[..., None] * (a - h * (a * h).mean(-1, keepdims=True))
    dpos = None
    if theta is not None:
        dpos = (b[..., 1::2] * u[..., 0::2] - b[..., 0::2] * u[..., 1::2]).sum(1) @ np.asarray(freq, np.float64)
    return dx, (b * h).sum((0, 1)), dpos


def edge_bucket(vec, borders):
    v, b = np.asarray(vec, np.float64), np.asarray(borders, np.float64)
    square = (v[:, 0] * v[:, 0] + v[:, 1] * v[:, 1]) + v[:, 2] * v[:, 2]
    return np.array([int((s >= b * b).sum()) for s in square], np.int32)


def edge_bias_backward(grad, bucket, n_buckets):
    table = np.zeros((n_buckets, grad.shape[1]))
    for e, b in enumerate(bucket):
        if 0 <= b < n_buckets:
            table[b] += grad[e]
    return table


def _rows(x, src):
    """x[src], zeros where the sender is none."""
    ok = (src >= 0) & (src < x.shape[0])
    return np.where(ok[:, None, None], x[np.where(ok, src, 0)] if x.shape[0] else np.zeros((len(src),) + x.shape[1:]), 0.0)


def _scores(q, k, bias, scale, i, src, rows):
    with np.errstate(invalid="ignore"):
        s = scale * np.einsum("hd,ehd->eh", q[i], _rows(k, src[rows]))
        if bias is not None:
            s = np.where(np.isneginf(bias[rows]), -np.inf, s + bias[rows])
    return s


def edge_attention(q, k, v, off, src, bias=None, scale=None):
    """(out [N, H, Dv], stats [N, H, 2])."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    bias = None if bias is None else np.asarray(bias, np.float64)
    n, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out, stats = np.zeros((n, H, v.shape[2])), np.zeros((n, H, 2))
    for i in range(n):
        rows = np.arange(off[i], off[i + 1])
        s = _scores(q, k, bias, scale, i, src, rows)
        vs = _rows(v, src[rows])
        for h in range(H):
            live = ~np.isneginf(s[:, h])
            if live.any():
                m = s[live, h].max()
                p = np.exp(s[live, h] - m)
                stats[i, h] = m, p.sum()
                out[i, h] = (p / p.sum()) @ vs[live, h]
    return out, stats


def edge_attention_backward(g, q, k, v, stats, off, src, bias=None, scale=None):
    """dict(q, k, v, bias) for the statistics given."""
    g, q, k, v, stats = (np.asarray(a, np.float64) for a in (g, q, k, v, stats))
    bias = None if bias is None else np.asarray(bias, np.float64)
    n, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    dq, dk, dv, db = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((len(src), H))
    for i in range(n):
        rows = np.arange(off[i], off[i + 1])
        s = _scores(q, k, bias, scale, i, src, rows)
        ks, vs = _rows(k, src[rows]), _rows(v, src[rows])
        for h in range(H):
            live = np.flatnonzero(~np.isneginf(s[:, h])) if stats[i, h, 1] != 0 else np.zeros(0, int)
            if not len(live):
                continue
            p = np.exp(s[live, h] - stats[i, h, 0]) / stats[i, h, 1]
            dp = vs[live, h] @ g[i, h]
            ds = p * (dp - (p * dp).sum())
            dq[i, h] = scale * ds @ ks[live, h]
            db[rows[live], h] = ds
            for e, w, d in zip(rows[live], p, ds):
                if 0 <= src[e] < k.shape[0]:
                    dk[src[e], h] += scale * d * q[i, h]
                    dv[src[e], h] += w * g[i, h]
    return dict(q=dq, k=dk, v=dv, bias=db)
