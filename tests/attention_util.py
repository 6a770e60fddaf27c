"""Graphs and error bounds for the tests of the attention over edges and of the head norm.

The bounds are worst cases of the fp32 arithmetic to first order, element by element, from u = 2^-24 and the number of
additions behind each sum, in any order; MARGIN covers the higher orders.  The exponential is CUDA's __expf, whose error
is at most 2 + 1.173 |x| units in the last place, each of which is at most 2 u of the value.  A result is off by half a
unit of its type more: u of it in fp32, 2^-8 in bf16.
"""
import numpy as np

from oracle import attention as at

U = 2.0 ** -24
MARGIN = 1.1
TINY = 1e-37


def half_unit(bf16):
    return 2.0 ** -8 if bf16 else U


def graph(rng, degrees, n_src):
    """(off, src, dst, send_off, send_edges), int32, senders drawn at random and sorted in a row."""
    off = np.concatenate([[0], np.cumsum(degrees)]).astype(np.int32)
    dst = np.repeat(np.arange(len(degrees)), degrees).astype(np.int32)
    src = rng.integers(0, max(n_src, 1), off[-1]).astype(np.int32)
    src = src[np.lexsort((src, dst))]
    order = np.argsort(src, kind="stable").astype(np.int32)
    send_off = np.searchsorted(src[order], np.arange(n_src + 1)).astype(np.int32)
    return off, src, dst, send_off, order


def exp_error(x):
    return 2 * U * (2 + 1.2 * np.abs(x))


def _by_row(values, off, reduce, empty=0.0):
    out = np.full((len(off) - 1,) + values.shape[1:], empty)
    for i in range(len(off) - 1):
        if off[i + 1] > off[i]:
            out[i] = reduce(values[off[i]:off[i + 1]], axis=0)
    return out


def _edges(q, k, off, src, bias, scale):
    """Per edge and head: scores (-inf where left out), the bound on their error, and 0 for senders that are none."""
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    dst = np.repeat(np.arange(len(off) - 1), np.diff(off))
    ks = at._rows(k, src)
    with np.errstate(invalid="ignore"):
        s = scale * np.einsum("ehd,ehd->eh", q[dst], ks)
        size = abs(scale) * np.einsum("ehd,ehd->eh", np.abs(q[dst]), np.abs(ks))
    b = np.zeros_like(s) if bias is None else np.asarray(bias, np.float64)
    dead = np.isneginf(b)
    s = np.where(dead, -np.inf, s + b)
    err = np.where(dead, 0.0, (D + 10) * U * size + 2 * U * np.abs(np.where(dead, 0.0, b)))
    return dst, ks, s, err, scale


def forward_bounds(q, k, v, off, src, bias, scale, bf16):
    """The oracle's out and stats, and bounds on their errors."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    out, stats = at.edge_attention(q, k, v, off, src, bias, scale)
    dst, _, s, es, _ = _edges(q, k, off, src, bias, scale)
    n = np.diff(off)[:, None]
    row_es = _by_row(es, off, np.max)
    live = np.isfinite(s)
    x = np.where(live, s - stats[dst, :, 0], 0.0)
    p = np.where(live, np.exp(x) / np.maximum(stats[dst, :, 1], 1e-300), 0.0)
    spread = _by_row(np.abs(x), off, np.max)
    # the running maximum moves at most n times, by no more than the spread in all
    rel = es + row_es[dst] + U * np.abs(x) + exp_error(x) + (2.4 * U * spread + 6 * U * n)[dst]
    rel_z = _by_row(p * rel, off, np.sum) + (n + 4) * U
    vs = np.abs(at._rows(v, src))
    vs = np.where(live[:, :, None], vs, 0.0)
    err = _by_row((p * (rel + rel_z[dst] + ((n + 6) * U)[dst]))[:, :, None] * vs, off, np.sum)
    d_stats = np.stack([row_es + U * np.abs(stats[:, :, 0]), stats[:, :, 1] * rel_z], 2)
    return (out, stats), (MARGIN * (err + half_unit(bf16) * np.abs(out)) + TINY, MARGIN * d_stats + TINY)


def backward_bounds(g, q, k, v, stats, off, src, bias, scale, bf16):
    """The oracle's gradients for the statistics given, and bounds on their errors."""
    g, q, k, v, stats = (np.asarray(a, np.float64) for a in (g, q, k, v, stats))
    want = at.edge_attention_backward(g, q, k, v, stats, off, src, bias, scale)
    dst, ks, s, es, scale = _edges(q, k, off, src, bias, scale)
    Dv, n = v.shape[2], np.diff(off)[:, None]
    live = np.isfinite(s) & (stats[dst, :, 1] != 0)
    x = np.where(live, s - stats[dst, :, 0], 0.0)
    p = np.where(live, np.exp(x) / np.where(live, stats[dst, :, 1], 1.0), 0.0)
    rel = es + U * np.abs(x) + exp_error(x) + 3 * U
    vs = np.where(live[:, :, None], at._rows(v, src), 0.0)
    ks = np.where(live[:, :, None], ks, 0.0)
    dp = np.einsum("ehd,ehd->eh", g[dst], vs)
    edp = (Dv + 4) * U * np.einsum("ehd,ehd->eh", np.abs(g[dst]), np.abs(vs))
    delta = _by_row(p * dp, off, np.sum)
    e_pdp = p * (np.abs(dp) * (rel + 2 * U) + edp)
    e_delta = _by_row(e_pdp + ((n + 3) * U)[dst] * p * np.abs(dp), off, np.sum)
    ds = np.abs(p * (dp - delta[dst]))
    eds = ds * rel + p * (edp + e_delta[dst] + 3 * U * (np.abs(dp) + np.abs(delta)[dst]))
    wide = lambda a: a[:, :, None]  # noqa: E731
    ak = np.abs(ks)
    chain = ((n + 5) * U)[dst]
    dq = _by_row(wide(e_pdp + chain * p * np.abs(dp)) * ak + wide(e_delta[dst] * p + np.abs(delta)[dst] * p * (rel + chain)) * ak,
                 off, np.sum)
    e_q = abs(scale) * dq
    sends = (src >= 0) & (src < k.shape[0])
    count = np.bincount(src[sends], minlength=k.shape[0])
    back = np.where(sends, count[np.where(sends, src, 0)] if k.shape[0] else 0, 0)[:, None]
    e_k, e_v = np.zeros_like(k), np.zeros_like(v)
    aq, ag = np.abs(q[dst]), np.abs(g[dst])
    np.add.at(e_k, src[sends], (abs(scale) * wide(eds + (back + 5) * U * ds) * np.where(wide(live), aq, 0.0))[sends])
    np.add.at(e_v, src[sends], (wide(p * (rel + (back + 5) * U)) * np.where(wide(live), ag, 0.0))[sends])
    half = half_unit(bf16)
    bounds = dict(q=e_q + half * np.abs(want["q"]), k=e_k + half * np.abs(want["k"]), v=e_v + half * np.abs(want["v"]),
                  bias=eds + U * np.abs(want["bias"]))
    return want, {name: MARGIN * b + TINY for name, b in bounds.items()}


def head_norm_bounds(x, w, eps, theta, d_theta, bf16):
    """(y, rstd) of the oracle and bounds; d_theta: the error of an angle."""
    x = np.asarray(x, np.float64)
    D = x.shape[2]
    y, r = at.head_norm(x, w, eps, theta)
    plain = np.abs(at.head_norm(x, w, eps)[0])
    rel_r = 0.5 * (D + 4) * U + 4 * U
    e_u = plain * (rel_r + 4 * U)
    if theta is not None:  # each value of a pair takes both
        both = plain[..., 0::2] + plain[..., 1::2]
        e = (e_u[..., 0::2] + e_u[..., 1::2]) + both * (3 * U + (d_theta + 4 * U)[:, None, :])
        e_u = np.repeat(e, 2, axis=-1)
    return (y, r), (MARGIN * (e_u + half_unit(bf16) * np.abs(y)) + TINY, MARGIN * r * rel_r + TINY)


def head_norm_backward_bounds(g, x, rstd, w, theta, freq, d_theta, bf16):
    """(dx, dw, dpos) of the oracle for the rstd given, and bounds."""
    g, x, r = (np.asarray(a, np.float64) for a in (g, x, rstd))
    N, H, D = x.shape
    want = at.head_norm_backward(g, x, r, w, theta, freq)
    ww = np.ones(D) if w is None else np.abs(np.asarray(w, np.float64))
    h = np.abs(x) * r[..., None]
    b, e_b = np.abs(g), np.zeros_like(g)
    if theta is not None:
        both = np.repeat(b[..., 0::2] + b[..., 1::2], 2, axis=-1)
        b = both  # bounds both values of a turned pair
        e_b = both * (3 * U + np.repeat(d_theta + 4 * U, 2, axis=-1)[:, None, :])
    a, e_a = b * ww, e_b * ww + U * b * ww
    mean = (a * h).mean(-1, keepdims=True)
    e_mean = (e_a * h + a * h * 2 * U).mean(-1, keepdims=True) + (D + 3) * U * mean
    dx = r[..., None] * (e_a + h * e_mean + 4 * U * (a + h * mean))
    rows = N * H
    dw = (e_b * h + b * h * (rows + 6) * U).sum((0, 1))
    dpos = None
    if theta is not None:
        u = h * ww
        t = (b[..., 1::2] * u[..., 0::2] + b[..., 0::2] * u[..., 1::2])
        e_t = e_b[..., 1::2] * u[..., 0::2] + e_b[..., 0::2] * u[..., 1::2] + t * (H + 6) * U
        dpos = (e_t + t * (D + 8) * U).sum(1) @ np.abs(np.asarray(freq, np.float64))
        dpos = MARGIN * dpos + TINY
    return want, (MARGIN * (dx + half_unit(bf16) * np.abs(want[0])) + TINY, MARGIN * dw + TINY, dpos)


def worst(got, want, bound):
    """The largest error in units of its bound (at most 1 when the bounds hold); NaN and infinities have to match."""
    got, want, bound = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(bound, np.float64)
    if got.size == 0:
        return 0.0
    odd = ~np.isfinite(want)
    if odd.any():
        assert np.array_equal(got[odd], want[odd], equal_nan=True)
        got, want, bound = got[~odd], want[~odd], bound[~odd]
    return float((np.abs(got - want) / bound).max()) if got.size else 0.0
