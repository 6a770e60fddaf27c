"""Pins of the attention oracle: finite differences, closed forms, invariances (CPU)."""
import numpy as np
import pytest

from oracle import attention as at
from tests.rotations import random_rotation, rotate_features, wigner_d_blocks


def _graph(rng, n, n_src, degrees):
    off = np.concatenate([[0], np.cumsum(degrees)]).astype(int)
    return off, rng.integers(0, n_src, off[-1])


def _differences(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("axes", [0, 1, 3])
def test_head_norm_gradients(axes):
    rng = np.random.default_rng(axes)
    x, w, g = rng.standard_normal((4, 3, 8)), rng.standard_normal(8), rng.standard_normal((4, 3, 8))
    pos = rng.standard_normal((4, axes)) if axes else None
    freq = rng.standard_normal((4, axes)) if axes else None
    loss = lambda x, w, pos: (at.head_norm(x, w, 1e-3, at.angles(pos, freq))[0] * g).sum()  # noqa: E731
    _, r = at.head_norm(x, w, 1e-3)
    dx, dw, dpos = at.head_norm_backward(g, x, r, w, at.angles(pos, freq), freq)
    for grad, base, f in ((dx, x, lambda t: loss(t, w, pos)), (dw, w, lambda t: loss(x, t, pos)),
                          (dpos, pos, lambda t: loss(x, w, t))):
        if grad is None:
            continue
        d = rng.standard_normal(base.shape)
        assert abs(_differences(f, base, d) - (grad * d).sum()) < 1e-7 * np.sqrt((grad ** 2).sum() * (d ** 2).sum())


def test_rotated_products_depend_on_the_difference_of_positions():
    rng = np.random.default_rng(1)
    q, k, freq = rng.standard_normal((1, 2, 6)), rng.standard_normal((1, 2, 6)), rng.standard_normal((3, 3))
    a, b, shift = rng.standard_normal((3, 1, 3))
    turn = lambda x, p: at.head_norm(x, None, 0.0, at.angles(p, freq))[0]  # noqa: E731
    here, there = ((turn(q, a + t) * turn(k, b + t)).sum(-1) for t in (0, shift))
    assert np.allclose(here, there, atol=1e-13)
    one = turn(np.tile([1.0, 0.0], 3)[None, None], a)[0, 0]  # unit pairs: cosines and sines, the root mean square divided out
    assert np.allclose(one, np.sqrt(2) * np.stack([np.cos(freq @ a[0]), np.sin(freq @ a[0])], 1).ravel())


def test_buckets_of_a_triple():
    vec = np.array([[3, 4, 0], [0, 0, 0], [2, 3, 6], [1e20, 0, 0]], np.float32)
    assert at.edge_bucket(vec, [5, 7, 8]).tolist() == [1, 0, 2, 3]
    assert at.edge_bucket(vec, np.nextafter(np.float32([5, 7]), np.float32(9))).tolist() == [0, 0, 1, 2]
    assert at.edge_bucket(vec, [0.0]).tolist() == [1, 1, 1, 1]
    grad = np.arange(8.0).reshape(4, 2)
    assert at.edge_bias_backward(grad, np.array([1, 0, 1, 9]), 3).tolist() == [[2, 3], [4, 6], [0, 0]]


def test_attention_gradients():
    rng = np.random.default_rng(2)
    n, ns, H, D, V = 5, 6, 2, 3, 4
    off, src = _graph(rng, n, ns, [0, 1, 4, 7, 3])
    src[3] = -1
    q, k, v = rng.standard_normal((n, H, D)), rng.standard_normal((ns, H, D)), rng.standard_normal((ns, H, V))
    bias, g = rng.standard_normal((len(src), H)), rng.standard_normal((n, H, V))
    bias[6] = -np.inf
    bias[12:, 1] = -np.inf  # the last row, one head
    args = dict(q=q, k=k, v=v, bias=bias)
    loss = lambda **a: (at.edge_attention(a["q"], a["k"], a["v"], off, src, a["bias"])[0] * g).sum()  # noqa: E731
    out, stats = at.edge_attention(q, k, v, off, src, bias)
    assert (out[0] == 0).all() and (out[4, 1] == 0).all() and (stats[4, 1] == 0).all()
    grads = at.edge_attention_backward(g, q, k, v, stats, off, src, bias)
    for name, base in args.items():
        d = rng.standard_normal(base.shape)
        diff = _differences(lambda t: loss(**{**args, name: t}), base, d)  # noqa: B023
        size = np.sqrt((grads[name] ** 2).sum() * (d ** 2).sum())
        assert abs(diff - (grads[name] * d).sum()) < 1e-7 * size, name
    assert (grads["bias"][np.isneginf(bias)] == 0).all()


def test_equal_scores_give_the_mean_and_masks_hide_anything():
    rng = np.random.default_rng(3)
    off, src = np.array([0, 4]), np.arange(4)
    v = rng.standard_normal((4, 1, 5))
    q, k = np.zeros((1, 1, 2)), rng.standard_normal((4, 1, 2))
    out, stats = at.edge_attention(q, k, v, off, src)
    assert np.allclose(out[0, 0], v.mean(0)) and stats.tolist() == [[[0, 4]]]
    low = np.full((4, 1), np.finfo(np.float32).min, np.float64)  # the lowest value is a number, not a mask
    assert np.allclose(at.edge_attention(q, k, v, off, src, low)[0], out)
    bias = np.zeros((4, 1))
    bias[2] = -np.inf
    v[2], k[2] = np.nan, np.inf
    out, stats = at.edge_attention(q, k, v, off, src, bias)
    assert np.allclose(out[0, 0], v[[0, 1, 3], 0].mean(0)) and stats[0, 0, 1] == 3


def test_equivariant_values_turn_with_the_frame():
    rng = np.random.default_rng(4)
    off, src = _graph(rng, 3, 4, [2, 3, 4])
    q, k, x = rng.standard_normal((3, 2, 3)), rng.standard_normal((4, 2, 3)), rng.standard_normal((4, 6, 16))
    blocks = wigner_d_blocks(random_rotation(5))
    run = lambda x: at.edge_attention(q, k, x.reshape(4, 2, 48), off, src)[0].reshape(3, 6, 16)  # noqa: E731
    assert np.allclose(run(rotate_features(x, blocks)), rotate_features(run(x), blocks), atol=1e-10)
