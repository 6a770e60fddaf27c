"""Pins of the oracle's dropout and norms: the generator's published vectors,
loops over single rows, finite differences and rotations (CPU only)."""
import numpy as np
import pytest

from oracle import norm
from tests.rotations import random_rotation, rotate_features, wigner_d_blocks


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    """The known-answer vectors published with the generator."""
    assert tuple(int(v) for v in norm.philox(counter, key)) == want


def test_drop_factor_places_and_rate():
    f = norm.drop_factor(200, 160, 0.25, seed=7, offset=(1 << 40) + 3)
    assert set(np.unique(f)) == {0.0, 65536 / 49152}
    kept = (f != 0).mean()
    assert abs(kept - 0.75) < 5 * np.sqrt(0.25 * 0.75 / f.size)
    # one element by hand
    r, c = 17, 93
    words = norm.philox((c // 8, r, 3, 1 << 8), (7, 0))
    draw = (int(words[(c % 8) // 2]) >> (16 * (c % 2))) & 0xFFFF
    assert (f[r, c] != 0) == (draw >= 16384)
    # rows of another first row, groups, the ends of the rate
    assert np.array_equal(norm.drop_factor(50, 160, 0.25, 7, (1 << 40) + 3, first_row=150), f[150:])
    g = norm.drop_factor(200, 160, 0.25, 7, (1 << 40) + 3, group=16)
    assert np.array_equal(g[:, ::16], f[:, :10]) and np.array_equal(g, np.repeat(g[:, ::16], 16, 1))
    assert np.all(norm.drop_factor(3, 5, 0.0, 1) == 1) and np.all(norm.drop_factor(3, 5, 1.0, 1) == 0)
    assert np.all(norm.drop_factor(3, 5, 2.0 ** -18, 1) == 1)
    assert np.isfinite(norm.apply_drop(np.full((200, 160), np.nan), f)[f == 0]).all()


def test_forward_is_the_layer_norm_of_a_row():
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((3, 7)) + 2, rng.standard_normal(7), rng.standard_normal(7)
    got = norm.forward(x, w, b, eps=0.1)
    for i in range(3):
        m = sum(x[i]) / 7
        v = sum((t - m) ** 2 for t in x[i]) / 7
        assert np.allclose(got["y"][i], [(t - m) / (v + 0.1) ** 0.5 * a + c for t, a, c in zip(x[i], w, b)])
        assert np.allclose(got["stats"][i], [m, (v + 0.1) ** -0.5])


@pytest.mark.parametrize("l_max", [3, 6])
def test_degree_norm_commutes_with_rotations(l_max):
    rng, K = np.random.default_rng(1), (l_max + 1) ** 2
    x, w, b = rng.standard_normal((5, 6, K)), rng.standard_normal((l_max + 1, 6)), rng.standard_normal(6)
    f = norm.drop_factor(5, 6 * K, 0.4, 3, group=K)
    blocks = wigner_d_blocks(random_rotation(4), l_max=l_max)
    rot = lambda t: rotate_features(t, blocks)  # noqa: E731
    got = norm.forward(rot(x), w, b, factor=f, residual=rot(x[::-1]))["y"]
    want = rot(norm.forward(x, w, b, factor=f, residual=x[::-1])["y"])
    assert np.allclose(got, want, atol=1e-10)
    # a plain layer norm over the row does not
    plain = lambda t: norm.forward(t.reshape(5, -1))["y"].reshape(t.shape)  # noqa: E731
    assert not np.allclose(plain(rot(x)), rot(plain(x)), atol=1e-3)


@pytest.mark.parametrize("shape", [(3, 5), (2, 3, 16), (2, 2, 49)])
def test_backward_matches_finite_differences(shape):
    rng = np.random.default_rng(2)
    l_max = int(round(np.sqrt(shape[2]))) - 1 if len(shape) == 3 else 0
    C, K = shape[1], (l_max + 1) ** 2
    x, res, g, gs = (rng.standard_normal(shape) for _ in range(4))
    w = rng.standard_normal((l_max + 1, C)) if len(shape) == 3 else rng.standard_normal(C)
    b = rng.standard_normal(C)
    f = norm.drop_factor(shape[0], C * K, 0.3, 11, group=K)

    def loss(x, res, w, b):
        got = norm.forward(x, w, b, eps=0.01, residual=res, factor=f)
        return float((got["y"] * g).sum() + (got["s"] * gs).sum())

    fw = norm.forward(x, w, b, eps=0.01, residual=res, factor=f)
    got = norm.backward(g, fw["s"], fw["stats"], w, gs, f)
    args = [x, res, w, b]
    for i, k in enumerate(("x", "r", "w", "b")):
        for _ in range(3):
            d = rng.standard_normal(args[i].shape)
            up, down = ([a + s * 1e-6 * d if j == i else a for j, a in enumerate(args)] for s in (1, -1))
            assert abs((loss(*up) - loss(*down)) / 2e-6 - (got[k] * d).sum()) < 1e-6 * max(1.0, np.abs(got[k]).sum()), k


def test_a_dropped_mean_term_is_seen():
    """The finite differences tell a backward pass without the mean of a."""
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 6)), rng.standard_normal((2, 6)) + 1
    fw = norm.forward(x)
    wrong = norm.backward(g, fw["s"], fw["stats"])["x"] + g.mean(1, keepdims=True) * fw["stats"][:, 1:]
    d = np.ones_like(x)
    assert abs((wrong * d).sum()) > 1.0  # the true gradient has no component along a shift of the row
    assert abs((norm.backward(g, fw["s"], fw["stats"])["x"] * d).sum()) < 1e-10


def test_c_entries_refuse_bad_arguments_before_any_launch():
    """The checks of the C entry points come before any CUDA call (no GPU needed)."""
    import ctypes

    import __graft_entry__

    __graft_entry__.build()
    import equivariant_gnn_message_gb300 as eq

    lib = eq.load_library()
    at = lambda k: ctypes.c_void_p((k + 1) << 20)  # noqa: E731  never dereferenced
    no, bad, unsup = eq._NO_DROP, eq.EQMP_ERR_INVALID_ARG, eq.EQMP_ERR_UNSUPPORTED

    def forward(x=at(0), ld=8, r=None, dtype=0, rows=4, cols=8, drop=no, w=None, eps=1e-5, s=None, y=at(1), stats=None):
        return lib.eqmp_layer_norm(x, ld, r, 8, dtype, rows, cols, drop, w, None, eps, s, y, stats, None)

    def drop(p, group=1):
        d = eq.Dropout(0.5, 1, group=group)
        d.p = p
        return d

    assert forward(rows=0) == eq.EQMP_OK and forward(y=None) == eq.EQMP_OK
    for kw in (dict(x=None), dict(ld=-1), dict(ld=(1 << 31) + 1), dict(dtype=2), dict(rows=-1), dict(cols=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(x=ctypes.c_void_p((1 << 20) + 2)), dict(y=at(0)), dict(s=at(1)),
               dict(w=ctypes.c_void_p(6)), dict(y=ctypes.c_void_p((1 << 20) + 4)), dict(drop=drop(-0.5)),
               dict(drop=drop(float("nan"))), dict(drop=drop(1.5)), dict(drop=drop(0.5, 3))):
        assert forward(**kw) == bad, kw
    assert forward(rows=(1 << 30) + 1) == unsup and forward(cols=(1 << 30) + 1) == unsup

    def backward(g=at(0), x=at(1), stats=at(2), gr=None, gx=at(3), gw=at(4), ws=at(5), nbytes=1 << 19, rows=4):
        return lib.eqmp_layer_norm_backward(g, 8, x, 8, None, 0, 0, rows, 8, no, None, stats, gr, gx, gw, None, ws, nbytes,
                                            None)

    assert backward(gx=None, gw=None) == eq.EQMP_OK
    for kw in (dict(g=None), dict(x=None), dict(stats=None), dict(ws=None), dict(nbytes=15), dict(gx=at(0)),
               dict(gr=at(3)), dict(ws=ctypes.c_void_p((6 << 20) + 4)), dict(rows=-1)):
        assert backward(**kw) == bad, kw
    assert lib.eqmp_layer_norm_backward_workspace_size(-1, 8) == -1
    assert lib.eqmp_degree_norm_backward_workspace_size(8, 8, 2) == -1
    degree = lambda l_max, d, c=8: lib.eqmp_degree_norm(at(0), None, 0, 4, c, l_max, d, None, None, 1e-5, None, at(1), None,  # noqa: E731
                                                        None)
    assert degree(2, no) == unsup and degree(7, no) == unsup and degree(3, no, 0) == bad
    assert degree(3, drop(0.5, 1)) == bad and degree(4, drop(0.5, 16)) == bad
    assert lib.eqmp_dropout(at(0), 8, 0, 4, 8, drop(0.5), ctypes.c_void_p((1 << 20) + 4), None) == bad
    assert lib.eqmp_dropout(at(0), 9, 0, 4, 8, drop(0.5), at(0), None) == bad
    assert lib.eqmp_dropout(None, 8, 0, 4, 8, drop(0.5), at(1), None) == bad
