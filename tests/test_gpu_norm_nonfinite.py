"""A NaN or an infinity in the norms by degree goes where the formula takes it and no further: every other degree and
row keeps its bits, and within the degree the places that stay finite are the oracle's (GPU)."""
import numpy as np
import pytest

from oracle import norm
from tests.gpu_util import host
from tests.test_gpu_norm import Case, eq  # noqa: F401

pytestmark = pytest.mark.gpu

# vectors of 16 bytes, with all of a pair's degrees (25, 49 components) or the first of four values (16, 36) possibly of
# degree 0; rows that begin anywhere (odd channels); single values (shift); several warps a row; rows of the plain kernels
SHAPES = [((9, 8, 16), 0), ((9, 8, 25), 0), ((9, 8, 36), 0), ((9, 8, 49), 0), ((9, 5, 25), 0), ((9, 7, 36), 0), ((9, 3, 49), 0),
          ((9, 6, 16), 1), ((9, 6, 49), 1), ((6, 128, 16), 0), ((6, 96, 49), 0), ((6, 520, 16), 0), ((6, 200, 49), 0)]
ROW, CHANNEL = 4, 2


def _put(t, k, value):
    t = t.clone() if t.storage_offset() == 0 else _shifted(t)
    t[ROW, CHANNEL, k] = value
    return t


def _shifted(t):
    """A copy that begins at the same place behind an aligned address."""
    import torch

    buf = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    v = buf[t.storage_offset():t.storage_offset() + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def _components(K):
    return [k for k in (0, 1, 2, 4, 6, 8, 9, 16, 24, 35, 48) if k < K]


def _same_elsewhere(got, clean, want, degree, what):
    """got against the call on clean values outside of (ROW, degree), and the oracle's finite places inside."""
    import torch

    l_max = int(round(got.shape[-1] ** 0.5)) - 1
    inside = torch.zeros(got.shape, dtype=torch.bool, device=got.device)
    inside[ROW, :, torch.from_numpy(norm.degrees(l_max)).cuda() == degree] = True
    assert torch.equal(got[~inside], clean[~inside]), what
    assert np.array_equal(np.isfinite(host(got)), np.isfinite(want)), what


def _h(t):
    return None if t is None else host(t)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("form", [dict(), dict(residual=True, p=0.3)], ids=["plain", "residual"])
@pytest.mark.parametrize("shape,shift", SHAPES, ids=str)
@np.errstate(all="ignore")
def test_forward_keeps_degrees_apart(eq, shape, shift, form, bf16):  # noqa: F811
    import torch

    c = Case(shape, bf16=bf16, shift=shift, **form)
    need = ("y", "s", "stats") if form else ("y", "stats")
    clean, x = c.forward(eq, need=need), c.x
    for k in _components(shape[2]):
        degree = int(k ** 0.5)
        for value in (float("nan"), float("inf"), -float("inf")):
            c.x = _put(x, k, value)
            got = c.forward(eq, need=need)
            want = norm.forward(_h(c.x), _h(c.w), _h(c.b), c.eps, _h(c.r), c.factor)
            for name in need:
                if name == "stats":
                    others = [i for i in range(c.l_max + 2) if not (i == 1 + degree or (i == 0 and k == 0))]
                    assert torch.equal(got["stats"][:, others], clean["stats"][:, others]), (k, value)
                    rows = [i for i in range(shape[0]) if i != ROW]
                    assert torch.equal(got["stats"][rows], clean["stats"][rows])
                    assert np.array_equal(np.isfinite(host(got["stats"])), np.isfinite(want["stats"])), (k, value)
                else:
                    _same_elsewhere(got[name], clean[name], want[name], degree, (name, k, value))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("form", [dict(), dict(residual=True, p=0.3)], ids=["plain", "residual"])
@pytest.mark.parametrize("shape,shift", SHAPES, ids=str)
@np.errstate(all="ignore")
def test_backward_keeps_degrees_apart(eq, shape, shift, form, bf16):  # noqa: F811
    """grad_y, s (with the statistics of the forward pass on it) and grad_s, one bad value in one of them at a time."""
    import torch

    c = Case(shape, bf16=bf16, shift=shift, **form)
    need = ("x", "r", "w", "b") if form else ("x", "w", "b")
    s = c.forward(eq, need=("s",))["s"] if form else c.x

    def stats_of(s):
        return (eq.eqmp_degree_norm(s, eps=c.eps, need=("stats",)))["stats"]

    stats, g, r = stats_of(s), c.g, c.r
    clean = c.backward(eq, s, stats, need=need)
    for k in _components(shape[2]):
        degree = int(k ** 0.5)
        for where in ("g", "s", "r")[:3 if form else 2]:
            for value in (float("nan"), float("inf")):
                c.g, c.r = _put(g, k, value) if where == "g" else g, _put(r, k, value) if where == "r" else r
                s2 = _put(s, k, value) if where == "s" else s
                st2 = stats_of(s2)
                got = c.backward(eq, s2, st2, need=need)
                want = norm.backward(_h(c.g), _h(s2), _h(st2), _h(c.w), _h(c.r), c.factor)
                what = (where, k, value)
                for name in need[:-2]:
                    _same_elsewhere(got[name], clean[name], want[name], degree, (name,) + what)
                others = [i for i in range(c.l_max + 1) if i != degree]
                assert torch.equal(got["w"][others], clean["w"][others]), what
                assert np.array_equal(np.isfinite(host(got["w"])), np.isfinite(want["w"])), what
                assert np.array_equal(np.isfinite(host(got["b"])), np.isfinite(want["b"])), what
                ok = torch.from_numpy(np.isfinite(want["b"])).cuda()
                assert torch.equal(got["b"][ok], clean["b"][ok]), what


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shape,shift", SHAPES, ids=str)
def test_a_bad_parameter_stays_in_its_channel(eq, shape, shift, bf16):  # noqa: F811
    import torch

    c = Case(shape, bf16=bf16, shift=shift)
    clean, w, b = c.forward(eq, need=("y",))["y"], c.w, c.b
    degrees = torch.from_numpy(norm.degrees(c.l_max)).cuda()
    for l in [None] + list(range(c.l_max + 1)):
        c.w, c.b = w.clone(), b.clone()
        (c.b if l is None else c.w[l])[CHANNEL] = float("nan")
        y = c.forward(eq, need=("y",))["y"]
        bad = torch.zeros(shape, dtype=torch.bool, device="cuda")
        bad[:, CHANNEL, degrees == (l or 0)] = True
        assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad]), l
