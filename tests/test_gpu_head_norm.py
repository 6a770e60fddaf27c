"""The head norm with its rotation against the float64 oracle, within worst-case bounds (GPU)."""
import numpy as np
import pytest

from oracle import attention as at
from tests.attention_util import U, head_norm_backward_bounds, head_norm_bounds, worst
from tests.gpu_util import host
from tests.test_gpu_attention import eq  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-6


def angle_error(pos, freq):
    """Of an angle reduced to half a turn: a few units of it, and the second float of a frequency in turns."""
    turns = np.abs(np.asarray(pos, np.float64)) @ np.abs(np.asarray(freq, np.float64)).T / (2 * np.pi)
    return 2 * np.pi * (6 * pos.shape[1] * U + turns * 2.0 ** -46)


class Problem:
    def __init__(self, n, hq, hk, dim, dtype, axes=0, pad=None, weights=True, seed=0, far=1.0):
        import torch

        rng = np.random.default_rng(seed)
        self.bf16, self.dtype = dtype == "bf16", torch.bfloat16 if dtype == "bf16" else torch.float32
        self.hk = hk
        up = lambda a, dt=torch.float32: torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dt).cuda()  # noqa: E731

        def pair():
            a = up(rng.standard_normal((n, (hq + hk) * dim + (pad or 0))), self.dtype)
            parts = a[:, :hq * dim].unflatten(1, (hq, dim)), a[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim)) if hk else None
            return parts if pad is not None else tuple(t if t is None else t.contiguous() for t in parts)

        (self.q, self.k), (self.gq, self.gk) = pair(), pair()
        self.wq, self.wk = (up(1 + 0.2 * rng.standard_normal(dim)) for _ in "qk") if weights else (None, None)
        self.pos = self.freq = None
        if axes:
            self.pos, self.freq = up(far * rng.standard_normal((n, axes))), up(rng.standard_normal((dim // 2, axes)))
        self.turn = dict(pos=self.pos, freq=self.freq)

    def forward(self, eq, **kw):  # noqa: F811
        return eq.eqmp_head_norm(self.q, self.k, self.wq, self.wk if self.hk else None, eps=EPS, **self.turn, **kw)

    def backward(self, eq, rstd, **kw):  # noqa: F811
        return eq.eqmp_head_norm_backward(self.gq, self.gk, self.q, self.k, rstd, self.wq, self.wk if self.hk else None, **self.turn,
                                          **kw)

    def check(self, eq):  # noqa: F811
        keys = ("q", "k") if self.hk else ("q",)
        got = self.forward(eq, need=keys + ("rstd",))
        theta = d_theta = freq = None
        if self.pos is not None:
            pos, freq = host(self.pos), host(self.freq)
            theta, d_theta = at.angles(pos, freq), angle_error(pos, freq)
        grads = self.backward(eq, got["rstd"], need=sum(((k, "w" + k) for k in keys), ()) + (("pos",) if theta is not None else ()))
        hq, dpos, dpos_bound = self.q.shape[1], 0.0, 0.0
        for name, x, g, w, r in (("q", self.q, self.gq, self.wq, got["rstd"][:, :hq]), ("k", self.k, self.gk, self.wk, got["rstd"][:, hq:])):
            if name not in keys:
                continue
            w = None if w is None else host(w)
            want, bound = head_norm_bounds(host(x), w, EPS, theta, d_theta, self.bf16)
            assert worst(host(got[name]), want[0], bound[0]) <= 1, name
            assert worst(host(r), want[1], bound[1]) <= 1, name
            want, bound = head_norm_backward_bounds(host(g), host(x), host(r), w, theta, freq, d_theta, self.bf16)
            assert worst(host(grads[name]), want[0], bound[0]) <= 1, name
            assert worst(host(grads["w" + name]), want[1], bound[1]) <= 1, name
            if theta is not None:
                dpos, dpos_bound = dpos + want[2], dpos_bound + bound[2]
        if theta is not None:
            assert worst(host(grads["pos"]), dpos, dpos_bound) <= 1
        return got, grads


SHAPES = [(1, 1, 0, 1), (64, 4, 4, 16), (37, 6, 2, 18), (5, 8, 8, 32), (130, 3, 1, 7), (9, 5, 5, 64), (11, 2, 1, 128), (3, 2, 2, 256),
          (700, 1, 1, 8), (33, 4, 3, 2), (6, 2, 2, 254), (4, 40, 9, 30), (2, 1, 1, 255)]


@pytest.mark.parametrize("shape,axes", [(s, a) for s in SHAPES for a in range(4) if a == 0 or s[3] % 2 == 0], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_against_the_oracle(eq, shape, dtype, axes):  # noqa: F811
    Problem(*shape, dtype, axes, weights=shape[0] != 5, seed=shape[0]).check(eq)


@pytest.mark.parametrize("pad", [0, 1, 5, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [16, 18])
def test_slices_of_a_projection(eq, dim, dtype, pad):  # noqa: F811
    Problem(50, 4, 2, dim, dtype, 3, pad=pad).check(eq)


@pytest.mark.parametrize("axes", [1, 3])
def test_far_positions(eq, axes):  # noqa: F811
    """A hundred thousand turns and more: the angle is as good as at the origin."""
    Problem(200, 2, 2, 16, "f32", axes, far=1e6).check(eq)


def test_many_nodes(eq):  # noqa: F811
    """More nodes than warps of a launch, so that each takes several; sums over all of them."""
    Problem(30000, 2, 1, 8, "f32", 3).check(eq)


def test_no_nodes(eq):  # noqa: F811
    p = Problem(0, 4, 2, 16, "f32", 1)
    got = p.forward(eq, need=("q", "k", "rstd"))
    g = p.backward(eq, got["rstd"], need=("q", "k", "wq", "wk", "pos"))
    assert g["q"].shape == (0, 4, 16) and not g["wq"].any() and not g["wk"].any() and g["pos"].shape == (0, 1)


def test_a_row_of_zeros_and_a_bad_one(eq):  # noqa: F811
    """Zeros stay zeros (eps > 0); a NaN reaches its own head, the weights' gradients and the node's position."""
    import torch

    p = Problem(20, 4, 2, 16, "f32", 3)
    p.q[3, 1] = 0
    p.check(eq)
    clean = p.forward(eq, need=("q", "k", "rstd"))
    grads = p.backward(eq, clean["rstd"], need=("q", "k", "wq", "wk", "pos"))
    p.q[7, 2, 5] = float("nan")
    got = p.forward(eq, need=("q", "k", "rstd"))
    bad = p.backward(eq, got["rstd"], need=("q", "k", "wq", "wk", "pos"))
    assert torch.isnan(got["q"][7, 2]).all() and torch.isnan(bad["q"][7, 2]).all()
    assert torch.isnan(bad["wq"]).all() and torch.isnan(bad["pos"][7]).all() and torch.equal(bad["wk"], grads["wk"])
    for a, b in ((got["q"], clean["q"]), (bad["q"], grads["q"])):
        a[7, 2] = b[7, 2]
        assert torch.equal(a, b)
    assert torch.equal(got["k"], clean["k"]) and torch.equal(bad["k"], grads["k"])


def test_the_same_again_and_captured(eq):  # noqa: F811
    import torch

    p = Problem(999, 8, 8, 32, "bf16", 3, pad=64)
    first = p.forward(eq, need=("q", "k", "rstd"))
    need = ("q", "k", "wq", "wk", "pos")
    grads = p.backward(eq, first["rstd"], need=need)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again, regrads = p.forward(eq, need=("q", "k", "rstd"), stream=side), p.backward(eq, first["rstd"], need=need, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(first[k], again[k]) for k in first) and all(torch.equal(grads[k], regrads[k]) for k in need)
    tape = torch.cuda.CUDAGraph()
    with torch.cuda.graph(tape):
        out = p.forward(eq, need=("q", "k", "rstd"))
        back = p.backward(eq, out["rstd"], need=need)
    tape.replay()
    assert all(torch.equal(first[k], out[k]) for k in out) and all(torch.equal(grads[k], back[k]) for k in need)


@pytest.mark.parametrize("need", [("q",), ("k",), ("wq",), ("wk",), ("pos",)], ids=str)
def test_each_gradient_alone(eq, need):  # noqa: F811
    import torch

    p = Problem(300, 4, 2, 16, "f32", 3)
    rstd = p.forward(eq, need=("rstd",))["rstd"]
    every = p.backward(eq, rstd, need=("q", "k", "wq", "wk", "pos"))
    assert torch.equal(p.backward(eq, rstd, need=need)[need[0]], every[need[0]])


def test_gradients_against_differences(eq):  # noqa: F811
    """By the float64 oracle's loss along random directions; 1e-3 of |grad| |d| covers the fp32 gradients' 1e-5 or so."""
    p = Problem(30, 3, 2, 12, "f32", 3)
    rstd = p.forward(eq, need=("rstd",))["rstd"]
    grads = p.backward(eq, rstd, need=("q", "k", "wq", "wk", "pos"))
    args = {k: host(getattr(p, k)) for k in grads}
    gq, gk, freq = host(p.gq), host(p.gk), host(p.freq)

    def loss(a):
        theta = at.angles(a["pos"], freq)
        return (at.head_norm(a["q"], a["wq"], EPS, theta)[0] * gq).sum() + (at.head_norm(a["k"], a["wk"], EPS, theta)[0] * gk).sum()

    rng = np.random.default_rng(0)
    for name, base in args.items():
        d = rng.standard_normal(base.shape)
        diff = (loss({**args, name: base + 1e-5 * d}) - loss({**args, name: base - 1e-5 * d})) / 2e-5
        grad = host(grads[name])
        assert abs(diff - (grad * d).sum()) <= 1e-3 * np.sqrt((grad ** 2).sum() * (d ** 2).sum() / grad.size), name
