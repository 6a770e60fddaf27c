"""Edges that have no sender, no receiver, or no place in the sender view: gradients of the attention (GPU)."""
import numpy as np
import pytest

from tests.attention_util import backward_bounds, worst
from tests.gpu_util import host
from tests.test_gpu_attention import LONG, MIXED, Problem, eq  # noqa: F401

pytestmark = pytest.mark.gpu

NEED = ("q", "k", "v", "bias")


def _up(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _stale(p, edges):
    """Results and a workspace that hold NaN before the call."""
    import torch

    nan = lambda s, dt=torch.float32: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out = dict(q=nan(p.q.shape, p.dtype), k=nan(p.k.shape, p.dtype), v=nan(p.v.shape, p.dtype), bias=nan((edges, p.q.shape[1])))
    return out


def _workspace(eq, p, edges, listed):  # noqa: F811
    import torch

    n = eq.eqmp_edge_attention_backward_workspace_size(p.q.shape[0], edges, listed, p.q.shape[1], p.q.shape[2], p.v.shape[2])
    return torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)


def _views(eq, src, n_src):  # noqa: F811
    """Sender views of the same edges: the library's own, one without the edges whose sender is none, and that one in a list of
    fixed length."""
    off, edges = eq.sender_view(src, n_src)
    listed = edges[off[0]:off[-1]]
    rest = np.full(len(src) - len(listed), -1, np.int32)
    return [(off, edges), (off - off[0], listed), (off - off[0], np.concatenate((listed, rest)))]


@pytest.mark.parametrize("masked", [0.0, 0.2])
@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
@pytest.mark.parametrize("shape,dtype", [((3, 8, 12), "f32"), ((3, 7, 9), "bf16"), ((40, 4, 8), "f32")], ids=str)
def test_every_edge_has_its_bias_gradient(eq, shape, dtype, degrees, masked):  # noqa: F811
    """Senders outside read as zeros, and their edges' scores have gradients, whatever else is asked for and whether the sender
    view lists them or not."""
    import torch

    p = Problem(*shape, dtype, degrees, seed=2, masked=masked)
    n, E = len(degrees), len(p.src)
    p.src[[0, 1, 40, 50, E - 1]] = [2 ** 31 - 1, -1, n, -2 ** 31, -1]
    if masked:
        p.bias[:2] = -float("inf")
    p.graph = (p.graph[0], _up(p.src))
    stats = p.forward(eq)["stats"]
    want, bound = backward_bounds(host(p.g), *p.host_args()[:3], host(stats), *p.host_args()[3:], None, p.bf16)
    alone = p.backward(eq, stats, need=("bias",), out=dict(bias=_stale(p, E)["bias"]))["bias"]
    for off, edges in _views(eq, p.src, n):
        p.senders = (p.senders[0], _up(off), _up(edges))
        got = p.backward(eq, stats, need=NEED, out=_stale(p, E), workspace=_workspace(eq, p, E, len(edges)))
        for name in NEED:
            assert worst(host(got[name]), want[name], bound[name]) <= 1, name
        assert torch.equal(got["bias"], alone)
        for need in (("k", "bias"), ("v", "bias")):
            assert torch.equal(p.backward(eq, stats, need=need, out=_stale(p, E))["bias"], alone)


def test_bias_gradients_of_no_receivers(eq):  # noqa: F811
    p = Problem(4, 16, 32, "f32", MIXED)
    E = len(p.src)
    got = eq.eqmp_edge_attention_backward(p.g[:0], p.q[:0], p.k, p.v, p.forward(eq)["stats"][:0], p.graph[0][:1], p.graph[1], *p.senders,
                                          need=("v", "bias"), out=dict(bias=_stale(p, E)["bias"]))
    assert not got["bias"].any() and not got["v"].any()


@pytest.mark.parametrize("H", [1, 5, 31, 32, 33, 1024])
def test_bias_gradients_of_any_number_of_heads(eq, H):  # noqa: F811
    """The pass over all edges at numbers of heads around a warp, with empty rows at both ends and edges outside the rows."""
    import torch

    p = Problem(H, 3, 2, "f32", [0, 0, 70, 1, 0, 33, 0], seed=6)
    stats = p.forward(eq)["stats"]
    want, bound = backward_bounds(host(p.g), *p.host_args()[:3], host(stats), *p.host_args()[3:], None, False)
    every = p.backward(eq, stats)["bias"]
    assert worst(host(every), want["bias"], bound["bias"]) <= 1
    for a, b in ((2, 4), (3, 6), (4, 5)):
        part = eq.eqmp_edge_attention_backward(p.g[a:b], p.q[a:b], p.k, p.v, stats[a:b], p.graph[0][a:b + 1], p.graph[1], None, None,
                                               None, bias=p.bias, need=("bias",), out=dict(bias=_stale(p, len(p.src))["bias"]))["bias"]
        lo, hi = int(p.off[a]), int(p.off[b])
        assert torch.equal(part[lo:hi], every[lo:hi]) and not part[:lo].any() and not part[hi:].any()


@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
@pytest.mark.parametrize("shape,dtype", [((4, 16, 32), "f32"), ((3, 7, 9), "bf16"), ((2, 65, 30), "f32")], ids=str)
def test_padded_edge_lists(eq, shape, dtype, degrees):  # noqa: F811
    """Lists of fixed length, with edges behind the last row and before the first that name real nodes and stand in the sender
    view: they are part of no receiver, so nothing has a gradient from them, whatever the workspace held."""
    import torch

    whole = Problem(*shape, dtype, degrees, seed=3)
    stats = whole.forward(eq)["stats"]
    want, bound = backward_bounds(host(whole.g), *whole.host_args()[:3], host(stats), *whole.host_args()[3:], None, whole.bf16)
    n, E = len(degrees), len(whole.src)
    rng = np.random.default_rng(1)
    for before, behind in ((0, 37), (5, 0), (70, 130)):
        p = Problem(*shape, dtype, degrees, seed=3)
        join = lambda a, fill: np.concatenate((fill(before), a, fill(behind)))  # noqa: B023,E731
        zeros, any_node = (lambda k: np.zeros(k, np.int32)), (lambda k: rng.integers(0, n, k).astype(np.int32))
        for fill in (zeros, any_node):
            src, dst = join(whole.src, fill), join(whole.dst, fill)
            off, edges = eq.sender_view(src, n)
            p.graph, p.senders = (_up(whole.off + before), _up(src)), (_up(dst), _up(off), _up(edges))
            pad = lambda k: torch.zeros(k, shape[0], device="cuda")  # noqa: E731
            p.bias = torch.cat((pad(before), whole.bias, pad(behind)))
            got = p.backward(eq, stats, out=_stale(p, len(src)), workspace=_workspace(eq, p, len(src), len(edges)))
            assert not got["bias"][:before].any() and not got["bias"][before + E:].any()
            got["bias"] = got["bias"][before:before + E]
            # long rows are cut where the whole list is: the same to the bounds
            for name in NEED:
                assert worst(host(got[name]), want[name], bound[name]) <= 1, name


@pytest.mark.parametrize("shape", [(4, 16, 128), (3, 6, 10), (2, 5, 49), (5, 7, 9), (2, 200, 300)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_only_edge_left_of_a_long_row(eq, shape, dtype):  # noqa: F811
    """Rows that are cut into parts, all edges but one masked, another one for each head: as the only edge of a short row."""
    import torch

    degrees, H = [700, 2, 300, 400, 65], shape[0]
    p = Problem(*shape, dtype, degrees, seed=4)
    left = np.array([[(97 * i + 263 * h + (0, d - 1)[h % 2]) % d for h in range(H)] for i, d in enumerate(degrees)]) + p.off[:-1, None]
    bias = torch.full_like(p.bias, -float("inf"))
    for i in range(len(degrees)):
        for h in range(H):
            bias[left[i, h], h] = p.bias[left[i, h], h]
    p.bias = bias
    got = p.forward(eq)
    for i in range(len(degrees)):
        for h in range(H):
            assert torch.equal(got["out"][i, h], p.v[int(p.src[left[i, h]]), h])
    for stats in (got["stats"], torch.stack((got["stats"][:, :, 0] * (1 + 2.0 ** -22), got["stats"][:, :, 1]), 2)):
        g = p.backward(eq, stats)
        assert not g["q"].any() and not g["k"].any() and not g["bias"].any() and g["v"].any()


@pytest.mark.parametrize("shape", [(4, 16, 128), (2, 5, 49), (3, 7, 9)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["g", "v", "k", "bias"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_the_only_edge_and_values_that_are_none(eq, shape, dtype, where, bad):  # noqa: F811
    """NaN and infinities around a receiver's only edge, of a short row and of a cut one: gradients are NaN where the formula's are."""
    H = shape[0]
    p = Problem(*shape, dtype, [1, 3, 1100], n_src=1104, seed=4)
    p.src[:] = np.arange(1104)  # each edge has its own sender
    p.graph = (p.graph[0], _up(p.src))
    off, edges = eq.sender_view(p.src, 1104)
    p.senders = (p.senders[0], _up(off), _up(edges))
    p.bias[1:4][:2] = -float("inf")
    p.bias[4:] = -float("inf")
    p.bias[777] = 0.5
    for row, edge in ((0, 0), (1, 3), (2, 777)):
        if where == "g":
            p.g[row, H // 2, 1] = bad
        elif where == "bias":
            p.bias[edge, H // 2] = bad
        elif where == "v":
            p.v[edge, H // 2, 1] = bad
        else:  # a score of plus infinity, or NaN
            p.k[edge, H // 2, 1] = bad if p.q[row, H // 2, 1] > 0 else -bad
    stats = p.forward(eq)["stats"]
    got = p.backward(eq, stats)
    with np.errstate(invalid="ignore"):
        want, bound = backward_bounds(host(p.g), *p.host_args()[:3], host(stats), *p.host_args()[3:], None, p.bf16)
    for name in NEED:
        b = np.where(np.isfinite(bound[name]), bound[name], 1e-37)  # masked edges beside a NaN: 0
        assert worst(host(got[name]), want[name], b) <= 1, name
