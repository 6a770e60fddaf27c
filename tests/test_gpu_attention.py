"""Attention over a receiver's edges against the float64 oracle, within worst-case bounds (GPU)."""
import numpy as np
import pytest

from oracle import attention as at
from tests.attention_util import backward_bounds, forward_bounds, graph, worst
from tests.gpu_util import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def eq():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    import equivariant_gnn_message_gb300 as eq

    torch.cuda.set_device(0)
    yield eq
    assert eq.eqmp_device_error() == 0


MIXED = [0, 1, 2, 3, 31, 32, 33, 0, 5, 19, 64, 65, 4, 7, 0]
LONG = [3, 700, 0, 300, 257, 256, 1, 128]  # split rows: blocks of 32 edges, cut at any place


class Problem:
    """Inputs on the GPU and as float64 arrays.  pad: columns behind the heads of a projection (None: separate tensors)."""

    def __init__(self, heads, dim, vdim, dtype, degrees, pad=None, n_src=None, masked=0.0, seed=0, biased=True):
        import torch

        rng = np.random.default_rng(seed)
        n = len(degrees)
        n_src = n if n_src is None else n_src
        self.bf16, self.dtype = dtype == "bf16", torch.bfloat16 if dtype == "bf16" else torch.float32
        self.off, self.src, self.dst, self.send_off, self.send_edges = graph(rng, degrees, n_src)
        H, E = heads, len(self.src)

        def heads_of(rows, cols):
            a = torch.from_numpy(rng.standard_normal((rows, H * cols + (pad or 0))).astype(np.float32)).to(self.dtype).cuda()
            return a[:, :H * cols].unflatten(1, (H, cols)) if pad is not None else a.reshape(rows, H, cols)

        self.q, self.k, self.v, self.g = heads_of(n, dim), heads_of(n_src, dim), heads_of(n_src, vdim), heads_of(n, vdim)
        self.bias = None
        if biased:
            b = rng.standard_normal((E, H)).astype(np.float32)
            if masked:
                b[rng.random((E, H)) < masked] = -np.inf
                b[self.off[2]:self.off[3]] = -np.inf  # a row without an edge left
            self.bias = torch.from_numpy(b).cuda()
        up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.graph = (up(self.off), up(self.src))
        self.senders = (up(self.dst), up(self.send_off), up(self.send_edges))

    def host_args(self):
        return [host(t) for t in (self.q, self.k, self.v)] + [self.off, self.src, None if self.bias is None else host(self.bias)]

    def forward(self, eq, **kw):
        return eq.eqmp_edge_attention(self.q, self.k, self.v, *self.graph, bias=self.bias, need=("out", "stats"), **kw)

    def backward(self, eq, stats, **kw):
        kw.setdefault("need", ("q", "k", "v", "bias"))
        return eq.eqmp_edge_attention_backward(self.g, self.q, self.k, self.v, stats, *self.graph, *self.senders, bias=self.bias,
                                               **kw)

    def check(self, eq, scale=None):
        got = self.forward(eq, scale=scale)
        want, bound = forward_bounds(*self.host_args(), scale, self.bf16)
        assert worst(host(got["out"]), want[0], bound[0]) <= 1
        assert worst(host(got["stats"]), want[1], bound[1]) <= 1
        grads = self.backward(eq, got["stats"], scale=scale)
        want, bound = backward_bounds(host(self.g), *self.host_args()[:3], host(got["stats"]), *self.host_args()[3:], scale, self.bf16)
        for name in ("q", "k", "v", "bias"):
            assert worst(host(grads[name]), want[name], bound[name]) <= 1, name
        return got, grads


SHAPES = [(1, 1, 1), (4, 18, 50), (2, 65, 30), (4, 6, 10), (4, 16, 128), (8, 32, 128), (3, 5, 49), (2, 64, 256), (5, 18, 100), (1, 256, 1024), (12, 8, 16),
          (6, 24, 72), (16, 4, 4), (2, 33, 300), (3, 128, 512), (8, 32, 256), (33, 8, 8)]


@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_the_oracle(eq, shape, dtype, degrees):
    Problem(*shape, dtype, degrees, seed=sum(shape)).check(eq)


@pytest.mark.parametrize("pad", [0, 1, 2, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_of_a_projection(eq, dtype, pad):
    Problem(4, 16, 48, dtype, MIXED, pad=pad).check(eq)


@pytest.mark.parametrize("masked", [0.1, 0.9])
@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
@pytest.mark.parametrize("shape", [(4, 16, 128), (3, 5, 49)], ids=str)
def test_masked_edges(eq, shape, degrees, masked):
    Problem(*shape, "f32", degrees, masked=masked).check(eq)


@pytest.mark.parametrize("degrees,n_src", [([0], 1), ([1], 1), ([0, 0, 0], 4), ([5], 9), ([2, 1], 1), ([700], 3), ([0, 400, 400], 500)],
                         ids=str)
def test_small_and_uneven_graphs(eq, degrees, n_src):
    """Rows of no and of one edge, other numbers of senders than of receivers, one long row, senders of many edges."""
    for dtype in ("f32", "bf16"):
        Problem(4, 16, 32, dtype, degrees, n_src=n_src).check(eq)
        Problem(3, 7, 9, dtype, degrees, n_src=n_src, biased=False).check(eq, scale=-0.3)


def test_no_receivers_or_no_senders(eq):
    import torch

    p = Problem(4, 16, 32, "f32", [0, 0])
    got = eq.eqmp_edge_attention(p.q[:0], p.k, p.v, p.graph[0][:1], p.graph[1], need=("out", "stats"))
    assert got["out"].shape == (0, 4, 32) and got["stats"].shape == (0, 4, 2)
    g = eq.eqmp_edge_attention_backward(p.g[:0], p.q[:0], p.k, p.v, got["stats"], p.graph[0][:1], p.graph[1], *p.senders)
    assert not g["k"].any() and not g["v"].any() and g["k"].shape == (2, 4, 16) and g["q"].shape == (0, 4, 16)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = eq.eqmp_edge_attention(p.q, p.k[:0], p.v[:0], p.graph[0], p.graph[1], need=("out", "stats"))
    assert not got["out"].any() and not got["stats"].any()
    g = eq.eqmp_edge_attention_backward(p.g, p.q, p.k[:0], p.v[:0], got["stats"], p.graph[0], p.graph[1], p.senders[0], one,
                                        p.senders[2])
    assert not g["q"].any() and g["k"].shape == (0, 4, 16)


@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
@pytest.mark.parametrize("shape", [(4, 16, 32), (3, 7, 9)], ids=str)
def test_what_masked_edges_hold_is_not_seen(eq, shape, degrees):
    """NaN and infinities in the rows of a sender whose edges are all masked, and in a receiver without an edge: no result
    of another row holds them, and everything else is as with zeros there, to the bit."""
    import torch

    a, b = (Problem(*shape, "f32", degrees, seed=5) for _ in range(2))
    hidden, empty = int(a.src[a.off[3]]), 1
    for p, bad in ((a, 0.0), (b, float("nan"))):
        p.bias[torch.from_numpy(p.src == hidden).cuda()] = -float("inf")
        p.bias[p.off[empty]:p.off[empty + 1]] = -float("inf")
        p.k[hidden], p.v[hidden] = bad, bad
        p.q[empty], p.g[empty] = bad, bad
    b.k[hidden, :, 0] = float("inf")
    x, y = a.forward(eq), b.forward(eq)
    gx, gy = a.backward(eq, x["stats"]), b.backward(eq, y["stats"])
    for name in x:
        assert torch.equal(x[name], y[name]), name
    for name in gx:
        assert torch.equal(gx[name], gy[name]), name
    assert not y["out"][empty].any() and not gy["q"][empty].any() and not gy["k"][hidden].any() and not gy["v"][hidden].any()


def test_masks_of_the_lowest_value_are_numbers(eq):
    """Rows of nothing but the lowest value are spread evenly, beside others they vanish; both passes."""
    import torch

    low = torch.finfo(torch.float32).min
    p = Problem(2, 8, 16, "f32", [4, 5], seed=1)
    p.bias.zero_()
    p.bias[:4] = low
    p.bias[4] = low
    got = p.forward(eq)
    for i, edges in ((0, range(4)), (1, range(5, 9))):
        vs = torch.stack([p.v[int(p.src[e])] for e in edges])
        if i == 0:  # the lowest value takes the scores in: equal weights
            assert torch.allclose(got["out"][0], vs.mean(0), rtol=1e-5, atol=1e-6)
            assert (got["stats"][0, :, 1] == 4).all()
        else:
            rest = eq.eqmp_edge_attention(p.q[1:], p.k, p.v, torch.tensor([0, 4], device="cuda", dtype=torch.int32),
                                          p.graph[1][5:].contiguous())
            assert torch.allclose(got["out"][1], rest["out"][0], rtol=1e-5, atol=1e-6)
    p.check(eq)


def test_nan_and_infinity_stay_in_their_row_and_head(eq):
    import torch

    for bad in (float("nan"), float("inf")):
        p = Problem(4, 16, 32, "f32", MIXED, seed=7)
        clean = p.forward(eq)
        row, head = 9, 2
        p.bias[p.off[row] + 3, head] = bad
        got = p.forward(eq)
        assert torch.isnan(got["out"][row, head]).all()
        got["out"][row, head] = clean["out"][row, head]
        assert torch.equal(got["out"], clean["out"])
        g = p.backward(eq, got["stats"])
        touched = torch.zeros(len(p.off) - 1, dtype=torch.bool, device="cuda")
        touched[torch.from_numpy(p.src[p.off[row]:p.off[row + 1]]).long().cuda()] = True
        assert torch.isnan(g["q"][row, head]).all() and torch.isfinite(g["q"][:row]).all() and torch.isfinite(g["v"][~touched]).all()
        assert torch.isfinite(g["v"][:, [0, 1, 3]]).all() and torch.isfinite(g["bias"][:, [0, 1, 3]]).all()


def test_senders_outside_read_as_zeros(eq):
    import torch

    p = Problem(3, 8, 12, "f32", MIXED, seed=2)
    p.src[[1, 40, 50]] = [-1, 15, 2 ** 31 - 1]
    p.graph = (p.graph[0], torch.from_numpy(p.src).cuda())
    got = p.forward(eq)
    want, bound = forward_bounds(*p.host_args(), None, False)
    assert worst(host(got["out"]), want[0], bound[0]) <= 1 and worst(host(got["stats"]), want[1], bound[1]) <= 1
    g = p.backward(eq, got["stats"], need=("q", "bias"))
    want, bound = backward_bounds(host(p.g), *p.host_args()[:3], host(got["stats"]), *p.host_args()[3:], None, False)
    assert worst(host(g["q"]), want["q"], bound["q"]) <= 1 and worst(host(g["bias"]), want["bias"], bound["bias"]) <= 1


@pytest.mark.parametrize("need", [("q",), ("k",), ("v",), ("bias",), ("q", "bias"), ("k", "v")], ids=str)
@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
def test_each_gradient_alone(eq, degrees, need):
    import torch

    p = Problem(4, 16, 32, "f32", degrees, masked=0.1)
    stats = p.forward(eq)["stats"]
    every, some = p.backward(eq, stats), p.backward(eq, stats, need=need)
    assert set(some) == set(need) and all(torch.equal(every[k], some[k]) for k in need)
    if "k" not in need and "v" not in need:  # the sender view is not needed
        some = eq.eqmp_edge_attention_backward(p.g, p.q, p.k, p.v, stats, *p.graph, None, None, None, bias=p.bias, need=need)
        assert all(torch.equal(every[k], some[k]) for k in need)


def test_receiver_ranges(eq):
    """Part of the receivers by pointer offsets, as the layer's shards: the same rows to the bit, gradients that add up, and
    zeros for the bias of other edges; what lies behind the results is left as it was."""
    import torch

    p = Problem(4, 16, 32, "f32", MIXED, seed=3)
    whole = p.forward(eq)
    grads = p.backward(eq, whole["stats"])
    n, total = len(MIXED), None
    for a, b in ((0, 6), (6, n)):
        room = torch.full((b - a + 3, 4, 32), 7.0, device="cuda")
        got = eq.eqmp_edge_attention(p.q[a:b], p.k, p.v, p.graph[0][a:b + 1], p.graph[1], bias=p.bias, need=("out", "stats"),
                                     out=dict(out=room[:b - a]))
        assert torch.equal(got["out"], whole["out"][a:b]) and torch.equal(got["stats"], whole["stats"][a:b])
        assert (room[b - a:] == 7).all()
        mine = (p.dst >= a) & (p.dst < b)
        edges = p.send_edges[mine[p.send_edges]]
        send_off = np.searchsorted(p.src[edges], np.arange(n + 1)).astype(np.int32)
        part = eq.eqmp_edge_attention_backward(p.g[a:b], p.q[a:b], p.k, p.v, got["stats"], p.graph[0][a:b + 1], p.graph[1],
                                               p.senders[0] - a, torch.from_numpy(send_off).cuda(), torch.from_numpy(edges).cuda(),
                                               bias=p.bias, need=("q", "k", "v", "bias"))
        mine = torch.from_numpy(mine).cuda()
        assert torch.equal(part["q"], grads["q"][a:b]) and torch.equal(part["bias"][mine], grads["bias"][mine])
        assert not part["bias"][~mine].any()
        alone = eq.eqmp_edge_attention_backward(p.g[a:b], p.q[a:b], p.k, p.v, got["stats"], p.graph[0][a:b + 1], p.graph[1], None,
                                                None, None, bias=p.bias, need=("bias",))
        assert torch.equal(alone["bias"], part["bias"])
        total = part if total is None else {k: total[k] + part[k] for k in ("k", "v")}
    assert all(torch.allclose(total[k], grads[k], rtol=1e-5, atol=1e-5) for k in ("k", "v"))


def test_one_node_for_all(eq):
    """Strides of 0: a query and an upstream gradient that every receiver shares."""
    import torch

    p = Problem(4, 16, 32, "f32", MIXED)
    p.q, p.g = p.q[3:4].expand(len(MIXED), -1, -1), p.g[3:4].expand(len(MIXED), -1, -1)
    p.check(eq)
    v = p.v.transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError, match="contiguous heads"):
        eq.eqmp_edge_attention(p.q, p.k, v, *p.graph)
    assert torch.equal(p.forward(eq)["out"], p.forward(eq)["out"])


def test_unaligned_memory(eq):
    """Tensors that begin anywhere, and the same values on 16 bytes: the same to the tolerance of both."""
    import torch

    p = Problem(4, 16, 32, "bf16", MIXED)
    off = lambda t: torch.cat((t.new_zeros(1), t.flatten()))[1:].view(t.shape)  # noqa: E731
    p.q, p.k, p.v, p.g = off(p.q), off(p.k), off(p.v), off(p.g)
    assert p.q.data_ptr() % 16
    p.check(eq)


def test_the_same_again_and_captured(eq):
    """Bitwise the same twice, on another stream, and replayed from a graph with new inputs in place."""
    import torch

    for degrees in (MIXED, LONG):
        p = Problem(8, 32, 128, "f32", degrees, masked=0.1)
        first = p.forward(eq)
        grads = p.backward(eq, first["stats"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        again = p.forward(eq, stream=side)
        regrads = p.backward(eq, again["stats"], stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], again[k]) for k in first) and all(torch.equal(grads[k], regrads[k]) for k in grads)
        tape = torch.cuda.CUDAGraph()
        with torch.cuda.graph(tape):
            out = p.forward(eq)
            back = p.backward(eq, out["stats"])
        tape.replay()
        assert all(torch.equal(first[k], out[k]) for k in out) and all(torch.equal(grads[k], back[k]) for k in back)
        p.q.mul_(0.5)
        tape.replay()
        want = p.forward(eq)
        assert torch.equal(out["out"], want["out"]) and not torch.equal(out["out"], first["out"])


def test_node_features_as_values(eq):
    """Features [N, C, 16] seen as [N, H, 16 C / H], rotated: the result turns with them."""
    import torch

    from tests.rotations import random_rotation, rotate_features, wigner_d_blocks

    p = Problem(4, 16, 128, "f32", MIXED, seed=8)
    n, blocks = len(MIXED), wigner_d_blocks(random_rotation(3))
    x = p.v.reshape(n, 32, 16)
    turned = torch.from_numpy(rotate_features(host(x), blocks).astype(np.float32)).cuda()
    out = eq.eqmp_edge_attention(p.q, p.k, x.view(n, 4, 128), *p.graph, bias=p.bias)["out"].view(n, 32, 16)
    out_turned = eq.eqmp_edge_attention(p.q, p.k, turned.view(n, 4, 128), *p.graph, bias=p.bias)["out"].view(n, 32, 16)
    # the rotation's rounding to fp32 and two results of bounded error: 1e-5 of values of order 1
    assert np.abs(host(out_turned) - rotate_features(host(out), blocks)).max() < 1e-5


def test_gradients_against_differences(eq):
    """Along random directions, by the float64 oracle's loss; 1e-3 of |grad| |d| covers the fp32 gradients' 1e-5 or so and the
    differences' 1e-8."""
    p = Problem(3, 8, 12, "f32", MIXED, masked=0.1, seed=4)
    got = p.forward(eq)
    grads = p.backward(eq, got["stats"])
    rng = np.random.default_rng(0)
    q, k, v, off, src, bias = p.host_args()
    args, g = dict(q=q, k=k, v=v, bias=bias), host(p.g)
    loss = lambda a: (at.edge_attention(a["q"], a["k"], a["v"], off, src, a["bias"])[0] * g).sum()  # noqa: E731
    for name in args:
        d = rng.standard_normal(args[name].shape)
        step = lambda t: loss({**args, name: args[name] + t * d})  # noqa: B023,E731
        diff, grad = (step(1e-5) - step(-1e-5)) / 2e-5, host(grads[name])
        assert abs(diff - (grad * d).sum()) <= 1e-3 * np.sqrt((grad ** 2).sum() * (d ** 2).sum() / grad.size), name


def test_edges_without_any_sender(eq):
    """Receivers with edges and no node that sends: all senders read as zeros, so the weights are those of the bias."""
    import torch

    p = Problem(4, 16, 32, "f32", [3, 0, 5])
    got = eq.eqmp_edge_attention(p.q, p.k[:0], p.v[:0], *p.graph, bias=p.bias, need=("out", "stats"))
    rows = [p.bias[:3], p.bias[3:8]]
    for i, b in ((0, rows[0]), (2, rows[1])):
        m = b.max(0).values
        assert torch.equal(got["stats"][i, :, 0], m)
        assert torch.allclose(got["stats"][i, :, 1], (b - m).exp().sum(0), rtol=1e-6)
    assert not got["out"].any() and not got["stats"][1].any()


def test_offsets_beyond_32_bits(eq):
    """Nodes whose keys and values lie more than 2^31 elements into their tensors, and rows more than 2^32 bytes apart."""
    import torch

    H, D, V, n = 8, 32, 1024, 300_000  # values: 2.4e9 elements
    v = torch.zeros(n, H, V, dtype=torch.bfloat16, device="cuda")
    far = [0, 1, 131072, 262143, n - 2, n - 1]
    gen = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.randn(len(far), H, V, generator=gen, device="cuda").bfloat16()
    v[far] = rows
    k = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
    k[far] = torch.randn(len(far), H, D, generator=gen, device="cuda").bfloat16()
    q = torch.randn(2, H, D, generator=gen, device="cuda").bfloat16()
    off, src = torch.tensor([0, 6, 6], dtype=torch.int32, device="cuda"), torch.tensor(far, dtype=torch.int32, device="cuda")
    got = eq.eqmp_edge_attention(q, k, v, off, src, need=("out", "stats"))
    near = eq.eqmp_edge_attention(q, k[far].contiguous(), rows, off, torch.arange(6, dtype=torch.int32, device="cuda"), need=("out", "stats"))
    assert torch.equal(got["out"], near["out"]) and torch.equal(got["stats"], near["stats"])
    # the same nodes as receivers of the gradients
    g = torch.randn(2, H, V, generator=gen, device="cuda").bfloat16()
    send_off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    for i, node in enumerate(far):
        send_off[node + 1:] = i + 1
    back = eq.eqmp_edge_attention_backward(g, q, k, v, got["stats"], off, src, torch.zeros(6, dtype=torch.int32, device="cuda"), send_off,
                                           torch.arange(6, dtype=torch.int32, device="cuda"), need=("v",))["v"]
    p = (q[0].float()[None] * k[far].float()).sum(2) * D ** -0.5
    p = torch.softmax(p, 0)[:, :, None] * g[0].float()
    assert torch.allclose(back[far].float(), p, rtol=2 ** -7, atol=1e-6)
    back[far] = 0
    assert not back.any()
    del back, v
    wide = torch.zeros(3, 2 ** 31, dtype=torch.bfloat16, device="cuda")  # 4 GB from row to row
    wide[:, :H * D] = torch.randn(3, H * D, generator=gen, device="cuda").bfloat16()
    kw = wide[:, :H * D].unflatten(1, (H, D))
    src3, off3 = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, 3, 3], dtype=torch.int32, device="cuda")
    vv = torch.randn(3, H, 64, generator=gen, device="cuda").bfloat16()
    a, b = (eq.eqmp_edge_attention(q, t, vv, off3, src3)["out"] for t in (kw, kw.contiguous()))
    assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-6)


def test_two_calls_at_once(eq):
    """Calls on two waiting streams and two recorded graphs replayed together: each has its own memory, results as alone."""
    import torch

    a, b = Problem(8, 32, 128, "f32", MIXED * 8, seed=1), Problem(8, 32, 128, "f32", LONG * 4, seed=2)
    want = []
    for p in (a, b):
        f = p.forward(eq)
        want.append((f, p.backward(eq, f["stats"])))
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        with torch.cuda.stream(s):
            torch.cuda._sleep(5_000_000)
    got = []
    for p, s in zip((a, b), sides):
        f = p.forward(eq, stream=s)
        got.append((f, p.backward(eq, f["stats"], stream=s)))
    torch.cuda.synchronize()
    tapes, held = [], []
    for p in (a, b):
        tape = torch.cuda.CUDAGraph()
        with torch.cuda.graph(tape):
            f = p.forward(eq)
            held.append((f, p.backward(eq, f["stats"])))
        tapes.append(tape)
    for tape, s in zip(tapes, sides):
        with torch.cuda.stream(s):
            torch.cuda._sleep(5_000_000)
            tape.replay()
    torch.cuda.synchronize()
    for results in (got, held):
        for (f, g), (f0, g0) in zip(results, want):
            assert all(torch.equal(f[k], f0[k]) for k in f0) and all(torch.equal(g[k], g0[k]) for k in g0)


def test_temporaries_outlive_the_call(eq):
    """The workspaces of calls that wait on a side stream are not handed to the current one."""
    import torch

    from tests.test_gpu_streams import _busy_sides

    p = Problem(4, 16, 32, "f32", LONG, masked=0.1)
    f = p.forward(eq)
    want = p.backward(eq, f["stats"])
    torch.cuda.synchronize()
    side, = _busy_sides(1)
    got = p.backward(eq, f["stats"], stream=side)
    E = len(p.src)
    sizes = [eq.eqmp_edge_attention_backward_workspace_size(len(LONG), E, E, 4, 16, 32)] * 4 + [v.numel() * 4 for v in want.values()] * 4
    taken = [torch.full((n // 4,), float("nan"), device="cuda") for n in sizes]
    torch.cuda.synchronize()
    assert all(torch.isnan(t).all() for t in taken) and all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("shape", [(4, 16, 32), (3, 7, 9)], ids=str)
def test_a_graph_that_is_none_does_no_harm(eq, shape):
    """Offsets that go up and down and lie outside, senders, receivers and edge numbers of any value: indices are clamped or
    their edges left out, so the results are some numbers and the next call is sound."""
    import torch

    p = Problem(*shape, "f32", LONG, seed=9)
    good = p.forward(eq)
    rng = np.random.default_rng(1)
    E, n = len(p.src), len(LONG)
    up = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    wild = lambda k: up(rng.integers(-2 ** 31, 2 ** 31, k))  # noqa: E731
    near = lambda lo, hi, k: up(rng.integers(lo, hi, k))  # noqa: E731
    for off, src, senders in ((near(-50, E + 50, n + 1), near(-3, n + 3, E), (near(-3, n + 3, E), near(-50, E + 50, n + 1), near(-9, E + 9, E))),
                              (wild(n + 1), wild(E), (wild(E), wild(n + 1), wild(E)))):
        got = eq.eqmp_edge_attention(p.q, p.k, p.v, off, src, bias=p.bias, need=("out", "stats"))
        back = eq.eqmp_edge_attention_backward(p.g, p.q, p.k, p.v, got["stats"], off, src, *senders, bias=p.bias,
                                               need=("q", "k", "v", "bias"))
        torch.cuda.synchronize()
        assert got["out"].shape == good["out"].shape and back["bias"].shape == (E, shape[0])
    again = p.forward(eq)
    assert torch.equal(again["out"], good["out"])


@pytest.mark.parametrize("shape", [(4, 16, 128), (3, 6, 10), (2, 5, 49), (5, 7, 9)], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_only_edge_of_a_receiver(eq, shape, dtype):
    """Its weight is 1 whatever the score: the value is the result, and nothing but the value has a gradient, with the pass's own
    statistics and with those of another order of the sums."""
    import torch

    p = Problem(*shape, dtype, [1, 1, 3, 1, 0, 1], seed=4)
    p.bias[2:4] = -float("inf")  # the third row keeps one of its three edges
    got = p.forward(eq)
    for i, e in enumerate([0, 1, 4, 5, None, 6]):
        if e is not None:
            assert torch.equal(got["out"][i], p.v[int(p.src[e])])
    for stats in (got["stats"], torch.stack((got["stats"][:, :, 0] * (1 + 2.0 ** -22), got["stats"][:, :, 1]), 2)):
        g = p.backward(eq, stats)
        assert not g["q"].any() and not g["k"].any() and not g["bias"].any() and g["v"].any()
