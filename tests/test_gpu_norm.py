"""GPU parity of dropout, the layer norm and the norm by degree, and of their
gradients, against the float64 oracle within derived bounds (norm_util)."""
import numpy as np
import pytest

from oracle import norm
from tests import norm_util as nu
from tests.gpu_util import host
from tests.rotations import random_rotation, rotate_features, wigner_d_blocks

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x9E3779B97F4A7C15, (1 << 40) + 5


@pytest.fixture(scope="module")
def eq():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    import equivariant_gnn_message_gb300 as m

    torch.cuda.set_device(0)
    return m


def _up(a, dtype, pad=0, shift=0):
    """a on the GPU, its rows `pad` elements apart and its first element `shift` elements behind an aligned address."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)
    if not pad and not shift:
        return t
    n = t.shape[0]
    width = t[0].numel() if n else int(np.prod(t.shape[1:]))
    buf = torch.full((n * (width + pad) + shift + 16,), float("nan"), device="cuda", dtype=dtype)
    v = buf[shift:shift + n * (width + pad)].view(n, width + pad)[:, :width]
    v.copy_(t.reshape(n, width))
    return v if t.dim() == 2 else v.view(t.shape) if pad == 0 else v


def _rows(shape, rng, scale=1.0):
    """Rows with a mean and a spread of their own; one constant and one zero row among several."""
    n = shape[0]
    a = rng.standard_normal(shape) * np.exp(0.5 * rng.standard_normal((n,) + (1,) * (len(shape) - 1)))
    if len(shape) == 2:
        a += 3 * rng.standard_normal((n, 1))
    if n > 4:
        a[2], a[3] = 0.75, 0.0
    return a * scale


class Case:
    """The inputs of one call on the host (as stored) and on the GPU."""

    def __init__(self, shape, bf16=False, residual=False, p=0.0, group=1, pad=0, shift=0, affine=True, seed=0):
        import torch

        rng = np.random.default_rng(seed + 1000 * shape[0] + shape[1])
        self.dtype = torch.bfloat16 if bf16 else torch.float32
        self.shape, self.bf16, self.p = shape, bf16, p
        K = shape[2] if len(shape) == 3 else 1
        self.l_max = int(round(np.sqrt(K))) - 1
        self.degree = len(shape) == 3
        group = K if self.degree else group
        up = lambda a: _up(a, self.dtype, pad, shift)  # noqa: E731
        self.x, self.r, self.g = (up(_rows(shape, rng, s)) for s in (1.0, 1.0, 0.3))
        self.r = self.r if residual else None
        f32 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
        wshape = (self.l_max + 1, shape[1]) if self.degree else (shape[1],)
        self.w = f32(1 + 0.5 * rng.standard_normal(wshape)) if affine else None
        self.b = f32(0.5 * rng.standard_normal(shape[1])) if affine else None
        self.eps = 1e-5
        self.factor = norm.drop_factor(shape[0], int(np.prod(shape[1:])), p, SEED, OFFSET, group) if p else None
        self.args = dict(p=p, seed=SEED, offset=OFFSET, group=group)

    def drop(self, eq):
        return eq.Dropout(**self.args) if self.p else None

    def forward(self, eq, need=("y", "s", "stats"), **kw):
        fn = eq.eqmp_degree_norm if self.degree else eq.eqmp_layer_norm
        return fn(self.x, self.w, self.b, eps=self.eps, residual=self.r, drop=self.drop(eq), need=need, **kw)

    def forward_bounds(self):
        h = lambda t: None if t is None else host(t)  # noqa: E731
        return nu.forward_bounds(host(self.x), h(self.w), h(self.b), self.eps, h(self.r), self.factor, self.bf16)

    def backward(self, eq, s, stats, need=("x", "r", "w", "b"), **kw):
        fn = eq.eqmp_degree_norm_backward if self.degree else eq.eqmp_layer_norm_backward
        return fn(self.g, s, stats, self.w, grad_s=self.r, drop=self.drop(eq), need=need, **kw)

    def backward_bounds(self, s, stats):
        h = lambda t: None if t is None else host(t)  # noqa: E731
        return nu.backward_bounds(host(self.g), host(s), host(stats), h(self.w), h(self.r), self.factor, self.bf16)


def _check(got, want, bounds):
    for k, v in got.items():
        assert tuple(v.shape) == want[k].shape, k
        e = nu.worst(host(v), want[k], bounds[k])
        assert e <= 1.0, f"{k}: {e:.3g} of its bound"


# rows, cols: one value, below and around each power of two of lanes, vector and scalar rows, several threads per row,
# more than a CTA holds
ROWS = [(1, 1), (7, 1), (300, 2), (5, 3), (129, 8), (64, 16), (33, 24), (500, 31), (64, 64), (9, 100), (65, 131), (40, 256),
        (31, 509), (19, 1000), (16, 1024), (5, 1025), (6, 2048), (4, 4096), (3, 4099), (2, 8192), (5, 8200), (3, 16392),
        (2, 20000), (1, 70001)]
FORMS = [dict(), dict(bf16=True), dict(residual=True, p=0.3), dict(bf16=True, residual=True, p=0.3),
         dict(p=0.5, affine=False), dict(bf16=True, residual=True, pad=8), dict(residual=True, p=0.1, pad=5),
         dict(bf16=True, residual=True, p=0.1, shift=1)]


def _id(v):
    return "_".join(f"{k}{x}" for k, x in v.items()) or "plain" if isinstance(v, dict) else None


@pytest.mark.parametrize("form", FORMS, ids=_id)
@pytest.mark.parametrize("rows,cols", ROWS)
def test_layer_norm_parity(eq, rows, cols, form):
    c = Case((rows, cols), **form)
    got = c.forward(eq)
    want, bounds = c.forward_bounds()
    _check(got, want, bounds)
    back = c.backward(eq, got["s"], got["stats"])
    _check(back, *c.backward_bounds(got["s"], got["stats"]))


@pytest.mark.parametrize("form", [dict(), dict(residual=True, p=0.2), dict(bf16=True, residual=True, p=0.2)], ids=_id)
@pytest.mark.parametrize("cols", [6148, 6852, 8064, 48, 96, 768, 900, 1024, 1536, 6147])
def test_widths_between_lane_counts(eq, cols, form):
    """Widths at which the number of values a lane holds changes, up to the most lanes that a row may have."""
    c = Case((301, cols), **form)
    got = c.forward(eq)
    _check(got, *c.forward_bounds())
    _check(c.backward(eq, got["s"], got["stats"]), *c.backward_bounds(got["s"], got["stats"]))


FEATURES = [(1, 1, 16), (7, 3, 16), (100, 8, 16), (33, 32, 16), (9, 128, 16), (3, 300, 16), (64, 5, 25), (17, 32, 25),
            (5, 64, 36), (31, 7, 36), (20, 32, 49), (3, 129, 49), (2, 400, 49), (700, 4, 16), (2, 1100, 16)]


@pytest.mark.parametrize("form", [f for f in FORMS if "pad" not in f], ids=_id)
@pytest.mark.parametrize("shape", FEATURES, ids=str)
def test_degree_norm_parity(eq, shape, form):
    c = Case(shape, **form)
    got = c.forward(eq)
    _check(got, *c.forward_bounds())
    back = c.backward(eq, got["s"], got["stats"])
    _check(back, *c.backward_bounds(got["s"], got["stats"]))


@pytest.mark.parametrize("cols,group", [(48, 16), (75, 25), (98, 49), (36, 3), (30, 2), (64, 64), (1000, 8), (1024, 4)])
@pytest.mark.parametrize("bf16", [False, True])
def test_layer_norm_dropout_groups(eq, cols, group, bf16):
    c = Case((50, cols), bf16=bf16, residual=True, p=0.4, group=group)
    got = c.forward(eq)
    _check(got, *c.forward_bounds())
    _check(c.backward(eq, got["s"], got["stats"]), *c.backward_bounds(got["s"], got["stats"]))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,cols,group", [(1, 1, 1), (3, 7, 1), (1000, 8, 1), (257, 64, 1), (33, 131, 1), (5, 1000, 8),
                                             (50, 512, 16), (20, 800, 25), (7, 49 * 32, 49), (2, 100003, 1), (3, 4096, 4096)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 0), (0, 1)])
def test_dropout_is_exact(eq, rows, cols, group, bf16, pad, shift):
    """A kept value is x times the scale, rounded once in fp32 (and once more to bf16); a dropped one is 0."""
    import torch

    dtype = torch.bfloat16 if bf16 else torch.float32
    x = _up(np.random.default_rng(cols).standard_normal((rows, cols)), dtype, pad, shift)
    out = eq.eqmp_dropout(x, eq.Dropout(p=0.25, seed=SEED, offset=OFFSET, group=group))
    f = torch.from_numpy(norm.drop_factor(rows, cols, 0.25, SEED, OFFSET, group)).cuda()
    assert out.is_contiguous() and torch.equal(out, torch.where(f > 0, x.float() * f.float(), 0.0).to(dtype))


def test_dropout_ends_of_the_rate_and_in_place(eq):
    import torch

    x = torch.randn(50, 33, device="cuda")
    x[0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0])
    assert torch.equal(eq.eqmp_dropout(x[1:], None), x[1:])
    assert torch.equal(eq.eqmp_dropout(x[1:], eq.Dropout(p=2.0 ** -18, seed=3)), x[1:])
    assert torch.equal(eq.eqmp_dropout(x, eq.Dropout(p=1.0, seed=3)), torch.zeros_like(x))
    d = eq.Dropout(p=0.5, seed=3, offset=9)
    want = eq.eqmp_dropout(x, d)
    kept = norm.drop_factor(50, 33, 0.5, 3, 9) > 0
    assert np.array_equal(np.isfinite(host(want[:1, :3])), ~kept[:1, :3])
    y = x.clone()
    assert eq.eqmp_dropout(y, d, out=y) is y and torch.equal(y.nan_to_num(), want.nan_to_num())
    with pytest.raises(eq.EqmpError):  # a shifted overlap is refused
        eq.eqmp_dropout(x[:49], d, out=x[1:])


def test_dropped_values_do_not_reach_the_norm(eq):
    """NaN and infinity in dropped places change nothing, forward and backward; elsewhere they stay in their row."""
    import torch

    c = Case((20, 64), residual=True, p=0.5)
    want = c.forward(eq)
    dead = torch.from_numpy(c.factor == 0).cuda()
    c.x = torch.where(dead, torch.tensor(float("nan"), device="cuda"), c.x)
    got = c.forward(eq)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    c.r = c.r.clone()
    c.r[5, 3], c.r[6, 3] = float("nan"), float("inf")
    got = c.forward(eq)
    ok = [i for i in range(20) if i not in (5, 6)]
    assert torch.equal(got["y"][ok], want["y"][ok]) and not got["y"][[5, 6]].isfinite().any()
    # the gradient of a dropped place is 0 whatever reaches it from the residual stream
    gs = torch.full((20, 64), float("inf"), device="cuda")
    got = eq.eqmp_layer_norm_backward(c.g, want["s"], want["stats"], c.w, grad_s=gs, drop=c.drop(eq), need=("x", "r"))
    assert (got["x"][dead] == 0).all() and got["x"][~dead].isinf().all() and got["r"].isinf().all()


@pytest.mark.parametrize("shape", [(1, 8), (64, 64), (3, 5000), (10, 7, 16), (4, 9, 49)], ids=str)
def test_gradients_match_differences(eq, shape):
    """Directional differences of the float64 forward pass against the GPU gradients: a quadratic error in the step
    (1e-5, third derivatives of order 1 to 100) and the gradients' own fp32 error leave 1e-4 of the gradient's size."""
    c = Case(shape, residual=True, p=0.3)
    c.eps = 0.1
    rng = np.random.default_rng(5)
    fw = c.forward(eq)
    x, r, w, b, g = (host(t) for t in (c.x, c.r, c.w, c.b, c.g))
    got = c.backward(eq, fw["s"], fw["stats"])  # c.r is also the gradient that reaches s

    def loss(x, r_in, w, b):
        f = norm.forward(x, w, b, c.eps, r_in, c.factor)
        return float((f["y"] * g).sum() + (f["s"] * r).sum())

    args = [x, r, w, b]
    for i, k in enumerate(("x", "r", "w", "b")):
        d = rng.standard_normal(args[i].shape)
        up, down = ([a + t * 1e-5 * d if j == i else a for j, a in enumerate(args)] for t in (1, -1))
        grad = host(got[k])
        assert abs((loss(*up) - loss(*down)) / 2e-5 - (grad * d).sum()) <= 1e-4 * np.sqrt((grad ** 2).sum() * (d ** 2).sum()), k


@pytest.mark.parametrize("l_max", [3, 6])
def test_degree_norm_commutes_with_rotations(eq, l_max):
    """norm(R x) = R norm(x) with whole channels dropped, to the fp32 error of rows of order 1 (100 u)."""
    c = Case((12, 16, (l_max + 1) ** 2), p=0.3)
    blocks = wigner_d_blocks(random_rotation(8), l_max=l_max)
    y = host(c.forward(eq, need=("y",))["y"])
    scale = np.abs(y).max()
    c.x = _up(rotate_features(host(c.x), blocks), c.dtype)
    assert np.abs(host(c.forward(eq, need=("y",))["y"]) - rotate_features(y, blocks)).max() <= 1e-4 * scale


def test_step_counter_and_graph_replay(eq):
    """A recorded graph draws another mask after its step counter was advanced: the one of that offset."""
    import torch

    x, step = torch.randn(40, 96, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    d = eq.Dropout(p=0.3, seed=5, offset=(1 << 32) - 2, step=step)
    out = eq.eqmp_dropout(x, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eq.eqmp_dropout(x, d, out=out)
        got = eq.eqmp_layer_norm(x, residual=x, drop=d, need=("y", "s", "stats"))
        back = eq.eqmp_layer_norm_backward(x, got["s"], got["stats"], drop=d)
    for k in (0, 1, 5):
        step.fill_(k)
        graph.replay()
        one = eq.Dropout(p=0.3, seed=5, offset=(1 << 32) - 2 + k)
        assert torch.equal(out, eq.eqmp_dropout(x, one))
        want = eq.eqmp_layer_norm(x, residual=x, drop=one, need=("y", "s", "stats"))
        assert all(torch.equal(got[n], want[n]) for n in want)
        wb = eq.eqmp_layer_norm_backward(x, want["s"], want["stats"], drop=one)
        assert all(torch.equal(back[n], wb[n]) for n in wb)


@pytest.mark.parametrize("shape", [(3000, 64), (700, 1030), (500, 32, 16), (300, 8, 49)], ids=str)
@pytest.mark.parametrize("bf16", [False, True])
def test_results_repeat_and_outputs_are_independent(eq, shape, bf16):
    """Bitwise the same again, with other results asked for, with the caller's buffers and a workspace of NaN, and on
    another stream."""
    import torch

    c = Case(shape, bf16=bf16, residual=True, p=0.2)
    a = c.forward(eq)
    for k in a:
        assert torch.equal(c.forward(eq, need=(k,))[k], a[k]), k
    g = c.backward(eq, a["s"], a["stats"])
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # NaN as fp32
    out = {k: torch.full_like(v, float("nan")) for k, v in g.items()}
    again = c.backward(eq, a["s"], a["stats"], out=out, workspace=ws)
    assert all(again[k] is out[k] and torch.equal(out[k], g[k]) for k in g)
    for k in g:
        assert torch.equal(c.backward(eq, a["s"], a["stats"], need=(k,))[k], g[k]), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = c.forward(eq)
        h = c.backward(eq, b["s"], b["stats"])
    other = c.forward(eq, stream=side)
    side.synchronize()
    assert all(torch.equal(a[k], b[k]) and torch.equal(a[k], other[k]) for k in a)
    assert all(torch.equal(g[k], h[k]) for k in g)


def test_broadcast_rows_and_no_rows(eq):
    import torch

    x = torch.randn(1, 96, device="cuda")
    y = eq.eqmp_layer_norm(x.expand(30, 96))["y"]  # a row stride of 0
    assert torch.equal(y, eq.eqmp_layer_norm(x)["y"].expand(30, 96))
    for dtype in (torch.float32, torch.bfloat16):  # a broadcast gradient, odd rows
        x, g = torch.randn(301, 77, device="cuda").to(dtype), torch.randn(1, 77, device="cuda").to(dtype)
        stats = eq.eqmp_layer_norm(x, need=("stats",))["stats"]
        got = eq.eqmp_layer_norm_backward(g.expand(301, 77), x, stats, grad_s=g.expand(301, 77), need=("x", "w", "b"))
        gg = host(g).repeat(301, 0)
        _check(got, *nu.backward_bounds(gg, host(x), host(stats), None, gg, None, dtype is torch.bfloat16))
    for shape in ((0, 96), (0, 8, 16)):
        c = Case(shape)
        got = c.forward(eq)
        assert got["y"].shape == shape and got["stats"].shape[0] == 0
        ones = {"w": torch.ones_like(c.w), "b": torch.ones_like(c.b)}
        c.backward(eq, got["s"], got["stats"], out=ones)
        assert not ones["w"].any() and not ones["b"].any()
    assert eq.eqmp_dropout(torch.empty(0, 5, device="cuda"), eq.Dropout(0.5, 1)).shape == (0, 5)


def test_many_rows_sum_of_gradients(eq):
    """200,003 rows: every CTA has many rows, and the sums over them keep their bounds."""
    for shape, bf16 in (((200003, 24), True), ((100001, 3, 16), False)):
        c = Case(shape, bf16=bf16)
        got = c.forward(eq)
        _check(c.backward(eq, got["s"], got["stats"]), *c.backward_bounds(got["s"], got["stats"]))


@pytest.mark.parametrize("form", [dict(), dict(residual=True, p=0.2), dict(bf16=True), dict(bf16=True, residual=True, p=0.2),
                                  dict(bf16=True, residual=True, p=0.2, pad=8), dict(p=0.2, pad=3)], ids=_id)
@pytest.mark.parametrize("rows,cols", [(20011, 37), (5003, 131), (6001, 509), (2503, 1022), (70001, 33), (1500, 4101)])
def test_rows_that_begin_anywhere(eq, rows, cols, form):
    """Rows of odd widths, many to a CTA: they begin at every place behind a 16-byte boundary."""
    c = Case((rows, cols), **form)
    got = c.forward(eq)
    _check(got, *c.forward_bounds())
    _check(c.backward(eq, got["s"], got["stats"]), *c.backward_bounds(got["s"], got["stats"]))


@pytest.mark.parametrize("group", [1, 3, 7, 11, 77])
@pytest.mark.parametrize("bf16", [False, True])
def test_dropout_groups_on_rows_that_begin_anywhere(eq, group, bf16):
    c = Case((3001, 231), bf16=bf16, residual=True, p=0.4, group=group)
    got = c.forward(eq)
    _check(got, *c.forward_bounds())
    _check(c.backward(eq, got["s"], got["stats"]), *c.backward_bounds(got["s"], got["stats"]))


@pytest.mark.parametrize("shape", [(3001, 5, 25), (2003, 7, 36), (1501, 13, 49), (999, 129, 25)], ids=str)
@pytest.mark.parametrize("bf16", [False, True])
def test_features_that_begin_anywhere(eq, shape, bf16):
    c = Case(shape, bf16=bf16, residual=True, p=0.3)
    got = c.forward(eq)
    _check(got, *c.forward_bounds())
    _check(c.backward(eq, got["s"], got["stats"]), *c.backward_bounds(got["s"], got["stats"]))


def test_neighbours_of_the_rows_are_not_touched(eq):
    """Results of odd rows in a larger buffer leave what lies around them, and NaN around the inputs does not enter."""
    import torch

    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(700, 203, device="cuda").to(dtype)
        wide = torch.full((700 * 203 + 64,), float("nan"), device="cuda", dtype=dtype)
        inside = wide[32:32 + x.numel()].view(700, 203)
        inside.copy_(x)
        out = torch.full_like(wide, 7.0)
        y = out[32:32 + x.numel()].view(700, 203)
        stats = torch.empty(700, 2, device="cuda")
        eq.eqmp_layer_norm(inside, need=("y", "stats"), out=dict(y=y, stats=stats))
        want = eq.eqmp_layer_norm(x, need=("y", "stats"))
        assert torch.equal(y, want["y"]) and torch.equal(stats, want["stats"])
        assert (out[:32] == 7).all() and (out[-32:] == 7).all()
        gx = out[32:32 + x.numel()].view(700, 203).fill_(7.0)
        got = eq.eqmp_layer_norm_backward(x, inside, stats, need=("x", "w"), out=dict(x=gx))
        ref = eq.eqmp_layer_norm_backward(x, x, stats, need=("x", "w"))
        assert torch.equal(gx, ref["x"]) and torch.equal(got["w"], ref["w"])
        assert (out[:32] == 7).all() and (out[-32:] == 7).all()
        pad = torch.full((700, 211 + (dtype is torch.float32)), float("nan"), device="cuda", dtype=dtype)
        pad[:, :203] = x
        # rows that lie otherwise may be summed in another order: equal within the bounds, not in every bit
        _check(eq.eqmp_layer_norm(pad[:, :203]),
               *nu.forward_bounds(host(x), None, None, 1e-5, None, None, dtype is torch.bfloat16))
        assert torch.equal(eq.eqmp_dropout(pad[:, :203], eq.Dropout(0.3, 1)), eq.eqmp_dropout(x, eq.Dropout(0.3, 1)))


def test_offsets_past_32_bits(eq):
    """More than 2^31 elements: the last rows against the oracle, and the sum of the gradient against its parts."""
    import torch

    rows, cols = 2_140_000, 1009  # 2.16e9 elements of bf16, odd rows
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for i in range(0, rows, 1 << 18):
        x[i:i + (1 << 18)].normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    got = eq.eqmp_layer_norm(x, need=("y", "stats"))
    tail = slice(rows - 100, rows)
    _check({k: got[k][tail] for k in got}, *nu.forward_bounds(host(x[tail]), None, None, 1e-5, None, None, True))
    g, stats = got.pop("y"), got.pop("stats")  # y as the gradient
    back = eq.eqmp_layer_norm_backward(g, x, stats, need=("x", "b"))
    _check(dict(x=back["x"][tail]), *nu.backward_bounds(host(g[tail]), host(x[tail]), host(stats[tail]), None, None, None, True))
    b = sum(g[i:i + (1 << 18)].double().sum(0) for i in range(0, rows, 1 << 18))
    size = sum(g[i:i + (1 << 18)].double().abs().sum(0) for i in range(0, rows, 1 << 18))
    assert ((back["b"].double() - b).abs() <= (64 + rows // 64) * nu.U * size).all()
    del back, g
    out = eq.eqmp_dropout(x, eq.Dropout(p=0.5, seed=SEED, offset=OFFSET))
    f = norm.drop_factor(100, cols, 0.5, SEED, OFFSET, first_row=rows - 100)
    assert np.array_equal(host(out[tail]), host(x[tail]) * f)


def test_refusals(eq):
    import torch

    f32 = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    x, feat = f32(4, 8), f32(4, 8, 16)
    d = eq.Dropout(p=0.1, seed=1)
    for bad, kind in ((dict(x=x.double()), TypeError), (dict(x=x.cpu()), ValueError), (dict(x=f32(4)), ValueError),
                      (dict(x=f32(4, 0)), ValueError), (dict(x=x.t()), ValueError), (dict(w=f32(7)), ValueError),
                      (dict(w=f32(8).bfloat16()), TypeError), (dict(b=f32(16)[::2]), ValueError),
                      (dict(residual=f32(3, 8)), ValueError), (dict(residual=x.bfloat16()), TypeError),
                      (dict(need=("z",)), ValueError), (dict(out={"y": f32(4, 9)}), ValueError),
                      (dict(eps=-1.0), eq.EqmpError), (dict(eps=float("nan")), eq.EqmpError),
                      (dict(drop=eq.Dropout(0.1, 1, group=3)), eq.EqmpError), (dict(out={"y": x}), eq.EqmpError),
                      (dict(need=("y", "s"), out={"y": (t := f32(4, 8)), "s": t}), eq.EqmpError)):
        with pytest.raises(kind):
            eq.eqmp_layer_norm(**{"x": x, **bad})
    for bad, kind in ((dict(x=f32(4, 8, 9)), ValueError), (dict(x=x), ValueError), (dict(x=feat.transpose(0, 1)), ValueError),
                      (dict(w=f32(4, 7)), ValueError), (dict(b=f32(4, 8)), ValueError), (dict(drop=d), eq.EqmpError)):
        with pytest.raises(kind):
            eq.eqmp_degree_norm(**{"x": feat, **bad})
    stats = f32(4, 2)
    for bad, kind in ((dict(stats=None), TypeError), (dict(stats=f32(4, 3)), ValueError), (dict(grad_y=f32(4, 9)), ValueError),
                      (dict(grad_s=x.bfloat16()), TypeError), (dict(need=("y",)), ValueError),
                      (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), eq.EqmpError),
                      (dict(out={"x": x}), eq.EqmpError)):
        with pytest.raises(kind):
            eq.eqmp_layer_norm_backward(**{"grad_y": f32(4, 8), "s": x, "stats": stats, **bad})
    for bad in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError):
            eq.Dropout(bad, 1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, offset=-1), dict(seed=1, group=0)):
        with pytest.raises(ValueError):
            eq.Dropout(0.5, **kw)
    with pytest.raises(TypeError):
        eq.Dropout(0.5, 1, step=torch.zeros(1, device="cuda"))
    with pytest.raises(TypeError):
        eq.eqmp_dropout(x.double(), d)
    with pytest.raises(TypeError):
        eq.eqmp_dropout(x, 0.1)
    with pytest.raises(TypeError):
        eq.eqmp_layer_norm(x, drop=0.1)
    row = torch.randn(1, 33, device="cuda")
    want = eq.eqmp_dropout(row, d)
    assert torch.equal(eq.eqmp_dropout(row.as_strided((1, 33), (40, 1)), d, out=row), want)  # one row, in place
    with pytest.raises(ValueError):
        eq.eqmp_dropout(x, d, out=f32(8, 4))
