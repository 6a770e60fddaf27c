"""What the entry points of the attention over edges refuse, and where the binding makes its memory: without a GPU, by
made-up addresses at the C calls (they fail their checks, or end with EQMP_ERR_CUDA) and by a stand-in under the binding."""
import itertools

import pytest
import torch

import equivariant_gnn_message_gb300 as eq
from tests.binding_util import FakeGpu
from tests.test_binding_cpu import _check_streams

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

N, NS, E, H, D, DV, B = 6, 5, 40, 4, 8, 16, 7
STEP = 1 << 22


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return eq.load_library()


class Call:
    """One entry point: its arguments by name, with defaults that pass every check, and the bytes of those in memory
    (written ones in `out`)."""

    def __init__(self, lib, name, sizes, out, order, **values):
        self.fn, self.name, self.sizes, self.out, self.order = getattr(lib, name), name, sizes, out, order
        self.values = {**{k: STEP * (i + 1) for i, k in enumerate(sizes)}, **values}

    def __call__(self, **kw):
        a = {**self.values, **kw}
        return self.fn(*[a[k] for k in self.order.split()])


def calls(lib, dtype=0):
    b = 4 if dtype == 0 else 2
    size = dict(N=N, NS=NS, E=E, H=H, D=D, DV=DV, dtype=dtype, st=0)
    yield Call(lib, "eqmp_head_norm", dict(q=N * H * D * b, k=N * 2 * D * b, wq=D * 4, wk=D * 4, pos=N * 12, freq=D // 2 * 12,
                                           oq=N * H * D * b, ok=N * 2 * D * b, rstd=N * (H + 2) * 4), ("oq", "ok", "rstd"),
               "q q_ld H k k_ld HK dtype N D wq wk eps pos freq axes oq ok rstd st", **size, q_ld=H * D, k_ld=2 * D, HK=2, eps=1e-6,
               axes=3)
    yield Call(lib, "eqmp_head_norm_backward",
               dict(yq=N * H * D * b, yk=N * 2 * D * b, q=N * H * D * b, k=N * 2 * D * b, wq=D * 4, wk=D * 4, rstd=N * (H + 2) * 4,
                    pos=N * 12, freq=D // 2 * 12, gq=N * H * D * b, gk=N * 2 * D * b, gwq=D * 4, gwk=D * 4, gpos=N * 12,
                    ws=lib.eqmp_head_norm_backward_workspace_size(N, D)), ("gq", "gk", "gwq", "gwk", "gpos", "ws"),
               "yq q_ld yk k_ld q q_ld H k k_ld HK dtype N D wq wk rstd pos freq axes gq gk gwq gwk gpos ws ws_bytes st", **size,
               q_ld=H * D, k_ld=2 * D, HK=2, axes=3, ws_bytes=lib.eqmp_head_norm_backward_workspace_size(N, D))
    yield Call(lib, "eqmp_edge_bias", dict(vec=E * 12, borders=(B - 1) * 4, table=B * H * 4, bias=E * H * 4, bucket=E * 4),
               ("bias", "bucket"), "vec E borders B table H bias bucket st", **size, B=B)
    big = 50000
    yield Call(lib, "eqmp_edge_bias_backward",
               dict(g=big * H * 4, bucket=big * 4, gt=B * H * 4, ws=lib.eqmp_edge_bias_backward_workspace_size(big, B, H)), ("gt", "ws"),
               "g bucket E B H gt ws ws_bytes st", **{**size, "E": big}, B=B,
               ws_bytes=lib.eqmp_edge_bias_backward_workspace_size(big, B, H))
    big = 1400
    rows = dict(q=N * H * D * b, k=NS * H * D * b, v=NS * H * DV * b)
    lds = dict(q_ld=H * D, v_ld=H * DV, scale=0.5)
    yield Call(lib, "eqmp_edge_attention",
               dict(rows, off=(N + 1) * 4, src=big * 4, bias=big * H * 4, o=N * H * DV * b, stats=N * H * 8,
                    ws=lib.eqmp_edge_attention_workspace_size(big, H, DV)), ("o", "stats", "ws"),
               "q q_ld k q_ld v v_ld dtype N NS E H D DV off src bias scale o stats ws ws_bytes st", **{**size, "E": big}, **lds,
               ws_bytes=lib.eqmp_edge_attention_workspace_size(big, H, DV))
    nbytes = lib.eqmp_edge_attention_backward_workspace_size(N, big, big, H, D, DV)
    yield Call(lib, "eqmp_edge_attention_backward",
               dict(rows, go=N * H * DV * b, off=(N + 1) * 4, src=big * 4, dst=big * 4, so=(NS + 1) * 4, se=big * 4, bias=big * H * 4,
                    stats=N * H * 8, gq=N * H * D * b, gk=NS * H * D * b, gv=NS * H * DV * b, gb=big * H * 4, ws=nbytes),
               ("gq", "gk", "gv", "gb", "ws"),
               "go v_ld q q_ld k q_ld v v_ld dtype N NS E H D DV off src dst so se ES bias scale stats gq gk gv gb ws ws_bytes st",
               **{**size, "E": big}, **lds, ES=big, ws_bytes=nbytes)


def _named(lib, dtype=0):
    return {c.name: c for c in calls(lib, dtype)}


NAMES = ("eqmp_head_norm", "eqmp_head_norm_backward", "eqmp_edge_bias", "eqmp_edge_bias_backward", "eqmp_edge_attention",
         "eqmp_edge_attention_backward")


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("name", NAMES)
def test_every_output_meets_nothing(lib, name, dtype):
    call = _named(lib, dtype)[name]
    assert call() == eq.EQMP_ERR_CUDA
    for a, b in itertools.combinations(call.sizes, 2):
        same = {b: call.values[a]}
        if a not in call.out and b not in call.out:
            assert call(**same) == eq.EQMP_ERR_CUDA, (a, b)
            continue
        assert call(**same) == eq.EQMP_ERR_INVALID_ARG, (a, b)
        for lower, upper in ((a, b), (b, a)):
            n = call.sizes[lower] // 16 * 16
            if n > 16:
                assert call(**{upper: call.values[lower] + n - 16}) == eq.EQMP_ERR_INVALID_ARG, (a, b)
            assert call(**{upper: call.values[lower] + (call.sizes[lower] + 15) // 16 * 16}) == eq.EQMP_ERR_CUDA, (a, b)


@pytest.mark.parametrize("name", NAMES)
def test_missing_and_misaligned_memory(lib, name):
    call = _named(lib)[name]
    optional = {"wq", "wk", "bias", "oq", "ok", "rstd", "bucket", "o", "stats", "gq", "gk", "gv", "gb", "gwq", "gwk", "gpos", "gt", "table"}
    must = {"eqmp_head_norm_backward": {"rstd"}, "eqmp_edge_attention_backward": {"stats"}, "eqmp_edge_bias": {"table"},
            "eqmp_edge_bias_backward": {"bucket"}}.get(name, set())
    for k in call.sizes:
        if k not in optional or k in must:
            assert call(**{k: None}) == eq.EQMP_ERR_INVALID_ARG, k
        elif k != "gt":
            assert call(**{k: None}) == eq.EQMP_ERR_CUDA, k
        assert call(**{k: call.values[k] + 2}) == eq.EQMP_ERR_INVALID_ARG, k
    assert call(**{k: None for k in call.out if k != "ws"}) == eq.EQMP_OK  # nothing asked for
    if "ws" in call.sizes:
        assert call(ws_bytes=call.values["ws_bytes"] - 1) == eq.EQMP_ERR_INVALID_ARG
        assert call(ws=call.values["ws"] + 8) == eq.EQMP_ERR_INVALID_ARG


BAD = dict(
    eqmp_head_norm=[dict(N=-1), dict(H=0), dict(HK=-1), dict(D=0), dict(D=7), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                    dict(eps=float("inf")), dict(axes=4), dict(axes=-1), dict(q_ld=-1), dict(q_ld=2 ** 31 + 1)],
    eqmp_head_norm_backward=[dict(N=-1), dict(H=0), dict(HK=-1), dict(D=7), dict(dtype=-1), dict(axes=0), dict(k_ld=-8)],
    eqmp_edge_bias=[dict(E=-1), dict(B=0), dict(H=0)],
    eqmp_edge_bias_backward=[dict(E=-1), dict(B=0), dict(H=0)],
    eqmp_edge_attention=[dict(N=-1), dict(NS=-1), dict(E=-1), dict(H=0), dict(D=0), dict(DV=0), dict(dtype=5), dict(q_ld=-1),
                         dict(v_ld=2 ** 31 + 1), dict(scale=float("inf")), dict(scale=float("nan"))],
    eqmp_edge_attention_backward=[dict(N=-1), dict(NS=-1), dict(E=-1), dict(ES=-1), dict(H=-2), dict(D=0), dict(DV=0), dict(dtype=3),
                                  dict(q_ld=-1), dict(scale=float("nan"))])
LARGE = dict(eqmp_head_norm=[dict(N=2 ** 30 + 1), dict(D=258), dict(H=65537)], eqmp_head_norm_backward=[dict(D=258)],
             eqmp_edge_bias=[dict(E=2 ** 30 + 1), dict(B=1025), dict(H=257)],
             eqmp_edge_bias_backward=[dict(E=2 ** 30 + 1), dict(B=1025), dict(H=257)],
             eqmp_edge_attention=[dict(N=2 ** 30 + 1), dict(NS=2 ** 30 + 1), dict(E=2 ** 30 + 1), dict(H=1025), dict(D=257), dict(DV=1025)],
             eqmp_edge_attention_backward=[dict(N=2 ** 30 + 1), dict(E=2 ** 30 + 1), dict(ES=2 ** 30 + 1), dict(H=1025), dict(D=257),
                                           dict(DV=1025)])


@pytest.mark.parametrize("name", NAMES)
def test_sizes(lib, name):
    call = _named(lib)[name]
    for bad in BAD[name]:
        assert call(**bad) == eq.EQMP_ERR_INVALID_ARG, bad
    for bad in LARGE[name]:
        assert call(**bad) == eq.EQMP_ERR_UNSUPPORTED, bad


def test_workspace_sizes(lib):
    assert lib.eqmp_edge_attention_workspace_size(1024, 8, 128) == 0 < lib.eqmp_edge_attention_workspace_size(1025, 8, 128)
    # the parts of a large graph stay small beside its rows
    assert lib.eqmp_edge_attention_workspace_size(1909372, 8, 128) < 20 << 20
    assert lib.eqmp_edge_attention_workspace_size(-1, 8, 128) == lib.eqmp_edge_attention_workspace_size(5, 8, 1025) == -1
    assert lib.eqmp_edge_attention_backward_workspace_size(5, 5, 2 ** 30 + 1, 8, 8, 8) == -1
    assert lib.eqmp_head_norm_backward_workspace_size(5, 257) == -1 and lib.eqmp_head_norm_backward_workspace_size(0, 8) == 0
    assert lib.eqmp_edge_bias_backward_workspace_size(32768, 64, 8) == 0 and lib.eqmp_edge_bias_backward_workspace_size(5, 0, 8) == -1


# ------------------------------------------------------------------ the binding
@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch, eq)


def _arguments(gpu):
    t, i32 = gpu.tensor, lambda *n: gpu.tensor(*n, dtype=torch.int32)
    q, k, v, o = t(N, H, D), t(NS, H, D), t(NS, H, DV), t(N, H, DV)
    graph, senders = (i32(N + 1), i32(E)), (i32(E), i32(NS + 1), i32(E))
    return t, i32, q, k, v, o, graph, senders


def _binding_calls(gpu):
    t, i32, q, k, v, o, graph, senders = _arguments(gpu)
    turn, rstd = dict(pos=t(N, 3), freq=t(D // 2, 3)), t(N, 2 * H)
    yield lambda s: eq.eqmp_head_norm(q, q, t(D), t(D), need=("q", "k", "rstd"), stream=s, **turn)
    yield lambda s: eq.eqmp_head_norm_backward(q, q, q, q, rstd, need=("q", "k", "wq", "wk", "pos"), stream=s, **turn)
    yield lambda s: eq.eqmp_edge_bias(t(E, 3), t(B - 1), t(B, H), stream=s)
    yield lambda s: eq.eqmp_edge_bias_backward(t(E, H), i32(E), B, stream=s)
    yield lambda s: eq.eqmp_edge_attention(q, k, v, *graph, bias=t(E, H), need=("out", "stats"), stream=s)
    yield lambda s: eq.eqmp_edge_attention_backward(o, q, k, v, t(N, H, 2), *graph, *senders, bias=t(E, H),
                                                    need=("q", "k", "v", "bias"), stream=s)


def test_memory_is_made_on_the_stream_of_the_call(gpu):
    _check_streams(gpu, _binding_calls(gpu))


def test_the_binding_refuses(gpu):
    t, i32, q, k, v, o, graph, senders = _arguments(gpu)
    half, rstd, stats, bf16 = t(N, H, D, dtype=torch.float16), t(N, 2 * H), t(N, H, 2), t(N, H, D, dtype=torch.bfloat16)
    attend = lambda q=q, k=k, v=v, off=graph[0], src=graph[1], **kw: eq.eqmp_edge_attention(q, k, v, off, src, **kw)  # noqa: E731

    def back(g=o, q=q, k=k, v=v, stats=stats, off=graph[0], src=graph[1], dst=senders[0], so=senders[1], se=senders[2], **kw):
        return eq.eqmp_edge_attention_backward(g, q, k, v, stats, off, src, dst, so, se, **kw)

    norm = lambda q=q, k=q, **kw: eq.eqmp_head_norm(q, k, **kw)  # noqa: E731
    for error, call in (
            (TypeError, lambda: norm(half)), (TypeError, lambda: norm(k=bf16)), (ValueError, lambda: norm(q[0])),
            (ValueError, lambda: norm(torch.ones(N, H, D))), (ValueError, lambda: norm(pos=t(N, 3))),
            (ValueError, lambda: norm(pos=t(N, 4), freq=t(4, 4))), (ValueError, lambda: norm(pos=t(N, 2), freq=t(4, 3))),
            (ValueError, lambda: norm(t(N, H, 7), t(N, H, 7), pos=t(N, 1), freq=t(3, 1))), (ValueError, lambda: norm(k=None, need=("k",))),
            (ValueError, lambda: norm(need=("out",))), (ValueError, lambda: norm(t(N, D, H).transpose(1, 2))),
            (ValueError, lambda: norm(wq=t(D + 1))), (TypeError, lambda: norm(wq=t(D, dtype=torch.bfloat16))),
            (ValueError, lambda: norm(t(N, H, D, gpu=1))), (ValueError, lambda: norm(wk=t(D, gpu=1))),
            (ValueError, lambda: norm(out=dict(q=t(N, H, D + 1)))),
            (ValueError, lambda: eq.eqmp_head_norm_backward(q, None, q, q, rstd)),
            (ValueError, lambda: eq.eqmp_head_norm_backward(q, q, q, q, rstd, need=("pos",))),
            (ValueError, lambda: eq.eqmp_head_norm_backward(q, q, q, q, t(N, H))),
            (ValueError, lambda: eq.eqmp_edge_bias(t(E, 2), t(B - 1), t(B, H))), (ValueError, lambda: eq.eqmp_edge_bias(t(E, 3), t(B), t(B, H))),
            (TypeError, lambda: eq.eqmp_edge_bias(t(E, 3), t(B - 1, dtype=torch.float64), t(B, H))),
            (ValueError, lambda: eq.eqmp_edge_bias(t(E, 3, gpu=1), t(B - 1), t(B, H))),
            (ValueError, lambda: eq.eqmp_edge_bias(t(E, 3), t(B - 1), t(B, H), need=("table",))),
            (TypeError, lambda: eq.eqmp_edge_bias_backward(t(E, H), t(E, dtype=torch.int64), B)),
            (ValueError, lambda: eq.eqmp_edge_bias_backward(t(E, H), i32(E), 0)),
            (ValueError, lambda: eq.eqmp_edge_bias_backward(t(E, H), i32(E + 1), B)),
            (TypeError, lambda: attend(k=bf16)), (ValueError, lambda: attend(k=t(NS, H, D + 1))), (ValueError, lambda: attend(v=t(NS, H + 1, DV))),
            (ValueError, lambda: attend(v=t(NS + 1, H, DV))), (TypeError, lambda: attend(src=t(E, dtype=torch.int64))),
            (ValueError, lambda: attend(off=i32(N))), (ValueError, lambda: attend(bias=t(E, H + 1))),
            (TypeError, lambda: attend(bias=t(E, H, dtype=torch.bfloat16))), (ValueError, lambda: attend(bias=t(E, H, gpu=1))),
            (ValueError, lambda: attend(v=t(NS, DV, H).transpose(1, 2))), (ValueError, lambda: attend(need=("lse",))),
            (ValueError, lambda: attend(workspace=t(1 << 16, dtype=torch.uint8, gpu=1))), (TypeError, lambda: attend(workspace=t(64))),
            (ValueError, lambda: back(g=q)), (ValueError, lambda: back(stats=t(N, H))), (ValueError, lambda: back(so=i32(NS))),
            (ValueError, lambda: back(se=None)), (TypeError, lambda: back(dst=t(E, dtype=torch.int64))),
            (ValueError, lambda: back(need=("out",))), (ValueError, lambda: back(out=dict(q=t(N, H, D, gpu=1))))):
        gpu.lib.calls.clear()
        with pytest.raises(error):
            call()
        assert not [name for name, _ in gpu.lib.calls if not name.endswith("_size")]
    # slices of a projection and one node for all are taken
    wide = t(N, 3 * H * D)
    eq.eqmp_edge_attention(wide[:, :H * D].unflatten(1, (H, D)), k, v, *graph)
    args = gpu.lib.calls[-1][1]
    assert args[1] == 3 * H * D and args[3] == H * D
    eq.eqmp_head_norm(q[:1].expand(N, H, D))
    assert gpu.lib.calls[-1][1][1] == 0
