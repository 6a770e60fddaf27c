"""What the Python binding allocates and refuses, without a GPU (binding_util stands in for it)."""
import pytest
import torch

import equivariant_gnn_message_gb300 as eq
from tests.binding_util import FakeGpu, FakeStream

SIDE = 11


@pytest.fixture
def gpu(monkeypatch):
    return FakeGpu(monkeypatch, eq)


def _norm_calls(gpu):
    """The norms' and dropout's entry points, each as a function of the stream."""
    t = gpu.tensor
    x, feat, w = t(5, 8), t(5, 8, 16), t(8)
    d = eq.Dropout(0.5, 1)
    yield lambda s: eq.eqmp_dropout(x, d, stream=s)
    yield lambda s: eq.eqmp_layer_norm(x, w, w, residual=x, need=("y", "s", "stats"), stream=s)
    yield lambda s: eq.eqmp_layer_norm_backward(x, x, t(5, 2), w, need=("x", "r", "w", "b"), stream=s)
    yield lambda s: eq.eqmp_degree_norm(feat, need=("y", "s", "stats"), stream=s)
    yield lambda s: eq.eqmp_degree_norm_backward(feat, feat, t(5, 5), need=("x", "r", "w", "b"), stream=s)


def _check_streams(gpu, calls):
    """On another stream than the current one everything that is made for a call is made on the call's stream: the memory
    of a temporary, freed when the call returns, must not go to the current stream's next allocation while the kernels
    still use it, and no fill of a result may run on another stream than its kernel.  Results are also recorded on the
    current stream, where they will be used."""
    for call in calls:
        for stream, want in ((None, 7), (gpu.current, 7), (FakeStream(SIDE), SIDE)):
            gpu.made.clear()
            gpu.lib.calls.clear()
            got = call(stream)
            results = [id(v) for v in (got.values() if isinstance(got, dict) else [got])]
            assert gpu.made and gpu.lib.calls[-1][1][-1] == want and gpu.current.cuda_stream == 7
            for t in gpu.made:
                assert gpu.given(t) and t.made_on == want
                if id(t) in results:
                    assert t.recorded == ((7,) if want == SIDE else ())


def test_norms_allocate_on_the_stream_of_the_call(gpu):
    _check_streams(gpu, _norm_calls(gpu))


def _layer_calls(gpu):
    t, i32 = gpu.tensor, lambda n: gpu.tensor(n, dtype=torch.int32)
    graph = (t(6, 3), t(4, 8, 16), i32(5), i32(6))
    back = graph + (i32(6), i32(5), i32(6), t(4, 8, 16))
    shared, radial = dict(w=t(34, 8)), dict(R=t(6, 8), M=t(8, 34 * 8))
    yield lambda s: eq.eqmp_sh(graph[0], stream=s)
    yield lambda s: eq.eqmp_tp_scatter(t(6, 16), *graph[1:], stream=s, **shared)
    for weights in (shared, radial):
        yield lambda s: eq.eqmp_fused(*graph, stream=s, **weights)
        yield lambda s: eq.eqmp_fused_so2(*graph, stream=s, **weights)
        yield lambda s: eq.eqmp_fused_backward(*back, need=("x", "w", "R", "M", "vec"), stream=s, **weights)
        yield lambda s: eq.eqmp_fused_backward_noalloc(*back, need=("x", "w", "R", "M", "vec"), stream=s, **weights)
    yield lambda s: eq.eqmp_fused_lmax(4, graph[0], t(4, 8, 25), *graph[2:], w=t(65, 8), stream=s)


def test_message_layers_allocate_on_the_stream_of_the_call(gpu):
    _check_streams(gpu, _layer_calls(gpu))


@pytest.mark.parametrize("box", [None, (9.0, 9.0, 9.0)])
def test_radius_graph_reads_its_count_on_the_stream_of_the_call(gpu, box):
    """The edge count is read in the order of the kernels, also when the call is repeated for more room."""
    for stream, want in ((None, 7), (FakeStream(SIDE), SIDE)):
        gpu.made.clear()
        gpu.lib.calls.clear()
        gpu.counts = [700, 700]
        out, E = eq.eqmp_radius_graph(gpu.tensor(10, 3), 1.0, dst=True, rev=True, stream=stream, box=box)
        assert E == 700 and out["src"].shape == (700,) and gpu.current.cuda_stream == 7
        runs = [args for name, args in gpu.lib.calls if not name.endswith("_size")]
        assert len(runs) == 2 and all(args[-1] == want for args in runs)
        read = [t for t in gpu.made if t.read_on is not None]
        assert len(read) == 1 and read[0].read_on == want
        for t in gpu.made:
            assert gpu.given(t) and t.made_on == want
        assert out["off"].recorded == ((7,) if want == SIDE else ())


def test_workspace_of_another_gpu_is_refused(gpu):
    t = gpu.tensor
    x, feat, ws = t(5, 8), t(5, 8, 16), lambda g: t(4096, dtype=torch.uint8, gpu=g)
    for call in (lambda ws: eq.eqmp_layer_norm_backward(x, x, t(5, 2), workspace=ws),
                 lambda ws: eq.eqmp_degree_norm_backward(feat, feat, t(5, 5), workspace=ws)):
        call(ws(0))
        gpu.lib.calls.clear()
        with pytest.raises(ValueError, match="workspace must be a CUDA tensor on the current device"):
            call(ws(1))
        assert not gpu.lib.calls


def test_step_counter_of_another_gpu_is_refused(gpu):
    t = gpu.tensor
    x, feat = t(5, 8), t(5, 8, 16)

    def drop(g, group=1):
        return eq.Dropout(0.5, 1, group=group, step=t(1, dtype=torch.int64, gpu=g))

    for call in (lambda g: eq.eqmp_dropout(x, drop(g)), lambda g: eq.eqmp_layer_norm(x, drop=drop(g)),
                 lambda g: eq.eqmp_layer_norm_backward(x, x, t(5, 2), drop=drop(g)),
                 lambda g: eq.eqmp_degree_norm(feat, drop=drop(g, 16)),
                 lambda g: eq.eqmp_degree_norm_backward(feat, feat, t(5, 5), drop=drop(g, 16))):
        call(0)
        gpu.lib.calls.clear()
        with pytest.raises(ValueError, match="step must be a CUDA tensor on the current device"):
            call(1)
        assert not [name for name, _ in gpu.lib.calls if not name.endswith("_size")]
