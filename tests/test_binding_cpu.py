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
