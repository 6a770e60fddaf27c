"""Calls on a stream that is not the current one (GPU)."""
import pytest

from tests.test_gpu_norm import Case, eq  # noqa: F401

pytestmark = pytest.mark.gpu

SLEEP = 20_000_000  # clocks, about 10 ms: the calls below are made before the first kernel runs


def _busy_sides(n):
    import torch

    sides = [torch.cuda.Stream() for _ in range(n)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(SLEEP)
    return sides


@pytest.mark.parametrize("shape", [(5000, 96), (70, 9000), (700, 16, 25)], ids=str)
def test_norm_temporaries_outlive_the_call(eq, shape):  # noqa: F811
    """Backward calls wait on two side streams while the current stream takes and overwrites memory of the sizes of their
    workspaces and results: the gradients are those of the lone call, to the bit."""
    import torch

    cases = [Case(shape, residual=True, p=0.2, seed=k) for k in (0, 1)]
    saved = [c.forward(eq) for c in cases]
    want = [c.backward(eq, a["s"], a["stats"]) for c, a in zip(cases, saved)]
    torch.cuda.synchronize()
    got = [c.backward(eq, a["s"], a["stats"], stream=s) for c, a, s in zip(cases, saved, _busy_sides(2))]
    size = getattr(eq, "eqmp_degree_norm_backward_workspace_size" if len(shape) == 3 else
                   "eqmp_layer_norm_backward_workspace_size")(*(shape[:2] + (4,) * (len(shape) == 3)))
    taken = [torch.full((n,), float("nan"), device="cuda")
             for n in [size // 4 + 4, size // 4] * 4 + [v.numel() for v in want[0].values()] * 4]
    torch.cuda.synchronize()
    assert all(torch.isnan(t).all() for t in taken)
    for g, w in zip(got, want):
        assert all(torch.equal(g[k], w[k]) for k in w)


@pytest.mark.parametrize("mode", ["shared", "radial"])
def test_layer_temporaries_outlive_the_call(eq, mode):  # noqa: F811
    """The message layer and its gradients on a waiting side stream, as above; the zeros that gradients begin with are
    written before the kernels add to them.  To the tolerance of the layer's parity tests, against the lone call."""
    import numpy as np
    import torch

    from equivariant_gnn_message_gb300.inputs import make_workload
    from tests.gpu_util import TOL, host, rel_err, to_device, weights_kw

    wl = make_workload(n_atoms=300, cutoff=5.0, channels=32, weights=mode, storage="f32", seed=3)
    d = to_device(wl)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    so, se = eq.sender_view(wl.src, wl.n_atoms)
    g = torch.randn(wl.n_atoms, 32, 16, device="cuda")
    need = ("x", "vec", "w") if mode == "shared" else ("x", "vec", "R", "M")
    back = (d["vec"], d["x"], d["off"], d["src"], up(wl.dst), up(so), up(se), g)
    calls = (lambda s: dict(out=eq.eqmp_fused(d["vec"], d["x"], d["off"], d["src"], stream=s, **weights_kw(d))),
             lambda s: eq.eqmp_fused_backward(*back, need=need, stream=s, **weights_kw(d)))
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        side, = _busy_sides(1)
        got = call(side)
        sizes = [v.numel() for v in want.values()] + [lib_size // 4 for lib_size in (
            eq.load_library().eqmp_fused_backward_workspace_size(wl.n_atoms, wl.n_edges, 32, int(mode == "radial")),)]
        taken = [torch.full((n,), float("nan"), device="cuda") for n in sizes * 4]
        torch.cuda.synchronize()
        assert eq.eqmp_device_error() == 0 and all(torch.isnan(t).all() for t in taken)
        for k in want:
            assert rel_err(host(got[k]), host(want[k])) <= TOL["f32"], k


@pytest.mark.parametrize("e_cap", [None, 100])
@pytest.mark.parametrize("box", [None, (12.0, 12.0, 12.0)])
def test_radius_graph_on_a_waiting_stream(eq, box, e_cap):  # noqa: F811
    """The count is that of this call, not what lay in its place: the same edges, to the bit, with room and without."""
    import torch

    pos = torch.rand(200, 3, device="cuda") * 12
    want, E = eq.eqmp_radius_graph(pos, 4.0, e_cap=e_cap, dst=True, rev=True, box=box)
    torch.cuda.synchronize()
    side, = _busy_sides(1)
    got, n = eq.eqmp_radius_graph(pos, 4.0, e_cap=e_cap, dst=True, rev=True, box=box, stream=side)
    torch.cuda.synchronize()
    assert n == E > 100 and set(got) == set(want)
    assert all(torch.equal(got[k], want[k]) for k in want)
