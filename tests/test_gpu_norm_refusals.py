"""Refusals of the norms' and dropout's entry points that look at memory and at devices (GPU)."""
import pytest

from tests.test_gpu_norm import eq  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_over_parameters_and_statistics(eq):  # noqa: F811
    """What a call would overwrite while it reads it is refused, and left as it was."""
    import torch

    slab = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    x = slab[:8192].view(torch.float32).view(64, 32).normal_()
    g, w, b = torch.randn(64, 32, device="cuda"), torch.randn(32, device="cuda"), torch.randn(32, device="cuda")
    stats = eq.eqmp_layer_norm(x, need=("stats",))["stats"]
    t = torch.zeros(32, device="cuda")
    before = [v.clone() for v in (x, g, w, b, stats)]
    with pytest.raises(eq.EqmpError):
        eq.eqmp_layer_norm(x, w, b, need=("stats",), out={"stats": x.view(-1)[:128].view(64, 2)})
    for kw in (dict(out={"w": w}), dict(out={"b": w}), dict(out={"w": t, "b": t}), dict(out={"w": x[0]}),
               dict(out={"b": stats.view(-1)[:32]}), dict(workspace=slab),
               dict(workspace=slab[8192:], out={"w": slab[16384:16512].view(torch.float32)})):
        with pytest.raises(eq.EqmpError) as err:
            eq.eqmp_layer_norm_backward(g, x, stats, w, **kw)
        assert err.value.status == eq.EQMP_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(v, u) for v, u in zip((x, g, w, b, stats), before))
    side = torch.zeros(128, device="cuda")  # side by side is fine
    got = eq.eqmp_layer_norm_backward(g, x, stats, w, out={"w": side[:32], "b": side[32:64]})
    want = eq.eqmp_layer_norm_backward(g, x, stats, w)
    assert all(torch.equal(got[k], want[k]) for k in want) and not side[64:].any()
