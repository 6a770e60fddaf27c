"""The example block: its gradients against differences of the float64 oracle, and a few training steps."""
import numpy as np
import pytest

from oracle import layer, norm
from tests.gpu_util import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    from examples import message_block

    torch.cuda.set_device(0)
    return message_block


def _loss(graph, x, target, prm, factors):
    """The block in float64 with the oracle's norms, dropout factors and message layer."""
    h = norm.forward(x, prm["pre_w"], prm["pre_b"])["y"]
    u = norm.forward(graph["rbf"] @ prm["w1"], prm["ln_w"], prm["ln_b"], factor=factors[0])["y"]
    R = (u / (1 + np.exp(-u))) @ prm["w2"]
    m = layer.message_pass(graph["vec"], h, graph["off"], graph["src"], R=R, M=prm["M"])
    y = norm.forward(m, prm["post_w"], prm["post_b"], residual=x, factor=factors[1])["y"]
    return 0.5 * ((y - target) ** 2).sum() / x.shape[0]


def test_gradients_match_differences(block):
    """Every gradient of a block with dropout, along a random direction: the difference of the float64 loss over a step
    of 1e-5 has an error of the step's square, and the fp32 gradients one of 1e-5 or so; 2e-3 of |g| |d| / sqrt(n), the
    expected size of the product, is well above both."""
    graph, x, target, prm = block.problem(40, 8, hidden=24, seed=3)
    drops = block.masks(0.2, 11, 5)
    loss, kept = block.forward(graph, x, target, prm, drops)
    grads = block.backward(graph, kept, prm, drops)
    g64 = {k: host(v) if k in ("vec", "rbf") else v.cpu().numpy() for k, v in graph.items()}
    p64 = {k: host(v) for k, v in prm.items()}
    x64, t64 = host(x), host(target)
    E = g64["rbf"].shape[0]
    factors = (norm.drop_factor(E, 24, 0.2, 11, 10), norm.drop_factor(40, 128, 0.2, 11, 11, group=16))
    f = lambda x, prm: _loss(g64, x, t64, prm, factors)  # noqa: E731
    assert abs(float(loss) - f(x64, p64)) < 1e-5 * abs(float(loss))
    rng = np.random.default_rng(0)
    for name, g in grads.items():
        base = x64 if name == "x" else p64[name]
        d = rng.standard_normal(base.shape)
        move = lambda t: f(x64 + t * d, p64) if name == "x" else f(x64, {**p64, name: base + t * d})  # noqa: E731
        diff = (move(1e-5) - move(-1e-5)) / 2e-5
        g = host(g)
        assert abs(diff - (g * d).sum()) <= 2e-3 * np.sqrt((g ** 2).sum() * (d ** 2).sum() / g.size), name


def test_a_few_steps_lower_the_loss(block):
    import equivariant_gnn_message_gb300 as eq

    before, after = block.train(n_atoms=200, channels=16, steps=30, p=0.1, rate=1e-2)
    assert after < before
    assert (before, after) == block.train(n_atoms=200, channels=16, steps=30, p=0.1, rate=1e-2)  # bitwise the same again
    assert eq.eqmp_device_error() == 0
