"""The example attention block: its gradients against differences of the float64 oracle, its rotations, and a few steps."""
import numpy as np
import pytest

from oracle import attention as at
from oracle import norm
from tests.gpu_util import host
from tests.rotations import random_rotation, rotate_features, wigner_d_blocks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    import torch

    import __graft_entry__

    __graft_entry__.build()
    from examples import attention_block

    torch.cuda.set_device(0)
    return attention_block


def _loss(graph, bucket, x, target, prm):
    """The block in float64 with the oracle's norms and attention."""
    heads = prm["table"].shape[1]
    h = norm.forward(x, prm["pre_w"], prm["pre_b"])["y"]
    both = (h[:, :, 0] @ prm["W"]).reshape(x.shape[0], 2 * heads, -1)
    theta = at.angles(graph["place"], graph["rates"])
    q, k = (at.head_norm(t, w, 1e-6, theta)[0] for t, w in ((both[:, :heads], prm["wq"]), (both[:, heads:], prm["wk"])))
    out, _ = at.edge_attention(q, k, h.reshape(x.shape[0], heads, -1), graph["off"], graph["src"], prm["table"][bucket])
    y = norm.forward(out.reshape(x.shape), prm["post_w"], prm["post_b"], residual=x)["y"]
    return 0.5 * ((y - target) ** 2).sum() / x.shape[0]


def test_gradients_match_differences(block):
    """Every gradient along a random direction: the difference of the float64 loss over a step of 1e-5 has an error of the
    step's square, and the fp32 gradients one of 1e-5 or so; 2e-3 of |g| |d| / sqrt(n), the expected size of the product,
    is well above both."""
    graph, x, target, prm = block.problem(40, 8, 2, seed=3)
    loss, kept = block.forward(graph, x, target, prm)
    grads = block.backward(graph, kept, prm)
    g64 = {k: host(v) if k in ("vec", "borders", "place", "rates") else v.cpu().numpy() for k, v in graph.items()}
    bucket = at.edge_bucket(g64["vec"], g64["borders"])
    assert np.array_equal(bucket, kept["bias"]["bucket"].cpu().numpy())
    p64, x64, t64 = {k: host(v) for k, v in prm.items()}, host(x), host(target)
    f = lambda x, prm: _loss(g64, bucket, x, t64, prm)  # noqa: E731
    assert abs(float(loss) - f(x64, p64)) < 1e-5 * abs(float(loss))
    rng = np.random.default_rng(0)
    assert set(grads) == set(prm) | {"x"}
    for name, g in grads.items():
        base = x64 if name == "x" else p64[name]
        d = rng.standard_normal(base.shape)
        move = lambda t: f(x64 + t * d, p64) if name == "x" else f(x64, {**p64, name: base + t * d})  # noqa: B023,E731
        diff, g = (move(1e-5) - move(-1e-5)) / 2e-5, host(g)
        assert abs(diff - (g * d).sum()) <= 2e-3 * np.sqrt((g ** 2).sum() * (d ** 2).sum() / g.size), name


def test_the_result_turns_with_the_frame(block):
    import torch

    graph, x, target, prm = block.problem(60, 8, 2, seed=4)
    turn = random_rotation(7)
    blocks = wigner_d_blocks(turn)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()  # noqa: E731
    y = host(block.forward(graph, x, target, prm)[1]["post"]["y"])
    turned = dict(graph, vec=up(host(graph["vec"]) @ turn.T))
    # rounding may put a turned edge on the other side of a border; the buckets of the test are those of the lengths as given
    assert torch.equal(block.eq.eqmp_edge_bias(turned["vec"], graph["borders"], prm["table"])["bucket"],
                       block.eq.eqmp_edge_bias(graph["vec"], graph["borders"], prm["table"])["bucket"])
    y_turned = host(block.forward(turned, up(rotate_features(host(x), blocks)), target, prm)[1]["post"]["y"])
    # fp32 values of order 1 through two norms and a softmax, and the rotation's own rounding: 1e-4
    assert np.abs(y_turned - rotate_features(y, blocks)).max() < 1e-4


def test_a_few_steps_run_the_same_again(block):
    import equivariant_gnn_message_gb300 as eq

    first = block.train(n_atoms=200, channels=16, heads=4, steps=10, rate=1e-2)
    assert np.isfinite(first).all() and first == block.train(n_atoms=200, channels=16, heads=4, steps=10, rate=1e-2)
    assert eq.eqmp_device_error() == 0
