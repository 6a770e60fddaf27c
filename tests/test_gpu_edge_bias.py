"""The bias by buckets of the edges' lengths against the oracle (GPU): buckets and biases exactly, the gradient within the
worst case of its sums."""
import numpy as np
import pytest

from oracle import attention as at
from tests.attention_util import MARGIN, TINY, U, worst
from tests.gpu_util import host
from tests.test_gpu_attention import eq  # noqa: F401

pytestmark = pytest.mark.gpu


def _up(a, dt=np.float32):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()


def _run(eq, vec, borders, table):  # noqa: F811
    got = eq.eqmp_edge_bias(_up(vec), _up(borders), _up(table))
    want = at.edge_bucket(vec, borders)
    assert np.array_equal(got["bucket"].cpu().numpy(), want)
    assert np.array_equal(got["bias"].cpu().numpy(), np.asarray(table, np.float32)[want])
    return got


@pytest.mark.parametrize("E,B,H", [(0, 4, 2), (1, 1, 1), (5, 2, 3), (512, 16, 4), (513, 17, 5), (3000, 64, 8), (2000, 1024, 7),
                                   (700, 300, 40), (100, 1024, 256), (1500, 33, 256), (32769, 64, 8),
                                   (40000, 33, 5), (33000, 1024, 18), (32768, 16, 6)])
def test_forward_and_gradient(eq, E, B, H):  # noqa: F811
    rng = np.random.default_rng(E + B)
    vec = 3 * rng.standard_normal((E, 3)).astype(np.float32)
    borders = np.sort(rng.random(B - 1) * 8).astype(np.float32)
    got = _run(eq, vec, borders, rng.standard_normal((B, H)).astype(np.float32))
    g = rng.standard_normal((E, H)).astype(np.float32)
    bucket = got["bucket"].cpu().numpy()
    table = host(eq.eqmp_edge_bias_backward(_up(g), got["bucket"], B)["table"])
    count = np.bincount(bucket, minlength=B)[:, None]
    size = at.edge_bias_backward(np.abs(g).astype(np.float64), bucket, B)
    # sums of `count` values in some order, through copies and parts that may be zeros, which add exactly
    assert worst(table, at.edge_bias_backward(g.astype(np.float64), bucket, B), MARGIN * count * U * size + TINY) <= 1


def test_lengths_at_the_borders(eq):  # noqa: F811
    """Exact triples at, a step below and a step above a border; zero, tiny, huge, infinite and NaN vectors."""
    triples = np.array([[3, 4, 0], [0, 0, 5], [2, 3, 6], [1, 2, 2], [0, 0, 0], [1e-30, 0, 0], [1e-42, 0, 0], [3e38, 3e38, 3e38],
                        [np.inf, 0, 0], [np.nan, 1, 1]], np.float32)
    rng = np.random.default_rng(0)
    signs = rng.choice([-1, 1], (10, 10, 3)).astype(np.float32)
    vec = (signs * triples).reshape(-1, 3)
    at_ = np.array([3, 5, 7], np.float32)
    for borders in (at_, np.nextafter(at_, np.float32(0)), np.nextafter(at_, np.float32(9)), np.array([0, 1e-42, 1e-30], np.float32),
                    np.array([5, 5, 5], np.float32), np.array([0, 3e38, np.inf], np.float32)):
        _run(eq, vec, borders, rng.standard_normal((4, 3)))


def test_lengths_next_to_a_border(eq):  # noqa: F811
    """Borders that are the rounded lengths themselves: fp32 squares would put many edges on the wrong side."""
    rng = np.random.default_rng(1)
    vec = rng.standard_normal((5000, 3)).astype(np.float32)
    lengths = np.sqrt((vec.astype(np.float64) ** 2).sum(1)).astype(np.float32)
    _run(eq, vec, np.sort(lengths[:1023]), rng.standard_normal((1024, 2)))


def test_buckets_outside_add_nothing_and_bad_values_stay(eq):  # noqa: F811
    import torch

    rng = np.random.default_rng(2)
    bucket = rng.integers(-2, 8, 4000).astype(np.int32)
    bucket[:4] = [-2 ** 31, 2 ** 31 - 1, 6, -1]
    g = rng.standard_normal((4000, 3)).astype(np.float32)
    g[bucket == 4, 1] = np.nan
    got = host(eq.eqmp_edge_bias_backward(_up(g), _up(bucket, np.int32), 6)["table"])
    want = at.edge_bias_backward(np.nan_to_num(g.astype(np.float64)), bucket, 6)
    assert np.isnan(got[4, 1])
    got[4, 1] = want[4, 1]
    assert np.abs(got - want).max() < 4000 * U * np.abs(np.nan_to_num(g)).sum()
    torch.cuda.synchronize()


def test_one_result_alone_and_the_same_again(eq):  # noqa: F811
    import torch

    rng = np.random.default_rng(3)
    vec, borders, table = _up(rng.standard_normal((300000, 3))), _up(np.linspace(0.1, 3, 31)), _up(rng.standard_normal((32, 8)))
    both = eq.eqmp_edge_bias(vec, borders, table)
    assert torch.equal(eq.eqmp_edge_bias(vec, borders, table, need=("bias",))["bias"], both["bias"])
    assert torch.equal(eq.eqmp_edge_bias(vec, borders, table, need=("bucket",))["bucket"], both["bucket"])
    g = torch.randn(300000, 8, device="cuda")
    first = eq.eqmp_edge_bias_backward(g, both["bucket"], 32)["table"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = eq.eqmp_edge_bias_backward(g, both["bucket"], 32, stream=side)["table"]
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    tape = torch.cuda.CUDAGraph()
    with torch.cuda.graph(tape):
        out = eq.eqmp_edge_bias(vec, borders, table)
        back = eq.eqmp_edge_bias_backward(g, out["bucket"], 32)["table"]
    tape.replay()
    assert torch.equal(out["bias"], both["bias"]) and torch.equal(back, first)
