"""The bias by buckets and the head norm at sizes where a CTA takes several tiles and a warp several nodes (GPU)."""
import numpy as np
import pytest

from oracle import attention as at
from tests.attention_util import MARGIN, TINY, U, worst
from tests.gpu_util import host
from tests.test_gpu_attention import eq  # noqa: F401
from tests.test_gpu_edge_bias import _up
from tests.test_gpu_head_norm import Problem

pytestmark = pytest.mark.gpu


def _check_table(got, g, bucket, n_buckets):
    """Sums of `count` values in some order, through copies and parts that may be zeros, which add exactly."""
    ok = (bucket >= 0) & (bucket < n_buckets)
    count = np.bincount(bucket[ok], minlength=n_buckets)[:, None]
    want, size = (np.stack([np.bincount(bucket[ok], w[ok], n_buckets) for w in f(g).T], 1) for f in (np.asarray, np.abs))
    assert worst(got, want, MARGIN * count * U * size + TINY) <= 1


@pytest.mark.parametrize("H", [3, 4])
def test_bias_of_several_tiles_a_cta(eq, H):  # noqa: F811
    """More edges than the CTAs of a launch take in their first tile, the last tile not full."""
    E, B = 1_400_003, 23
    rng = np.random.default_rng(H)
    vec = rng.standard_normal((E, 3), dtype=np.float32)
    borders = np.sort(rng.random(B - 1) * 4).astype(np.float32)
    table = rng.standard_normal((B, H)).astype(np.float32)
    v, b = vec.astype(np.float64), borders.astype(np.float64)
    bucket = np.searchsorted(b * b, (v[:, 0] * v[:, 0] + v[:, 1] * v[:, 1]) + v[:, 2] * v[:, 2], side="right").astype(np.int32)
    some = rng.integers(0, E, 500)
    assert np.array_equal(bucket[some], at.edge_bucket(vec[some], borders))
    got = eq.eqmp_edge_bias(_up(vec), _up(borders), _up(table))
    assert np.array_equal(got["bucket"].cpu().numpy(), bucket) and np.array_equal(got["bias"].cpu().numpy(), table[bucket])
    g = rng.standard_normal((E, H), dtype=np.float32)
    _check_table(host(eq.eqmp_edge_bias_backward(_up(g), got["bucket"], B)["table"]), g, bucket, B)


@pytest.mark.parametrize("E", [4000, 50_000])  # one launch, two
@pytest.mark.parametrize("H", [3, 4])
def test_buckets_outside_add_nothing(eq, E, H):  # noqa: F811
    """To the bound of each sum: an edge too many or too few would show."""
    rng = np.random.default_rng(E + H)
    bucket = rng.integers(-2, 8, E).astype(np.int32)
    bucket[[0, 1, 2, E // 2, E - 1]] = [-2 ** 31, 2 ** 31 - 1, 6, -1, 1 << 20]
    g = rng.standard_normal((E, H)).astype(np.float32)
    g[(bucket < 0) | (bucket > 5)] += 100
    _check_table(host(eq.eqmp_edge_bias_backward(_up(g), _up(bucket, np.int32), 6)["table"]), g.astype(np.float64), bucket, 6)


@pytest.mark.parametrize("n", [19_457, 29_186, 38_915])  # two, three and four nodes a warp, and fewer in the last
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,dim,axes,pad", [(2, 1, 16, 3, None), (3, 2, 18, 1, 5), (1, 0, 7, 0, None), (2, 2, 64, 2, 8), (1, 1, 100, 3, None)])
def test_head_norm_of_several_nodes_a_warp(eq, n, dtype, hq, hk, dim, axes, pad):  # noqa: F811
    Problem(n, hq, hk, dim, dtype, axes=axes, pad=pad, seed=n).check(eq)
