"""The attention at the ends of fp32's range (GPU)."""
import numpy as np
import pytest

from tests.attention_util import forward_bounds, worst
from tests.gpu_util import host
from tests.test_gpu_attention import LONG, MIXED, Problem, eq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("degrees", [MIXED, LONG], ids=["mixed", "long"])
@pytest.mark.parametrize("shape,dtype", [((4, 16, 128), "f32"), ((4, 16, 128), "bf16"), ((3, 6, 10), "f32"), ((3, 7, 9), "bf16"),
                                         ((2, 65, 30), "f32")], ids=str)
@pytest.mark.parametrize("size", [3e38, 1e-30])
def test_values_near_the_ends_of_the_range(eq, shape, dtype, degrees, size):  # noqa: F811
    """Rows whose values sum to almost the largest number, or are tiny, with scores that rise by up to 8 along the row: a weight
    above 1 would overflow."""
    import torch

    E = int(np.sum(degrees))
    p = Problem(*shape, dtype, degrees, n_src=E, seed=3)
    p.src[:] = np.arange(E)  # each edge has its own sender
    p.graph = (p.graph[0], torch.from_numpy(p.src).cuda())
    rng = np.random.default_rng(0)
    each = np.repeat(np.maximum(degrees, 1), degrees)[:, None, None]
    v = rng.uniform(-1, 1, (E,) + shape[0::2]) * size / (each if size > 1 else 1)
    p.v = torch.from_numpy(v.astype(np.float32)).to(p.dtype).cuda()
    rise = np.concatenate([np.linspace(0, 7.9, d) for d in degrees] + [[]])
    p.q.zero_()
    p.bias = torch.from_numpy(np.repeat(rise[:, None], shape[0], 1).astype(np.float32)).cuda()
    p.bias[:, 0] = p.bias[:, 0].flip(0)
    got = p.forward(eq)
    want, bound = forward_bounds(*p.host_args(), None, p.bf16)
    # a mean of values of at most `size`, rounded to their type by 2^-8 of it at most
    assert np.abs(want[0]).max() <= size * (1 + 2.0 ** -8)
    assert worst(host(got["out"]), want[0], bound[0]) <= 1 and worst(host(got["stats"]), want[1], bound[1]) <= 1
