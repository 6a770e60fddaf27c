"""The attention on graphs large enough for the forms and splits that small ones do not get (GPU)."""
import numpy as np
import pytest

from tests import attention_forms as forms
from tests.attention_util import backward_bounds, forward_bounds, worst
from tests.gpu_util import host
from tests.test_gpu_attention import Problem, eq  # noqa: F401

pytestmark = pytest.mark.gpu

NEED = ("q", "k", "v", "bias")


def _check_heads(eq, p, heads):  # noqa: F811
    """Both passes of `p` against the oracle in the heads given."""
    cut = lambda a: a[:, heads]  # noqa: E731
    got = p.forward(eq)
    grads = p.backward(eq, got["stats"])
    q, k, v, off, src, bias = p.host_args()
    args = (cut(q), cut(k), cut(v), off, src, cut(bias))
    want, bound = forward_bounds(*args, None, p.bf16)
    for name, w, b in zip(("out", "stats"), want, bound):
        assert worst(cut(host(got[name])), w, b) <= 1, name
    want, bound = backward_bounds(cut(host(p.g)), *args[:3], cut(host(got["stats"])), *args[3:], None, p.bf16)
    for name in NEED:
        assert worst(cut(host(grads[name])), want[name], bound[name]) <= 1, name


def test_wide_heads_in_few_blocks(eq):  # noqa: F811
    """Parts of so many values that there are fewer blocks than 2048, and different ones in each pass."""
    degrees = [20, 15_000, 0, 3, 8_000, 90, 6_800, 87]
    p = Problem(512, 4, 16, "f32", degrees, n_src=40, masked=0.1, seed=2)
    assert eq.eqmp_edge_attention_workspace_size(30_000, 512, 16) == 2 * 469 * 512 * 18 * 4
    _check_heads(eq, p, [0, 1, 255, 511])


@pytest.mark.parametrize("shape,dtype", [((3, 4, 4), "f32"), ((3, 7, 9), "bf16")], ids=str)
def test_blocks_of_more_than_32_edges(eq, shape, dtype):  # noqa: F811
    rng = np.random.default_rng(5)
    degrees = [int(d) for d in np.concatenate(([70_000], rng.integers(0, 300, 100), [129, 128, 127, 20_000, 0, 257]))]
    p = Problem(*shape, dtype, degrees, n_src=50, masked=0.05, seed=3)
    _check_heads(eq, p, list(range(shape[0])))


@pytest.mark.parametrize("name", forms.cases())
def test_forms_of_large_graphs(eq, name):  # noqa: F811
    """Each form against the oracle, several rows a warp among them; and the case gets the form that it is for."""
    p = forms.problem(eq, name)
    H = p.q.shape[1]
    _check_heads(eq, p, sorted({0, 1, H // 2, H - 1}))
    rows, form, each = forms.cases()[name][4:]
    found = forms.forms(lambda: p.backward(eq, p.forward(eq)["stats"]))
    assert set(found) == {"fwd", "recv", "send"}
    for ring, numbers, ctas in found.values():
        assert ring == (each is not None) and numbers == form
        if ring:  # a CTA for each block of 32 edges, and for each few rows
            assert ctas == -(-len(p.src) // 32) + -(-rows // each)
