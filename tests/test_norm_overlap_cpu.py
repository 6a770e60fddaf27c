"""The norms' and dropout's refusals of memory that meets other memory, at the C entry points.  The checks come before
any CUDA call, so the addresses are made up and the calls that pass end with EQMP_ERR_CUDA: not run where there is a GPU."""
import itertools

import pytest
import torch

import equivariant_gnn_message_gb300 as eq

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

ROWS, C, L = 6, 8, 3
K = (L + 1) ** 2
STEP = 1 << 20  # between the arguments' addresses


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__

    __graft_entry__.build()
    return eq.load_library()


def _drop(step):
    d = eq.Dropout(0.25, 1, group=K)
    d.step_ptr = step
    return d


def _sizes(degree, rows, bytes_):
    """name -> (bytes read or written, whether it is written) of a forward and of a backward call."""
    cols, l = (C * K, L) if degree else (C * K, 0)
    c = C if degree else cols
    row, w, stats = rows * cols * bytes_, (l + 1) * c * 4, rows * (l + 2) * 4
    ws = min(rows, 608) * (l + 2) * c * 4
    return (dict(x=(row, 0), r=(row, 0), w=(w, 0), b=(c * 4, 0), step=(8, 0), s=(row, 1), y=(row, 1), stats=(stats, 1)),
            dict(x=(row, 0), g=(row, 0), r=(row, 0), w=(w, 0), stats=(stats, 0), step=(8, 0), gr=(row, 1), gx=(row, 1),
                 gw=(w, 1), gb=(c * 4, 1), ws=(ws, 1)))


def _forward(lib, degree, rows, dtype, a):
    d, cols = _drop(a["step"]), C * K
    if degree:
        return lib.eqmp_degree_norm(a["x"], a["r"], dtype, rows, C, L, d, a["w"], a["b"], 1e-5, a["s"], a["y"], a["stats"], 0)
    return lib.eqmp_layer_norm(a["x"], cols, a["r"], cols, dtype, rows, cols, d, a["w"], a["b"], 1e-5, a["s"], a["y"],
                               a["stats"], 0)


def _backward(lib, degree, rows, dtype, a):
    d, cols = _drop(a["step"]), C * K
    if degree:
        return lib.eqmp_degree_norm_backward(a["g"], a["x"], a["r"], dtype, rows, C, L, d, a["w"], a["stats"], a["gr"],
                                             a["gx"], a["gw"], a["gb"], a["ws"], 1 << 18, 0)
    return lib.eqmp_layer_norm_backward(a["g"], cols, a["x"], cols, a["r"], cols, dtype, rows, cols, d, a["w"], a["stats"],
                                        a["gr"], a["gx"], a["gw"], a["gb"], a["ws"], 1 << 18, 0)


@pytest.mark.parametrize("degree", [False, True], ids=["layer", "degree"])
@pytest.mark.parametrize("dtype,bytes_", [(0, 4), (1, 2)])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
def test_every_output_meets_nothing(lib, backward, dtype, bytes_, degree):
    sizes, call = _sizes(degree, ROWS, bytes_)[backward], _backward if backward else _forward
    assert (eq.EQMP_F32, eq.EQMP_BF16) == (0, 1)
    apart = {k: STEP * (i + 1) for i, k in enumerate(sizes)}
    assert call(lib, degree, ROWS, dtype, apart) == eq.EQMP_ERR_CUDA
    for a, b in itertools.combinations(sizes, 2):
        if not (sizes[a][1] or sizes[b][1]):  # two inputs may be one
            assert call(lib, degree, ROWS, dtype, {**apart, b: apart[a]}) == eq.EQMP_ERR_CUDA, (a, b)
            continue
        assert call(lib, degree, ROWS, dtype, {**apart, b: apart[a]}) == eq.EQMP_ERR_INVALID_ARG, (a, b)
        for lower, upper in ((a, b), (b, a)):
            n = sizes[lower][0]
            if n % 16 == 0 and n > 16:  # the last 16 bytes of one; then side by side
                assert call(lib, degree, ROWS, dtype, {**apart, upper: apart[lower] + n - 16}) == eq.EQMP_ERR_INVALID_ARG, (a, b)
                assert call(lib, degree, ROWS, dtype, {**apart, upper: apart[lower] + n}) == eq.EQMP_ERR_CUDA, (a, b)


def test_skipped_outputs_meet_nothing(lib):
    sizes = _sizes(True, ROWS, 4)[1]
    apart = {k: STEP * (i + 1) for i, k in enumerate(sizes)}
    assert _backward(lib, True, ROWS, 0, {**apart, "gw": None, "gb": None, "ws": apart["gr"]}) == eq.EQMP_ERR_CUDA
    assert _forward(lib, True, ROWS, 0, {**apart, "b": None, "s": None, "y": STEP * 30}) == eq.EQMP_ERR_CUDA


def test_no_rows(lib):
    """The zeros of the sums over no rows are refused over w, and rows of no length meet nothing."""
    sizes = _sizes(True, 0, 4)[1]
    apart = {k: STEP * (i + 1) for i, k in enumerate(sizes)}
    assert _backward(lib, True, 0, 0, {**apart, "gw": apart["w"]}) == eq.EQMP_ERR_INVALID_ARG
    assert _backward(lib, True, 0, 0, {**apart, "gw": apart["x"], "gb": None}) == eq.EQMP_ERR_CUDA


def test_dropout_in_place_and_its_counter(lib):
    d = _drop(STEP)
    call = lambda x, ld, out, rows=ROWS: lib.eqmp_dropout(x, ld, 0, rows, C * K, d, out, 0)  # noqa: E731
    assert call(2 * STEP, C * K, 3 * STEP) == eq.EQMP_ERR_CUDA
    assert call(2 * STEP, C * K, 2 * STEP) == eq.EQMP_ERR_CUDA  # in place
    assert call(2 * STEP, C * K, 2 * STEP + 4) == eq.EQMP_ERR_INVALID_ARG
    assert call(2 * STEP, 2 * C * K, 2 * STEP) == eq.EQMP_ERR_INVALID_ARG
    assert call(2 * STEP, C * K, STEP - 8) == eq.EQMP_ERR_INVALID_ARG  # over the counter
    assert call(2 * STEP, C * K, STEP + 8) == eq.EQMP_ERR_CUDA
