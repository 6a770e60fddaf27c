"""GPU parity of the norms in each form that their kernels are made in, against the float64 oracle within the derived
bounds (norm_util).

A row kernel is made for a type, a degree, a width of the vectors, a number of vectors a lane, a place where rows begin
and a mode (nothing beside the norm; residual sum and dropout by units; dropout drawn lane by lane).  The number of vectors
hangs on the width and on whether rows are few, so each width stands with enough rows for its own; the plain mode runs
only where neither s nor, backward, a second gradient is asked for."""
import pytest

from tests.test_gpu_norm import Case, _check, eq  # noqa: F401

pytestmark = pytest.mark.gpu

# rows, columns: few rows (8 values a lane); then 16 values, or 12, 24 and 32 in the forward pass; rows of 16 warps
ALIGNED = [(301, 64), (12007, 48), (12007, 64), (6007, 96), (1009, 768), (1501, 1000), (1501, 1024), (607, 1536), (12, 6144),
           (12, 8192)]
ODD = [(301, 77), (12007, 37), (3001, 131), (1501, 509), (1009, 767), (1009, 1021), (503, 1537), (12, 4223), (12, 6147),
       (12, 8099)]
# inputs that lie otherwise than the outputs: padded rows
APART = [(301, 77), (12007, 37), (3001, 131), (1501, 509), (1009, 767), (503, 1536), (12, 4223), (12, 6147), (12, 8099)]
# outputs that do not begin on 16 bytes: single values
SINGLE = [(301, 77), (301, 64), (12, 8099)]
LAYER = ([("aligned", *s) for s in ALIGNED] + [("odd", *s) for s in ODD] + [("apart", *s) for s in APART] +
         [("single", *s) for s in SINGLE])
# atoms, channels (None: about 6100 values a row)
FEATURES = [("aligned", 301, 8), ("aligned", 2503, 8), ("aligned", 1303, 32), ("aligned", 7, None), ("odd", 301, 5),
            ("odd", 2503, 7), ("odd", 1303, 31), ("odd", 7, None), ("single", 33, 6), ("single", 7, None)]


def _behind(like, by=1):
    """An empty tensor like `like` that begins `by` elements behind an aligned address."""
    import torch

    return torch.empty(like.numel() + 16, dtype=like.dtype, device=like.device)[by:by + like.numel()].view(like.shape)


def _both_passes(eq, c, plain, single=False):  # noqa: F811
    like = c.x.new_empty(c.shape)
    fneed, bneed = (("y", "stats"), ("x", "w", "b")) if plain else (("y", "s", "stats"), ("x", "r", "w", "b"))
    out = (lambda names: {k: _behind(like) for k in names}) if single else (lambda names: None)
    got = c.forward(eq, need=fneed, out=out([k for k in fneed if k != "stats"]))
    _check(got, *c.forward_bounds())
    s = c.x if plain else got["s"]
    back = c.backward(eq, s, got["stats"], need=bneed, out=out([k for k in bneed if k in "xr"]))
    _check(back, *c.backward_bounds(s, got["stats"]))


def _divisor(n):
    return next((d for d in range(2, n) if n % d == 0), n)


@pytest.mark.parametrize("form", ["plain", "elements", "units"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("place,rows,cols", LAYER)
def test_layer_norm_forms(eq, place, rows, cols, bf16, form):  # noqa: F811
    kw = dict(plain=dict(), elements=dict(residual=True, p=0.3),
              units=dict(residual=True, p=0.3, group=8 if cols % 8 == 0 else _divisor(cols)))[form]
    _both_passes(eq, Case((rows, cols), bf16=bf16, pad=5 if place == "apart" else 0, **kw), form == "plain", place == "single")


@pytest.mark.parametrize("form", ["plain", "channels"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("l_max", [3, 4, 5, 6])
@pytest.mark.parametrize("place,atoms,channels", FEATURES)
def test_degree_norm_forms(eq, place, atoms, channels, l_max, bf16, form):  # noqa: F811
    K = (l_max + 1) ** 2
    if channels is None:
        channels = 6144 // K // 8 * 8 if place == "aligned" else 6100 // K | 1
    kw = dict(residual=True, p=0.3) if form == "channels" else {}
    _both_passes(eq, Case((atoms, channels, K), bf16=bf16, shift=int(place == "single"), **kw), form == "plain")


@pytest.mark.parametrize("form", [dict(), dict(residual=True, p=0.3), dict(residual=True, p=0.3, group=2), dict(residual=True)],
                         ids=lambda f: "_".join(f"{k}{v}" for k, v in f.items()) or "plain")
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rows,cols", [(301, 64), (12007, 64), (1501, 1000), (1501, 1024), (12, 8192)])
@pytest.mark.parametrize("by", [0, 1])
def test_parameters_at_any_place(eq, rows, cols, bf16, form, by):  # noqa: F811
    """w and b off 16-byte boundaries (by 1), and without them (by 0), at each number of values a lane."""
    c = Case((rows, cols), bf16=bf16, affine=bool(by), **form)
    if by:
        c.w, c.b = _behind(c.w).copy_(c.w), _behind(c.b).copy_(c.b)
    _both_passes(eq, c, not form)
