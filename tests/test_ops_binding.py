"""The Python side of the token-side operators, without a GPU: what it accepts, what it does
around a call and what it says when it refuses."""
import pytest
import torch

from activation_implicit_gemm_gb300 import _build, _ops


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    _ops._start()


# ------------------------------------------------------------------------ forms of positions

def rope_plan(shape, sections, batch=2, tokens=6):
    q = torch.zeros(batch, tokens, 3, 16)
    freq = torch.ones(8 if sections is None else sum(sections))
    return _ops._rope_plan(q, None, torch.zeros(shape, dtype=torch.int32), freq, sections, "half",
                           False, q, None, -1)


@pytest.mark.parametrize("shape", [(6,), (6, 1), (1, 6), (2, 6), (1, 6, 1), (2, 6, 1)])
@pytest.mark.parametrize("sections", [None, (8,)])
def test_positions_of_one_axis(shape, sections):
    rope_plan(shape, sections)


@pytest.mark.parametrize("shape", [(6, 2), (1, 6, 2), (2, 6, 2)])
def test_positions_of_two_axes(shape):
    rope_plan(shape, (3, 5))


@pytest.mark.parametrize("shape,sections", [
    ((5,), None), ((3, 6), None), ((6, 2), None), ((2, 6, 2), None), ((6,), (3, 5)),
    ((2, 6), (3, 5)), ((1, 6), (3, 5)), ((6, 3), (3, 5)), ((3, 6, 2), (3, 5)), ((), None),
    ((1, 2, 6, 1), None)])
def test_positions_that_do_not_fit(shape, sections):
    with pytest.raises(ValueError, match="positions"):
        rope_plan(shape, sections)


def test_positions_of_one_token_a_sequence():
    """Two axes of length one are the same thing either way round."""
    for shape in ((4,), (4, 1), (1, 4)):
        rope_plan(shape, None, batch=1, tokens=4)
    for shape in ((1,), (1, 1), (4, 1), (1, 1, 1), (4, 1, 1)):
        rope_plan(shape, None, batch=4, tokens=1)
