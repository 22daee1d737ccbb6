"""What the entries of a serving step refuse, and do not, where arguments share memory.
Pointers are fake addresses that are never touched: what passes the checks ends with the
launch's error on a machine without a GPU, and is not tried on one with it."""
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from test_step_abi import A, BAD, D, assign  # noqa: E402

here = pytest.mark.skipif(torch.cuda.is_available(), reason="calls that pass the checks would run on fake addresses")


@pytest.mark.parametrize("kw", [dict(first=A + 0x1000), dict(own_len=A + 0x1000), dict(q_start=A + 0x1000),
                                dict(free_left=A + 0x1000), dict(positions=A + 0x1000)])
def test_counts_are_not_written(kw):
    """count is read only: no output may be it, not even as a whole."""
    assert assign(**kw) == BAD


@here
@pytest.mark.parametrize("kw", [{}, dict(own_len=A), dict(free_left=D)])
def test_lengths_and_list_in_place(kw):
    assert assign(**kw) == bl.ERR_LAUNCH
