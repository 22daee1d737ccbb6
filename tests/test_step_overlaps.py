"""What the entries of a serving step refuse, and do not, where arguments share memory.
Pointers are fake addresses that are never touched: what passes the checks ends with the
launch's error on a machine without a GPU, and is not tried on one with it."""
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from test_step_abi import A, BAD, D, F, G, assign, tree  # noqa: E402

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


@here
def test_a_column_of_a_wider_tree():
    """Rows of a tree hold ceil(min(max_q, tokens) / 64) words: what lies behind the last row's is not the tree's, and may
    be an output."""
    column = G - (5 * 4 + 1) * 8  # six rows of one word, four words apart, that end where O begins
    assert tree(tree=column, ld_tree=4) == bl.ERR_LAUNCH
    assert tree(tree=column + 8, ld_tree=4) == BAD
    assert tree(tree=column, ld_tree=4, lse=column + 5 * 32) == BAD
    two = G - (69 * 4 + 2) * 8  # 70 tokens: two words
    more = dict(tokens=70, seqs=1, max_q=70, ldo_token=1024, q_start=F + 0x200, lse=None, ld_tree=4, ws=G + 0x2000000)
    assert tree(tree=two, **more) == bl.ERR_LAUNCH
    assert tree(tree=two + 8, **more) == BAD
