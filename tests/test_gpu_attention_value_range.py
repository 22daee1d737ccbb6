"""Attention where V_scales are zero, very small or very large, for all of a row's keys or
for those that it meets first: the header's promise, that a bf16 call of many rows rounds a
weight p V_scale to 11 bits or to 2^-27 of the row's largest, holds whichever keys come
first.  The bounds are those of test_gpu_attention_masked.py, whose terms are all relative
to the row's own p |v| and p V_scale."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402
from ternary_weight_linear_forward_amd import synth  # noqa: E402

from gpu_helpers import to_dev  # noqa: E402
from test_gpu_attention import Setup  # noqa: E402
from test_gpu_attention_masked import call, compare, reference, tree_sight, window_sight, words  # noqa: E402

pytestmark = pytest.mark.gpu

ROWS = [(8, 128, 1, "bf16"), (8, 128, 60, "bf16"), (4, 64, 40, "bf16"), (8, 256, 20, "bf16"), (8, 128, 60, "f32"),
        (8, 64, 60, "f32"), (8, 128, 2, "f32")]  # heads, D, query tokens


def near_ones(n, heads, D, dtype):
    """Queries near (1, 1, ..), so that a key of equal bytes has a high score with all of them."""
    x = (1.0 + 0.1 * synth.activations_f32(n * heads, D, 3)).astype(np.float32).reshape(n, heads, D)
    bits = synth.to_bf16_bits(x) if dtype == "bf16" else x
    return to_dev(bits), synth.bf16_bits_to_f32(bits).reshape(x.shape) if dtype == "bf16" else x


def own_key(st, t, byte=None, vs=None):
    page, at = st.lists[1][t // st.page], t % st.page
    if byte is not None:
        st.k[page, :, at] = byte
        st.ks[page, :, at] = 0.03
    if vs is not None:
        st.vs[page, :, at] = vs


def both(st, heads, D, n, dtype, window, sinks):
    own = st.own[0]
    qt, q = near_ones(n, heads, D, dtype)
    o, lse = call(st, qt, [n], entry=bl.attention_window, window=window, sinks=sinks)
    compare(o, lse, reference(st, q, [n], lambda b: window_sight(0, own, n, window, sinks), D ** -0.5, dtype))
    bits = np.random.default_rng(n).random((n, n)) < 0.5
    o, lse = call(st, qt, [n], entry=bl.attention_tree, tree=to_dev(words([bits], n)))
    compare(o, lse, reference(st, q, [n], lambda b: tree_sight(0, own, n, bits), D ** -0.5, dtype))


@pytest.mark.parametrize("heads,D,n,dtype", ROWS)
@pytest.mark.parametrize("sinks,nats", [(1, 14), (4, 20), (3, 60), (2, 150)])
def test_first_tokens_without_a_value(heads, D, n, dtype, sinks, nats):
    """First tokens that draw much of the softmax and whose values are zero, as trained models have them."""
    print("zero sinks", heads, D, n, dtype, sinks, nats, flush=True)
    st = Setup(1, D, 64, 0, [500], seed=D + n)
    for t in range(sinks):  # score: D^-1/2 0.03 byte D
        own_key(st, t, byte=0, vs=0.0)
        page = st.lists[1][0]
        st.k[page, :, t] = 100
        st.ks[page, :, t] = nats / (D ** 0.5 * 100)
    both(st, heads, D, n, dtype, 300, sinks)


@pytest.mark.parametrize("heads,D,n,dtype", ROWS)
@pytest.mark.parametrize("zeros,rest", [(32, 1e-8), (64, 0.02), (64, 1e-8), (200, 1e-12), (31, 2.0 ** -80)])
def test_values_that_come_late(heads, D, n, dtype, zeros, rest):
    """The first keys' values are zero, those of the rest small; scores of one size."""
    print("late values", heads, D, n, dtype, zeros, rest, flush=True)
    st = Setup(1, D, 64, 0, [500], seed=D + n)
    for t in range(500):
        own_key(st, t, vs=0.0 if t < zeros else rest)
    both(st, heads, D, n, dtype, 400, 64)


@pytest.mark.parametrize("heads,D,n,dtype", ROWS)
@pytest.mark.parametrize("sizes", [[-60], [-66], [-90], [60], [90], [-90, -7, -60], [-7, -90], [90, -7], [-90, 60], [0, None, -70],
                                   [None, -50, None, -3]])
def test_values_of_any_size(heads, D, n, dtype, sizes):
    """V_scales near 2^size by blocks of 64 keys (None: zero)."""
    print("value sizes", heads, D, n, dtype, sizes, flush=True)
    st = Setup(1, D, 64, 0, [450], seed=D + n)
    for j, page in enumerate(st.lists[1]):
        e = sizes[j % len(sizes)]
        st.vs[page] *= np.float32(0.0 if e is None else 2.0 ** (e + 5))
    both(st, heads, D, n, dtype, 300, 70)


@pytest.mark.parametrize("dtype,n", [("bf16", 60), ("f32", 60), ("bf16", 2)])
@pytest.mark.parametrize("small", [0.0, 2.0 ** -70])
def test_parts_that_begin_without_a_value(dtype, n, small):
    """A long cache, cut into parts: parts whose keys have values of zero (or very small ones) throughout, and parts that
    begin with them, under high and low scores."""
    print("parts", dtype, n, small, flush=True)
    own, D = 6500, 64
    st = Setup(1, D, 64, 0, [own], seed=n)
    rng = np.random.default_rng(7)
    for j, page in enumerate(st.lists[1]):
        if j % 7 in (0, 1, 2) or 30 <= j < 60:
            st.vs[page] = np.where(np.isnan(st.vs[page]), st.vs[page], np.float32(small))
            st.ks[page] *= np.float32(rng.choice([0.3, 3.0]))
    both(st, 8, D, n, dtype, 6000, 100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_grow_over_values_that_shrink(dtype):
    """Every block's scores far above the last one's and its values far below, to 2^-100, and the other way round: sums
    and weights run apart by more than either type's range allows in one unit."""
    D, n, own = 64, 60, 900
    for turn in (1, -1):
        st = Setup(1, D, 64, 0, [own], seed=4)
        for j, page in enumerate(st.lists[1][::turn]):
            st.k[page] = 90
            st.ks[page] = np.where(np.isnan(st.ks[page]), st.ks[page], np.float32(0.005 + 0.008 * j))
            st.vs[page] *= np.float32(2.0 ** (-6 * j))
        both(st, 8, D, n, dtype, 800, 50)
