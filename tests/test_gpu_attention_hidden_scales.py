"""A hidden key whose scales are -inf reaches no row: keys outside every window, drafted
tokens that a row does not see, the unwritten rest of a sequence's last block.  The bounds are those of the calls without such keys."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev  # noqa: E402
from test_gpu_attention import Setup, queries  # noqa: E402
from test_gpu_attention_masked import call, compare, grown_tree, reference, tree_sight, window_sight, words  # noqa: E402

pytestmark = pytest.mark.gpu
NOWHERE = float("-inf")


def blank(st):
    """Every place that holds no key: -inf."""
    st.ks[np.isnan(st.ks)] = NOWHERE
    st.vs[np.isnan(st.vs)] = NOWHERE


def put(st, which, tokens):
    """Scales of -inf at own tokens; what they were."""
    kept = st.ks.copy(), st.vs.copy()
    for t in tokens:
        page = st.lists[which][t // st.page]
        st.ks[page, :, t % st.page] = st.vs[page, :, t % st.page] = NOWHERE
    return kept


@pytest.mark.parametrize("heads,D,n,dtype", [(8, 128, 1, "bf16"), (8, 128, 80, "bf16"), (8, 64, 80, "bf16"), (8, 256, 80, "bf16"),
                                             (8, 128, 1, "f32"), (8, 128, 80, "f32"), (8, 64, 80, "f32"), (8, 64, 10, "f32"),
                                             (4, 200, 80, "f32")])
def test_hidden_scales_of_minus_infinity(heads, D, n, dtype):
    print("hidden -inf", heads, D, n, dtype, flush=True)
    own, window, sinks = 1000, 200, 65
    qt, q = queries(n, heads, D, 5, dtype)
    # outside every window, and behind the last key
    st = Setup(1, D, 64, 150, [own], seed=n + D)
    see = window_sight(150, own, n, window, sinks)
    kept = put(st, 1, [t for t in range(own) if not see[:, 150 + t].any()])
    blank(st)
    o, lse = call(st, qt, [n], entry=bl.attention_window, window=window, sinks=sinks)
    st.ks, st.vs = kept
    compare(o, lse, reference(st, q, [n], lambda b: see, D ** -0.5, dtype))
    # drafted tokens that no row sees
    st = Setup(1, D, 64, 0, [own], seed=n + D + 1)
    bits = grown_tree(np.random.default_rng(n), n)
    bits[:, n // 2] = False
    kept = put(st, 1, [own - n + n // 2])
    blank(st)
    o, lse = call(st, qt, [n], entry=bl.attention_tree, tree=to_dev(words([bits], n)))
    st.ks, st.vs = kept
    compare(o, lse, reference(st, q, [n], lambda b: tree_sight(0, own, n, bits), D ** -0.5, dtype))
