"""Attention calls at their host bounds: bounds larger than what a call holds, rows
of very different sizes in one tile, long causal prompts.  The reference and its
error bound are those of test_gpu_attention."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402
from test_gpu_attention import Setup, check, queries, reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kvh,D,prefix,nq,max_q,dtype", [
    (64, 8, 128, 3000, [5, 0, 6, 1], 13, "bf16"),
    (8, 8, 128, 3000, [30, 1, 60, 5], 100, "bf16"),
    (8, 8, 64, 1600, [1, 9, 0, 20] * 2, 100, "f32"),
])
def test_max_q_above_the_tokens(heads, kvh, D, prefix, nq, max_q, dtype):
    """max_q is a bound: a call with fewer tokens than it gives what a tight bound gives."""
    print("attention max_q", heads, kvh, D, prefix, nq, max_q, dtype, flush=True)
    own = [n + 7 * b for b, n in enumerate(nq)]
    st = Setup(kvh, D, 64, prefix, own, seed=D + max_q)
    qt, q = queries(sum(nq), heads, D, 12, dtype)
    start = to_dev(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32))
    for max_own in (max(own), 0):
        ln = own if max_own else [0] * len(own)
        o, lse = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array(ln, np.int32)), max_own,
                              prefix_pages=to_dev(st.prefix_pages), prefix_len=prefix, q_start=start, max_q=max_q,
                              return_lse=True)
        torch.cuda.synchronize()
        if max_own == 0:
            st.own = ln
        want, bound, wl, wb = reference(st, q, nq, D ** -0.5, dtype)
        check(o, want, bound)
        assert np.all(np.abs(to_host(lse) - wl) <= wb)
