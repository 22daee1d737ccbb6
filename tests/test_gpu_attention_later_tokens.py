"""Causal attention of a prompt with a token whose scales are -inf: the queries before it,
which do not see it, are within the bounds of the call without it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_host  # noqa: E402
from test_gpu_attention import Setup, check, queries, reference  # noqa: E402
from test_gpu_attention_hidden_scales import blank, put  # noqa: E402
from test_gpu_attention_masked import call  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kvh,D,prefix,own,nq,at,dtype", [
    (8, 1, 128, 70, 300, 90, 260, "bf16"), (8, 1, 128, 0, 64, 64, 33, "bf16"), (2, 2, 128, 200, 70, 40, 40, "f32"),
    (8, 2, 64, 10, 130, 100, 127, "f32"), (4, 4, 100, 0, 90, 20, 75, "bf16"), (8, 1, 256, 30, 50, 50, 20, "bf16")])
def test_later_tokens_of_a_prompt(heads, kvh, D, prefix, own, nq, at, dtype):
    print("later -inf", heads, kvh, D, prefix, own, nq, at, dtype, flush=True)
    st = Setup(kvh, D, 64, prefix, [own], seed=D + at)
    qt, q = queries(nq, heads, D, 15, dtype)
    want, bound, wl, wb = reference(st, q, [nq], D ** -0.5, dtype)
    put(st, 1, [at])
    blank(st)
    o, lse = call(st, qt, [nq], max_q=nq, entry=bl.attention)
    free = at - (own - nq)  # queries 0 .. free - 1 see keys 0 .. at - 1 at most
    check(o[:free], want[:free], bound[:free])
    assert np.all(np.abs(to_host(lse)[:free] - wl[:free]) <= wb[:free])
