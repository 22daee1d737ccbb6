"""A query row that holds a NaN gets NaN as its output and as its lse, however the call is
cut, and no other row is touched."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402
from test_gpu_attention import Setup, check, queries  # noqa: E402
from test_gpu_attention_masked import call, reference, tree_sight, window_sight, words  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", ["attention", "window", "tree"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kvh,D,prefix,own,nq", [
    (8, 1, 128, 0, [60], [9]),              # one part
    (8, 1, 128, 0, [200, 90], [80, 40]),
    (8, 2, 64, 0, [6500], [2]),             # parts, joined
    (8, 1, 64, 0, [6500, 900], [40, 40]),
    (8, 1, 128, 7000, [20, 30], [3, 4]),    # a prefix of its own pass
    (4, 1, 200, 100, [900], [70]),
])
def test_a_nan_stays_in_its_row(entry, dtype, heads, kvh, D, prefix, own, nq):
    print("nan", entry, dtype, heads, kvh, D, prefix, own, nq, flush=True)
    st = Setup(kvh, D, 64, prefix, own, seed=D + sum(nq))
    tokens = sum(nq)
    qt, q = queries(tokens, heads, D, 6, dtype)
    rng = np.random.default_rng(tokens)
    bad = np.zeros((tokens, heads), bool)
    for t in (0, tokens // 2, tokens - 1):
        h = int(rng.integers(heads))
        bad[t, h] = True
        if t % 2:
            qt[t, h, int(rng.integers(D))] = float("nan")
        else:
            qt[t, h] = float("nan")
    bits = [np.tril(np.ones((n, n), bool)) for n in nq]
    kw = dict(attention={}, window=dict(window=max(own) + prefix - 1, sinks=3), tree=dict(tree=to_dev(words(bits, max(nq)))))
    fn = dict(attention=bl.attention, window=bl.attention_window, tree=bl.attention_tree)[entry]
    o, lse = call(st, qt, nq, max_q=max(nq), entry=fn, **kw[entry])
    see = (lambda b: tree_sight(prefix, own[b], nq[b], bits[b])) if entry == "tree" else \
        (lambda b: window_sight(prefix, own[b], nq[b], max(own) + prefix - (entry == "window"), 3))
    o64, bound, wl, wb = reference(st, q, nq, see, D ** -0.5, dtype)
    keep = to_dev(~bad)
    check(torch.where(keep[..., None], o, torch.zeros_like(o)), np.where(bad[..., None], 0.0, o64), bound)
    got = to_host(lse)
    assert np.all(np.abs(got - wl)[~bad] <= wb[~bad])
    assert bool(torch.isnan(o)[~keep].all()) and np.isnan(got[bad]).all()
