"""Queries of any size that their type holds, with a scale to match: bf16 rows of up to 2^120
whose products with the keys would pass binary32's range, and of 2^-100.  Scores, and so the
bounds, are those of ordinary queries."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402
from test_gpu_attention import Setup, check, queries  # noqa: E402
from test_gpu_attention_masked import call, compare, reference, tree_sight, window_sight, words  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D,n", [(8, 128, 1), (8, 128, 60), (8, 64, 60), (8, 256, 20)])
@pytest.mark.parametrize("size", [120, 100, 62, 58, -100])
def test_queries_of_any_size(dtype, heads, D, n, size):
    print("query size", dtype, heads, D, n, size, flush=True)
    st = Setup(1, D, 64, 0, [400], seed=D + n)
    qt, q = queries(n, heads, D, 7, dtype)
    qt, q = qt * 2.0 ** size, (q * np.float32(2.0 ** size)).astype(np.float32)  # (powers of two: exact)
    assert bool(torch.isfinite(qt).all()) and np.isfinite(q).all()
    scale = float(np.float32(D ** -0.5 * 2.0 ** -size))
    for sign in (1.0, -1.0):
        o, lse = call(st, qt, [n], entry=bl.attention_window, window=300, sinks=4, scale=sign * scale)
        compare(o, lse, reference(st, q, [n], lambda b: window_sight(0, 400, n, 300, 4), sign * scale, dtype))
    bits = np.random.default_rng(n).random((n, n)) < 0.5
    o, lse = call(st, qt, [n], entry=bl.attention_tree, tree=to_dev(words([bits], n)), scale=scale)
    compare(o, lse, reference(st, q, [n], lambda b: tree_sight(0, 400, n, bits), scale, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D,n", [(8, 128, 1), (8, 128, 60), (8, 64, 60), (8, 256, 20)])
def test_a_scale_of_zero(dtype, heads, D, n):
    """All keys alike: the values' mean; a NaN in a query still shows."""
    print("scale 0", dtype, heads, D, n, flush=True)
    st = Setup(1, D, 64, 0, [400], seed=D + n)
    qt, q = queries(n, heads, D, 7, dtype)
    qt[n - 1, 3, 5] = float("nan")
    bad = np.zeros((n, heads), bool)
    bad[n - 1, 3] = True
    o, lse = call(st, qt, [n], entry=bl.attention_window, window=300, sinks=4, scale=0.0)
    o64, bound, wl, wb = reference(st, q, [n], lambda b: window_sight(0, 400, n, 300, 4), 0.0, dtype)
    keep = to_dev(~bad)
    check(torch.where(keep[..., None], o, torch.zeros_like(o)), np.where(bad[..., None], 0.0, o64), bound)
    got = to_host(lse)
    assert np.all(np.abs(got - wl)[~bad] <= wb[~bad])
    assert bool(torch.isnan(o)[~keep].all()) and np.isnan(got[bad]).all()
