"""Positions up to 2^31, the most that prefix_len and max_own allow, over a cache of one long
page that the page lists name again and again."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402
from test_gpu_attention import PLACE, U, check, queries  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,dtype,window,sinks", [(128, "bf16", 10, 0), (128, "f32", 10, 0), (128, "bf16", 63, 5), (4, "bf16", 10, 0),
                                                      (128, "bf16", 200, 70)])
def test_a_window_at_the_end(heads, dtype, window, sinks):
    """The last query of 2^30 own keys behind a prefix of 2^30 sees its window's keys and the first ones alone."""
    print("far", heads, dtype, window, sinks, flush=True)
    D, page, far = 16, 1 << 20, 1 << 30
    rng = np.random.default_rng(3)
    k = rng.integers(-128, 128, (1, 1, page, D)).astype(np.int8)
    v = rng.integers(-128, 128, (1, 1, page // 64, D, 64)).astype(np.int8)
    ks, vs = [(0.02 + 0.02 * rng.random((1, 1, page))).astype(np.float32) for _ in range(2)]
    cache = bl.KVCache(to_dev(k), to_dev(v), to_dev(ks), to_dev(vs), D)
    pages = torch.zeros(far // page, dtype=torch.int32, device="cuda")
    qt, q = queries(1, heads, D, 5, dtype)
    o, lse = bl.attention_window(cache, qt, pages[None], torch.tensor([far], dtype=torch.int32, device="cuda"), far, window,
                                 sinks, prefix_pages=pages, prefix_len=far, return_lse=True)
    torch.cuda.synchronize()
    t = np.concatenate([np.arange(sinks), np.arange(page - window, page)])  # (2^31 and 0 are multiples of the page)
    kk = k[0, 0, t].astype(np.float64) * ks[0, 0, t].astype(np.float64)[:, None]
    vv = v[0, 0, t // 64, :, PLACE[t % 64]].astype(np.float64) * vs[0, 0, t].astype(np.float64)[:, None]
    s = D ** -0.5 * (q[0].astype(np.float64) @ kk.T)
    A = (D ** -0.5 * (np.abs(q[0].astype(np.float64)) @ np.abs(kk).T)).max(1)
    w = np.exp(s - s.max(1)[:, None])
    p = w / w.sum(1)[:, None]
    want, n = p @ vv, len(t)
    e = (D + 16) * U * A + 2.0 ** -21 * A + 8 * U * (A + np.abs(s).max(1))
    rel = 2 * e + (n + 16) * U + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21)
    bound = rel[:, None] * (p @ np.abs(vv)) + (2.0 ** -8 if dtype == "bf16" else U) * np.abs(want)
    if dtype == "bf16":
        bound += (n * 2.0 ** -20 * (p * vs[0, 0, t]).max(1))[:, None]
    check(o, want[None], bound[None])
    wl = s.max(1) + np.log(w.sum(1))
    assert np.all(np.abs(to_host(lse)[0] - wl) <= 2 * e + (n + 16) * U + 4 * U * np.abs(wl))
