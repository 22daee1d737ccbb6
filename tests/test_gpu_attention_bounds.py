"""Attention calls at their host bounds: bounds larger than what a call holds, rows
of very different sizes in one tile, long causal prompts.  The reference and its
error bound are those of test_gpu_attention."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402
from test_gpu_attention import U, Setup, check, queries, reference  # noqa: E402

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


@pytest.mark.parametrize("heads,kvh,D,nq,prefix,dtype", [
    (8, 1, 128, [1] * 28, 6500, "bf16"), (8, 1, 100, [1] * 14, 6500, "bf16"), (8, 2, 64, [1] * 38, 6500, "f32"),
    (8, 1, 128, [40, 3], 70, "bf16"), (8, 2, 128, [2] * 3, 70, "bf16"), (4, 1, 50, [50], 0, "f32")])
@pytest.mark.parametrize("stray", [1e38, float("inf"), float("nan")])
def test_rows_do_not_touch_one_another(heads, kvh, D, nq, prefix, dtype, stray):
    """Rows of one tile belong to different tokens, those of the prefix also to different sequences: queries of very
    different sizes, and tokens of no sequence (the first and the last) that hold anything, leave every other row
    within its own bound."""
    tokens = sum(nq) + 2
    print("attention stray", heads, kvh, D, tokens, prefix, dtype, stray, flush=True)
    own = [n + 5 * b % 70 for b, n in enumerate(nq)]
    st = Setup(kvh, D, 64, prefix, own, seed=D + tokens)
    qt, q = queries(tokens, heads, D, 13, dtype)
    sizes = np.array([1.0, 2.0 ** -30, 8.0, 2.0 ** -9, 2.0 ** 7, 2.0 ** -7, 2.0 ** -100])[np.arange(tokens) % 7]
    q = q * sizes[:, None, None].astype(np.float32)  # (powers of two: exact)
    qt = qt * torch.tensor(sizes, dtype=qt.dtype, device="cuda")[:, None, None]
    qt[0], qt[-1] = stray, -stray
    qt[-1, :, ::3] = 1.0
    start = to_dev((1 + np.concatenate([[0], np.cumsum(nq)])).astype(np.int32))
    out = torch.full((tokens, heads, D), -9.0, dtype=qt.dtype, device="cuda")
    _, lse = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array(own, np.int32)), max(own),
                          prefix_pages=to_dev(st.prefix_pages), prefix_len=prefix, q_start=start, max_q=max(nq),
                          out=out, return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q[1:-1], nq, D ** -0.5, dtype)
    check(out[1:-1], want, bound)
    assert np.all(np.abs(to_host(lse)[1:-1] - wl) <= wb)
    assert bool((out[0] == -9).all()) and bool((out[-1] == -9).all())


def test_a_million_places_in_the_batch():
    """2^20 sequences of 256 heads, 64 of them with a token: workgroups and join rows past 2^32 threads."""
    print("attention 2^20 sequences", flush=True)
    seqs, heads, kvh, D, prefix = 1 << 20, 256, 4, 16, 100
    lens = [(7 * b) % 64 for b in range(64)]
    st = Setup(kvh, D, 64, prefix, lens, seed=3)
    qt, q = queries(64, heads, D, 14, "bf16")
    where = np.sort(np.random.default_rng(5).permutation(seqs)[:64])  # the sequences that have their one token
    where[0], where[-1] = 0, seqs - 1
    has = np.zeros(seqs, np.int64)
    has[where] = 1
    start = to_dev(np.concatenate([[0], np.cumsum(has)]).astype(np.int32))
    own = np.full(seqs, 64, np.int32)
    own[where] = lens
    table = np.full((seqs, 1), -1, np.int32)
    table[where] = st.table[:, :1]
    o, lse = bl.attention(st.cache(), qt, to_dev(table), to_dev(own), 64, prefix_pages=to_dev(st.prefix_pages),
                          prefix_len=prefix, q_start=start, max_q=1, return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q, [1] * 64, D ** -0.5, "bf16")
    check(o, want, bound)
    assert np.all(np.abs(to_host(lse) - wl) <= wb)


@pytest.mark.parametrize("heads,kvh,D,prefix,own,nq,at,dtype", [
    (8, 1, 128, 70, 300, 90, 260, "bf16"), (8, 1, 128, 0, 64, 64, 33, "bf16"), (2, 2, 128, 200, 70, 40, 40, "f32"),
    (8, 2, 64, 10, 130, 100, 127, "f32"), (4, 4, 100, 0, 90, 20, 75, "bf16"), (8, 1, 256, 30, 50, 50, 20, "bf16")])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_hidden_keys_may_hold_anything(heads, kvh, D, prefix, own, nq, at, dtype, bad):
    """A prompt's token whose key and value are not finite: the queries before it, which do not see it, are as if it
    were not there."""
    print("attention hidden", heads, kvh, D, prefix, own, nq, at, dtype, bad, flush=True)
    st = Setup(kvh, D, 64, prefix, [own], seed=D + at)
    qt, q = queries(nq, heads, D, 15, dtype)
    page = st.lists[1][at // 64]
    cache = st.cache()
    cache.k_scale[page, :, at % 64] = bad
    cache.v_scale[page, :, at % 64] = bad
    o, lse = bl.attention(cache, qt, to_dev(st.table), to_dev(np.array([own], np.int32)), own,
                          prefix_pages=to_dev(st.prefix_pages), prefix_len=prefix, max_q=nq, return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q, [nq], D ** -0.5, dtype)
    free = at - (own - nq)  # queries 0 .. free - 1 see keys 0 .. own - nq + free - 1 = at - 1 at most
    check(o[:free], want[:free], bound[:free])
    assert np.all(np.abs(to_host(lse)[:free] - wl[:free]) <= wb[:free])


@pytest.mark.parametrize("heads,kvh,D,nq,dtype", [(4, 2, 64, 1, "f32"), (8, 1, 128, 1, "bf16"), (8, 1, 128, 40, "bf16")])
def test_lengths_are_cut_to_their_bound(heads, kvh, D, nq, dtype):
    """own_len past max_own counts as max_own, also inside keys that are there, and below 0 as 0."""
    print("attention cut", heads, kvh, D, nq, dtype, flush=True)
    st = Setup(kvh, D, 64, 40, [300, 90, 300], seed=D + nq)
    qt, q = queries(3 * nq, heads, D, 16, dtype)
    o = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array([1 << 30, -(1 << 31), 151], np.int32)), 150,
                     prefix_pages=to_dev(st.prefix_pages), prefix_len=40, max_q=nq)
    torch.cuda.synchronize()
    st.own = [150, 0, 150]
    want, bound, _, _ = reference(st, q, [nq] * 3, D ** -0.5, dtype)
    check(o, want, bound)


@pytest.mark.parametrize("heads,kvh,D,n,prefix,dtype", [(2, 1, 128, 2048, 0, "bf16"), (2, 2, 64, 1100, 0, "f32"),
                                                        (2, 1, 128, 900, 300, "f32"), (1, 1, 256, 800, 0, "bf16")])
def test_a_prompt_into_an_empty_cache(heads, kvh, D, n, prefix, dtype):
    """Every token of a sequence is a query: the first sees one key of its own, the last all of them."""
    print("attention causal", heads, kvh, D, n, prefix, dtype, flush=True)
    st = Setup(kvh, D, 64, prefix, [n], seed=D + n)
    qt, q = queries(n, heads, D, 17, dtype)
    o, lse = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array([n], np.int32)), n,
                          prefix_pages=to_dev(st.prefix_pages), prefix_len=prefix, max_q=n, return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q, [n], D ** -0.5, dtype)
    check(o, want, bound)
    assert np.all(np.abs(to_host(lse) - wl) <= wb)


@pytest.mark.parametrize("heads,kvh,D,tokens", [(64, 8, 160, 400), (64, 8, 64, 1500), (64, 8, 64, 12), (32, 32, 100, 700)])
def test_every_weight_of_fp32_queries_has_22_bits(heads, kvh, D, tokens):
    """Rows of seven keys with values (and 63 of value 0 before them), so that a single weight off by a step of its
    first term shows: among hundreds of thousands of weights some lie at the middle between two binary16 numbers,
    where both terms have to agree on the first."""
    print("attention terms", heads, kvh, D, tokens, flush=True)
    n, G = 70, heads // kvh
    worst = 0.0
    for seed in range(4):
        st = Setup(kvh, D, 64, n, [0], seed=100 + seed)
        st.vs[st.lists[0][0], :, 1:] = 0.0
        qt, q = queries(tokens, heads, D, 20 + seed, "f32")
        o = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array([0], np.int32)), 0,
                         prefix_pages=to_dev(st.prefix_pages), prefix_len=n, max_q=tokens)
        torch.cuda.synchronize()
        k, v = st.rows(st.lists[0], n)
        qq = q.astype(np.float64).reshape(tokens, kvh, G, D)
        s = D ** -0.5 * np.einsum("thgd,nhd->thgn", qq, k)
        A = D ** -0.5 * np.einsum("thgd,nhd->thgn", np.abs(qq), np.abs(k)).max(-1)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        want, size = np.einsum("thgn,nhd->thgd", p, v), np.einsum("thgn,nhd->thgd", p, np.abs(v))
        e = (D + 16) * U * A + 2.0 ** -21 * A + 8 * U * (A + np.abs(s).max(-1))
        bound = (2 * e + (n + 16) * U + 2.0 ** -21)[..., None] * size + U * np.abs(want)
        err = np.abs(to_host(o).astype(np.float64).reshape(want.shape) - want)
        worst = max(worst, (err / bound).max())
    assert worst <= 1.0
