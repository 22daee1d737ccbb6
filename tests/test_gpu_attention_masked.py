"""Attention with a sliding window and with a tree of drafts over the int8 cache,
against a plain binary64 softmax over the values the cache stands for.

The bound is that of the causal form (test_gpu_attention.py), which takes the keys
that a row sees, whichever they are: with u = 2^-24 and A = scale * sum |q_d k_d|, a
score is off by at most e = (D + 16) u A + 2^-21 A + 8 u S, S <= A + max; a weight by
2 e, sums over n keys by (n + 16) u, the weights' rounding to 11 bits (bf16) or 22
(fp32), and one rounding of the output.

With bf16 queries and many rows a weight w = p V_scale is one binary16 number in units
that bring the largest of a row's first ones to 2^2 (and, when later ones outgrow that,
the largest so far), so that it is off by 2^-11 of itself or by half of binary16's least step, 2^-25 of those
units: at most 2^-27 of the row's largest w.  A value is w times a byte of at most 128,
and o their sum over the n keys: another n 128 2^-27 max(p V_scale), which shows only in
columns where the keys with large weights hold zeros."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402
from test_gpu_attention import U, Setup, check, queries  # noqa: E402

pytestmark = pytest.mark.gpu


def window_sight(P, own, n, window, sinks):
    """Who sees which of P + own keys: [n, P + own]."""
    x = np.arange(P + own)
    end = P + np.clip(own - n + 1 + np.arange(n), 0, own)[:, None]
    return (x < end) & ((x >= end - window) | (x < sinks))


def tree_sight(P, own, n, bits):
    x = np.arange(P + own)
    node = x - (P + own - n)
    see = np.ones((n, P + own), bool)
    for k in np.nonzero((x >= P) & (node >= 0))[0]:
        see[:, k] = bits[:, node[k]]
    return see


def value_scales(st, which, n):
    t = np.arange(n)
    p = np.array(st.lists[which], np.int64)[t // st.page] if n else t
    return st.vs[p, :, t % st.page].astype(np.float64)


def reference(st, q, nq, sight, scale, dtype):
    """(o, bound, lse, lse bound) in binary64; sight(b): [n, keys]."""
    heads, D = q.shape[1:]
    G = heads // st.H
    kp, vp = st.rows(st.lists[0], st.prefix)
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lbound = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    at = 0
    for b, n in enumerate(nq):
        ko, vo = st.rows(st.lists[1 + b], st.own[b])
        k, v, see = np.concatenate([kp, ko]), np.concatenate([vp, vo]), sight(b)
        rows = np.nonzero(see.any(1))[0]
        for h in range(heads if len(rows) else 0):
            kk, vv, qq, m = k[:, h // G], v[:, h // G], q[at + rows, h].astype(np.float64), see[rows]
            s = np.where(m, scale * (qq @ kk.T), -np.inf)
            A = np.where(m, abs(scale) * (np.abs(qq) @ np.abs(kk).T), 0.0).max(1)
            top = s.max(1)
            w = np.exp(s - top[:, None])
            total, seen = w.sum(1), m.sum(1)
            p = w / total[:, None]
            e = (D + 16) * U * A + 2.0 ** -21 * A + 8 * U * (A + np.abs(np.where(m, s, 0.0)).max(1))
            rel = 2 * e + (seen + 16) * U + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21)
            o[at + rows, h] = p @ vv
            bound[at + rows, h] = rel[:, None] * (p @ np.abs(vv)) + (2.0 ** -8 if dtype == "bf16" else U) * np.abs(p @ vv)
            if dtype == "bf16":
                vs = np.concatenate([value_scales(st, 0, st.prefix), value_scales(st, 1 + b, st.own[b])])[:, h // G]
                bound[at + rows, h] += (seen * 2.0 ** -20 * (p * np.where(m, vs, 0.0)).max(1))[:, None]
            lse[at + rows, h] = top + np.log(total)
            lbound[at + rows, h] = 2 * e + (seen + 16) * U + 4 * U * np.abs(lse[at + rows, h])
        at += n
    return o, bound, lse, lbound


def compare(o, lse, want):
    o64, bound, wl, wb = want
    check(o, o64, bound)
    got, empty = to_host(lse), np.isneginf(wl)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - wl[~empty]) <= wb[~empty])


def call(st, qt, nq, max_q=None, entry=None, **kw):
    start = to_dev(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32))
    one = all(n == 1 for n in nq) and max_q is None
    out = entry(st.cache(), qt, to_dev(st.table), to_dev(np.array(st.own, np.int32)), max(st.own),
                prefix_pages=to_dev(st.prefix_pages), prefix_len=st.prefix, q_start=None if one else start,
                max_q=max_q or max(nq), return_lse=True, **kw)
    torch.cuda.synchronize()
    return out


WINDOWS = [  # heads, kv heads, D, page, prefix, own, query tokens, window, sinks, dtype
    (1, 1, 1, 64, 0, [1], [1], 1, 0, "f32"),
    (8, 1, 128, 64, 0, [1, 64, 65, 0, 200], [1] * 5, 64, 0, "bf16"),
    (8, 1, 128, 64, 0, [1, 64, 65, 0, 200], [1] * 5, 1, 1, "bf16"),
    (4, 4, 100, 64, 77, [40, 0], [1, 1], 50, 4, "f32"),        # windows into the prefix
    (64, 8, 128, 128, 300, [5, 129, 0, 64, 900], [1] * 5, 130, 300, "bf16"),
    (64, 8, 128, 128, 300, [5, 129, 0, 64, 900], [1] * 5, 130, 333, "bf16"),  # first tokens past the prefix
    (25, 5, 128, 64, 0, [3000, 2000], [1, 1], 700, 5, "f32"),
    (16, 2, 200, 64, 64, [1000], [1], 257, 64, "bf16"),
    (40, 2, 256, 64, 130, [700, 1], [1, 1], 128, 0, "f32"),
    (8, 2, 64, 64, 0, [5000], [1], 3000, 4, "bf16"),           # parts, joined
    (1, 1, 64, 64, 3000, [0, 10], [1, 1], 100, 7, "f32"),      # a query behind the prefix alone
    (5, 5, 17, 64, 64, [65, 0], [1, 1], 1000, 3, "bf16"),      # a window over everything
    (4, 1, 64, 64, 0, [700], [600], 100, 3, "f32"),
    (8, 2, 128, 64, 90, [130, 5, 64], [100, 5, 64], 33, 10, "bf16"),
    (3, 3, 100, 64, 33, [200, 0, 7], [64, 0, 1], 20, 0, "bf16"),
    (16, 2, 128, 128, 400, [600, 300], [350, 1], 64, 500, "f32"),
    (5, 1, 256, 64, 0, [400, 90], [400, 33], 70, 1, "bf16"),
    (2, 2, 48, 64, 10, [3], [9], 2, 1, "f32"),                 # more queries than own keys
    (2, 2, 48, 64, 0, [3], [9], 2, 1, "bf16"),
    (8, 1, 128, 64, 0, [900], [900], 1, 0, "bf16"),            # every query its own key alone
    (8, 1, 128, 64, 100, [900, 500], [900, 77], 300, 0, "bf16"),
    (32, 4, 64, 64, 0, [900], [333], 129, 65, "bf16"),
    (32, 4, 64, 64, 0, [900], [333], 129, 65, "f32"),
]


@pytest.mark.parametrize("heads,kvh,D,page,prefix,own,nq,window,sinks,dtype", WINDOWS)
def test_window(heads, kvh, D, page, prefix, own, nq, window, sinks, dtype):
    print("window", heads, kvh, D, prefix, own, nq, window, sinks, dtype, flush=True)
    st = Setup(kvh, D, page, prefix, own, seed=D + prefix + sum(own))
    qt, q = queries(sum(nq), heads, D, 4, dtype)
    o, lse = call(st, qt, nq, entry=bl.attention_window, window=window, sinks=sinks)
    compare(o, lse, reference(st, q, nq, lambda b: window_sight(prefix, own[b], nq[b], window, sinks), D ** -0.5, dtype))


def grown_tree(rng, n):
    """Ancestors of n drafted tokens, themselves among them, [n, n]."""
    bits = np.zeros((n, n), bool)
    for i in range(n):
        p = int(rng.integers(-1, i)) if i and rng.random() < 0.9 else -1
        if p >= 0:
            bits[i] = bits[p]
        bits[i, i] = True
    return bits


def words(trees, most, extra=0):
    """Rows of int64 words of the trees, bits past a tree's tokens set (they are ignored)."""
    w = max(1, (most + 63) // 64) + extra
    out = []
    for bits in trees:
        full = np.ones((len(bits), 64 * w), bool)
        full[:, :len(bits)] = bits
        out.append(np.packbits(full, axis=1, bitorder="little").view(np.int64))
    return np.concatenate(out) if out else np.zeros((0, w), np.int64)


TREES = [  # heads, kv heads, D, page, prefix, own, query tokens, dtype
    (1, 1, 1, 64, 0, [1], [1], "f32"),
    (4, 4, 100, 64, 77, [140], [7], "f32"),
    (8, 1, 128, 64, 0, [100, 64, 130, 70], [12, 64, 2, 6], "bf16"),   # 16 rows and more, a tree that is all there is
    (64, 8, 128, 64, 500, [200, 33, 129, 65], [25, 25, 1, 13], "bf16"),
    (64, 8, 128, 128, 3000, [5, 90], [5, 30], "bf16"),                # a prefix of its own pass
    (8, 2, 64, 64, 1, [130, 0], [65, 0], "f32"),
    (25, 5, 128, 64, 0, [300, 250], [63, 129], "bf16"),
    (8, 1, 128, 64, 0, [6000], [200], "bf16"),
    (16, 2, 128, 64, 130, [400], [127], "f32"),
    (5, 1, 256, 64, 10, [300, 90], [250, 40], "bf16"),
    (2, 2, 48, 64, 10, [3], [9], "f32"),     # fewer own keys than drafted tokens
    (2, 2, 48, 64, 0, [70], [130], "bf16"),
    (2, 2, 48, 64, 0, [0], [5], "bf16"),
    (32, 4, 64, 192, 64, [640], [300], "bf16"),
]


@pytest.mark.parametrize("heads,kvh,D,page,prefix,own,nq,dtype", TREES)
def test_tree(heads, kvh, D, page, prefix, own, nq, dtype):
    print("tree", heads, kvh, D, prefix, own, nq, dtype, flush=True)
    st = Setup(kvh, D, page, prefix, own, seed=D + prefix + sum(own))
    rng = np.random.default_rng(sum(nq))
    trees = [grown_tree(rng, n) for n in nq]
    qt, q = queries(sum(nq), heads, D, 4, dtype)
    o, lse = call(st, qt, nq, entry=bl.attention_tree, tree=to_dev(words(trees, max(nq))))
    compare(o, lse, reference(st, q, nq, lambda b: tree_sight(prefix, own[b], nq[b], trees[b]), D ** -0.5, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,D,n", [(4, 64, 70), (8, 128, 20), (16, 128, 70), (2, 200, 70)])
def test_any_bits(heads, D, n, dtype):
    """Rows that see nothing at all, everything, later tokens, or a single key, in no order; nothing before the tree, and
    a bound of query tokens far above what there is."""
    rng = np.random.default_rng(D)
    for own in (n, n + 40):
        st = Setup(1, D, 64, 0, [own], seed=own)
        bits = rng.random((n, n)) < rng.choice([0.0, 0.02, 0.5, 1.0], (n, 1))
        bits[0], bits[1], bits[n - 1] = False, True, False
        qt, q = queries(n, heads, D, 5, dtype)
        o, lse = call(st, qt, [n], max_q=4 * n, entry=bl.attention_tree, tree=to_dev(words([bits], n, extra=1)))
        compare(o, lse, reference(st, q, [n], lambda b: tree_sight(0, own, n, bits), D ** -0.5, dtype))


def test_a_chain_is_causal():
    """A tree whose tokens see all before them is causal attention; a window over everything is attention's own call, and
    gives its bits."""
    for heads, kvh, D, own, nq, dtype in ((8, 1, 128, [90, 300], [12, 12], "bf16"), (16, 2, 128, [900], [200], "bf16"),
                                          (4, 4, 100, [70, 9], [5, 9], "f32"), (8, 1, 64, [700], [100], "f32")):
        st = Setup(kvh, D, 64, 40, own, seed=D)
        qt, q = queries(sum(nq), heads, D, 6, dtype)
        chain = [np.tril(np.ones((n, n), bool)) for n in nq]
        want = call(st, qt, nq, entry=bl.attention)
        o, lse = call(st, qt, nq, entry=bl.attention_tree, tree=to_dev(words(chain, max(nq))))
        compare(o, lse, reference(st, q, nq, lambda b: window_sight(40, own[b], nq[b], 1 << 30, 0), D ** -0.5, dtype))
        got = call(st, qt, nq, entry=bl.attention_window, window=40 + max(own), sinks=3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,D,n", [("bf16", 128, 1), ("bf16", 128, 60), ("f32", 128, 1), ("f32", 64, 60), ("bf16", 64, 200)])
def test_scores_that_move(dtype, D, n):
    """Keys and values of very different sizes from block to block, so that rows meet their first large key in other
    blocks than their neighbours, and weights leave binary16's range on both sides."""
    own, window, sinks = 900, 130, 70
    st = Setup(1, D, 64, 100, [own], seed=D + n)
    sizes = np.array([1.0, 0.05, 6.0, 0.3, 12.0, 0.01, 20.0, 3.0])
    values = np.array([1.0, 1e-6, 1.0, 300.0, 1e-3, 1.0, 1e4, 1e-9])
    for mine in st.lists:
        for j, page in enumerate(mine):
            st.ks[page] *= np.float32(sizes[j % 8])
            st.vs[page] *= np.float32(values[j % 8])
    qt, q = queries(n, 8, D, 11, dtype, size=2.0)
    o, lse = call(st, qt, [n], entry=bl.attention_window, window=window, sinks=sinks)
    compare(o, lse, reference(st, q, [n], lambda b: window_sight(100, own, n, window, sinks), D ** -0.5, dtype))
    rng = np.random.default_rng(n)
    bits = rng.random((n, n)) < 0.1
    o, lse = call(st, qt, [n], entry=bl.attention_tree, tree=to_dev(words([bits], n)))
    compare(o, lse, reference(st, q, [n], lambda b: tree_sight(100, own, n, bits), D ** -0.5, dtype))


@pytest.mark.parametrize("dtype,D,n", [("bf16", 128, 60), ("bf16", 64, 200), ("bf16", 256, 40), ("f32", 128, 60),
                                       ("f32", 64, 60), ("f32", 256, 40)])
def test_scores_that_grow(dtype, D, n):
    """Keys that grow from block to block, to scores of a hundred and more: every row's weights outgrow its first keys'
    again and again, in blocks of its own.  With values of even sizes, and values that shrink as the keys grow."""
    own = 900
    for shrink in (False, True):
        st = Setup(1, D, 64, 0, [own], seed=D + n)
        for j, page in enumerate(st.lists[1]):
            st.ks[page] *= np.float32(0.05 + 2.5 * j)
            if shrink:
                st.vs[page] *= np.float32(2.0 ** -j)
        qt, q = queries(n, 8, D, 13, dtype, size=2.0)
        o, lse = call(st, qt, [n], entry=bl.attention_window, window=700, sinks=90)
        compare(o, lse, reference(st, q, [n], lambda b: window_sight(0, own, n, 700, 90), D ** -0.5, dtype))
        bits = np.random.default_rng(n).random((n, n)) < 0.3
        o, lse = call(st, qt, [n], entry=bl.attention_tree, tree=to_dev(words([bits], n)))
        compare(o, lse, reference(st, q, [n], lambda b: tree_sight(0, own, n, bits), D ** -0.5, dtype))


@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("bf16", 80), ("f32", 1), ("f32", 80)])
def test_hidden_keys_reach_nobody(dtype, n):
    """Keys outside every window hold scales that are not finite, and their pages' entries name pages of such keys;
    drafted tokens nobody sees do too."""
    own, window, sinks, heads, D = 1000, 200, 65, 8, 128
    st = Setup(1, D, 64, 150, [own], seed=n)
    see = window_sight(150, own, n, window, sinks)
    clean = [x.copy() for x in (st.ks, st.vs)]
    for t in range(150 + own):
        page, at = (st.lists[0], t) if t < 150 else (st.lists[1], t - 150)
        if not see[:, t].any():
            st.ks[page[at // 64], :, at % 64], st.vs[page[at // 64], :, at % 64] = (np.nan, np.inf)[t % 2], (np.inf, np.nan)[t % 2]
    spare = [p for p in range(len(st.k)) if p not in st.lists[0] and p not in st.lists[1]]
    assert spare and np.isnan(st.ks[spare[0]]).all()
    for j in range((own + 63) // 64):
        if not see[:, 150 + 64 * j:150 + min(own, 64 * j + 64)].any():
            st.table[0, j] = spare[0]
    qt, q = queries(n, heads, D, 5, dtype)
    o, lse = call(st, qt, [n], entry=bl.attention_window, window=window, sinks=sinks)
    st.ks, st.vs = [x.copy() for x in clean]
    compare(o, lse, reference(st, q, [n], lambda b: see, D ** -0.5, dtype))
    if n > 1:
        st = Setup(1, D, 64, 0, [own], seed=n)
        bits = grown_tree(np.random.default_rng(n), n)
        bits[:, 3] = bits[:, 40] = False
        clean = [x.copy() for x in (st.ks, st.vs)]
        for x in (3, 40):
            t = own - n + x
            st.ks[st.lists[1][t // 64], :, t % 64] = st.vs[st.lists[1][t // 64], :, t % 64] = np.nan
        o, lse = call(st, qt, [n], entry=bl.attention_tree, tree=to_dev(words([bits], n)))
        st.ks, st.vs = clean
        compare(o, lse, reference(st, q, [n], lambda b: tree_sight(0, own, n, bits), D ** -0.5, dtype))


def test_bad_pages_padding_and_strides():
    """Pages outside the cache hide their keys; tokens of no sequence keep their output; strided rows of queries, output
    and tree."""
    st = Setup(2, 64, 64, 0, [300, 200], seed=9)
    nq = [3, 2]
    qt, q = queries(7, 4, 64, 6, "f32", odd=True)
    trees = [grown_tree(np.random.default_rng(1), n) for n in nq]
    table = st.table.copy()
    table[0, 3], table[1, 1] = -1, len(st.k)
    start = to_dev(np.array([0, 3, 5], np.int32))
    wide = np.zeros((7, 5), np.int64)
    wide[:5, 1:2] = words(trees, 3)
    hidden = {0: slice(192, 256), 1: slice(64, 128)}

    def sight(b, see):
        see = see.copy()
        see[:, hidden[b]] = False
        return see

    for entry, kw, see in (
            (bl.attention_window, dict(window=150, sinks=70), lambda b: window_sight(0, st.own[b], nq[b], 150, 70)),
            (bl.attention_tree, dict(tree=to_dev(wide)[:, 1:2]), lambda b: tree_sight(0, st.own[b], nq[b], trees[b]))):
        buf = torch.full((4, 7, 66), -9.0, device="cuda")
        out = buf[:, :, 1:65].transpose(0, 1)
        entry(st.cache(), qt, to_dev(table), to_dev(np.array(st.own, np.int32)), 300, q_start=start, max_q=3, out=out, **kw)
        torch.cuda.synchronize()
        o, bound, _, _ = reference(st, q[:5], nq, lambda b: sight(b, see(b)), 64 ** -0.5, "f32")
        check(out[:5].contiguous(), o, bound)
        assert bool((buf[:, 5:] == -9).all()) and bool((buf[:, :, 0] == -9).all()) and bool((buf[:, :, 65] == -9).all())


@pytest.mark.parametrize("which", ["window", "tree"])
def test_graph_and_stream(which):
    """In a graph, replayed with other lengths, queries and trees in the same buffers; and on a side stream."""
    st = Setup(2, 128, 64, 100, [400, 700], seed=11)
    cache, table, pp = st.cache(), to_dev(st.table), to_dev(st.prefix_pages)
    n, heads = 9, 16
    qs = [queries(2 * n, heads, 128, s, "bf16")[0] for s in (6, 7)]
    masks = [to_dev(words([grown_tree(np.random.default_rng(s + b), n) for b in range(2)], n)) for s in (0, 5)]
    q, mask, ln = qs[0].clone(), masks[0].clone(), to_dev(np.array([400, 700], np.int32))
    out = torch.empty_like(q)
    sizes = (2 * n, heads, 2, 128, 2, n, 700, 100)
    nws = bl.bitlinear_attention_window_workspace_bytes(*sizes, 300, 4) if which == "window" else \
        bl.bitlinear_attention_tree_workspace_bytes(*sizes)
    ws = torch.empty(max(16, nws), dtype=torch.uint8, device="cuda")
    kw = dict(prefix_pages=pp, prefix_len=100, max_q=n, ws=ws)
    kw.update(dict(window=300, sinks=4) if which == "window" else dict(tree=mask))
    entry = bl.attention_window if which == "window" else bl.attention_tree
    run = lambda **more: entry(cache, q, table, ln, 700, **{**kw, **more})  # noqa: E731
    run(out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out=out)
    for r in range(3):
        q.copy_(qs[r % 2])
        mask.copy_(masks[r % 2])
        ln.copy_(torch.tensor([400 - 30 * r, 700 - 250 * r], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = run()
        torch.cuda.synchronize()
        assert torch.equal(got, want), r
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    for _ in range(4):
        torch.empty_like(out).fill_(7)
    got = run(stream=side, ws=None)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("G,n,dtype", [(8, 8, "bf16"), (8, 9, "bf16"), (4, 8, "f32"), (4, 9, "f32")])
def test_parts_of_uneven_sequences(G, n, dtype):
    """The most rows of a short tile and the fewest of a long one, on sequences of which some have none of the keys, some
    none of the tokens, of a split's later parts."""
    own, nq = [6500, 70, 0, 2100, n, 3], [n, n - 1, n, 0, n, n]
    st = Setup(2, 64, 128, 0, own, seed=n)
    rng = np.random.default_rng(n)
    trees = [grown_tree(rng, k) for k in nq]
    qt, q = queries(sum(nq), 2 * G, 64, 4, dtype)
    o, lse = call(st, qt, nq, entry=bl.attention_tree, tree=to_dev(words(trees, n)))
    compare(o, lse, reference(st, q, nq, lambda b: tree_sight(0, own[b], nq[b], trees[b]), 64 ** -0.5, dtype))
    o, lse = call(st, qt, nq, entry=bl.attention_window, window=2500, sinks=65)
    compare(o, lse, reference(st, q, nq, lambda b: window_sight(0, own[b], nq[b], 2500, 65), 64 ** -0.5, dtype))


@pytest.mark.parametrize("n,dtype", [(3, "bf16"), (40, "bf16"), (40, "f32")])
def test_graphs_that_share_a_workspace(n, dtype):
    """Two captured calls with the same workspace, replayed in turn with eager calls between them."""
    st = Setup(1, 128, 64, 0, [6500, 900], seed=n)
    cache, table, ln = st.cache(), to_dev(st.table), to_dev(np.array(st.own, np.int32))
    mask = to_dev(words([grown_tree(np.random.default_rng(b), n) for b in range(2)], n))
    q, start = queries(2 * n, 8, 128, 5, dtype)[0], to_dev(np.array([0, n, 2 * n], np.int32))
    nws = max(bl.bitlinear_attention_window_workspace_bytes(2 * n, 8, 1, 128, 2, n, 6500, 0, 4000, 9),
              bl.bitlinear_attention_tree_workspace_bytes(2 * n, 8, 1, 128, 2, n, 6500, 0))
    assert nws > 0
    ws = torch.full((nws,), 255, dtype=torch.uint8, device="cuda")
    kw = dict(q_start=start, max_q=n)
    calls = [lambda **more: bl.attention_tree(cache, q, table, ln, 6500, mask, **kw, **more),
             lambda **more: bl.attention_window(cache, q, table, ln, 6500, 4000, 9, **kw, **more)]
    wants = [c() for c in calls]
    outs = [torch.zeros_like(q) for _ in calls]
    for c, out in zip(calls, outs):
        c(out=out, ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for c, out in zip(calls, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c(out=out, ws=ws)
    for r in range(6):
        outs[r % 2].zero_()
        graphs[r % 2].replay()
        calls[1 - r % 2](ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(outs[r % 2], wants[r % 2]), r


def test_a_step_of_drafts():
    """The operators together, as a step of drafts uses them: places for the drafts, their keys and values, attention of
    the tree and of a layer with a window; then a path is accepted, its keys move together, the rest goes back, and the
    next step's token sees what a cache without drafts would hold."""
    rng = np.random.default_rng(3)
    H, heads, D, page, seqs, window, sinks = 2, 8, 64, 64, 3, 90, 4
    lens, n = [50, 120, 7], [20, 33, 5]
    cache = bl.KVCache.empty(24, H, D, page)
    for t in (cache.k, cache.v):
        t.zero_()
    for t in (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))
    table = torch.full((seqs, 5), -1, dtype=torch.int32, device="cuda")
    free, nfree = to_dev(rng.permutation(24).astype(np.int32)), to_dev(np.array([24], np.int32))
    held = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    tokens = lambda m: to_dev(rng.standard_normal((m, H, D)).astype(np.float32))  # noqa: E731

    def place(count, room=None):
        _, first, start, slots, pos, _ = bl.cache_assign(held, to_dev(np.array(count, np.int32)), table, free, nfree,
                                                         sum(max(c, 0) for c in count) if room is None else room, page,
                                                         own_len=held, free_left=nfree)
        return first, start, slots, pos

    def content(b, m):
        t = np.arange(m)
        p = to_host(table)[b, t // page].astype(np.int64)
        k, v = bl.cache_read(cache, to_dev(p * page + t % page), dtype=torch.float32)
        return to_host(k).astype(np.float64), to_host(v).astype(np.float64)

    def expect(q, nq, sight):
        class Held:
            H, D, prefix, own, lists = 2, 64, 0, [len(content(b, int(m))[0]) for b, m in enumerate(to_host(held))], [None, 0, 1, 2]

            def rows(self, which, m):
                return content(which, m) if which is not None else (np.zeros((0, 2, 64)), np.zeros((0, 2, 64)))
        return reference(Held(), q, nq, sight, D ** -0.5, "f32")

    _, _, slots, pos = place(lens)
    assert np.array_equal(to_host(pos), np.concatenate([np.arange(m) for m in lens]))
    bl.cache_write(cache, tokens(sum(lens)), tokens(sum(lens)), slots)
    # the drafts
    _, start, slots, _ = place(n)
    kd, vd = tokens(sum(n)), tokens(sum(n))
    bl.cache_write(cache, kd, vd, slots)
    trees = [grown_tree(rng, m) for m in n]
    qt, q = queries(sum(n), heads, D, 4, "f32")
    o, lse = bl.attention_tree(cache, qt, table, held, 5 * page, to_dev(words(trees, max(n))), q_start=start, max_q=max(n),
                               return_lse=True)
    torch.cuda.synchronize()
    compare(o, lse, expect(q, n, lambda b: tree_sight(0, lens[b] + n[b], n[b], trees[b])))
    o, lse = bl.attention_window(cache, qt, table, held, 5 * page, window, sinks, q_start=start, max_q=max(n), return_lse=True)
    torch.cuda.synchronize()
    compare(o, lse, expect(q, n, lambda b: window_sight(0, lens[b] + n[b], n[b], window, sinks)))
    # the deepest path of each tree is accepted
    path = [np.nonzero(t[t.sum(1).argmax()])[0] for t in trees]
    width, at, s = max(map(len, path)), to_host(start), to_host(slots)
    src, dst = np.full((2, seqs, width), -1, np.int64)
    for b, p in enumerate(path):
        src[b, :len(p)], dst[b, :len(p)] = s[at[b] + p], s[at[b]:at[b] + len(p)]
    want = bl.cache_read(cache, to_dev(np.concatenate([s[at[b] + p] for b, p in enumerate(path)])), dtype=torch.float32)
    bl.cache_move(cache, to_dev(src), to_dev(dst))
    got = bl.cache_read(cache, to_dev(np.concatenate([s[at[b]:at[b] + len(p)] for b, p in enumerate(path)])), dtype=torch.float32)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    before = int(to_host(nfree)[0])
    place([len(p) - m for p, m in zip(path, n)])
    lens = [a + len(p) for a, p in zip(lens, path)]
    torch.cuda.synchronize()
    assert list(to_host(held)) == lens
    assert int(to_host(nfree)[0]) == 24 - sum((m + 63) // 64 for m in lens) >= before
    # the next step: a token each, causal and with the window
    _, start, slots, pos = place([1] * seqs)
    assert list(to_host(pos)) == lens
    bl.cache_write(cache, tokens(seqs), tokens(seqs), slots)
    qt, q = queries(seqs, heads, D, 8, "f32")
    o, lse = bl.attention_window(cache, qt, table, held, 5 * page, window, sinks, return_lse=True)
    torch.cuda.synchronize()
    compare(o, lse, expect(q, [1] * seqs, lambda b: window_sight(0, lens[b] + 1, 1, window, sinks)))
    o, lse = bl.attention(cache, qt, table, held, 5 * page, return_lse=True)
    torch.cuda.synchronize()
    compare(o, lse, expect(q, [1] * seqs, lambda b: np.ones((1, lens[b] + 1), bool)))
