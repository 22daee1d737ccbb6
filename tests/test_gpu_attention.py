"""Attention over the int8 cache with a shared prefix, against a plain binary64
softmax over the values the cache stands for.

The bound.  With u = 2^-24 and A = scale * sum |q_d k_d| of a score: queries are
carried to 22 bits or their own 8 (2^-22 A), the sum over head_dim adds (D + 8) u A,
and the exponent's argument a few u of its size S <= A + max: a score is off by at
most e = (D + 16) u A + 2^-21 A + 8 u S.  A weight p is then off by 2 e (its own
and the maximum's), sums over n keys by (n + 16) u, and weights are rounded to 11
bits for bf16 (2^-11) or 22 for fp32 (2^-21).  o is off by the sum of p |v| times
all that, and one rounding of the output."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402
from ternary_weight_linear_forward_amd import synth  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
PLACE = np.array([16 * ((t % 16) // 4) + 8 * (t // 32) + 4 * ((t % 32) // 16) + t % 4 for t in range(64)])


class Setup:
    """A cache of random pages: places no sequence uses hold random bytes and NaN scales."""

    def __init__(self, H, D, page, prefix, own, seed, spread=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.D, self.page, self.prefix, self.own = H, D, page, prefix, own
        Dp = (D + 15) // 16 * 16
        need = lambda n: (n + page - 1) // page  # noqa: E731
        pages = need(prefix) + sum(need(n) for n in own) + 2
        self.k = rng.integers(-128, 128, (pages, H, page, Dp)).astype(np.int8)
        self.v = rng.integers(-128, 128, (pages, H, page // 64, Dp, 64)).astype(np.int8)
        self.ks = np.full((pages, H, page), np.nan, np.float32)
        self.vs = np.full((pages, H, page), np.nan, np.float32)
        ids = list(rng.permutation(pages))
        self.lists, table = [], max([need(n) for n in own] + [1])
        for n in [prefix] + list(own):
            mine = [ids.pop() for _ in range(need(n))]
            self.lists.append(mine)
            for t in range(n):
                p = mine[t // page]
                self.ks[p, :, t % page] = (0.02 + 0.02 * rng.random(H)) * spread ** rng.standard_normal(H)
                self.vs[p, :, t % page] = (0.02 + 0.02 * rng.random(H)) * spread ** rng.standard_normal(H)
        self.table = np.full((len(own), table + 1), 1 << 30, np.int32)
        for b, mine in enumerate(self.lists[1:]):
            self.table[b, :len(mine)] = mine
        self.prefix_pages = np.array(self.lists[0], np.int32)

    def cache(self):
        return bl.KVCache(to_dev(self.k), to_dev(self.v), to_dev(self.ks), to_dev(self.vs), self.D)

    def rows(self, pages, n):
        """Keys and values [n, H, D] of the first n tokens of a list of pages, binary64."""
        t = np.arange(n)
        p, t = np.array(pages, np.int64)[t // self.page] if n else t, t % self.page
        k = self.k[p, :, t, :self.D].astype(np.float64) * self.ks[p, :, t].astype(np.float64)[..., None]
        v = self.v[p, :, t // 64, :self.D, PLACE[t % 64]].astype(np.float64) * self.vs[p, :, t].astype(np.float64)[..., None]
        return k, v


def reference(st, q, nq, scale, dtype, hidden_pages=()):
    """(o, error bound, lse, lse bound) per token and head in binary64."""
    heads, D = q.shape[1:]
    G = heads // st.H
    kp, vp = st.rows(st.lists[0], st.prefix)
    o, bound = np.zeros(q.shape), np.zeros(q.shape)
    lse, lbound = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    at = 0
    for b, n in enumerate(nq):
        ko, vo = st.rows(st.lists[1 + b], st.own[b])
        k, v = np.concatenate([kp, ko]), np.concatenate([vp, vo])
        seen0 = np.ones(len(k), bool)
        for j, p in enumerate(st.lists[1 + b]):
            if p in hidden_pages:
                seen0[st.prefix + j * st.page:st.prefix + (j + 1) * st.page] = False
        for i in range(n):
            limit = st.prefix + max(0, st.own[b] - n + i + 1)
            seen = seen0[:limit].nonzero()[0]
            if len(seen) == 0:
                continue
            for h in range(heads):
                kk, vv, qq = k[seen, h // G], v[seen, h // G], q[at + i, h].astype(np.float64)
                s = scale * (kk @ qq)
                A = (abs(scale) * (np.abs(kk) @ np.abs(qq))).max()
                top = s.max()
                w = np.exp(s - top)
                p = w / w.sum()
                o[at + i, h] = p @ vv
                S = A + np.abs(s).max()
                e = (D + 16) * U * A + 2.0 ** -21 * A + 8 * U * S
                rel = 2 * e + (len(seen) + 16) * U + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21)
                bound[at + i, h] = rel * (p @ np.abs(vv)) + (2.0 ** -8 if dtype == "bf16" else U) * np.abs(o[at + i, h])
                lse[at + i, h] = top + np.log(w.sum())
                lbound[at + i, h] = 2 * e + (len(seen) + 16) * U + 4 * U * abs(lse[at + i, h])
        at += n
    return o, bound, lse, lbound


def queries(tokens, heads, D, seed, dtype, odd=False, size=1.0):
    x = (synth.activations_f32(tokens * heads, D, seed) * np.float32(size)).reshape(tokens, heads, D)
    bits = synth.to_bf16_bits(x) if dtype == "bf16" else x
    v = synth.bf16_bits_to_f32(bits).reshape(x.shape) if dtype == "bf16" else x
    if not odd:
        return to_dev(bits), v
    buf = np.zeros((heads, tokens, D + 3), bits.dtype)  # head-major rows with odd gaps
    buf[:, :, 1:D + 1] = bits.transpose(1, 0, 2)
    return to_dev(buf)[:, :, 1:D + 1].transpose(0, 1), v


def check(got, want, bound):
    got = synth.bf16_bits_to_f32(to_host(got)) if got.dtype == torch.bfloat16 else to_host(got)
    err = np.abs(got.astype(np.float64) - want)
    assert np.isfinite(got).all()
    assert np.all(err <= bound + 1e-30), (err - bound).max()


CASES = [  # heads, kv heads, D, page, prefix, own lengths, dtype, odd strides
    (1, 1, 1, 64, 0, [1], "f32", False),
    (8, 1, 128, 64, 0, [1, 64, 65, 0], "bf16", False),
    (4, 4, 100, 64, 77, [40, 0], "f32", False),
    (64, 8, 128, 128, 300, [5, 129, 0, 64, 200], "bf16", False),
    (8, 2, 64, 64, 1, [63], "f32", True),
    (6, 2, 80, 192, 500, [1, 2, 3, 191, 192, 193], "bf16", True),
    (24, 1, 128, 64, 200, [100, 3], "bf16", False),
    (40, 2, 256, 64, 130, [70, 1], "f32", False),
    (5, 5, 17, 64, 64, [65, 0], "bf16", True),
    (16, 2, 200, 128, 1000, [10], "bf16", False),
    (32, 4, 128, 256, 3000, [300, 1, 77, 0, 256, 257, 5, 9], "f32", False),
    (64, 8, 128, 64, 20000, [33, 200], "bf16", False),
    (2, 1, 128, 64, 0, [5000, 17], "bf16", False),
    (25, 5, 128, 64, 700, [20] * 40, "bf16", False),
    (8, 8, 64, 64, 0, [0, 0], "bf16", False),
]


@pytest.mark.parametrize("heads,kvh,D,page,prefix,own,dtype,odd", CASES)
def test_one_token_each(heads, kvh, D, page, prefix, own, dtype, odd):
    print("attention", heads, kvh, D, page, prefix, own[:6], dtype, flush=True)
    st = Setup(kvh, D, page, prefix, own, seed=D + prefix)
    qt, q = queries(len(own), heads, D, 3, dtype, odd)
    o, lse = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array(own, np.int32)), max(own),
                          prefix_pages=to_dev(st.prefix_pages), prefix_len=prefix, return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q, [1] * len(own), D ** -0.5, dtype)
    check(o, want, bound)
    got = to_host(lse)
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - wl[~empty]) <= wb[~empty])


PROMPTS = [  # heads, kv heads, D, page, prefix, own, query tokens, dtype
    (4, 1, 64, 64, 0, [70], [70], "f32"),
    (8, 2, 128, 64, 90, [130, 5, 64], [100, 5, 64], "bf16"),
    (3, 3, 100, 64, 33, [200, 0, 7], [64, 0, 1], "bf16"),
    (16, 2, 128, 128, 400, [300, 300], [150, 1], "f32"),
    (5, 1, 256, 64, 0, [40, 90], [40, 33], "bf16"),
    (2, 2, 48, 64, 10, [3], [9], "f32"),  # more queries than own keys: the first ones see the prefix alone
    (2, 2, 48, 64, 0, [3], [9], "bf16"),  # ... or nothing
    (1, 1, 128, 64, 0, [700], [600], "bf16"),
]


@pytest.mark.parametrize("heads,kvh,D,page,prefix,own,nq,dtype", PROMPTS)
def test_prompts(heads, kvh, D, page, prefix, own, nq, dtype):
    print("attention prompt", heads, kvh, D, prefix, own, nq, dtype, flush=True)
    st = Setup(kvh, D, page, prefix, own, seed=D + prefix + sum(nq))
    qt, q = queries(sum(nq), heads, D, 4, dtype)
    start = to_dev(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32))
    o, lse = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array(own, np.int32)), max(own),
                          prefix_pages=to_dev(st.prefix_pages), prefix_len=prefix, q_start=start, max_q=max(nq),
                          return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q, nq, D ** -0.5, dtype)
    check(o, want, bound)
    got, empty = to_host(lse), np.isneginf(wl)
    assert np.array_equal(np.isneginf(got), empty)
    assert np.all(np.abs(got[~empty] - wl[~empty]) <= wb[~empty])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sharp_and_flat_softmax(dtype):
    """Scores that let one key win, scores of zero, and scales over many orders of magnitude."""
    for size, spread in ((12.0, 1.0), (0.0, 1.0), (0.05, 8.0)):
        st = Setup(2, 128, 64, 260, [90, 3], seed=5, spread=spread)
        qt, q = queries(2, 8, 128, 6, dtype, size=size)
        o = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array([90, 3], np.int32)), 90,
                         prefix_pages=to_dev(st.prefix_pages), prefix_len=260)
        torch.cuda.synchronize()
        want, bound, _, _ = reference(st, q, [1, 1], 128 ** -0.5, dtype)
        check(o, want, bound)


@pytest.mark.parametrize("tokens,heads,kvh,D,dtype", [
    (12, 8, 1, 128, "bf16"), (13, 16, 2, 64, "bf16"), (16, 8, 1, 128, "bf16"), (17, 8, 1, 100, "bf16"),
    (40, 8, 1, 128, "bf16"), (12, 8, 1, 64, "f32"), (13, 8, 1, 64, "f32"), (40, 16, 2, 50, "f32"),
    (40, 8, 1, 128, "f32"), (33, 8, 1, 256, "bf16")])
def test_row_counts(tokens, heads, kvh, D, dtype):
    """Rows of a prefix below and past every row tile's size (8 to a token), with references that have to move:
    scores and values of a key block are small or large, block by block, so that weights leave the range of
    binary16 on both sides of the first block's."""
    print("attention rows", tokens, heads, kvh, D, dtype, flush=True)
    own = [(7 * b) % 90 for b in range(tokens)]
    st = Setup(kvh, D, 64, 700, own, seed=tokens + D)
    sizes = np.array([1.0, 0.05, 6.0, 0.3, 12.0, 0.01, 20.0, 3.0])
    values = np.array([1.0, 1e-6, 1.0, 300.0, 1e-3, 1.0, 1e4, 1e-9])
    for j, page in enumerate(st.lists[0]):
        st.ks[page] *= np.float32(sizes[j % 8])
        st.vs[page] *= np.float32(values[j % 8])
    qt, q = queries(tokens, heads, D, 11, dtype, size=2.0)
    o, lse = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array(own, np.int32)), max(own),
                          prefix_pages=to_dev(st.prefix_pages), prefix_len=700, return_lse=True)
    torch.cuda.synchronize()
    want, bound, wl, wb = reference(st, q, [1] * tokens, D ** -0.5, dtype)
    check(o, want, bound)
    assert np.all(np.abs(to_host(lse) - wl) <= wb)


def test_zero_value_scales():
    """Tokens whose values are all zero (scale 0) take their share of the softmax."""
    st = Setup(1, 64, 64, 70, [10], seed=8)
    st.vs[st.lists[0][0], :, :64] = 0.0
    qt, q = queries(1, 4, 64, 6, "bf16")
    o = bl.attention(st.cache(), qt, to_dev(st.table), to_dev(np.array([10], np.int32)), 10,
                     prefix_pages=to_dev(st.prefix_pages), prefix_len=70)
    st2 = Setup(1, 64, 64, 70, [10], seed=8)
    st2.vs[:] = 0.0
    o2 = bl.attention(st2.cache(), qt, to_dev(st2.table), to_dev(np.array([10], np.int32)), 10,
                      prefix_pages=to_dev(st2.prefix_pages), prefix_len=70)
    torch.cuda.synchronize()
    want, bound, _, _ = reference(st, q, [1], 64 ** -0.5, "bf16")
    check(o, want, bound)
    assert not to_host(o2).any()


def test_bad_pages_and_lengths_are_not_followed():
    """A page outside the cache hides its keys, lengths are cut to their host bounds, tokens of no sequence are left."""
    st = Setup(2, 64, 64, 40, [150, 100], seed=9)
    qt, q = queries(3, 4, 64, 6, "f32")
    hidden = st.lists[1][1]
    table = st.table.copy()
    table[0, 1] = [-1, 1 << 30][0]
    out = torch.full((3, 4, 64), -9.0, device="cuda")
    start = to_dev(np.array([0, 1, 2], np.int32))
    bl.attention(st.cache(), qt, to_dev(table), to_dev(np.array([150, 1 << 30], np.int32)), 150,
                 prefix_pages=to_dev(st.prefix_pages), prefix_len=40, q_start=start, max_q=1, out=out)
    torch.cuda.synchronize()
    want, bound, _, _ = reference(st, q, [1, 1], 64 ** -0.5, "f32", hidden_pages=(hidden,))
    check(out[:1], want[:1], bound[:1])
    assert bool((out[2] == -9.0).all())
    # sequence 1: cut to 150 keys, whose third page lies outside the cache: its first two pages count as written
    k = bl.attention(st.cache(), qt[1:2], to_dev(st.table[1:2]), to_dev(np.array([100], np.int32)), 100,
                     prefix_pages=to_dev(st.prefix_pages), prefix_len=40)
    torch.cuda.synchronize()
    assert np.all(np.isfinite(to_host(k)))


def test_strided_output_and_other_stream():
    st = Setup(2, 64, 64, 100, [30, 70], seed=10)
    qt, q = queries(2, 4, 64, 6, "bf16")
    args = (st.cache(), qt, to_dev(st.table), to_dev(np.array([30, 70], np.int32)), 70)
    kw = dict(prefix_pages=to_dev(st.prefix_pages), prefix_len=100)
    want = bl.attention(*args, **kw)
    buf = torch.full((4, 2, 66), -9.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bl.attention(*args, **kw, out=buf[:, :, 1:65].transpose(0, 1), stream=side)
    side.synchronize()
    assert torch.equal(buf[:, :, 1:65].transpose(0, 1), want)
    assert bool((buf[:, :, 0] == -9).all()) and bool((buf[:, :, 65] == -9).all())


def test_graph_replay():
    """The call in a graph, replayed with other lengths and queries in the same buffers."""
    st = Setup(2, 128, 64, 500, [30, 170], seed=11)
    q1, q2 = queries(2, 16, 128, 6, "bf16")[0], queries(2, 16, 128, 7, "bf16")[0]
    cache, table, pp = st.cache(), to_dev(st.table), to_dev(st.prefix_pages)
    q, ln = q1.clone(), to_dev(np.array([30, 170], np.int32))
    out = torch.empty_like(q)
    ws = torch.empty(max(16, bl.bitlinear_attention_workspace_bytes(2, 16, 2, 128, 2, 1, 170, 500)), dtype=torch.uint8,
                     device="cuda")
    run = lambda: bl.attention(cache, q, table, ln, 170, prefix_pages=pp, prefix_len=500, out=out, ws=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for r in range(3):
        q.copy_(q1 if r % 2 == 0 else q2)
        ln.copy_(torch.tensor([30 - r, 170 - 60 * r], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, out), r
