"""Places of new tokens and moves in the int8 cache, against lists on the host: whole
numbers and bytes, equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

from gpu_helpers import to_dev, to_host  # noqa: E402

pytestmark = pytest.mark.gpu


def assigned(held, count, table, free, nfree, tokens, page, cap, prefix):
    """What bitlinear_cache_assign gives, with lists."""
    up = lambda n: (n + page - 1) // page  # noqa: E731
    table, free = table.copy(), free.copy()
    held, count = [min(max(int(h), 0), cap) for h in held], [int(c) for c in count]
    stack = list(free[:min(max(nfree, 0), len(free))])
    for b, (h, c) in enumerate(zip(held, count)):
        if c < 0:
            stack += list(table[b, up(max(0, h + c)):up(h)])
    stack = stack[:len(free)]
    free[:len(stack)] = stack
    length, first, start, slots, pos, asked, had = [], [], [0], [], [], 0, len(stack)
    for b, (h, c) in enumerate(zip(held, count)):
        begin, end = start[-1], start[-1] + max(0, c)
        start.append(end)
        if c <= 0:
            length.append(max(0, h + c))
            first.append(length[-1])
            continue
        fits = h + c <= cap and end <= tokens
        need = up(h + c) - up(h) if fits else 0
        asked += need
        if not fits or (need and asked > had):
            length.append(h)
            first.append(-1)
            slots += [-1] * (min(end, tokens) - min(begin, tokens))
            pos += [-1] * (min(end, tokens) - min(begin, tokens))
            continue
        for x in range(need):
            table[b, up(h) + x] = stack.pop()
        length.append(h + c)
        first.append(h)
        t = np.arange(h, h + c)
        slots += list(table[b, t // page].astype(np.int64) * page + t % page)
        pos += list(prefix + t)
    pad = [-1] * (tokens - len(slots))
    i32 = lambda x: np.array(x, np.int32)  # noqa: E731
    return {"own_len": i32(length), "first": i32(first), "q_start": i32(np.minimum(start, tokens)),
            "slots": np.array(slots + pad, np.int64), "positions": i32(pos + pad), "left": i32([len(stack)]), "table": table,
            "free": free}


def state(rng, seqs, page, cap, spare, cols=None):
    """Random lengths in pages of their own, and a list of 'spare' more with room for all."""
    cols = (cap + page - 1) // page if cols is None else cols
    held = rng.integers(0, cap + 1, seqs)
    used = (held + page - 1) // page
    ids = rng.permutation(int(used.sum()) + spare).astype(np.int32)
    table, at = np.full((seqs, cols), -7, np.int32), 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    free = np.full(len(ids) + 3, -9, np.int32)
    free[:spare] = ids[at:]
    return held.astype(np.int32), table, free


def run(held, count, table, free, nfree, tokens, page, cap, prefix=0, in_place=False, stream=None):
    d = {k: to_dev(np.ascontiguousarray(v)) for k, v in (("held", held), ("count", count), ("table", table), ("free", free),
                                                         ("n", np.array([nfree], np.int32)))}
    kw = dict(own_len=d["held"], free_left=d["n"]) if in_place else {}
    torch.cuda.synchronize()
    out = bl.cache_assign(d["held"], d["count"], d["table"], d["free"], d["n"], tokens, page, cap, prefix_len=prefix,
                          stream=stream, **kw)
    torch.cuda.synchronize()
    names = ("own_len", "first", "q_start", "slots", "positions", "left")
    got = {k: to_host(t) for k, t in zip(names, out)}
    if not in_place:
        assert np.array_equal(to_host(d["held"]), held) and to_host(d["n"])[0] == nfree
    got["table"], got["free"] = to_host(d["table"]), to_host(d["free"])
    return got


def compare(got, want):
    for k, w in want.items():
        assert got[k].shape == w.shape and np.array_equal(got[k], w), (k, got[k], w)


@pytest.mark.parametrize("seqs,page,cap,most,back,spare", [
    (1, 64, 100, 1, 0.0, 3), (1, 64, 64, 64, 0.0, 0), (16, 64, 600, 1, 0.0, 20), (3, 128, 1000, 300, 0.3, 30),
    (63, 64, 500, 5, 0.5, 4), (64, 192, 700, 70, 0.2, 100), (65, 64, 300, 40, 0.2, 9), (257, 64, 400, 3, 0.3, 50),
    (300, 64, 4000, 250, 0.2, 2000), (1023, 64, 200, 9, 0.4, 300), (1024, 64, 200, 3, 0.0, 100), (1025, 64, 200, 20, 0.3, 2000),
    (2500, 256, 900, 30, 0.4, 10), (40, 64, 30000, 4000, 0.1, 3000), (5, 1 << 20, 3 << 20, 100, 0.3, 2), (700, 64, 64, 1, 1.0, 0),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_places(seqs, page, cap, most, back, spare, in_place):
    """Tokens in one launch and in two, lists that last and that do not, sequences that give tokens back, idle ones,
    and ones past their capacity."""
    print("assign", seqs, page, cap, most, back, spare, in_place, flush=True)
    rng = np.random.default_rng(seqs + page + most)
    held, table, free = state(rng, seqs, page, cap, spare)
    count = rng.integers(0, most + 1, seqs)
    gives = rng.random(seqs) < back
    count[gives] = -rng.integers(1, cap + 1, int(gives.sum()))
    count = count.astype(np.int32)
    tokens = int(np.maximum(count, 0).sum()) + int(rng.integers(0, 3)) * 5
    want = assigned(held, count, table, free, spare, tokens, page, cap, 77)
    compare(run(held, count, table, free, spare, tokens, page, cap, 77, in_place), want)


def test_tokens_are_a_bound():
    """Sequences whose tokens pass the room for them get nothing; none at all is allowed."""
    held, table, free = state(np.random.default_rng(3), 6, 64, 300, 40)
    held[:] = [0, 64, 63, 1, 128, 10]
    count = np.array([3, 0, 5, 4, 2, 1], np.int32)
    for tokens in (15, 14, 12, 8, 7, 3, 2, 0):
        want = assigned(held, count, table, free, 40, tokens, 64, 300, 0)
        compare(run(held, count, table, free, 40, tokens, 64, 300), want)


def test_extreme_values():
    """Lengths and counts far outside, lists that claim more than their room, a full list that is given more."""
    rng = np.random.default_rng(4)
    held, table, free = state(rng, 5, 64, 300, 4)
    big = np.iinfo(np.int32)
    for h, c, n, room in (([big.max, -5, 300, 0, 64], [1, 3, -1, big.max, big.min], 4, None),
                          ([big.min, 0, 10, 299, 300], [big.min, big.max, 0, 1, 1], big.max, None),
                          ([64, 128, 192, 256, 300], [-64, -300, -1, -65, big.min], -3, None),
                          ([300, 300, 300, 300, 300], [-300] * 5, 6, 8), ([300, 64, 0, 0, 0], [-300, -64, 64, 200, 64], 0, 3),
                          ([10, 20, 0, 0, 0], [54, 44, 0, 0, 1], 9, 0)):
        h, c = np.array(h, np.int32), np.array(c, np.int32)
        table[:] = rng.permutation(25).reshape(5, 5)
        f = free if room is None else free[:room].copy()
        want = assigned(h, c, table, f, n, 700, 64, 300, 0)
        compare(run(h, c, table, f, n, 700, 64, 300), want)


def test_page_table_of_wider_rows():
    """A block table that is a part of a larger one, and a capacity of zero."""
    rng = np.random.default_rng(5)
    held, table, free = state(rng, 7, 64, 500, 30)
    wide = np.full((7, 20), -3, np.int32)
    wide[:, 4:12] = table
    count = np.array([5, 70, -3, 0, 200, 1, 1], np.int32)
    want = assigned(held, count, table, free, 30, 300, 64, 500, 0)
    d = to_dev(wide)
    f = to_dev(free)
    out = bl.cache_assign(to_dev(held), to_dev(count), d[:, 4:12], f, to_dev(np.array([30], np.int32)), 300, 64, 500)
    torch.cuda.synchronize()
    got = to_host(d)
    assert np.array_equal(got[:, 4:12], want["table"]) and np.all(got[:, :4] == -3) and np.all(got[:, 12:] == -3)
    assert np.array_equal(to_host(out[3]), want["slots"])
    none = run(np.zeros(2, np.int32), np.array([0, 3], np.int32), np.zeros((2, 1), np.int32), free, 30, 4, 64, 0)
    compare(none, assigned(np.zeros(2), [0, 3], np.zeros((2, 1), np.int32), free, 30, 4, 64, 0, 0))


@pytest.mark.parametrize("many", [False, True])
def test_steps_in_a_graph(many):
    """A captured step in place, replayed: lengths, tables and the list go on from replay to replay, as by lists."""
    rng = np.random.default_rng(6)
    seqs, page, cap = 20, 64, 5000
    held, table, free = state(rng, seqs, page, 300, 600, cols=(cap + page - 1) // page)
    tokens = 5000 if many else 400
    d = [to_dev(x) for x in (held, np.zeros(seqs, np.int32), table, free, np.array([600], np.int32))]
    step = lambda: bl.cache_assign(*d, tokens, page, cap, own_len=d[0], free_left=d[4])  # noqa: E731
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    n = 600
    for r in range(4):
        count = (rng.integers(-200, 20, seqs) if r == 2 else rng.integers(0, 240 if many else 20, seqs)).astype(np.int32)
        want = assigned(held, count, table, free, n, tokens, page, cap, 0)
        d[1].copy_(torch.from_numpy(count))
        g.replay()
        torch.cuda.synchronize()
        got = dict(zip(("own_len", "first", "q_start", "slots", "positions", "left"), map(to_host, out)))
        compare({**got, "table": to_host(d[2]), "free": to_host(d[3])}, want)
        held, table, free, n = want["own_len"], want["table"], want["free"], int(want["left"][0])


def test_on_another_stream():
    """Outputs on a side stream while the caller's stream still writes memory of their sizes that it has freed."""
    rng = np.random.default_rng(8)
    held, table, free = state(rng, 50, 64, 500, 90)
    count = rng.integers(0, 30, 50).astype(np.int32)
    want = assigned(held, count, table, free, 90, 2000, 64, 500, 0)
    d = [to_dev(x) for x in (held, count, table, free, np.array([90], np.int32))]
    first = bl.cache_assign(*d, 2000, 64, 500)
    d = [to_dev(x) for x in (held, count, table, free, np.array([90], np.int32))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    for t in first:
        for _ in range(4):
            torch.empty_like(t).fill_(7)
    got = bl.cache_assign(*d, 2000, 64, 500, stream=side)
    del first
    torch.cuda.synchronize()
    compare(dict(zip(("own_len", "first", "q_start", "slots", "positions", "left"), map(to_host, got))),
            {k: want[k] for k in ("own_len", "first", "q_start", "slots", "positions", "left")})


# ---- moves ------------------------------------------------------------------
PLACE = np.array([16 * ((t % 16) // 4) + 8 * (t // 32) + 4 * ((t % 32) // 16) + t % 4 for t in range(64)])


def random_cache(rng, pages, H, page, D):
    Dp = (D + 15) // 16 * 16
    return (rng.integers(-128, 128, (pages, H, page, Dp)).astype(np.int8),
            rng.integers(-128, 128, (pages, H, page // 64, Dp, 64)).astype(np.int8),
            rng.random((pages, H, page)).astype(np.float32), rng.random((pages, H, page)).astype(np.float32))


def moved(c, src, dst, page):
    """The cache after the moves of every group, read before any is written, the last to a slot counting."""
    c = [x.copy() for x in c]
    n = c[0].shape[0] * page
    for s, d in zip(src, dst):
        ok = [(a, b) for a, b in zip(s, d) if 0 <= a < n and 0 <= b < n]
        read = [(c[0][a // page, :, a % page].copy(), c[1][a // page, :, a % page // 64, :, PLACE[a % 64]].copy(),
                 c[2][a // page, :, a % page].copy(), c[3][a // page, :, a % page].copy()) for a, _ in ok]
        for (_, b), (k, v, ks, vs) in zip(ok, read):
            c[0][b // page, :, b % page] = k
            c[1][b // page, :, b % page // 64, :, PLACE[b % 64]] = v
            c[2][b // page, :, b % page] = ks
            c[3][b // page, :, b % page] = vs
    return c


@pytest.mark.parametrize("H,D,page,pages,groups,width", [
    (1, 1, 64, 1, 1, 1), (8, 128, 64, 40, 8, 5), (2, 100, 128, 30, 20, 13), (3, 17, 192, 9, 7, 64), (1, 256, 64, 70, 60, 64),
    (32, 100, 64, 30, 3, 33), (5, 80, 256, 4, 1, 2), (2, 64, 64, 900, 800, 1),
])
def test_moves(H, D, page, pages, groups, width):
    """Groups of their own pages each: moves that overlap, in both directions, onto themselves, to one slot several
    times, from and to slots outside."""
    print("move", H, D, page, pages, groups, width, flush=True)
    rng = np.random.default_rng(D + width)
    c = random_cache(rng, pages, H, page, D)
    own = pages * page // groups  # slots of a group
    src = rng.integers(0, own, (groups, width)) + np.arange(groups)[:, None] * own
    dst = np.sort(rng.integers(0, own, (groups, width)), 1) + np.arange(groups)[:, None] * own
    if width > 4:
        src[:, 1], dst[:, 2] = dst[:, 0], src[:, 3]          # a slot that another move writes or reads
        dst[:, 4] = dst[:, 0]                                # the same target twice
        src[::2, 3], dst[::3, 1] = pages * page, -1          # outside
        src[0, 0], dst[0, -1] = -(1 << 62), (1 << 62)
    cache = bl.KVCache(*[to_dev(x) for x in c], D)
    bl.cache_move(cache, to_dev(src), to_dev(dst))
    torch.cuda.synchronize()
    want = moved(c, src, dst, page)
    for got, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
        assert np.array_equal(to_host(got), w)


def test_move_runs_together():
    """A path of a tree moved to the tree's start, where several of its tokens already lie, one-dimensional; then the same
    in a captured graph, replayed with other slots."""
    rng = np.random.default_rng(2)
    c = random_cache(rng, 3, 2, 64, 128)
    cache = bl.KVCache(*[to_dev(x) for x in c], 128)
    src, dst = np.array([60, 61, 64, 70, 71, 100]), np.arange(60, 66)
    s, d = to_dev(src), to_dev(dst)
    bl.cache_move(cache, s, d)
    bl.cache_move(cache, s[:0], d[:0])
    torch.cuda.synchronize()
    want = moved(c, src[None], dst[None], 64)
    assert all(np.array_equal(to_host(t), w) for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bl.cache_move(cache, s, d)
    for r in range(3):
        src, dst = rng.integers(-5, 200, 6), rng.permutation(200)[:6]
        s.copy_(torch.from_numpy(src))
        d.copy_(torch.from_numpy(dst))
        g.replay()
        torch.cuda.synchronize()
        want = moved(want, src[None], dst[None], 64)
        assert all(np.array_equal(to_host(t), w) for t, w in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want)), r
