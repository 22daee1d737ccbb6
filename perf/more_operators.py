"""Cases of the operators of a serving step around the int8 cache, in their plain form and through the library.

Four operators that a step with drafted tokens runs one after the other:
  assign  places of the step's new tokens: pages from a free list into block tables, slots, positions, lengths; sequences
          that give tokens back return their pages;
  window  attention with a sliding window and a few first tokens that stay visible, over the paged int8 cache;
  tree    attention of a tree of drafted tokens over the paged int8 cache;
  move    the keys and values of accepted drafts moved together in the cache.

run() computes a case with elementary torch operations in 32 bits (whole numbers in 64), or, where `own` is true, with
ternary_weight_linear_forward_amd.bitlinear.  exact() is the definition in 64 bits, written apart from it.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# The cache holds the values of 64 consecutive tokens of a head transposed: row d of such a block is 64 bytes, and
# token t of the block is byte 16 * ((t % 16) // 4) + 8 * (t // 32) + 4 * ((t % 32) // 16) + t % 4 of it.
BLOCK = 64
PLACE = [16 * ((t % 16) // 4) + 8 * (t // 32) + 4 * ((t % 32) // 16) + t % 4 for t in range(BLOCK)]


def listed():
    return [
        # one decode step of a batch: 16 sequences, a token each
        {"name": "assign_16x1", "op": "assign", "B": 16, "page": 64, "own": 600, "most": 1, "back": 0.0, "short": False},
        # a mixed step: prompts of up to 250 tokens, single tokens, sequences that end or drop drafts
        {"name": "assign_300_mixed", "op": "assign", "B": 300, "page": 64, "own": 4000, "most": 250, "back": 0.2,
         "short": False},
        # 5 accepted drafts of each of 8 sequences, 70B k/v width
        {"name": "move_8x5_8x128", "op": "move", "B": 8, "width": 5, "nodes": 64, "heads": 8, "D": 128, "page": 64},
        # the 70B model's largest batch with long accepted paths, 32 heads of 100
        {"name": "move_176x13_32x100", "op": "move", "B": 176, "width": 13, "nodes": 60, "heads": 32, "D": 100, "page": 128},
        # a single conversation of 5000 tokens in a layer with a window of 1024, one token
        {"name": "window_1x64x128_bf16", "op": "window", "B": 1, "heads": 64, "kv_heads": 8, "D": 128, "page": 64,
         "prefix": 77, "own": 5000, "max_q": 1, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # decode of a batch of long conversations, a window of 4096
        {"name": "window_48x64x128_bf16", "op": "window", "B": 48, "heads": 64, "kv_heads": 8, "D": 128, "page": 128,
         "prefix": 0, "own": 8000, "max_q": 1, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # ragged prompts of the 3B model's head layout in fp32, window across the shared prefix
        {"name": "window_3x32x100_q300_f32", "op": "window", "B": 3, "heads": 32, "kv_heads": 32, "D": 100, "page": 64,
         "prefix": 200, "own": 900, "max_q": 300, "window": 500, "sinks": 16, "dtype": "f32"},
        # long prompts into a layer with a window
        {"name": "window_2x64x128_q4096_bf16", "op": "window", "B": 2, "heads": 64, "kv_heads": 8, "D": 128, "page": 256,
         "prefix": 0, "own": 4500, "max_q": 4096, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # a chain-like draft of 7 tokens in fp32, 3B head layout, short conversation
        {"name": "tree_1x7_32x100_f32", "op": "tree", "B": 1, "heads": 32, "kv_heads": 32, "D": 100, "page": 64,
         "prefix": 77, "own": 140, "max_q": 7, "dtype": "f32"},
        # trees of up to 25 drafts of a batch behind a system prompt
        {"name": "tree_16x25_64x128_bf16", "op": "tree", "B": 16, "heads": 64, "kv_heads": 8, "D": 128, "page": 64,
         "prefix": 1000, "own": 2100, "max_q": 25, "dtype": "bf16"},
        # wide trees over long conversations
        {"name": "tree_4x200_64x128_bf16", "op": "tree", "B": 4, "heads": 64, "kv_heads": 8, "D": 128, "page": 256,
         "prefix": 0, "own": 9000, "max_q": 200, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(64, 8, 128), (32, 32, 100), (25, 5, 128), (50, 50, 64), (8, 1, 256), (40, 40, 80)]


def draw(rng):
    op = rng.choice(["assign", "move", "window", "window", "tree", "tree"])
    page = rng.choice([64, 128, 256])
    if op == "assign":
        B, most = _log(rng, 1, 600), rng.choice([1, _log(rng, 2, 400)])
        return {"op": op, "B": B, "page": page, "own": max(most, _log(rng, 1, 4000)),
                "most": most if B * most <= 75000 else 1, "back": rng.choice([0.0, 0.2, 0.5]), "short": rng.random() < 0.3}
    if op == "move":
        heads, D = rng.choice([(8, 128), (32, 100), (25, 128), (50, 64), (4, 256), (3, 80)])
        width = _log(rng, 1, 20)
        return {"op": op, "B": max(1, min(_log(rng, 1, 176), 6000000 // (width * heads * D))), "width": width,
                "nodes": rng.randint(3 * width, 64), "heads": heads, "D": D, "page": page}
    heads, kv_heads, D = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "f32"])
    max_q = rng.choice([1, 1, _log(rng, 2, 1500)]) if op == "window" else _log(rng, 1, 250)
    B = _log(rng, 1, 48 if max_q < 30 else 6)
    own_len = max(max_q, _log(rng, 1, 9000))
    prefix = rng.choice([0, 0, 1, _log(rng, 2, 2000)])
    c = {"op": op, "B": B, "heads": heads, "kv_heads": kv_heads, "D": D, "page": page, "prefix": prefix, "own": own_len,
         "max_q": max_q, "dtype": dtype}
    if op == "window":
        c["window"], c["sinks"] = _log(rng, 1, 4096), rng.choice([0, 1, 4, _log(rng, 5, 300)])
    while work(c)["flops"] > 60e9 or work(c)["bytes"] > 3e8 or c["B"] * c["own"] * kv_heads * D > 5e8:
        if c["B"] > 1:
            c["B"] = c["B"] // 2
        else:
            c["own"], c["max_q"] = max(1, c["own"] // 2), max(1, c["max_q"] // 2)
            c["own"] = max(c["own"], c["max_q"])
    return c


def _case_rng(c):
    return random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))


def _lengths(c):
    """New tokens and own keys of every sequence of an attention case, from the case alone."""
    r = _case_rng(c)
    nq = [c["max_q"] if b == 0 else r.randint(max(1, c["max_q"] // 2), c["max_q"]) for b in range(c["B"])]
    ln = [c["own"] if b == 0 else r.randint(nq[b], c["own"]) for b in range(c["B"])]
    if c["max_q"] == 1 and c["B"] > 2:
        ln[-1] = 0  # an idle place of the batch: nothing of its own yet
    return nq, ln


def _trees(c):
    """Ancestors (itself among them) of every drafted token, as bits of a whole number."""
    r, out = _case_rng(c), []
    for n in _lengths(c)[0]:
        seen = []
        for i in range(n):
            # drafts hang on one of the last few tokens or anywhere, some start at the root
            p = -1 if i == 0 or r.random() < 0.1 else r.randint(max(0, i - 6), i - 1) if r.random() < 0.7 else r.randint(0, i - 1)
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        out.append(seen)
    return out


def _batch(c):
    """Lengths before, counts, capacity of an assign case."""
    r = _case_rng(c)
    held, count = [], []
    for b in range(c["B"]):
        h = r.randint(0, c["own"])
        if r.random() < c["back"] and h:
            n = -h if r.random() < 0.5 else -r.randint(1, min(h, 12))
        elif c["most"] > 1 and r.random() < 0.4:
            n = r.randint(0, c["most"])
        else:
            n = 1
        held.append(h)
        count.append(n)
    return held, count, c["own"] + c["most"] - (1 if c["short"] else 0)


def _pad16(D):
    return (D + 15) // 16 * 16


def _blank_cache(pages, heads, page, D):
    d = _pad16(D)
    return {"k": torch.zeros(pages, heads, page, d, dtype=torch.int8, device=DEV),
            "ks": torch.zeros(pages, heads, page, device=DEV),
            "v": torch.zeros(pages, heads, page // BLOCK, d, BLOCK, dtype=torch.int8, device=DEV),
            "vs": torch.zeros(pages, heads, page, device=DEV)}


def _filled_cache(g, pages, heads, page, D):
    ca = _blank_cache(pages, heads, page, D)
    for n in ("k", "v"):
        # (a page at a time: the binary32 copy of a large cache would not be small)
        for p in range(0, pages, 256):
            part = ca[n][p:p + 256]
            q = (torch.randn(part.shape, generator=g, device=DEV) * 35.0).round_().clamp_(-127, 127)
            if n == "k":
                q[..., D:] = 0
            else:
                q[..., D:, :] = 0
            part.copy_(q)
        ca[n + "s"] = 0.02 + 0.02 * torch.rand(ca[n + "s"].shape, generator=g, device=DEV)
    return ca


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    c = case
    s = {"case": dict(case), "place": torch.tensor(PLACE, device=DEV)}
    page, B = c["page"], c["B"]
    if c["op"] == "assign":
        held, count, cap = _batch(c)
        cols = (cap + page - 1) // page
        used = [(h + page - 1) // page for h in held]
        grow = sum((max(h, h + n) + page - 1) // page - u for h, n, u in zip(held, count, used))
        spare = max(1, grow // 2 if c["short"] else grow + B)  # (short: the list does not cover the step)
        total = sum(used) + spare
        ids = torch.randperm(total, generator=host).to(torch.int32)
        table, at = torch.full((B, cols), -1, dtype=torch.int32), 0
        for b, u in enumerate(used):
            table[b, :u] = ids[at:at + u]
            at += u
        free = torch.zeros(total, dtype=torch.int32)
        free[:spare] = ids[at:]
        s.update(held=_i32(held), count=_i32(count), table=table.to(DEV), free=free.to(DEV), nfree=_i32([spare]),
                 tokens=sum(max(n, 0) for n in count) + (7 if c["most"] > 1 else 0), cap=cap)  # (padded tokens at the end)
        return s
    if c["op"] == "move":
        # a tree of drafts of every sequence lies behind its tokens; the path's drafts go to the first places
        n, w = c["nodes"], c["width"]
        base = torch.randint(0, 3 * page, (B,), generator=host)
        cols = 3 + (n + 2 * page - 1) // page
        pages = torch.randperm(B * cols + 1, generator=host)[:B * cols].reshape(B, cols)
        path = torch.stack([torch.randperm(n - w, generator=host)[:w].sort().values + w for _ in range(B)])

        def slots(t):
            return (pages.gather(1, t // page) * page + t % page).to(DEV)

        s["src"], s["dst"] = slots(base[:, None] + path), slots(base[:, None] + torch.arange(w))
        s["cache"] = _filled_cache(g, B * cols + 1, c["heads"], page, c["D"])
        return s
    nq, ln = _lengths(c)
    npre = (c["prefix"] + page - 1) // page
    cols = max(1, (c["own"] + page - 1) // page)
    used = [(n + page - 1) // page for n in ln]
    pages = npre + sum(used) + 1
    ids = torch.randperm(pages, generator=host).to(torch.int32)
    table, at = torch.full((B, cols), -1, dtype=torch.int32), npre
    for b in range(B):
        table[b, :used[b]] = ids[at:at + used[b]]
        at += used[b]
    s["cache"] = _filled_cache(g, pages, c["kv_heads"], page, c["D"])
    s["q"] = (1.5 * torch.randn(sum(nq), c["heads"], c["D"], generator=g, device=DEV)).to(DTYPES[c["dtype"]])
    s["own_pages"], s["own_len"] = table.to(DEV), _i32(ln)
    s["prefix_pages"] = ids[:npre].to(DEV)
    s["q_start"] = torch.tensor([0] + nq).cumsum(0).to(torch.int32).to(DEV)
    if c["op"] == "tree":
        words = (c["max_q"] + 63) // 64
        rows = [[(m >> 64 * w & (1 << 64) - 1) for w in range(words)] for seen in _trees(c) for m in seen]
        s["tree"] = torch.tensor([[x - (1 << 64) if x >> 63 else x for x in row] for row in rows], dtype=torch.int64,
                                 device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _assign(s):
    page, cap, table, free = s["case"]["page"], s["cap"], s["table"], s["free"]
    held, count, B = s["held"].long(), s["count"].long(), s["case"]["B"]
    new = count.clamp(min=0)
    q_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    fits = held + new <= cap
    have = (held + page - 1) // page
    # pages given back, in order, go on top of the free list
    left = torch.where(count < 0, (held + count).clamp(min=0), held)
    keep = (left + page - 1) // page
    col = torch.arange(table.shape[1], device=DEV)
    back = (col >= keep[:, None]) & (col < have[:, None])
    rank = back.flatten().cumsum(0).reshape(back.shape) - 1
    top = s["nfree"].long() + back.sum()
    # (places that are not written go to one extra place)
    pushed = torch.cat([free, free.new_zeros(1)])
    pushed[torch.where(back, s["nfree"].long() + rank, free.shape[0])] = table
    free.copy_(pushed[:-1])
    # pages taken from the top, in order, as long as they last
    need = torch.where(fits, (held + new + page - 1) // page - have, 0).clamp(min=0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= top))
    taken = torch.where(ok, need, 0).sum()
    new_col = (col >= have[:, None]) & (col < (have + need)[:, None]) & ok[:, None]
    place = top - 1 - ((upto - need)[:, None] + col - have[:, None])
    table.copy_(torch.where(new_col, free[place.clamp(min=0, max=free.shape[0] - 1)], table))
    length = torch.where(ok, left + new, left)
    first = torch.where((count > 0) & ~ok, -1, left)
    j = torch.arange(s["tokens"], device=DEV)
    b = torch.bucketize(j, q_start[1:], right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    live = live & (first[b] >= 0)
    pos = torch.where(live, first[b] + j - q_start[b], -1)
    at = pos.clamp(min=0)
    slots = torch.where(live, table[b, at // page].long() * page + at % page, -1)
    return {"own_len": length.int(), "first": first.int(), "q_start": q_start.int(), "slots": slots,
            "positions": pos.int(), "left": (top - taken).int(), "own_pages": table, "free": free}


def _at(s, slots):
    page = s["case"]["page"]
    t = slots % page
    return slots // page, t, t // BLOCK, s["place"][t % BLOCK]


def _move(s):
    ca, D = s["cache"], s["case"]["D"]
    p, t, blk, pos = _at(s, s["src"])
    k, v = ca["k"][p, :, t], ca["v"][p, :, blk, :, pos]
    ks, vs = ca["ks"][p, :, t], ca["vs"][p, :, t]
    p, t, blk, pos = _at(s, s["dst"])
    ca["k"][p, :, t] = k
    ca["v"][p, :, blk, :, pos] = v
    ca["ks"][p, :, t] = ks
    ca["vs"][p, :, t] = vs
    return {"k": ca["k"][p, :, t, :D].float() * ca["ks"][p, :, t].unsqueeze(-1),
            "v": ca["v"][p, :, blk, :D, pos].float() * ca["vs"][p, :, t].unsqueeze(-1)}


def _keys(s, b, at):
    """Keys and values [kv_heads, n, D] of sequence b at positions 'at' (the prefix's first), in fp32."""
    c, ca = s["case"], s["cache"]
    D, page, P = c["D"], c["page"], c["prefix"]
    mine = (at - P).clamp(min=0)
    p, t = s["own_pages"][b].long()[mine // page], mine % page
    if P:
        pre = at < P
        p = torch.where(pre, s["prefix_pages"].long()[at.clamp(max=P - 1) // page], p)
        t = torch.where(pre, at % page, t)
    k = ca["k"][p, :, t, :D].float() * ca["ks"][p, :, t].unsqueeze(-1)
    v = ca["v"][p, :, t // BLOCK, :D, s["place"][t % BLOCK]].float() * ca["vs"][p, :, t].unsqueeze(-1)
    return k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous()


def _attend(s, masks):
    """Attention sequence by sequence; masks(b, n, ln): positions of the keys and who sees which ([n, keys])."""
    c = s["case"]
    D, Hk, G = c["D"], c["kv_heads"], c["heads"] // c["kv_heads"]
    nq, ln = _lengths(c)
    out, at = [], 0
    for b in range(c["B"]):
        n = nq[b]
        q = s["q"][at:at + n].float().reshape(n, Hk, G, D).permute(1, 0, 2, 3).reshape(Hk, n * G, D) * (D ** -0.5)
        pos, seen = masks(b, n, ln[b], at)
        at += n
        if pos.numel() == 0:
            out.append(torch.zeros(n, c["heads"], D, dtype=s["q"].dtype, device=DEV))
            continue
        k, v = _keys(s, b, pos)
        sc = torch.bmm(q, k.transpose(1, 2).contiguous()).reshape(Hk, n, G, -1)
        sc = torch.where(seen[None, :, None], sc, -math.inf)
        top = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - torch.where(top > -math.inf, top, 0.0))
        total = p.sum(-1, keepdim=True)
        o = torch.bmm(p.reshape(Hk, n * G, -1), v).reshape(Hk, n, G, D)
        o = torch.where(total > 0, o / total, 0.0).permute(1, 0, 2, 3).reshape(n, c["heads"], D)
        out.append(o.to(s["q"].dtype))
    return {"o": torch.cat(out)}


def _window(s):
    c = s["case"]
    P, W, S = c["prefix"], c["window"], c["sinks"]

    def masks(b, n, ln, at):
        lim = P + (ln - n + 1 + torch.arange(n, device=DEV)).clamp(min=0, max=ln)  # keys up to each query
        lo = max(0, P + max(0, ln - n + 1) - W)                                   # the first query's window
        pos = torch.cat([torch.arange(min(S, lo), device=DEV), torch.arange(lo, P + ln, device=DEV)])
        return pos, (pos < lim[:, None]) & ((pos >= lim[:, None] - W) | (pos < S))
    return _attend(s, masks)


def _tree(s):
    c = s["case"]
    P = c["prefix"]

    def masks(b, n, ln, at):
        pos = torch.arange(P + ln, device=DEV)
        node = pos - (P + ln - n)
        j = node.clamp(min=0)
        bit = (s["tree"][at:at + n][:, j // 64] >> (j % 64)) & 1
        return pos, (pos < P) | (node < 0) | (bit == 1)
    return _attend(s, masks)


# ---------------------------------------------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    from ternary_weight_linear_forward_amd import bitlinear as bl

    c = s["case"]
    if c["op"] == "assign":
        ln, first, q_start, slots, positions, left = bl.cache_assign(
            s["held"], s["count"], s["table"], s["free"], s["nfree"], s["tokens"], c["page"], s["cap"])
        return {"own_len": ln, "first": first, "q_start": q_start, "slots": slots, "positions": positions, "left": left,
                "own_pages": s["table"], "free": s["free"]}
    ca = s["cache"]
    cache = bl.KVCache(ca["k"], ca["v"], ca["ks"], ca["vs"], c["D"])
    if c["op"] == "move":
        bl.cache_move(cache, s["src"], s["dst"])
        k, v = bl.cache_read(cache, s["dst"].flatten(), dtype=torch.float32)
        return {"k": k.view(*s["dst"].shape, *k.shape[1:]), "v": v.view(*s["dst"].shape, *v.shape[1:])}
    kw = dict(prefix_pages=s["prefix_pages"], prefix_len=c["prefix"], q_start=None if c["max_q"] == 1 else s["q_start"],
              max_q=c["max_q"])
    if c["op"] == "window":
        return {"o": bl.attention_window(cache, s["q"], s["own_pages"], s["own_len"], c["own"], c["window"], c["sinks"], **kw)}
    return {"o": bl.attention_tree(cache, s["q"], s["own_pages"], s["own_len"], c["own"], s["tree"], **kw)}


PLAIN = {"assign": _assign, "move": _move, "window": _window, "tree": _tree}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    if c["op"] == "assign":  # lengths, counts in and lengths, starts out; table entries, slots and positions of the tokens
        tokens = sum(max(n, 0) for n in _batch(c)[1])
        return {"bytes": 20 * c["B"] + 12 * tokens + 8 * (tokens // c["page"] + 1), "flops": 10 * (c["B"] + tokens)}
    if c["op"] == "move":    # a token's row of K, column of V and scales in and out, slots; the values written back out
        n = c["B"] * c["width"]
        return {"bytes": n * (16 + c["heads"] * (4 * (_pad16(c["D"]) + 4) + 2 * (c["D"] + 4) + 8 * c["D"])),
                "flops": 2 * n * c["heads"] * c["D"]}
    es = 2 if c["dtype"] == "bf16" else 4
    nq, ln = _lengths(c)
    P = c["prefix"]
    if c["op"] == "window":
        W, S = c["window"], c["sinks"]
        keys = pairs = shared = 0
        for n, l in zip(nq, ln):
            ends = (P + max(0, min(l, l - n + i + 1)) for i in range(n))
            pairs += sum(min(e, W + min(S, max(0, e - W))) for e in ends)
            lo = max(0, P + max(0, l - n + 1) - W)
            keys += P + l - max(P, lo) + max(0, min(S, lo) - P)
            shared = max(shared, P - min(P, lo) + min(S, lo, P))
        keys += shared
    else:
        keys = P + sum(ln)
        pairs = sum(n * (P + l - n) for n, l in zip(nq, ln)) + sum(bin(m).count("1") for t in _trees(c) for m in t)
    return {"bytes": 2 * keys * c["kv_heads"] * (c["D"] + 4) + 2 * sum(nq) * c["heads"] * c["D"] * es,
            "flops": 4 * pairs * c["heads"] * c["D"]}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_assign(s):
    page, cap = s["case"]["page"], s["cap"]
    held, count, n = s["held"].tolist(), s["count"].tolist(), s["nfree"].item()
    table, room = s["table"].cpu(), s["free"].cpu()
    stack = room[:n].tolist()
    up = lambda x: (x + page - 1) // page  # noqa: E731
    for b, (h, d) in enumerate(zip(held, count)):
        if d < 0:
            stack += table[b, up(max(0, h + d)):up(h)].tolist()
    room[:len(stack)] = torch.tensor(stack, dtype=torch.int32)
    asked, had, start = 0, len(stack), [0]
    length, first, slots, positions = [], [], [], []
    for b, (h, d) in enumerate(zip(held, count)):
        start.append(start[-1] + max(0, d))
        if d <= 0:
            length.append(max(0, h + d))
            first.append(length[-1])
            continue
        need = up(h + d) - up(h) if h + d <= cap else 0
        asked += need
        if h + d > cap or (need and asked > had):
            length.append(h)
            first.append(-1)
            slots += [-1] * d
            positions += [-1] * d
            continue
        for x in range(need):
            table[b, up(h) + x] = stack.pop()
        length.append(h + d)
        first.append(h)
        for t in range(h, h + d):
            slots.append(table[b, t // page].item() * page + t % page)
            positions.append(t)
    pad = [-1] * (s["tokens"] - len(slots))
    return {"own_len": _i32(length), "first": _i32(first), "q_start": _i32(start),
            "slots": torch.tensor(slots + pad, dtype=torch.int64, device=DEV), "positions": _i32(positions + pad),
            "left": _i32([len(stack)]), "own_pages": table.to(DEV), "free": room.to(DEV)}


def _exact_rows(ca, pages, n, D):
    """The first n keys and values held by a list of pages, in 64 bits: [n, heads, D] each."""
    page = ca["k"].shape[2]
    t = torch.arange(n, device=DEV)
    p, t = torch.as_tensor(pages, device=DEV).long()[t // page], t % page
    byte = 16 * (t % 16 // 4) + 8 * (t % 64 // 32) + 4 * (t % 32 // 16) + t % 4
    k = ca["k"][p, :, t, :D].double() * ca["ks"][p, :, t].double()[..., None]
    v = ca["v"][p, :, t // 64, :D, byte].double() * ca["vs"][p, :, t].double()[..., None]
    return k, v


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "assign":
        return _exact_assign(s)
    if c["op"] == "move":
        page, ca, D = c["page"], s["cache"], c["D"]
        x = s["src"]
        t = x % page
        byte = 16 * (t % 16 // 4) + 8 * (t % 64 // 32) + 4 * (t % 32 // 16) + t % 4
        return {"k": ca["k"][x // page, :, t, :D].double() * ca["ks"][x // page, :, t].double()[..., None],
                "v": ca["v"][x // page, :, t // 64, :D, byte].double() * ca["vs"][x // page, :, t].double()[..., None]}
    nq, ln = _lengths(c)
    D, G, P = c["D"], c["heads"] // c["kv_heads"], c["prefix"]
    trees = _trees(c) if c["op"] == "tree" else None
    kp, vp = _exact_rows(s["cache"], s["prefix_pages"], P, D) if P else (None, None)
    out, at = [], 0
    for b in range(c["B"]):
        k, v = _exact_rows(s["cache"], s["own_pages"][b].clamp(min=0), ln[b], D)
        if P:
            k, v = torch.cat([kp, k]), torch.cat([vp, v])
        n, keys = nq[b], k.shape[0]
        k, v = k.permute(1, 2, 0).contiguous(), v.permute(1, 0, 2).contiguous()
        for i0 in range(0, n, 256):  # (a piece of a prompt at a time)
            m = min(256, n - i0)
            q = s["q"][at + i0:at + i0 + m].double().reshape(m, -1, G, D)
            x = torch.arange(keys, device=DEV)
            if c["op"] == "window":
                # (a query of a batch's idle place stands at the prefix's end)
                r = (P + ln[b] - n + i0 + torch.arange(m, device=DEV)[:, None]).clamp(min=P - 1)
                hidden = (x > r) | ((x <= r - c["window"]) & (x >= c["sinks"]))
            else:
                hidden = torch.zeros(m, keys, dtype=torch.bool)
                for i in range(m):
                    for j in range(n):
                        if ln[b] - n + j >= 0 and not trees[b][i0 + i] >> j & 1:
                            hidden[i, P + ln[b] - n + j] = True
                hidden = hidden.to(DEV)
            if not keys:
                out.append(torch.zeros(m, c["heads"], D, dtype=torch.float64, device=DEV))
                continue
            sc = torch.matmul(q.permute(1, 2, 0, 3).reshape(-1, G * m, D), k) / math.sqrt(D)
            sc = sc.reshape(-1, G, m, keys).masked_fill(hidden, -math.inf)
            pr = torch.softmax(sc, -1).nan_to_num(0.0)
            o = torch.matmul(pr.reshape(-1, G * m, keys), v).reshape(-1, G, m, D)
            out.append(o.permute(2, 0, 1, 3).reshape(m, c["heads"], D))
        at += n
    return {"o": torch.cat(out)}
