"""Refusals of the entries of a serving step (places, moves, window and tree
attention): every argument is checked on the host before any HIP call.  Pointer
arguments are fake addresses that are never touched."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402

A, B, C, D, E, F, G = (0x10000 + i * 0x40000000 for i in range(7))  # far apart, 16-byte aligned
BAD, WS = bl.ERR_INVALID_ARG, bl.ERR_WORKSPACE
NAN = float("nan")


def cache(**kw):
    a = dict(K=A, K_scale=B, V=C, V_scale=D, pages=10, page_tokens=64, heads=2, head_dim=128)
    a.update(kw)
    return bl.Cache(**a)


def assign(**kw):
    a = dict(seqs=5, page_tokens=64, held=A, count=A + 0x1000, max_own=1000, own_pages=B, ld_pages=16, free_pages=C,
             max_free=100, free_count=D, free_left=D + 0x100, own_len=E, first=E + 0x1000, q_start=E + 0x2000, slots=F,
             positions=G, tokens=40, prefix_len=70, stream=None)
    a.update(kw)
    return bl.bitlinear_cache_assign(**a)


@pytest.mark.parametrize("kw", [
    dict(seqs=0), dict(seqs=65537), dict(page_tokens=0), dict(page_tokens=65), dict(page_tokens=1 << 21), dict(max_own=-1),
    dict(max_own=(1 << 30) + 1, ld_pages=1 << 30), dict(ld_pages=15), dict(ld_pages=1 << 41), dict(max_free=-1),
    dict(max_free=1 << 31), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(prefix_len=-1), dict(prefix_len=(1 << 30) + 1),
    dict(held=None), dict(count=None), dict(own_pages=None), dict(free_pages=None), dict(free_count=None),
    dict(free_left=None), dict(own_len=None), dict(first=None), dict(q_start=None), dict(slots=None),
    dict(held=A + 2), dict(count=A + 0x1002), dict(own_pages=B + 2), dict(free_pages=C + 1), dict(free_count=D + 2),
    dict(free_left=D + 0x102), dict(own_len=E + 2), dict(first=E + 0x1001), dict(q_start=E + 0x2002), dict(slots=F + 4),
    dict(positions=G + 2),
    # an output on an input or on another output; in place only as a whole
    dict(own_len=A + 4), dict(own_len=A + 0x1000), dict(first=A), dict(q_start=A), dict(slots=A), dict(positions=A),
    dict(own_pages=A), dict(free_pages=A), dict(free_left=A), dict(first=E), dict(first=E + 16), dict(q_start=E),
    dict(slots=B), dict(slots=C), dict(positions=F), dict(positions=B + 64), dict(free_pages=B + 4 * (4 * 16 + 15)),
    dict(free_count=C), dict(free_left=C + 4 * 99), dict(own_len=D), dict(free_left=E), dict(q_start=E + 0x1000 + 16),
])
def test_cache_assign_rejects(kw):
    assert assign(**kw) == BAD


def move(c=None, **kw):
    a = dict(src=E, dst=F, groups=3, width=5, stream=None)
    a.update(kw)
    return bl.bitlinear_cache_move(c or cache(), **a)


@pytest.mark.parametrize("kw", [dict(src=None), dict(dst=None), dict(groups=-1), dict(groups=(1 << 20) + 1), dict(width=0),
                                dict(width=65), dict(src=E + 4), dict(dst=F + 4), dict(src=A), dict(dst=D), dict(dst=B)])
def test_cache_move_rejects(kw):
    assert move(**kw) == BAD


def test_no_groups_do_nothing():
    assert move(groups=0) == bl.OK and move(cache(pages=0), groups=0) == BAD
    assert bl.bitlinear_cache_move(ctypes.POINTER(bl.Cache)(), E, F, 0, 5, None) == BAD


def common(**kw):
    a = dict(Q=E, dtype=bl.BF16, tokens=6, heads=8, ldq_token=1024, ldq_head=128, seqs=3, q_start=None, max_q=2,
             own_pages=F, ld_pages=2, own_len=F + 0x1000, max_own=100, prefix_pages=F + 0x2000, prefix_len=70, scale=0.1,
             O=G, ldo_token=1024, ldo_head=128, lse=G + 0x1000000, ws=G + 0x2000000, ws_bytes=1 << 28, stream=None)
    a.update(kw)
    return a


def window(c=None, **kw):
    return bl.bitlinear_attention_window(c or cache(), **common(**{**dict(window=30, sinks=4), **kw}))


def tree(c=None, **kw):
    return bl.bitlinear_attention_tree(c or cache(), **common(**{**dict(tree=F + 0x3000, ld_tree=1), **kw}))


SHARED = [
    dict(Q=None), dict(O=None), dict(own_len=None), dict(own_pages=None), dict(prefix_pages=None), dict(dtype=bl.I32),
    dict(scale=NAN), dict(tokens=0), dict(tokens=5), dict(heads=7), dict(heads=0), dict(seqs=0), dict(max_q=0),
    dict(max_own=-1), dict(prefix_len=-1), dict(max_own=(1 << 30) + 1), dict(ld_pages=1), dict(Q=E + 1), dict(O=G + 1),
    dict(own_len=F + 2), dict(lse=G + 0x1000002), dict(ldo_token=900), dict(ldo_head=0), dict(ldq_token=-1), dict(O=E),
    dict(O=A), dict(lse=G), dict(lse=B), dict(O=F), dict(tokens=-1), dict(tokens=1 << 21), dict(max_q=-1),
]


@pytest.mark.parametrize("kw", SHARED)
def test_masked_attention_rejects(kw):
    assert window(**kw) == BAD and tree(**kw) == BAD


@pytest.mark.parametrize("kw", [dict(window=0), dict(window=-1), dict(window=(1 << 31) + 1), dict(sinks=-1),
                                dict(sinks=(1 << 30) + 1)])
def test_window_rejects(kw):
    assert window(**kw) == BAD
    sizes = (6, 8, 2, 128, 3, 2, 100, 70, kw.get("window", 30), kw.get("sinks", 4))
    assert bl.bitlinear_attention_window_workspace_bytes(*sizes) == -1


@pytest.mark.parametrize("kw", [
    dict(tree=None), dict(tree=F + 0x3004), dict(ld_tree=0), dict(ld_tree=-1), dict(tree=G), dict(O=F + 0x3000),
    dict(lse=F + 0x3000), dict(ld_tree=1 << 41),
    dict(tokens=200, seqs=2, max_q=100), dict(tokens=70, seqs=1, max_q=1000, q_start=F + 0x200),  # (65 bits and more)
])
def test_tree_rejects(kw):
    assert tree(**kw) == BAD


def test_workspaces():
    args = (6, 8, 2, 128, 3, 2, 100, 70)
    for i, v in [(0, 0), (1, 7), (2, 0), (3, 257), (4, 0), (5, 0), (6, -1), (7, -1)]:
        bad = list(args)
        bad[i] = v
        assert bl.bitlinear_attention_window_workspace_bytes(*bad, 30, 4) == -1, (i, v)
        assert bl.bitlinear_attention_tree_workspace_bytes(*bad) == -1, (i, v)
    # a window over everything is the plain call's plan
    assert bl.bitlinear_attention_window_workspace_bytes(*args, 170, 4) == bl.bitlinear_attention_workspace_bytes(*args)
    # a long cache with a short window is not split as a long one
    long = (1, 8, 1, 128, 1, 1, 1 << 20, 0)
    assert bl.bitlinear_attention_window_workspace_bytes(*long, 64, 4) < bl.bitlinear_attention_workspace_bytes(*long)
    need = bl.bitlinear_attention_tree_workspace_bytes(1, 8, 2, 128, 1, 1, 100000, 0)
    assert need > 0
    one = dict(tokens=1, seqs=1, max_q=1, max_own=100000, ld_pages=2000, prefix_len=0, prefix_pages=None)
    big = cache(pages=4000)
    for kw, st in ((dict(ws=None), WS), (dict(ws_bytes=need - 1), WS), (dict(ws=G + 0x2000004), BAD), (dict(ws=E), BAD),
                   (dict(ws=F + 0x3000), BAD)):
        assert tree(big, **{**one, **kw}) == st, kw
    need = bl.bitlinear_attention_window_workspace_bytes(1, 8, 2, 128, 1, 1, 100000, 0, 20000, 4)
    assert need > 0
    assert window(big, **{**one, **dict(window=20000, ws_bytes=need - 1)}) == WS
    assert window(big, **{**one, **dict(window=20000, ws=None)}) == WS


# --- torch helpers -----------------------------------------------------------
i32, i64 = torch.int32, torch.int64


def zeros(*s, dtype=i32):
    return torch.zeros(s, dtype=dtype)


@pytest.fixture
def no_launch(monkeypatch):
    """A library that counts its calls: a refusal makes none."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_bytes"):
                    return 64
                if name.endswith("_string"):
                    return b"refused"
                calls.append(name)
                return bl.OK
            return call

    monkeypatch.setattr(bl, "_lib", Lib())
    monkeypatch.setattr(bl, "_stream", lambda s=None: 0)
    return calls


def kv():
    return bl.KVCache(zeros(4, 2, 64, 64, dtype=torch.int8), zeros(4, 2, 1, 64, 64, dtype=torch.int8),
                      torch.zeros(4, 2, 64), torch.zeros(4, 2, 64), 50)


ASSIGN = dict(held=zeros(3), count=zeros(3), own_pages=zeros(3, 4), free_pages=zeros(9), free_count=zeros(1), tokens=5,
              page_tokens=64)


@pytest.mark.parametrize("kw", [
    {}, dict(held=zeros(3, dtype=i64)), dict(held=zeros(3, 1)), dict(count=zeros(4)), dict(count=zeros(6)[::2]),
    dict(count=torch.zeros(3)), dict(own_pages=zeros(12)), dict(own_pages=zeros(2, 4)), dict(own_pages=zeros(3, 8)[:, ::2]),
    dict(own_pages=zeros(3, 4, dtype=i64)), dict(own_pages=zeros(3, 1).expand(3, 4)), dict(own_pages=zeros(1, 4).expand(3, 4)),
    dict(free_pages=zeros(9, dtype=i64)), dict(free_pages=zeros(3, 3)), dict(free_pages=zeros(18)[::2]),
    dict(free_count=zeros(2)), dict(free_count=zeros(1, dtype=i64)), dict(tokens=-1), dict(page_tokens=0), dict(max_own=257),
    dict(own_len=zeros(2)), dict(own_len=zeros(3, dtype=i64)), dict(free_left=zeros(2)), dict(free_left=torch.zeros(1)),
])
def test_cache_assign_helper_rejects(no_launch, monkeypatch, kw):  # (the first: tensors of the host)
    if kw:
        monkeypatch.setattr(bl, "_here", lambda *_: None)
    with pytest.raises(bl.BitlinearError):
        bl.cache_assign(**{**ASSIGN, **kw})
    assert no_launch == []


@pytest.mark.parametrize("src,dst", [
    (zeros(2, 3, dtype=i64), zeros(2, 3, dtype=i64)), (zeros(2, 3, dtype=i64), zeros(3, 2, dtype=i64)),
    (zeros(2, 3), zeros(2, 3)), (zeros(2, 3, dtype=i64), zeros(2, 3)), (zeros(2, 6, dtype=i64)[:, ::2], zeros(2, 3, dtype=i64)),
    (zeros(1, 2, 3, dtype=i64), zeros(1, 2, 3, dtype=i64)), (zeros(2, 3, dtype=i64), zeros(2, 6, dtype=i64)[:, ::2]),
])
def test_cache_move_helper_rejects(no_launch, monkeypatch, src, dst):
    if src.shape != (2, 3) or dst.dtype != src.dtype or src.dtype != i64 or not (src.is_contiguous() and dst.is_contiguous()):
        monkeypatch.setattr(bl, "_here", lambda *_: None)
    with pytest.raises(bl.BitlinearError):
        bl.cache_move(kv(), src, dst)
    assert no_launch == []


@pytest.mark.parametrize("kw", [
    {}, dict(tree=zeros(6, dtype=i64)), dict(tree=zeros(6, 1)), dict(tree=zeros(5, 1, dtype=i64)),
    dict(tree=zeros(6, 0, dtype=i64)), dict(tree=zeros(6, 4, dtype=i64)[:, ::2]),
])
def test_tree_helper_rejects(no_launch, monkeypatch, kw):  # (the first: tensors of the host)
    if kw:
        monkeypatch.setattr(bl, "_here", lambda *_: None)
    a = dict(cache=kv(), Q=torch.zeros(6, 4, 50), own_pages=zeros(3, 2), own_len=zeros(3), max_own=100, max_q=2)
    with pytest.raises(bl.BitlinearError):
        bl.attention_tree(**{**a, **dict(tree=zeros(6, 1, dtype=i64)), **kw})
    assert no_launch == []


@pytest.mark.parametrize("kw", [
    {}, dict(Q=torch.zeros(6, 4, 49)), dict(Q=torch.zeros(6, 4, 50).half()), dict(own_pages=zeros(3)), dict(own_pages=zeros(2, 2)),
    dict(own_pages=zeros(3, 1)), dict(own_len=zeros(3, dtype=i64)), dict(q_start=zeros(3)), dict(q_start=zeros(4, dtype=i64)),
    dict(prefix_len=65, prefix_pages=zeros(1)), dict(prefix_len=1), dict(out=torch.zeros(6, 4, 50).bfloat16()),
])
def test_window_helper_rejects(no_launch, monkeypatch, kw):
    if kw:
        monkeypatch.setattr(bl, "_here", lambda *_: None)
    a = dict(cache=kv(), Q=torch.zeros(6, 4, 50), own_pages=zeros(3, 2), own_len=zeros(3), max_own=100, max_q=2, window=30)
    with pytest.raises(bl.BitlinearError):
        bl.attention_window(**{**a, **kw})
    assert no_launch == []
