"""How attention calls are cut into workgroups (csrc/attn_plan.h), checked on the
host: what every launch assumes of its tiles, over sizes with all their bounds
larger and smaller than what the call holds."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ternary_weight_linear_forward_amd", "csrc")
SHIM = """
#include "attn_plan.h"
extern "C" int cut(const int64_t *x, int64_t *out)
{
    const bl::AttnPlan p = bl::attn_plan(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], x[8] != 0);
    bl::AttnLaunch l[2];
    const int n = bl::attn_launches(p, l);
    for (int i = 0; i < n; ++i) {
        const int64_t v[] = {l[i].rows, l[i].waves, l[i].first, l[i].wgs};
        for (int k = 0; k < 4; ++k) out[4 * i + k] = v[k];
    }
    const int64_t v[] = {p.tiles_own, p.chunk_prefix, p.splits_prefix, p.chunk_own, p.splits_own, p.wgs_prefix,
                         p.wgs_own, p.joint, p.direct, p.ml_off};
    for (int k = 0; k < 10; ++k) out[8 + k] = v[k];
    return n;
}
extern "C" int64_t pieces(int64_t wgs, int64_t *out)
{
    int64_t n = 0;
    bl::attn_pieces(wgs, 0, [&](int64_t first, int64_t count) { out[2 * n] = first; out[2 * n++ + 1] = count; return 0; });
    return n;
}
extern "C" int64_t join_rows(int64_t tokens, int64_t heads, int64_t seqs, int64_t max_q)
{
    return bl::attn_join_rows(tokens, heads, seqs, max_q);
}
"""
NAMES = ("tiles_own", "chunk_prefix", "splits_prefix", "chunk_own", "splits_own", "wgs_prefix", "wgs_own", "joint",
         "direct", "ml_off")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, out = str(d / "cut.cpp"), str(d / "cut.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.fixture(scope="module")
def cut(lib):
    fn = lib.cut

    def call(*sizes):
        out = (ctypes.c_int64 * 18)()
        n = fn((ctypes.c_int64 * 9)(*sizes), out)
        return [tuple(out[4 * i:4 * i + 4]) for i in range(n)], dict(zip(NAMES, out[8:]))
    return call


def up(x, y):
    return (x + y - 1) // y


def check(cut, tokens, heads, kvh, D, seqs, max_q, max_own, prefix, f32):
    what = dict(tokens=tokens, heads=heads, kv_heads=kvh, D=D, seqs=seqs, max_q=max_q, max_own=max_own, prefix=prefix,
                f32=f32)
    launches, p = cut(tokens, heads, kvh, D, seqs, max_q, max_own, prefix, f32)
    G, most = heads // kvh, min(max_q, tokens)  # (a sequence has at most 'most' query tokens)
    nbp, nbo = up(prefix, 64), up(max_own, 64)
    at = 0
    for rows, waves, first, wgs in launches:
        assert first == at, what
        at += wgs
        if wgs == 0:
            continue
        # the kernel the tile size selects is started with the waves it is written for
        if rows == 16:
            assert waves in (1, 2, 4), what
        else:
            assert rows in (128, 256) and waves == rows // 32 and (D <= 64 or (D <= 128 and not f32)), what
            assert rows == 128 or D > 64, what
        # prefix workgroups: every tile has rows of its own, and the tiles cover all rows
        here = max(0, min(p["wgs_prefix"], first + wgs) - first)
        if here:
            tiles, rest = divmod(p["wgs_prefix"], kvh * p["splits_prefix"])
            assert rest == 0 and here == p["wgs_prefix"], what
            assert (tiles - 1) * rows < tokens * G <= tiles * rows, what
            assert p["splits_prefix"] * p["chunk_prefix"] >= nbp > (p["splits_prefix"] - 1) * p["chunk_prefix"], what
        if here < wgs:
            assert p["wgs_own"] == seqs * p["tiles_own"] * kvh * p["splits_own"], what
            assert (p["tiles_own"] - 1) * rows < most * G <= p["tiles_own"] * rows, what
            blocks = nbo + (nbp if p["joint"] else 0)
            assert p["splits_own"] * p["chunk_own"] >= blocks > (p["splits_own"] - 1) * p["chunk_own"], what
    assert at == p["wgs_prefix"] + p["wgs_own"] < 1 << 31, what
    assert (p["wgs_prefix"] > 0) == (prefix > 0 and not p["joint"]), what
    if p["direct"]:
        assert p["wgs_prefix"] == 0 and p["splits_own"] == 1, what


HEADS = [(1, 1), (8, 8), (32, 32), (64, 8), (8, 1), (25, 5), (96, 1)]


@pytest.mark.parametrize("heads,kvh", HEADS)
@pytest.mark.parametrize("f32", [False, True])
def test_tiles_have_rows(cut, heads, kvh, f32):
    """Every tile of every launch, with max_q at, above and far above the tokens there are."""
    for D in (50, 64, 128, 256):
        for tokens in (1, 3, 12, 13, 33, 60, 96, 97, 128, 400):
            for max_q in sorted({1, 2, 12, 13, 14, 16, 32, 97, 100, 128, 400, 5000}):
                for seqs in (1, 4, tokens):
                    for max_own, prefix in ((0, 8000), (333, 60001), (100, 4000), (64, 0), (0, 0), (700, 77)):
                        check(cut, tokens, heads, kvh, D, seqs, max_q, max_own, prefix, f32)


def test_the_bound_of_a_captured_call(cut):
    """A fixed max_q above the tokens of this call, with a prefix of its own pass."""
    for own in (0, 333):
        check(cut, 12, 64, 8, 128, 4, 13, own, 60001, False)
        check(cut, 96, 32, 32, 128, 4, 100, own, 4000, False)
        check(cut, 60, 32, 32, 64, 4, 100, own, 8000, True)


def test_launches_hold_fewer_than_2_32_threads(cut, lib):
    """At the largest sizes the header allows, and around a piece's size: the pieces are one after the other, hold
    every workgroup once, and none has 2^32 threads."""
    wgs = {1, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, 3 << 22, (1 << 30) + 5}
    for heads, kvh in ((256, 256), (256, 4), (4096, 4096), (17, 1), (34, 2), (1, 1)):
        for seqs, max_q, tokens in ((1 << 20, 1, 64), (1 << 20, 1, 1 << 20), (1 << 10, 1 << 10, 1 << 20), (1, 1 << 20, 1 << 20),
                                    (1 << 20, 1 << 20, 1), (256, 8192, 8192), (1 << 16, 1 << 20, 1 << 12)):
            if max(seqs * max_q, tokens) * heads > 1 << 28:
                continue
            for D, f32 in ((16, False), (128, False), (128, True), (256, False)):
                for prefix, own in ((0, 64), (100, 64), (1 << 30, 1 << 30), (60000, 0)):
                    check(cut, tokens, heads, kvh, D, seqs, max_q, own, prefix, f32)
                    launches, p = cut(tokens, heads, kvh, D, seqs, max_q, own, prefix, f32)
                    wgs |= {x[3] for x in launches if x[3]}
                    lib.join_rows.restype = ctypes.c_int64
                    rows = lib.join_rows(*(ctypes.c_int64(v) for v in (tokens, heads, seqs, max_q)))
                    assert rows == seqs * min(max_q, tokens) * heads <= 1 << 28
                    wgs |= {up(rows, 256 // lanes) for lanes in (16, 32, 64)}
    lib.pieces.restype = ctypes.c_int64
    for n in wgs:
        out = (ctypes.c_int64 * 1024)()
        k = lib.pieces(ctypes.c_int64(n), out)
        at = 0
        for i in range(k):
            assert out[2 * i] == at and 0 < out[2 * i + 1] * 512 < 1 << 32
            at += out[2 * i + 1]
        assert at == n
