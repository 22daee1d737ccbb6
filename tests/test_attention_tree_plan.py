"""The cut of attention calls with a tree of drafts (csrc/attn_plan.h), checked on the host:
prefix and own keys are covered by parts that the limits allow, tiles cover the rows, and
workgroups stay below 2^31 at the documented limits."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ternary_weight_linear_forward_amd", "csrc")
FIELDS = ("rows_prefix rows_own waves_prefix waves_own tiles_own chunk_prefix splits_prefix chunk_own splits_own wgs_prefix "
          "wgs_own joint together direct ml_off").split()
SHIM = """
#include "attn_plan.h"
extern "C" void cut(const int64_t *x, int64_t *out)
{
    const bl::AttnPlan p = bl::attn_plan(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], x[8] != 0, true);
    const int64_t v[] = {%s};
    for (int k = 0; k < %d; ++k) out[k] = v[k];
}
""" % (", ".join("p." + f for f in FIELDS), len(FIELDS))


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, out = str(d / "cut.cpp"), str(d / "cut.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", out], check=True)
    lib = ctypes.CDLL(out)

    def cut(tokens, heads, kvh, D, seqs, max_q, own, prefix, f32):
        v = (ctypes.c_int64 * len(FIELDS))()
        lib.cut((ctypes.c_int64 * 9)(tokens, heads, kvh, D, seqs, max_q, own, prefix, f32), v)
        return dict(zip(FIELDS, v))
    return cut


def up(x, y):
    return (x + y - 1) // y


def check(p, tokens, heads, kvh, D, seqs, max_q, own, prefix, f32):
    G, most = heads // kvh, min(max_q, tokens)
    nbp, nbo = up(prefix, 64), up(own, 64)
    for rows, waves, tiles in ((p["rows_own"], p["waves_own"], p["tiles_own"]),) + \
            (((p["rows_prefix"], p["waves_prefix"], None),) if p["wgs_prefix"] else ()):
        assert (rows == 16 and waves in (1, 2, 4)) or (rows in (128, 256) and waves == 4)
        assert rows < 256 or (f32 and D <= 64)
        assert tiles is None or tiles == up(most * G, rows)
    # the prefix in a pass of its own, or before each sequence's own keys
    blocks = nbo + (nbp if p["joint"] else 0)
    assert p["chunk_own"] * p["splits_own"] >= blocks and 0 <= p["splits_own"] <= 64
    assert blocks == 0 or (p["splits_own"] - 1) * p["chunk_own"] < blocks  # (no part that no sequence can have)
    if nbp and not p["joint"]:
        assert p["chunk_prefix"] * p["splits_prefix"] >= nbp and 1 <= p["splits_prefix"] <= 64
        assert p["wgs_prefix"] == up(tokens * G, p["rows_prefix"]) * kvh * p["splits_prefix"]
    else:
        assert p["wgs_prefix"] == 0 and p["splits_prefix"] == 0
    assert p["wgs_own"] == seqs * p["tiles_own"] * kvh * p["splits_own"]
    assert 0 <= p["wgs_prefix"] < 2 ** 31 and 0 <= p["wgs_own"] < 2 ** 31 and p["wgs_prefix"] + p["wgs_own"] < 2 ** 31
    parts = p["splits_prefix"] + p["splits_own"]
    assert p["direct"] == (p["splits_own"] == 1 and parts == 1)
    assert p["ml_off"] == (0 if p["direct"] else parts * tokens * heads * up(D, 16) * 16)
    if p["rows_own"] != 16 and blocks and seqs * p["tiles_own"] * kvh <= 1024:
        assert p["chunk_own"] <= 48 or p["splits_own"] == 64  # (the rule for sequences of uneven lengths)


@pytest.mark.parametrize("heads,kvh", [(1, 1), (32, 32), (64, 8), (25, 5), (96, 1), (4096, 1)])
def test_parts_cover_the_keys(cut, heads, kvh):
    for D, f32 in ((1, True), (64, False), (64, True), (128, False), (128, True), (256, False), (256, True)):
        for seqs, max_q in ((1, 1), (48, 1), (1, 7), (16, 8), (16, 25), (4, 200), (1, 4096), (300, 5)):
            for own in (0, 1, 64, 2000, 9000, 100000):
                for prefix in (0, 1, 500, 3000, 60000):
                    x = (seqs * max_q, heads, kvh, D, seqs, max_q, own, prefix, f32)
                    try:
                        check(cut(*x), *x)
                    except AssertionError as e:
                        raise AssertionError((x, cut(*x))) from e


def test_a_bound_of_tokens_far_above_the_batch(cut):
    """A captured call keeps the bound of its largest batch."""
    for f32 in (False, True):
        for tokens, max_q in ((1, 4096), (70, 4096), (600, 4096)):
            x = (tokens, 64, 8, 128, 4, max_q, 5000, 100, f32)
            check(cut(*x), *x)


@pytest.mark.parametrize("x", [
    (1 << 20, 256, 256, 1, 1, 1 << 20, 1 << 30, 1 << 30), (1 << 20, 256, 1, 256, 1 << 20, 1, 64, 0),
    (1 << 16, 4096, 4096, 1, 1 << 16, 1, 1 << 30, 0), (1 << 16, 4096, 1, 1, 1, 1 << 16, 1 << 30, 1 << 30),
    (1 << 16, 4096, 1, 1, 1 << 16, 1, 0, 1 << 30), (1, 4096, 4096, 16, 1, 1, 1 << 30, 1 << 30),
])
def test_the_limits(cut, x):
    for f32 in (False, True):
        check(cut(*x, f32), *x, f32)
