"""The cut of attention calls with a sliding window (csrc/attn_plan.h), checked on
the host: the parts cover every block that a tile's rows see, counted one by one."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ternary_weight_linear_forward_amd", "csrc")
SHIM = """
#include "attn_plan.h"
extern "C" void cut(const int64_t *x, int64_t *out)
{
    const bl::AttnPlan p = bl::attn_plan(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], x[8] != 0, true, x[9], x[10]);
    const int64_t v[] = {p.rows_own, p.tiles_own, p.chunk_own, p.splits_own, p.wgs_prefix, p.wgs_own, p.joint, p.direct,
                         p.waves_own};
    for (int k = 0; k < 9; ++k) out[k] = v[k];
}
extern "C" int64_t blocks(int64_t prefix, int64_t max_own, int64_t queries, int64_t window, int64_t sinks)
{
    return bl::attn_window_blocks(prefix, max_own, queries, window, sinks);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, out = str(d / "cut.cpp"), str(d / "cut.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.blocks.restype = ctypes.c_int64
    lib.blocks.argtypes = [ctypes.c_int64] * 5
    return lib


def up(x, y):
    return (x + y - 1) // y


def met(prefix, ends, window, sinks):
    """Blocks (of the prefix's list, then of the own one) with a key that a query of 'ends' (keys up to it) sees."""
    nbp, out = up(prefix, 64), set()
    block = lambda p: p // 64 if p < prefix else nbp + (p - prefix) // 64  # noqa: E731
    for e in ends:
        for lo, hi in ((0, min(sinks, e)), (max(0, e - window), e)):
            if hi > lo:
                out |= set(range(block(lo), block(hi - 1) + 1))
    return out


def test_blocks_of_a_tile(lib):
    """The bound holds for every place of a tile's queries, and is at most three blocks too many."""
    for prefix in (0, 1, 63, 64, 65, 200):
        for own in (1, 64, 65, 300, 700):
            for queries in (1, 2, 33, 65):
                for window in (1, 2, 63, 64, 65, 130, 500):
                    for sinks in (0, 1, 64, 65, 100, 300):
                        bound, most = lib.blocks(prefix, own, queries, window, sinks), 0
                        for last in {1, 2, queries, 64, 65, 66, own // 2, own - 1, own}:
                            if not 0 <= last <= own:
                                continue
                            ends = [prefix + max(0, last - i) for i in range(min(queries, last + 1))]
                            most = max(most, len(met(prefix, ends, window, sinks)))
                        assert bound >= most, (prefix, own, queries, window, sinks, bound, most)
                        if queries <= own // 2:  # (overlapping first tokens and windows are counted twice)
                            assert bound <= min(up(prefix, 64) + up(own, 64),
                                                up(sinks, 64) + up(window + queries, 64) + 4), (prefix, own, queries, window, sinks)


@pytest.mark.parametrize("heads,kvh", [(1, 1), (32, 32), (64, 8), (25, 5), (96, 1)])
def test_parts_cover_the_blocks(lib, heads, kvh):
    G = heads // kvh
    for D, f32 in ((64, False), (64, True), (128, False), (128, True), (256, False)):
        for seqs, max_q in ((1, 1), (48, 1), (3, 300), (2, 4096), (1, 7)):
            for own, prefix in ((5000, 77), (8192, 0), (0, 3000), (max_q, 1)):
                for window, sinks in ((1, 0), (64, 4), (1024, 4), (4096, 300), (3000, 8000)):
                    if window >= prefix + own:
                        continue
                    out = (ctypes.c_int64 * 9)()
                    lib.cut((ctypes.c_int64 * 11)(seqs * max_q, heads, kvh, D, seqs, max_q, own, prefix, f32, window, sinks), out)
                    rows, tiles, chunk, splits, wgs_prefix, wgs, joint, direct, waves = out
                    what = (heads, kvh, D, f32, seqs, max_q, own, prefix, window, sinks, list(out))
                    assert wgs_prefix == 0 and joint == (prefix > 0) and direct == (splits == 1), what
                    assert wgs == seqs * tiles * kvh * splits and tiles == up(max_q * G, rows), what
                    assert (rows == 16 and waves in (1, 2, 4)) or (rows in (128, 256) and waves == 4), what
                    assert rows < 256 or (f32 and D <= 64), what
                    for tile in {0, tiles // 2, tiles - 1}:
                        first, last = tile * rows // G, (min((tile + 1) * rows, max_q * G) - 1) // G
                        ends = [prefix + max(0, min(own, own - max_q + i + 1)) for i in (first, last)]
                        # every end between them: the blocks are those of the first one's window to the last
                        seen = met(prefix, ends, window, sinks) | met(prefix, ends[1:], window + ends[1] - ends[0], sinks)
                        assert chunk * splits >= len(seen), what
