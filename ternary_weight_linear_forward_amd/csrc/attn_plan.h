// attn_plan.h -- how an attention call (attention.hip) is cut into workgroups, and
// the launches that follow from it.  Host only, no HIP: a test compiles it alone.
#pragma once

#include <algorithm>
#include <stdint.h>

namespace bl {

constexpr int ATTN_BLOCK = 64; // keys of a block (CACHE_BLOCK)

// How a call is cut: the prefix's workgroups (row tiles x kv heads x splits of
// chunk_prefix blocks of 64 keys), then the sequences'.
struct AttnPlan {
    int rows_prefix, rows_own;   // rows of a workgroup (16: k_attn_stream, 128, 256: k_attn_tile)
    int waves_prefix, waves_own; // and its waves
    int tiles_own;               // row tiles of a sequence
    int chunk_prefix, splits_prefix, chunk_own, splits_own;
    int wgs_prefix, wgs_own;
    int wg0;        // first workgroup of the launch
    bool joint;     // the sequences' workgroups go over the prefix too (none of its own)
    bool together;  // prefix and sequences in one launch
    bool direct;    // one part in all: the workgroups write the result
    int64_t ml_off; // floats of o sums before the (m, l) pairs
};

inline int64_t div_up(int64_t x, int64_t y) { return (x + y - 1) / y; }

// (Times in this file are of kernels in their first launches after an idle time, both
// sides alike; sustained ones are up to an eighth lower.)

// Rows a workgroup takes: 16 with k_attn_stream, 128 or 256 (four or eight waves)
// with k_attn_tile.  Row tiles that read the cache again from L2 cost less than a
// mostly empty tile of 128: bf16, 8 kv heads of 128, keys x rows, us of k_attn_stream
// and of k_attn_tile: 60001 x 24: 48, 81; x 64: 69, 82; x 96: 95, 86; 12000 x 96: 37,
// 50; x 128: 40, 52; x 256: 62, 59; x 1024: 187, 108.  With the registers of fp32
// queries (two terms) and head_dim past 64, or of head_dim past 128, k_attn_stream
// won at every size (400 query tokens x 4 on 2100 keys, heads of 256, bf16: 738, 838;
// of 128, fp32: 813, 1109).  Eight waves share a conversion of the keys and need
// registers for two waves a SIMD (fp32 queries do not leave them).
constexpr int64_t kStreamRows = 96;

inline int tile_rows(int64_t rows, int64_t head_dim, bool f32)
{
    if (rows <= kStreamRows || head_dim > 128 || (f32 && head_dim > 64)) return 16;
    return rows <= 128 || head_dim <= 64 ? 128 : 256;
}

// How 'wgs' workgroups' passes over 'blocks' key blocks are split: blocks of a
// part, parts, waves of a workgroup.
struct AttnCut {
    int chunk, splits, waves;
};

// The cut with the least time, in eighths of a block, of all rounds of the card: a
// wave (of k_attn_stream, whose waves take blocks in turn) or workgroup (of
// k_attn_tile) costs its blocks and about four more for its start and end; waves
// that join their sums cost half a block, a part's sums on their way through memory
// 'part', and the join itself, where there would be none (joined), four blocks.
// waves: those of k_attn_stream, 0 for any; others: workgroups of the same launch.
// 2^20 workgroups are a thousand rounds of the card, which no split makes shorter: no
// more parts than that asks for, so that workgroups are numbered in 31 bits.
inline AttnCut choose_cut(int64_t wgs, int64_t blocks, int rows, int64_t head_dim, int waves, int64_t others,
                          int64_t part, bool joined)
{
    AttnCut best{0, 0, waves ? waves : 4};
    if (blocks == 0) return best;
    const int dc = head_dim <= 64 ? 1 : head_dim <= 128 ? 2 : 4;
    const bool stream = rows == 16;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(64, (int64_t(1) << 20) / wgs));
    int64_t least = -1;
    for (int w = 1; w <= 8; w *= 2) {
        if (stream ? w > 4 || (waves && w != waves) : w != rows / 32) continue;
        const bool alone = stream ? dc == 4 : rows == 256; // one wave a SIMD, one workgroup a CU; or two
        const int64_t slots = stream ? 256 * (4 / w) * (alone ? 1 : 2) : 256 * (alone ? 1 : 2);
        for (int64_t s = 1; s <= most && (s == 1 || div_up(blocks, s) >= (stream ? w : 2)); ++s) {
            const int64_t c = div_up(blocks, s), n = div_up(blocks, c);
            const int64_t cost =
                8 * div_up(wgs * n + others, slots) * ((stream ? div_up(c, w) : c) + 4) +
                (stream && w > 1 ? 4 : 0) + (n > 1 || joined ? n * part : 0) + (n > 1 && !joined ? 32 : 0);
            if (least < 0 || cost < least) {
                least = cost;
                best = AttnCut{static_cast<int>(c), static_cast<int>(n), w};
            }
        }
    }
    return best;
}

// Reading the prefix again for each sequence costs less than a launch and a join
// of their own up to about this many bytes (a launch and its join are near 8 us).
constexpr int64_t kJointBytes = int64_t(16) << 20;

inline AttnPlan attn_plan(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs,
                          int64_t max_q, int64_t max_own, int64_t prefix, bool f32)
{
    AttnPlan p;
    const int64_t G = heads / kv_heads, dp = div_up(head_dim, 16) * 16;
    const int64_t nbp = div_up(prefix, ATTN_BLOCK), nbo = div_up(max_own, ATTN_BLOCK);
    // (max_q is a bound, which a captured call keeps from its largest batch: a sequence has no more
    // query tokens than the call, so its tiles are never larger than the prefix's)
    max_q = std::min(max_q, tokens);
    p.rows_prefix = tile_rows(tokens * G, head_dim, f32);
    p.rows_own = tile_rows(max_q * G, head_dim, f32);
    p.tiles_own = static_cast<int>(div_up(max_q * G, p.rows_own));
    // one pass over prefix and own keys where a sequence fills row tiles of its own anyway (4 x 400 query
    // tokens x 8 rows on 2100 keys: 207 us, with a pass of its own for the prefix 222 + 25), or the prefix is
    // short
    p.joint = nbp > 0 && (max_q * G >= 128 || 2 * prefix * kv_heads * dp * (seqs - 1) <= kJointBytes);
    const int64_t tp = p.joint || nbp == 0 ? 0 : div_up(tokens * G, p.rows_prefix);
    // with the same kernel for both, one launch (5 x 8 rows on 60001 keys with 333 of their own: 54 us
    // for both, 52 + 12 one after the other)
    p.together = tp > 0 && p.rows_prefix == 16 && p.rows_own == 16;
    // a part's sums, written and read at a copy's rate, in eighths of a block's 2.6 us
    const int64_t part = 1 + tokens * heads * dp * 6 / 1000000;
    // workgroups with rows at most: a sequence's last tile is its own.  With both, 2 x 300 query tokens x 64
    // heads on 5000 keys are split (158 -> 135 us) and 4 x 400 on 2100 are not (204; split 222)
    const int64_t busy = std::min(seqs * p.tiles_own, div_up(tokens * G, p.rows_own) + seqs) * kv_heads;
    AttnCut cut{0, 0, 4};
    if (tp > 0)
        cut = choose_cut(tp * kv_heads, nbp, p.rows_prefix, head_dim, 0,
                         p.together && nbo > 0 ? busy : 0, part, true);
    p.chunk_prefix = cut.chunk;
    p.splits_prefix = cut.splits;
    p.waves_prefix = cut.waves;
    p.wgs_prefix = static_cast<int>(tp * kv_heads * p.splits_prefix);
    cut = choose_cut(busy, p.joint ? nbp + nbo : nbo, p.rows_own, head_dim,
                     p.together ? p.waves_prefix : 0, p.together ? p.wgs_prefix : 0, part, tp > 0);
    p.chunk_own = cut.chunk;
    p.splits_own = cut.splits;
    p.waves_own = cut.waves;
    p.wgs_own = static_cast<int>(seqs * p.tiles_own * kv_heads * p.splits_own);
    p.wg0 = 0;
    const int64_t parts = p.splits_prefix + p.splits_own;
    p.direct = parts == 1 && p.splits_own == 1;
    p.ml_off = p.direct ? 0 : parts * tokens * heads * dp;
    return p;
}

// The launches of a plan's parts, in order: workgroups first .. first + wgs - 1 in
// tiles of 'rows' rows by 'waves' waves.  Returns how many (some may be of no workgroup).
struct AttnLaunch {
    int rows, waves;
    int64_t first, wgs;
};

inline int attn_launches(const AttnPlan &p, AttnLaunch (&l)[2])
{
    if (p.together) {
        l[0] = {p.rows_own, p.waves_own, 0, int64_t(p.wgs_prefix) + p.wgs_own};
        return 1;
    }
    l[0] = {p.rows_prefix, p.waves_prefix, 0, p.wgs_prefix};
    l[1] = {p.rows_own, p.waves_own, p.wgs_prefix, p.wgs_own};
    return 2;
}

// Rows the join goes through: every query a sequence may have.
inline int64_t attn_join_rows(int64_t tokens, int64_t heads, int64_t seqs, int64_t max_q)
{
    return seqs * std::min(max_q, tokens) * heads;
}

// A launch holds fewer than 2^32 threads, workgroups here at most 512: larger ones go
// out in pieces of 2^22 workgroups, f(first, workgroups) each, until f gives something
// other than 'ok'.
constexpr int64_t kMaxWorkgroups = int64_t(1) << 22;

template <class R, class F>
R attn_pieces(int64_t wgs, R ok, const F &f)
{
    for (int64_t at = 0; at < wgs; at += kMaxWorkgroups) {
        const R r = f(at, std::min(wgs - at, kMaxWorkgroups));
        if (r != ok) return r;
    }
    return ok;
}

} // namespace bl
