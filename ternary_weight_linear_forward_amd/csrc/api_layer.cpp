// api_layer.cpp -- the C entry points around the BitLinears of a decoder layer
// (norm, int8 cache, attention; declared in include/bitlinear.h).  Validates
// every argument on the host, then enqueues the kernels; nothing is launched
// when validation fails.  No allocation, no synchronisation, no state.
#include "bitlinear.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "checks.h"
#include "launch.h"

namespace {

bool float_dtype(int dt) { return dt == BITLINEAR_F32 || dt == BITLINEAR_BF16; }
bool aligned_to(const void *p, int a) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a) == 0; }

// Byte span of rows [tokens x heads] of D elements with two strides.
Span rows_span(const void *p, int64_t tokens, int64_t heads, int64_t ld_t, int64_t ld_h, int64_t D, int es)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + static_cast<uintptr_t>(((tokens - 1) * ld_t + (heads - 1) * ld_h + D) * es)};
}

// Two-stride rows: strides in [0, 2^40] whose extents stay within 2^44
// elements; rows that are written may not overlap each other.
bool rows_ok(int64_t tokens, int64_t heads, int64_t ld_t, int64_t ld_h, int64_t D, bool written)
{
    if (ld_t < 0 || ld_h < 0 || ld_t > kMaxLd || ld_h > kMaxLd) return false;
    if ((ld_t && tokens - 1 > kMaxSpan / ld_t) || (ld_h && heads - 1 > kMaxSpan / ld_h)) return false;
    if (!written) return true;
    const bool inner_h = (heads == 1 || ld_h >= D) && (tokens == 1 || ld_t >= (heads - 1) * ld_h + D);
    const bool inner_t = (tokens == 1 || ld_t >= D) && (heads == 1 || ld_h >= (tokens - 1) * ld_t + D);
    return inner_h || inner_t;
}

// The spans of a cache's four arrays.
struct CacheSpans {
    Span s[4];
};

int check_cache(const bitlinear_cache_t *c, bl::CacheView *v, CacheSpans *sp)
{
    if (!c || !c->K || !c->V || !c->K_scale || !c->V_scale) return BITLINEAR_ERR_INVALID_ARG;
    const int64_t bytes = bitlinear_cache_bytes(c->pages, c->page_tokens, c->heads, c->head_dim);
    if (bytes < 0) return BITLINEAR_ERR_INVALID_ARG;
    if (!aligned16(c->K) || !aligned16(c->V) || !aligned16(c->K_scale) || !aligned16(c->V_scale))
        return BITLINEAR_ERR_INVALID_ARG;
    const int64_t n = c->pages * c->heads * c->page_tokens;
    sp->s[0] = span_of(c->K, 1, bytes, bytes, 1);
    sp->s[1] = span_of(c->V, 1, bytes, bytes, 1);
    sp->s[2] = span_of(c->K_scale, 1, n, n, 4);
    sp->s[3] = span_of(c->V_scale, 1, n, n, 4);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (overlap(sp->s[i], sp->s[j])) return BITLINEAR_ERR_INVALID_ARG;
    v->K = c->K;
    v->V = c->V;
    v->Ks = c->K_scale;
    v->Vs = c->V_scale;
    v->slots = c->pages * c->page_tokens;
    v->pages = static_cast<int>(c->pages);
    v->page_tokens = static_cast<int>(c->page_tokens);
    v->heads = static_cast<int>(c->heads);
    v->D = static_cast<int>(c->head_dim);
    v->Dp = static_cast<int>(round_up(c->head_dim, 16));
    return BITLINEAR_OK;
}

bool hits(const CacheSpans &c, Span s)
{
    for (const Span &x : c.s)
        if (overlap(x, s)) return true;
    return false;
}

constexpr int64_t kMaxCacheTokens = int64_t(1) << 24; // of one write or read
constexpr int64_t kMaxQueries = int64_t(1) << 20, kMaxKeys = int64_t(1) << 30, kMaxHeads = 4096,
                  kMaxRows = int64_t(1) << 28; // (query, head) rows of one call

bool attn_sizes_ok(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs, int64_t max_q,
                   int64_t max_own, int64_t prefix_len)
{
    return tokens >= 1 && tokens <= kMaxQueries && seqs >= 1 && seqs <= kMaxQueries && max_q >= 1 &&
           max_q <= kMaxQueries && kv_heads >= 1 && heads >= kv_heads && heads <= kMaxHeads && heads % kv_heads == 0 &&
           head_dim >= 1 && head_dim <= BITLINEAR_MAX_HEAD_DIM && max_own >= 0 && max_own <= kMaxKeys &&
           prefix_len >= 0 && prefix_len <= kMaxKeys && seqs * max_q <= kMaxRows / heads &&
           tokens <= kMaxRows / heads;
}

} // namespace

extern "C" {

int bitlinear_norm_quantize(const void *X, int x_dtype, int64_t M, int64_t K, int64_t ldx, const void *R, int64_t ldr,
                            const float *w, float eps, void *H, int h_dtype, int64_t ldh, void *Xq, int q_dtype,
                            int64_t ldq, int layout, float *beta, void *stream)
{
    if (!X || !Xq || !beta || !float_dtype(x_dtype)) return BITLINEAR_ERR_INVALID_ARG;
    if ((R || H) && !float_dtype(h_dtype)) return BITLINEAR_ERR_INVALID_ARG;
    if (q_dtype != BITLINEAR_I8 && q_dtype != BITLINEAR_I8_TILED) return BITLINEAR_ERR_INVALID_ARG;
    const bool tiled = q_dtype == BITLINEAR_I8_TILED;
    if (tiled && !valid_layout(layout)) return BITLINEAR_ERR_INVALID_ARG;
    if (M < 1 || M > BITLINEAR_MAX_M || K < 1 || K > BITLINEAR_MAX_K || ldx < K || !stride_ok(M, ldx) ||
        (R && (ldr < K || !stride_ok(M, ldr))) || (H && (ldh < K || !stride_ok(M, ldh))) ||
        (!tiled && (ldq < K || ldq % 16 || !stride_ok(M, ldq))))
        return BITLINEAR_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return BITLINEAR_ERR_INVALID_ARG;
    const int xs = dtype_size(x_dtype), hs = (R || H) ? dtype_size(h_dtype) : 4;
    if (!aligned16(Xq) || !aligned_to(X, xs) || !aligned_to(R, hs) || !aligned_to(H, hs) || !aligned_to(w, 4) ||
        !aligned_to(beta, 4))
        return BITLINEAR_ERR_INVALID_ARG;
    const int64_t tb = bl::tiled_bytes(M, K, tiled ? layout : 0);
    const Span sx = span_of(X, M, ldx, K, xs), sb = span_of(beta, 1, M, M, 4),
               sq = tiled ? span_of(Xq, 1, tb, tb, 1) : span_of(Xq, M, ldq, ldq, 1);
    if (overlap(sq, sx) || overlap(sb, sx) || overlap(sq, sb)) return BITLINEAR_ERR_INVALID_ARG;
    if (R) {
        const Span sr = span_of(R, M, ldr, K, hs);
        if (overlap(sq, sr) || overlap(sb, sr)) return BITLINEAR_ERR_INVALID_ARG;
    }
    if (w) {
        const Span sw = span_of(w, 1, K, K, 4);
        if (overlap(sq, sw) || overlap(sb, sw)) return BITLINEAR_ERR_INVALID_ARG;
    }
    if (H) {
        const Span sh = span_of(H, M, ldh, K, hs);
        if (overlap(sh, sq) || overlap(sh, sb) || (w && overlap(sh, span_of(w, 1, K, K, 4))))
            return BITLINEAR_ERR_INVALID_ARG;
        const bool is_r = R && H == R && ldh == ldr, is_x = H == X && ldh == ldx && h_dtype == x_dtype;
        if ((!is_x && overlap(sh, sx)) || (R && !is_r && overlap(sh, span_of(R, M, ldr, K, hs))))
            return BITLINEAR_ERR_INVALID_ARG;
    }
    if (tiled && K > kTiledMaxK) return BITLINEAR_ERR_UNSUPPORTED;
    bl::NormArgs a;
    a.X = X;
    a.x_dtype = x_dtype;
    a.M = M;
    a.K = K;
    a.ldx = ldx;
    a.R = R;
    a.ldr = ldr;
    a.w = w;
    a.eps = eps;
    a.H = H;
    a.h_dtype = (R || H) ? h_dtype : x_dtype;
    a.ldh = ldh;
    a.Xq = static_cast<int8_t *>(Xq);
    a.layout = tiled ? layout : -1;
    a.ldq = ldq;
    a.beta = beta;
    (void)hipGetLastError();
    return status_of(bl::launch_norm_quantize(a, as_stream(stream)));
}

int bitlinear_dequantize_act(const int8_t *Xq, int64_t ldq, const float *beta, int64_t M, int64_t K, void *V,
                             int v_dtype, int64_t ldv, void *stream)
{
    if (!Xq || !beta || !V || !float_dtype(v_dtype)) return BITLINEAR_ERR_INVALID_ARG;
    if (M < 1 || M > BITLINEAR_MAX_M || K < 1 || K > BITLINEAR_MAX_K || ldq < K || ldv < K || !stride_ok(M, ldq) ||
        !stride_ok(M, ldv))
        return BITLINEAR_ERR_INVALID_ARG;
    const int vs = dtype_size(v_dtype);
    if (!aligned_to(beta, 4) || !aligned_to(V, vs)) return BITLINEAR_ERR_INVALID_ARG;
    const Span sv = span_of(V, M, ldv, K, vs);
    if (overlap(sv, span_of(Xq, M, ldq, K, 1)) || overlap(sv, span_of(beta, 1, M, M, 4)))
        return BITLINEAR_ERR_INVALID_ARG;
    (void)hipGetLastError();
    return status_of(bl::launch_dequantize_act(Xq, ldq, beta, M, K, V, v_dtype, ldv, as_stream(stream)));
}

int64_t bitlinear_norm_backward_workspace_bytes(int64_t M, int64_t K, int dw)
{
    if (M < 1 || M > BITLINEAR_MAX_M || K < 1 || K > BITLINEAR_MAX_K) return -1;
    return dw ? bl::norm_bwd_parts(M, K) * K * 4 : 0;
}

int bitlinear_norm_backward(const float *dY, int64_t lddy, const void *H, int h_dtype, int64_t ldh, const float *w,
                            float eps, const void *dH, int64_t lddh, int64_t M, int64_t K, void *dX, int64_t lddx,
                            float *dW, void *ws, int64_t ws_bytes, void *stream)
{
    if (!dY || !H || !dX || !float_dtype(h_dtype)) return BITLINEAR_ERR_INVALID_ARG;
    if (M < 1 || M > BITLINEAR_MAX_M || K < 1 || K > BITLINEAR_MAX_K || lddy < K || ldh < K || lddx < K ||
        (dH && lddh < K) || !stride_ok(M, lddy) || !stride_ok(M, ldh) || !stride_ok(M, lddx) ||
        (dH && !stride_ok(M, lddh)))
        return BITLINEAR_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return BITLINEAR_ERR_INVALID_ARG;
    const int hs = dtype_size(h_dtype);
    if (!aligned_to(dY, 4) || !aligned_to(H, hs) || !aligned_to(w, 4) || !aligned_to(dH, hs) || !aligned_to(dX, hs) ||
        !aligned_to(dW, 4))
        return BITLINEAR_ERR_INVALID_ARG;
    const int64_t need = bitlinear_norm_backward_workspace_bytes(M, K, dW != nullptr);
    if (need > 0 && (!ws || ws_bytes < need)) return BITLINEAR_ERR_WORKSPACE;
    if (need > 0 && !aligned16(ws)) return BITLINEAR_ERR_INVALID_ARG;
    // inputs, then outputs: an output may overlap nothing, but dX may be dH
    const Span in[] = {span_of(dY, M, lddy, K, 4), span_of(H, M, ldh, K, hs), w ? span_of(w, 1, K, K, 4) : Span{0, 0}};
    const Span sdx = span_of(dX, M, lddx, K, hs), sdw = dW ? span_of(dW, 1, K, K, 4) : Span{0, 0},
               sws = need > 0 ? span_of(ws, 1, need, need, 1) : Span{0, 0},
               sdh = dH ? span_of(dH, M, lddh, K, hs) : Span{0, 0};
    for (const Span &s : in)
        if (overlap(sdx, s) || overlap(sdw, s) || overlap(sws, s)) return BITLINEAR_ERR_INVALID_ARG;
    if (overlap(sdx, sdw) || overlap(sdx, sws) || overlap(sdw, sws) || overlap(sdh, sdw) || overlap(sdh, sws))
        return BITLINEAR_ERR_INVALID_ARG;
    if (dH && overlap(sdx, sdh) && !(dX == dH && lddx == lddh)) return BITLINEAR_ERR_INVALID_ARG;
    bl::NormBwdArgs a;
    a.dY = dY;
    a.H = H;
    a.h_dtype = h_dtype;
    a.w = w;
    a.eps = eps;
    a.dH = dH;
    a.dX = dX;
    a.M = M;
    a.K = K;
    a.lddy = lddy;
    a.ldh = ldh;
    a.lddh = lddh;
    a.lddx = lddx;
    a.dW = dW;
    a.part = static_cast<float *>(ws);
    (void)hipGetLastError();
    return status_of(bl::launch_norm_backward(a, as_stream(stream)));
}

int64_t bitlinear_cache_bytes(int64_t pages, int64_t page_tokens, int64_t heads, int64_t head_dim)
{
    if (pages < 1 || heads < 1 || heads > kMaxHeads || page_tokens < 64 || page_tokens % 64 ||
        page_tokens > (int64_t(1) << 20) || head_dim < 1 || head_dim > BITLINEAR_MAX_HEAD_DIM || pages > INT32_MAX ||
        pages > (int64_t(1) << 36) / page_tokens)
        return -1;
    if (pages * heads * (page_tokens / 64) > INT32_MAX) return -1; // (kernels number the blocks in 32 bits)
    return pages * heads * page_tokens * round_up(head_dim, 16);
}

int bitlinear_cache_write(const bitlinear_cache_t *cache, const void *K, int64_t ldk_token, int64_t ldk_head,
                          const void *V, int64_t ldv_token, int64_t ldv_head, int dtype, int64_t tokens,
                          const int64_t *slots, void *stream)
{
    bl::CacheView c;
    CacheSpans cs;
    const int st = check_cache(cache, &c, &cs);
    if (st != BITLINEAR_OK) return st;
    if (!float_dtype(dtype) || tokens < 0 || tokens > kMaxCacheTokens) return BITLINEAR_ERR_INVALID_ARG;
    if (tokens == 0) return BITLINEAR_OK;
    const int es = dtype_size(dtype);
    if (!K || !V || !slots || !aligned_to(K, es) || !aligned_to(V, es) || !aligned_to(slots, 8) ||
        !rows_ok(tokens, c.heads, ldk_token, ldk_head, c.D, false) ||
        !rows_ok(tokens, c.heads, ldv_token, ldv_head, c.D, false))
        return BITLINEAR_ERR_INVALID_ARG;
    if (hits(cs, rows_span(K, tokens, c.heads, ldk_token, ldk_head, c.D, es)) ||
        hits(cs, rows_span(V, tokens, c.heads, ldv_token, ldv_head, c.D, es)) ||
        hits(cs, span_of(slots, 1, tokens, tokens, 8)))
        return BITLINEAR_ERR_INVALID_ARG;
    const bl::CacheRows r = {const_cast<void *>(K), const_cast<void *>(V), ldk_token, ldk_head, ldv_token, ldv_head};
    (void)hipGetLastError();
    return status_of(bl::launch_cache_write(c, r, dtype, tokens, slots, as_stream(stream)));
}

int bitlinear_cache_read(const bitlinear_cache_t *cache, const int64_t *slots, int64_t tokens, void *K,
                         int64_t ldk_token, int64_t ldk_head, void *V, int64_t ldv_token, int64_t ldv_head, int dtype,
                         void *stream)
{
    bl::CacheView c;
    CacheSpans cs;
    const int st = check_cache(cache, &c, &cs);
    if (st != BITLINEAR_OK) return st;
    if (!float_dtype(dtype) || tokens < 0 || tokens > kMaxCacheTokens) return BITLINEAR_ERR_INVALID_ARG;
    if (tokens == 0) return BITLINEAR_OK;
    const int es = dtype_size(dtype);
    if (!K || !V || !slots || !aligned_to(K, es) || !aligned_to(V, es) || !aligned_to(slots, 8) ||
        !rows_ok(tokens, c.heads, ldk_token, ldk_head, c.D, true) ||
        !rows_ok(tokens, c.heads, ldv_token, ldv_head, c.D, true))
        return BITLINEAR_ERR_INVALID_ARG;
    const Span sk = rows_span(K, tokens, c.heads, ldk_token, ldk_head, c.D, es),
               sv = rows_span(V, tokens, c.heads, ldv_token, ldv_head, c.D, es),
               ss = span_of(slots, 1, tokens, tokens, 8);
    if (hits(cs, sk) || hits(cs, sv) || overlap(sk, sv) || overlap(sk, ss) || overlap(sv, ss))
        return BITLINEAR_ERR_INVALID_ARG;
    const bl::CacheRows r = {K, V, ldk_token, ldk_head, ldv_token, ldv_head};
    (void)hipGetLastError();
    return status_of(bl::launch_cache_read(c, r, dtype, tokens, slots, as_stream(stream)));
}

int64_t bitlinear_attention_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                            int64_t seqs, int64_t max_q, int64_t max_own, int64_t prefix_len)
{
    if (!attn_sizes_ok(tokens, heads, kv_heads, head_dim, seqs, max_q, max_own, prefix_len)) return -1;
    return bl::attn_workspace_bytes(tokens, heads, kv_heads, head_dim, seqs, max_q, max_own, prefix_len);
}

int bitlinear_attention(const bitlinear_cache_t *cache, const void *Q, int dtype, int64_t tokens, int64_t heads,
                        int64_t ldq_token, int64_t ldq_head, int64_t seqs, const int32_t *q_start, int64_t max_q,
                        const int32_t *own_pages, int64_t ld_pages, const int32_t *own_len, int64_t max_own,
                        const int32_t *prefix_pages, int64_t prefix_len, float scale, void *O, int64_t ldo_token,
                        int64_t ldo_head, float *lse, void *ws, int64_t ws_bytes, void *stream)
{
    bl::AttnArgs a;
    CacheSpans cs;
    const int st = check_cache(cache, &a.c, &cs);
    if (st != BITLINEAR_OK) return st;
    if (!Q || !O || !own_len || !float_dtype(dtype) || !isfinite(scale) ||
        !attn_sizes_ok(tokens, heads, a.c.heads, a.c.D, seqs, max_q, max_own, prefix_len))
        return BITLINEAR_ERR_INVALID_ARG;
    if (!q_start && tokens != seqs * max_q) return BITLINEAR_ERR_INVALID_ARG;
    const int64_t np = (prefix_len + a.c.page_tokens - 1) / a.c.page_tokens,
                  no = (max_own + a.c.page_tokens - 1) / a.c.page_tokens;
    if ((np > 0 && !prefix_pages) || (no > 0 && !own_pages) || ld_pages < no || !stride_ok(seqs, ld_pages + 1))
        return BITLINEAR_ERR_INVALID_ARG;
    const int es = dtype_size(dtype);
    if (!aligned_to(Q, es) || !aligned_to(O, es) || !aligned_to(q_start, 4) || !aligned_to(own_pages, 4) ||
        !aligned_to(own_len, 4) || !aligned_to(prefix_pages, 4) || !aligned_to(lse, 4) ||
        !rows_ok(tokens, heads, ldq_token, ldq_head, a.c.D, false) ||
        !rows_ok(tokens, heads, ldo_token, ldo_head, a.c.D, true))
        return BITLINEAR_ERR_INVALID_ARG;
    const int64_t need =
        bl::attn_workspace_bytes(tokens, heads, a.c.heads, a.c.D, seqs, max_q, max_own, prefix_len);
    if (need > 0 && (!ws || ws_bytes < need)) return BITLINEAR_ERR_WORKSPACE;
    if (need > 0 && !aligned16(ws)) return BITLINEAR_ERR_INVALID_ARG;
    const Span so = rows_span(O, tokens, heads, ldo_token, ldo_head, a.c.D, es),
               sl = lse ? span_of(lse, 1, tokens * heads, tokens * heads, 4) : Span{0, 0},
               sw = need > 0 ? span_of(ws, 1, need, need, 1) : Span{0, 0};
    const Span in[] = {rows_span(Q, tokens, heads, ldq_token, ldq_head, a.c.D, es),
                       q_start ? span_of(q_start, 1, seqs + 1, seqs + 1, 4) : Span{0, 0},
                       no > 0 ? span_of(own_pages, seqs, ld_pages, no, 4) : Span{0, 0},
                       span_of(own_len, 1, seqs, seqs, 4),
                       np > 0 ? span_of(prefix_pages, 1, np, np, 4) : Span{0, 0},
                       cs.s[0], cs.s[1], cs.s[2], cs.s[3]};
    for (const Span &s : in)
        if (overlap(so, s) || overlap(sl, s) || overlap(sw, s)) return BITLINEAR_ERR_INVALID_ARG;
    if (overlap(so, sl) || overlap(so, sw) || overlap(sl, sw)) return BITLINEAR_ERR_INVALID_ARG;
    a.Q = Q;
    a.O = O;
    a.lse = lse;
    a.q_start = q_start;
    a.own_pages = own_pages;
    a.own_len = own_len;
    a.prefix_pages = prefix_pages;
    a.ldq_t = ldq_token;
    a.ldq_h = ldq_head;
    a.ldo_t = ldo_token;
    a.ldo_h = ldo_head;
    a.ld_pages = ld_pages;
    a.dtype = dtype;
    a.tokens = static_cast<int>(tokens);
    a.heads = static_cast<int>(heads);
    a.seqs = static_cast<int>(seqs);
    a.max_q = static_cast<int>(max_q);
    a.max_own = static_cast<int>(max_own);
    a.prefix = static_cast<int>(prefix_len);
    a.scale = scale;
    a.ws = static_cast<float *>(ws);
    (void)hipGetLastError();
    return status_of(bl::launch_attention(a, as_stream(stream)));
}

} // extern "C"
