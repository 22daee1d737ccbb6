// assign.hip -- places of a step's new tokens in the paged cache: pages given back and
// taken, lengths, query starts, slots and positions (bitlinear_cache_assign).
//
// Everything follows from sums over the sequences in order: pages given back, pages
// asked for, new tokens.  One workgroup forms them, 1024 sequences at a time, and the
// work behind a sum (pages of a list, tokens of a batch) is shared evenly by its threads,
// each of which finds its sequence by halving.  A sequence gets its pages iff the pages
// asked for up to it are no more than there are, so those that are granted are the first
// of all that are asked for: page p of them is the p-th from the top of the stack.
// Bound: latency, a chain of loads, sums over the waves and searches in LDS: 16 sequences of a token 5.1 us, 300 that
// take and give 13000 tokens 10.4 and 4.1 us.  One workgroup: sums across several would cost a second launch, which is
// as long as this one takes.
#include "common.h"
#include "launch.h"

namespace bl {

namespace {

constexpr int ASSIGN_SEQS = 1024; // sequences a pass, and threads

// Inclusive sum over the workgroup's threads, in order; the whole in 'total'.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t *waves, int64_t &total)
{
    const int lane = lane_id(), wave = wave_id(), n = blockDim.x / 64;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const int64_t o = __shfl_up(v, s);
        v += lane >= s ? o : 0;
    }
    __syncthreads(); // (the last sums are read)
    if (lane == 63) waves[wave] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int w = 0; w < n; ++w) {
        before += w < wave ? waves[w] : 0;
        total += waves[w];
    }
    return v + before;
}

// The sequence of 0 .. n - 1 whose share holds item x: the first with upto > x.
template <class T>
__device__ __forceinline__ int owner(const T *upto, int n, T x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (upto[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ void put(const AssignArgs &a, int j, int page, int pos)
{
    const bool none = pos < 0;
    a.slots[j] = none ? -1 : static_cast<int64_t>(page) * a.page_tokens + pos % a.page_tokens;
    if (a.positions) a.positions[j] = none ? -1 : a.prefix + pos;
}

} // namespace

// fill: the tokens' slots too.
__global__ __launch_bounds__(ASSIGN_SEQS) void k_assign(const AssignArgs a, bool fill)
{
    __shared__ int64_t waves[16], upto[ASSIGN_SEQS], token_upto[ASSIGN_SEQS];
    __shared__ int had[ASSIGN_SEQS]; // own tokens before, -1: gets nothing
    __shared__ unsigned long long granted;
    const int tid = threadIdx.x, step = blockDim.x, page = a.page_tokens;
    auto pages = [&](int64_t n) { return (n + page - 1) / page; };
    // held tokens and count of sequence b0 + tid; those of the first pass, which the others seldom follow, are read once
    struct Seq {
        int h, c;
    };
    auto read = [&](int b) { return b < a.seqs ? Seq{min(max(a.held[b], 0), a.max_own), a.count[b]} : Seq{0, 0}; };
    const Seq seq0 = read(tid);
    if (tid == 0) granted = 0;

    // pages given back, on top of the list
    int64_t top = a.free_count ? min(max(*a.free_count, 0), a.max_free) : 0;
    for (int b0 = 0; b0 < a.seqs; b0 += step) {
        const int n = min(step, a.seqs - b0);
        const Seq q = b0 ? read(b0 + tid) : seq0;
        int64_t back = 0;
        int keep = 0;
        if (q.c < 0) {
            keep = static_cast<int>(pages(max<int64_t>(static_cast<int64_t>(q.h) + q.c, 0)));
            back = pages(q.h) - keep;
        }
        if (!__syncthreads_or(back > 0)) continue;
        int64_t total;
        upto[tid] = scan(back, waves, total);
        had[tid] = keep;
        __syncthreads();
        for (int64_t p = tid; p < total && top + p < a.max_free; p += step) {
            const int s = owner<int64_t>(upto, n, p);
            const int64_t col = had[s] + p - (s ? upto[s - 1] : 0);
            a.free_pages[top + p] = a.own_pages[(b0 + s) * a.ld_pages + col];
        }
        top = min<int64_t>(top + total, a.max_free);
        __syncthreads();
    }

    // pages and places taken
    int64_t asked = 0, tokens = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += step) {
        const int b = b0 + tid, n = min(step, a.seqs - b0);
        const Seq q = b0 ? read(b) : seq0;
        const int64_t h = q.h, c = q.c;
        int64_t need = 0, all_need, all_new;
        const int64_t fresh = max<int64_t>(c, 0), token_end = tokens + scan(fresh, waves, all_new);
        const bool fits = h + fresh <= a.max_own && token_end <= a.tokens;
        if (fits) need = pages(h + fresh) - pages(h);
        const int64_t end = asked + scan(need, waves, all_need);
        const bool ok = fits && (need == 0 || end <= top);
        upto[tid] = end;
        token_upto[tid] = token_end;
        had[tid] = ok ? static_cast<int>(h) : -1;
        if (b < a.seqs) {
            const int64_t len = c < 0 ? max<int64_t>(h + c, 0) : ok ? h + c : h;
            a.own_len[b] = static_cast<int>(len);
            a.first[b] = c > 0 ? (ok ? static_cast<int>(h) : -1) : static_cast<int>(len);
            a.q_start[b] = static_cast<int>(min<int64_t>(token_end - fresh, a.tokens));
            if (b == a.seqs - 1) a.q_start[a.seqs] = static_cast<int>(min<int64_t>(token_end, a.tokens));
            if (ok && need > 0) atomicMax(&granted, static_cast<unsigned long long>(end));
        }
        __syncthreads();
        for (int64_t p = asked + tid; p < asked + all_need && p < top; p += step) {
            const int s = owner<int64_t>(upto, n, p);
            if (had[s] < 0) continue;
            const int64_t col = pages(had[s]) + p - (s ? upto[s - 1] : asked);
            a.own_pages[(b0 + s) * a.ld_pages + col] = a.free_pages[top - 1 - p];
        }
        if (fill) {
            for (int64_t j = tokens + tid; j < tokens + all_new && j < a.tokens; j += step) {
                const int s = owner<int64_t>(token_upto, n, j);
                int pos = -1, where = 0;
                if (had[s] >= 0) {
                    pos = had[s] + static_cast<int>(j - (s ? token_upto[s - 1] : tokens));
                    const int64_t col = pos / page, old = pages(had[s]); // (a new page is read where it comes from)
                    where = col < old ? a.own_pages[(b0 + s) * a.ld_pages + col]
                                      : a.free_pages[top - 1 - ((s ? upto[s - 1] : asked) + col - old)];
                }
                put(a, static_cast<int>(j), where, pos);
            }
        }
        asked += all_need;
        tokens += all_new;
        __syncthreads();
    }
    if (fill)
        for (int64_t j = tokens + tid; j < a.tokens; j += step) put(a, static_cast<int>(j), 0, -1);
    if (tid == 0) *a.free_left = static_cast<int>(top - static_cast<int64_t>(granted));
}

// Slots of many tokens, from the starts and tables that k_assign wrote.
__global__ __launch_bounds__(256) void k_assign_slots(const AssignArgs a)
{
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= a.tokens) return;
    int pos = -1, where = 0;
    if (j < a.q_start[a.seqs]) {
        const int s = owner<int32_t>(a.q_start + 1, a.seqs, j), first = a.first[s];
        if (first >= 0) {
            pos = first + (j - a.q_start[s]);
            where = a.own_pages[s * a.ld_pages + pos / a.page_tokens];
        }
    }
    put(a, j, where, pos);
}

hipError_t launch_cache_assign(const AssignArgs &a, hipStream_t stream)
{
    // One workgroup fills the slots of a few tokens itself, a second kernel those of many: 300 sequences of 1200 tokens 9.2
    // us, with a second kernel 11.2; 16 of 1024 7.9 and 8.1; 16 of 4096 10.8 and 8.3.
    constexpr int kFillTokens = 2048;
    const bool fill = a.tokens <= kFillTokens;
    const int threads = a.seqs <= 256 && (!fill || a.tokens <= 1024) ? 256 : ASSIGN_SEQS;
    hipLaunchKernelGGL(k_assign, dim3(1), dim3(threads), 0, stream, a, fill);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || fill) return e;
    hipLaunchKernelGGL(k_assign_slots, dim3((a.tokens + 255) / 256), dim3(256), 0, stream, a);
    return hipGetLastError();
}

} // namespace bl
