// A step's tables from the requests' lengths (gdn_build_step_tables), gfx950.
//
// Everything follows from three running sums over the requests: tokens, pages
// taken, descriptors.  Each output element is then independent: it finds its
// request by a binary search in the running sums.
//
// The work is a few kilobytes of integers, bound by latency: launch, one load
// of the lengths, the sums, one dependent load (a page), one store.  So one
// launch does it all: every workgroup forms the sums of all requests for
// itself (at most GDN_STEP_MAX_SEQS, 32 KB from the L2) and keeps them in the
// LDS, which costs less than a second launch or a grid-wide wait; then the
// workgroups share out the output elements, each kind of them from another
// wave on, so that the few of a small step do not wait for each other.
//
// Measured: 4.4 us for 32 decode requests, as long as any kernel that writes a
// line (12 us with 64-bit sums, the four kinds one after the other and the
// lengths read again for each element); 11.0 us for 4,096 requests of 16,288
// tokens (19 us).
#include "serving_internal.h"

namespace gdn {

// Requests of a thread (eight, with half the threads: 13.7 us for 4,096 requests
// against 12.3), and threads of a workgroup for up to 1,024 requests and for more
// (32 requests: 4.7 us with 256, 6.1 with 1,024).
constexpr int kTablesPer = 4;
constexpr int kTablesSmall = 256, kTablesLarge = 1024;
static_assert(kTablesLarge * kTablesPer >= GDN_STEP_MAX_SEQS, "");
constexpr unsigned kMost = 0x7fffffffu;

// Sums stay at 2^31 - 1 once they reach it (in any order: no term is negative).
__device__ __forceinline__ unsigned add(unsigned a, unsigned b) { return min(a + b, kMost); }
__device__ __forceinline__ int saturated(long long v) { return (int)min(v, (long long)kMost); }

struct Sums {
    unsigned tokens, pages, chunks;
};
__device__ __forceinline__ Sums add(const Sums &a, const Sums &b) {
    return {add(a.tokens, b.tokens), add(a.pages, b.pages), add(a.chunks, b.chunks)};
}

// the index of the last entry <= x of the non-decreasing sums at[0 .. n], at[0] == 0
__device__ __forceinline__ int owner(const int *at, int n, int x) {
    int lo = 0, hi = n;          // at[lo] <= x, and at[hi] > x wherever x < at[n]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void step_tables_kernel(StepTablesArgs a) {
    constexpr int MAX = THREADS * kTablesPer, WAVES = THREADS / 64;
    __shared__ int tok[MAX + 1], pag[MAX + 1], chk[MAX + 1], before[MAX];   // exclusive sums; tokens before the step
    __shared__ Sums wave_sum[WAVES];
    __shared__ unsigned long long more;           // pages past the rows' ends; all, where their sum is at its end
    const int S = a.num_seqs, page = 1 << a.page_shift;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto pages_of = [&](long long tokens) { return (tokens + page - 1) >> a.page_shift; };
    auto in_row = [&](long long pages) { return (int)min(pages, (long long)a.max_pages); };

    const int n_free = min(max(a.num_free[0], 0), a.free_capacity);
    int ctx[kTablesPer] = {}, len[kTablesPer] = {};
    if (S > 0) {                 // all loads at once: none behind a branch of its own
#pragma unroll
        for (int i = 0; i < kTablesPer; ++i) {
            const int s = min(tid * kTablesPer + i, S - 1);
            ctx[i] = a.context_lens[s];
            len[i] = a.query_lens[s];
        }
#pragma unroll
        for (int i = 0; i < kTablesPer; ++i) {
            const bool in = tid * kTablesPer + i < S;
            ctx[i] = in ? max(ctx[i], 0) : 0;
            len[i] = in ? max(len[i], 0) : 0;
        }
    }
    if (tid == 0) more = 0;
    Sums own[kTablesPer], mine = {0, 0, 0};
    unsigned long long want = 0, past = 0;
#pragma unroll
    for (int i = 0; i < kTablesPer; ++i) {
        const long long seq = (long long)ctx[i] + len[i], h = pages_of(ctx[i]), w = pages_of(seq);
        own[i] = {(unsigned)len[i], (unsigned)(in_row(w) - in_row(h)),
                  (unsigned)(((long long)len[i] + GDN_CONV_CHUNK_TOKENS - 1) / GDN_CONV_CHUNK_TOKENS)};
        want += (unsigned long long)(w - h);
        past += (unsigned long long)(w - h) - own[i].pages;
        mine = add(mine, own[i]);
        const int s = tid * kTablesPer + i;
        if (s < S) {
            before[s] = ctx[i];
            if (blockIdx.x == 0) a.seq_lens[s] = saturated(seq);
        }
    }
    // running sums: each thread's requests, then threads, then waves
    Sums inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const Sums up = {__shfl_up(inc.tokens, d, 64), __shfl_up(inc.pages, d, 64), __shfl_up(inc.chunks, d, 64)};
        if (lane >= d) inc = add(inc, up);
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    // what lies before this thread's requests.  (Not inc - mine: a sum that has
    // reached its end cannot be taken back.)
    Sums base = {__shfl_up(inc.tokens, 1, 64), __shfl_up(inc.pages, 1, 64), __shfl_up(inc.chunks, 1, 64)}, total = {0, 0, 0};
    if (lane == 0) base = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const Sums x = wave_sum[w];
        if (w < wave) base = add(base, x);
        total = add(total, x);
    }
    const bool end = total.pages == kMost;
    if (blockIdx.x == 0 && (end ? want : past)) atomicAdd(&more, end ? want : past);      // hardly ever
#pragma unroll
    for (int i = 0; i < kTablesPer; ++i) {
        const int s = tid * kTablesPer + i;
        if (s <= S) {
            tok[s] = (int)base.tokens;
            pag[s] = (int)base.pages;
            chk[s] = (int)base.chunks;
            if (blockIdx.x == 0) a.query_start_loc[s] = (int)base.tokens;
        }
        base = add(base, own[i]);
    }
    if (S == MAX && tid == THREADS - 1) {
        tok[S] = (int)total.tokens;
        pag[S] = (int)total.pages;
        chk[S] = (int)total.chunks;
        if (blockIdx.x == 0) a.query_start_loc[S] = (int)total.tokens;
    }
    __syncthreads();

    const int n_tok = (int)total.tokens, n_pag = (int)total.pages, n_chk = (int)total.chunks;
    // the p-th page taken in this step, or -1 when the free list has run out
    auto taken = [&](int p) { return p < n_free ? a.free_pages[n_free - 1 - p] : -1; };
    const int threads = gridDim.x * THREADS, me = blockIdx.x * THREADS + tid;
    // the first element of the k-th kind for this thread
    auto first = [&](int k) { return (long long)(me >= 64 * k ? me - 64 * k : me + threads - 64 * k); };

    for (long long i = first(0); i < a.num_tokens; i += threads) {
        const int t = (int)i;
        int pos = -1;
        long long slot = -1;
        if (t < n_tok) {
            const int s = owner(tok, S, t);
            const long long c = before[s], p = c + (t - tok[s]), pi = p >> a.page_shift;
            pos = saturated(p);
            if (pi < a.max_pages) {
                const int have = in_row(pages_of(c));
                const int id = pi >= have ? taken(pag[s] + (int)pi - have) : a.block_table[s * a.block_table_stride + pi];
                if (id >= 0) slot = ((long long)id << a.page_shift) + (p & (page - 1));
            }
        }
        a.positions[t] = pos;
        a.slot_mapping[t] = slot;
    }
    for (long long i = first(1); i < n_pag; i += threads) {
        const int p = (int)i, s = owner(pag, S, p);
        a.block_table[s * a.block_table_stride + in_row(pages_of(before[s])) + (p - pag[s])] = taken(p);
    }
    for (long long i = first(2); i < a.n_chunks; i += threads) {
        const int c = (int)i;
        gdn_conv_chunk d = {-1, 0};
        if (c < n_chk) {
            d.seq = owner(chk, S, c);
            d.chunk = c - chk[d.seq];
        }
        a.chunks[c] = d;
    }
    if (me == 64 * 3) {
        const int got = min(n_pag, n_free);
        a.counts[0] = n_tok;
        a.counts[1] = n_chk;
        a.counts[2] = got;
        a.counts[3] = saturated((long long)(more + (end ? 0 : total.pages)) - got);
    }
}

hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t stream) {
    const int threads = a.num_seqs <= kTablesSmall * kTablesPer ? kTablesSmall : kTablesLarge;
    // an output element per thread (two: 13.5 us for 4,096 requests, 12.3 so)
    const long long most = (long long)max(a.num_tokens, a.n_chunks);
    const int blocks = (int)max(min((most + threads - 1) / threads, 256LL), 1LL);
    if (threads == kTablesSmall)
        hipLaunchKernelGGL(step_tables_kernel<kTablesSmall>, dim3(blocks), dim3(threads), 0, stream, a);
    else
        hipLaunchKernelGGL(step_tables_kernel<kTablesLarge>, dim3(blocks), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
