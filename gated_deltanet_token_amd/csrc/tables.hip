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
// workgroups share out the output elements.
#include "serving_internal.h"

namespace gdn {

constexpr int kTablesThreads = 1024;
constexpr int kTablesWaves = kTablesThreads / 64;
// output elements per thread that make another workgroup worth its start
constexpr int kTablesPerBlock = 2 * kTablesThreads;

struct Sums {
    long long tokens, pages, chunks, missing;
};

__device__ __forceinline__ long long shfl_up_ll(long long v, int d) {
    return __shfl_up(v, d, 64);
}

__device__ __forceinline__ int saturated(long long v) { return (int)(v < 0x7fffffffLL ? v : 0x7fffffffLL); }

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

__global__ __launch_bounds__(kTablesThreads) void step_tables_kernel(StepTablesArgs a) {
    extern __shared__ int lds[];
    const int S = a.num_seqs;
    int *tok = lds, *pag = lds + (S + 1), *chk = lds + 2 * (S + 1);   // exclusive sums, [S + 1] each
    __shared__ Sums wave_sum[kTablesWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

    // what request s adds to each sum (nothing past the last one)
    auto of_request = [&](int s, long long &ctx, long long &seq, int &have, int &want) {
        Sums d = {0, 0, 0, 0};
        ctx = seq = have = want = 0;
        if (s < S) {
            ctx = max(a.context_lens[s], 0);
            const long long n = max(a.query_lens[s], 0);
            seq = ctx + n;
            const int page = 1 << a.page_shift;
            const long long have_all = (ctx + page - 1) >> a.page_shift;
            const long long want_all = (seq + page - 1) >> a.page_shift;
            have = (int)min(have_all, (long long)a.max_pages);
            want = (int)min(want_all, (long long)a.max_pages);
            d.tokens = n;
            d.pages = want - have;
            d.chunks = (n + GDN_CONV_CHUNK_TOKENS - 1) / GDN_CONV_CHUNK_TOKENS;
            d.missing = (want_all - have_all) - (want - have);
        }
        return d;
    };

    // running sums: each thread a run of consecutive requests, then threads, then waves
    const int per = (S + kTablesThreads - 1) / kTablesThreads;
    long long ctx, seq;
    int have, want;
    Sums mine = {0, 0, 0, 0};
    for (int i = 0; i < per; ++i) {
        const Sums d = of_request(tid * per + i, ctx, seq, have, want);
        mine.tokens += d.tokens;
        mine.pages += d.pages;
        mine.chunks += d.chunks;
        mine.missing += d.missing;
    }
    Sums inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const Sums up = {shfl_up_ll(inc.tokens, d), shfl_up_ll(inc.pages, d), shfl_up_ll(inc.chunks, d),
                         shfl_up_ll(inc.missing, d)};
        if (lane >= d) {
            inc.tokens += up.tokens;
            inc.pages += up.pages;
            inc.chunks += up.chunks;
            inc.missing += up.missing;
        }
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    Sums base = {0, 0, 0, 0}, total = {0, 0, 0, 0};
    for (int w = 0; w < kTablesWaves; ++w) {
        const Sums x = wave_sum[w];
        if (w < wave) {
            base.tokens += x.tokens;
            base.pages += x.pages;
            base.chunks += x.chunks;
        }
        total.tokens += x.tokens;
        total.pages += x.pages;
        total.chunks += x.chunks;
        total.missing += x.missing;
    }
    base.tokens += inc.tokens - mine.tokens;
    base.pages += inc.pages - mine.pages;
    base.chunks += inc.chunks - mine.chunks;
    for (int i = 0; i < per; ++i) {
        const int s = tid * per + i;
        if (s >= S) break;
        tok[s] = saturated(base.tokens);
        pag[s] = saturated(base.pages);
        chk[s] = saturated(base.chunks);
        const Sums d = of_request(s, ctx, seq, have, want);
        base.tokens += d.tokens;
        base.pages += d.pages;
        base.chunks += d.chunks;
    }
    if (tid == 0) {
        tok[S] = saturated(total.tokens);
        pag[S] = saturated(total.pages);
        chk[S] = saturated(total.chunks);
    }
    __syncthreads();

    const int n_tok = tok[S], n_pag = pag[S], n_chk = chk[S];
    const int n_free = min(max(a.num_free[0], 0), a.free_capacity);
    // the p-th page taken in this step, or -1 when the free list has run out
    auto taken = [&](int p) { return p < n_free ? a.free_pages[n_free - 1 - p] : -1; };
    const long long first = (long long)blockIdx.x * kTablesThreads + tid, step = (long long)gridDim.x * kTablesThreads;

    for (long long i = first; i < a.num_tokens; i += step) {
        const int t = (int)i;
        int pos = -1;
        long long slot = -1;
        if (t < n_tok) {
            const int s = owner(tok, S, t);
            of_request(s, ctx, seq, have, want);
            const long long p = ctx + (t - tok[s]);
            const long long pi = p >> a.page_shift;
            pos = saturated(p);
            if (pi < a.max_pages) {
                const int id = pi >= have ? taken(pag[s] + (int)pi - have) : a.block_table[s * a.block_table_stride + pi];
                if (id >= 0) slot = ((long long)id << a.page_shift) + (p & ((1 << a.page_shift) - 1));
            }
        }
        a.positions[t] = pos;
        a.slot_mapping[t] = slot;
    }
    for (long long i = first; i < n_pag; i += step) {
        const int p = (int)i, s = owner(pag, S, p);
        of_request(s, ctx, seq, have, want);
        a.block_table[s * a.block_table_stride + have + (p - pag[s])] = taken(p);
    }
    for (long long i = first; i < a.n_chunks; i += step) {
        const int c = (int)i;
        gdn_conv_chunk d = {-1, 0};
        if (c < n_chk) {
            d.seq = owner(chk, S, c);
            d.chunk = c - chk[d.seq];
        }
        a.chunks[c] = d;
    }
    for (long long i = first; i <= S; i += step) {
        a.query_start_loc[i] = tok[i];
        if (i < S) {
            of_request((int)i, ctx, seq, have, want);
            a.seq_lens[i] = saturated(seq);
        }
    }
    if (first == 0) {
        const int got = min(n_pag, n_free);
        a.counts[0] = n_tok;
        a.counts[1] = n_chk;
        a.counts[2] = got;
        a.counts[3] = saturated(total.missing + (total.pages - got));
    }
}

hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t stream) {
    const long long most = (long long)max(max(a.num_tokens, a.n_chunks), a.num_seqs + 1);
    const int blocks = (int)min((most + kTablesPerBlock - 1) / kTablesPerBlock, 256LL);
    const size_t lds = (size_t)3 * (a.num_seqs + 1) * sizeof(int);
    hipLaunchKernelGGL(step_tables_kernel, dim3(blocks), dim3(kTablesThreads), lds, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
