// What the attentions over a paged cache share, whatever its format (gfx950):
// which rows and keys a workgroup has, how a call's keys are divided, where
// partial results lie, and helpers across lanes.
#pragma once

#include "attention_keys.h"
#include "attention_plan.h"
#include "gdn_device.h"
#include "serving_internal.h"

namespace gdn {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ Request request_of(const AttentionArgs &a, int s) {
    Request r;
    int end;
    clamp_range(a.qsl[s], a.qsl[s + 1], a.num_tokens, r.begin, end);
    r.n = end - r.begin;
    r.len = max(a.seq_lens[s], 0);
    r.L = (int)min((long long)r.len, (long long)a.max_pages * a.page);
    return r;
}

__device__ __forceinline__ void key_range(const AttentionArgs &a, const Request &r, int i, int &jb, int &je) {
    key_range(a.causal, a.window, r, i, jb, je);
}

// the token within its request of a row, and the last one of up to `rows` rows
// from `row` on, of n
__device__ __forceinline__ int token_of(int row, int G) { return (int)((unsigned)row / (unsigned)G); }
__device__ __forceinline__ int last_row(int row, int rows, int n) { return (int)min((unsigned)row + rows, (unsigned)n) - 1; }

// Row tiles without a list: request s owns the tile numbers from
// floor(query_start_loc[s] * G / rows) + s * each on, G rows per token.  With
// each = 1 that is as many as it needs or more, with each = 0 as many as it
// needs behind its first one.  `up` rounds the first number up: then, with each =
// 0, a request of more than `rows` rows owns at least one number per `rows` of
// them, and the others one at most.  Returns the last request whose first number is at
// or before `tile` (64 candidates per step), and the tile's place in it.
__device__ __forceinline__ int find_request(const AttentionArgs &a, long long tile, int group, int rows, int each, bool up,
                                            int &within) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.num_seqs;
    const int add = up ? rows - 1 : 0;
    auto first = [&](int s) { return (long long)(((unsigned long long)max(a.qsl[s], 0) * group + add) / rows) + s * each; };
    while (n > 1) {
        const int step = (n + 63) / 64;
        const bool in = lane * step < n && first(lo + lane * step) <= tile;
        const unsigned long long b = __ballot(in);
        const int k = b ? 63 - __builtin_clzll(b) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    within = (int)(tile - first(lo));
    return lo;
}

// the request of token t, or the last one that begins before it, 64 candidates per step
__device__ __forceinline__ int find_token(const AttentionArgs &a, int t) {
    const int lane = threadIdx.x & 63;
    int s = 0, n = a.num_seqs;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const unsigned long long b = __ballot(lane * step < n && a.qsl[s + lane * step] <= t);
        const int k = b ? 63 - __builtin_clzll(b) : 0;
        s += k * step;
        n = min(step, n - k * step);
    }
    return s;
}

// The larger of a lane's value and that of the lane 32 (16) further or back: the
// swap of half-waves (of neighbouring rows of 16) between two copies leaves both
// lanes' values in each.  (The compiler must not see that they are copies: it
// then takes the two results for equal.)
__device__ __forceinline__ float max_over32(float x) {
    uint32_t u = __builtin_bit_cast(uint32_t, x), v = u;
    asm("" : "+v"(v));
    const auto r = __builtin_amdgcn_permlane32_swap(u, v, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float max_over16(float x) {
    uint32_t u = __builtin_bit_cast(uint32_t, x), v = u;
    asm("" : "+v"(v));
    const auto r = __builtin_amdgcn_permlane16_swap(u, v, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// 8 bf16 from packed pairs
__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const i32x4 v = {(int)a, (int)b, (int)c, (int)d};
    return __builtin_bit_cast(bf16x8, v);
}

// In this many keys of a workgroup's part a row's sums follow every new maximum;
// behind them each format lets some pass.
constexpr int kLateKeys = 256;

// A launch's division of its requests' keys, and its partial results: a row's D
// sums per split, and behind all of them a maximum and a sum of weights per
// (row, split).  Rows are (token, q head), or for the small requests alone
// (request, row of kSmallRows, kv head).
struct Division {
    int chunk, splits;
    bool by_rows;       // many rows: a tile number per kSmallRows rows, else one per kManyRows and one per request
    float *sums, *stats;
};
__device__ __forceinline__ float *part_o(const Division &v, int d, long long row, int split) {
    return v.sums + (row * v.splits + split) * d;
}
__device__ __forceinline__ float *part_ml(const Division &v, long long row, int split) {
    return v.stats + (row * v.splits + split) * 2;
}
template <Take TAKE>
__device__ __forceinline__ long long part_row(const AttentionArgs &a, int s, int t, int h, long long row, int hk) {
    return TAKE == Take::kSmall ? ((long long)s * kSmallRows + row) * a.num_kv_heads + hk
                                : (long long)t * a.num_q_heads + h;
}

// A workgroup's share of a many-rows launch.
struct ManyShare {
    int s, hk, split;
    Request rq;
    int row0, n_rows;
    int k_lo, k_hi;        // its keys
    bool whole;            // no other split has any
};
// The last tiles see the most keys and go first; a kv head's workgroups are
// num_kv_heads apart, so that with eight heads an XCD keeps to one.
template <int ROWS = kManyRows>
__device__ __forceinline__ bool many_share(const AttentionArgs &a, const Division &v, int block, int blocks, ManyShare &w) {
    const int G = a.num_q_heads / a.num_kv_heads;
    const unsigned units = (unsigned)blocks / (unsigned)v.splits, unit = (unsigned)block / (unsigned)v.splits, hks = a.num_kv_heads;
    w.split = block - (int)(unit * v.splits);
    const int tile = (int)(units / hks - 1 - unit / hks);
    w.hk = (int)(unit % hks);
    int within;
    w.s = v.by_rows ? find_request(a, tile, G, kSmallRows, 0, true, within) : find_request(a, tile, G, ROWS, 1, false, within);
    w.rq = request_of(a, w.s);
    w.n_rows = w.rq.n * G;
    if (within < 0 || (long long)within * ROWS >= w.n_rows || w.n_rows <= kSmallRows) return false;
    w.row0 = within * ROWS;
    int lo, hi, x;
    key_range(a, w.rq, token_of(w.row0, G), lo, x);
    key_range(a, w.rq, token_of(last_row(w.row0, ROWS, w.n_rows), G), x, hi);
    const Splits sp = splits_of(lo, hi, v.chunk, v.splits);
    if (w.split != sp.first && (w.split < sp.first || w.split > sp.last)) return false;
    w.whole = sp.last <= sp.first;
    w.k_lo = max(lo, w.split * v.chunk);
    w.k_hi = w.split == v.splits - 1 ? hi : min(hi, (w.split + 1) * v.chunk);
    return true;
}

// The keys [lo, hi) of [k_lo, k_hi) that some of `rows` rows from `row` on see,
// and those [all0, all1) that each of them sees.
struct WaveKeys {
    int lo, hi, all0, all1;
};
__device__ __forceinline__ WaveKeys wave_keys(const AttentionArgs &a, const ManyShare &w, int row, int rows) {
    const int G = a.num_q_heads / a.num_kv_heads;
    WaveKeys k{0, 0, 0, 0};
    if (row < w.n_rows) {
        key_range(a, w.rq, token_of(row, G), k.lo, k.all1);
        key_range(a, w.rq, token_of(last_row(row, rows, w.n_rows), G), k.all0, k.hi);
        k.lo = max(k.lo, w.k_lo);
        k.hi = min(k.hi, w.k_hi);
        k.all0 = max(k.all0, w.k_lo);
        k.all1 = min(k.all1, w.k_hi);
    }
    return k;
}

// the partial results of a launch at `ws`
inline Division division(const Launch &p, bool by_rows, int d, float *ws) {
    return {p.chunk, p.splits, by_rows, ws, ws + p.rows * p.splits * d};
}

// joins the splits of a launch, where it has any
void launch_join(Take take, const AttentionArgs &a, const Launch &p, const Division &v, int tile_rows, hipStream_t stream);

}  // namespace gdn
