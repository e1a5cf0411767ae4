// How an attention call's keys are divided, and the parts joined (gfx950).
#include "attention_split.h"

namespace gdn {

// ---------------------------------------------------------------------------
// The splits of a row joined: one wave per row of the launch that made them,
// its splits' sums brought to the common maximum.
// ---------------------------------------------------------------------------
template <int D, Take TAKE>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, Division v, int rows, int tile_rows) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    const unsigned part = blockIdx.x * 4u + (threadIdx.x >> 6);
    if (part >= (unsigned)rows) return;
    const int G = a.num_q_heads / a.num_kv_heads;
    int s, t, h;
    int r;                                  // the row within its request and kv head
    if constexpr (TAKE == Take::kSmall) {
        const unsigned of = part / (unsigned)a.num_kv_heads;
        r = (int)(of % kSmallRows);
        s = (int)(of / kSmallRows);
        h = (int)(part - of * a.num_kv_heads) * G + r % G;
        t = 0;
    } else {
        t = (int)(part / (unsigned)a.num_q_heads);
        h = (int)(part - (unsigned)t * a.num_q_heads);
        s = find_token(a, t);
    }
    const Request rq = request_of(a, s);
    const int n_rows = rq.n * G;
    if constexpr (TAKE == Take::kSmall) {
        if (n_rows > kSmallRows || r >= n_rows) return;
        t = rq.begin + token_of(r, G);
    } else {
        if (t < rq.begin || t >= rq.begin + rq.n || (TAKE == Take::kLarge && n_rows <= kSmallRows)) return;
        r = (t - rq.begin) * G + h % G;
    }
    // the keys of the row's tile decide which splits wrote
    const int r0 = r - r % tile_rows;
    int k_lo, k_hi, x;
    key_range(a, rq, token_of(r0, G), k_lo, x);
    key_range(a, rq, token_of(last_row(r0, tile_rows, n_rows), G), x, k_hi);
    const Splits sp = splits_of(k_lo, k_hi, v.chunk, v.splits);
    if (sp.last <= sp.first) return;
    float m = kNegInf, l = 0.f, o[E] = {};
    for (int i = sp.first; i <= sp.last; ++i) m = fmaxf(m, part_ml(v, part, i)[0]);
    const float at = m == kNegInf ? 0.f : m;
    for (int i = sp.first; i <= sp.last; ++i) {
        const float *ml = part_ml(v, part, i), *p = part_o(v, D, part, i);
        const float f = __builtin_amdgcn_exp2f(ml[0] - at);
        l = __builtin_fmaf(ml[1], f, l);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = __builtin_fmaf(p[lane * E + e], f, o[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *op = a.o + (long long)t * a.o_stride + (long long)h * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) op[e] = f32_to_bf16(o[e] * inv);
}

// ---------------------------------------------------------------------------
// With at most a token per request on average the few-rows kernel takes
// everything; else it takes the requests of up to kSmallRows rows, and the
// many-rows kernel the others (16 rows of a wave cost it as much as 32, and it
// reads a key once for 128 rows).  Keys are split until there is a workgroup for
// every CU, or as many of the many-rows kernel's as fit at once, but into parts of
// the rules' least keys or more.
// ---------------------------------------------------------------------------
static Launch divide(long long tiles, long long busy, long long rows, int kv_heads, int d, int max_seq_len, int aim,
                     long long min_chunk) {
    Launch p{tiles * kv_heads, rows, 0x40000000, 1, 0};
    busy *= kv_heads;
    long long want = busy > 0 ? aim / busy : 1;
    const long long most = max_seq_len / min_chunk;
    if (want > most) want = most;
    if (want > 1) {
        const long long chunk = ((max_seq_len + want - 1) / want + kTileKeys - 1) / kTileKeys * kTileKeys;
        p.splits = (int)((max_seq_len + chunk - 1) / chunk);
        if (p.splits > 1) {
            p.chunk = (int)chunk;
            p.floats = rows * p.splits * (d + 2);
        }
    }
    return p;
}

Plan plan_of(const SplitRules &rules, long long T, long long S, int q_heads, int kv_heads, int d, int max_seq_len, int window) {
    const long long G = q_heads / kv_heads;
    // few rows that see no more than one part's keys are not split, wherever these lie
    const int few_len = window > 0 && window <= rules.min_chunk ? window : max_seq_len;
    Plan p{};
    if (T <= S) {
        p.few_takes = Take::kAll;
        const long long full = T * G / kTileRows;
        const long long busy = full > T ? full : T;
        p.few = divide(full + S, busy, T * q_heads, kv_heads, d, few_len, kCUs,
                       busy * kv_heads * 4 <= kCUs ? rules.idle_chunk : rules.min_chunk);
    } else {
        p.few_takes = Take::kSmall;
        const long long full = T * G / rules.many_rows, busy = full > 1 ? full : 1, room = rules.room;
        // the small requests' parts need not be shorter than what the other
        // workgroups take anyway: at least this many keys one after the other, where
        // a small request's waves share theirs
        const long long anyway = busy * kv_heads * (T / S) / 2 / room * rules.waves;
        p.few = divide(S * (kSmallRows / kTileRows), S, S * kSmallRows * kv_heads, kv_heads, d, few_len, kCUs,
                       anyway > rules.min_chunk ? anyway : rules.min_chunk);
        // the fewer tile numbers of two ways that are enough (a request of many rows has
        // more than kSmallRows): 29 decode rows and 16 tokens take 23 us with 3 per kv
        // head, 32 with 31
        const long long by_rows = T * G / kSmallRows + 1;
        p.by_rows = by_rows < full + S;
        p.many = divide(p.by_rows ? by_rows : full + S, busy, T * q_heads, kv_heads, d, max_seq_len, room, rules.many_chunk);
    }
    return p;
}

template <Take TAKE>
static void launch_join_of(const AttentionArgs &a, const Launch &p, const Division &v, int tile_rows, hipStream_t stream) {
    const dim3 grid((unsigned)((p.rows + 3) / 4)), block(256);
    switch (a.d) {
        case 64: hipLaunchKernelGGL((attention_join_kernel<64, TAKE>), grid, block, 0, stream, a, v, (int)p.rows, tile_rows); break;
        case 128: hipLaunchKernelGGL((attention_join_kernel<128, TAKE>), grid, block, 0, stream, a, v, (int)p.rows, tile_rows); break;
        default: hipLaunchKernelGGL((attention_join_kernel<256, TAKE>), grid, block, 0, stream, a, v, (int)p.rows, tile_rows);
    }
}

void launch_join(Take take, const AttentionArgs &a, const Launch &p, const Division &v, int tile_rows, hipStream_t stream) {
    if (p.splits <= 1) return;
    switch (take) {
        case Take::kAll: return launch_join_of<Take::kAll>(a, p, v, tile_rows, stream);
        case Take::kSmall: return launch_join_of<Take::kSmall>(a, p, v, tile_rows, stream);
        case Take::kLarge: return launch_join_of<Take::kLarge>(a, p, v, tile_rows, stream);
    }
}

}  // namespace gdn
