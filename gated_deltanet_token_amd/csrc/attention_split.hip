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
