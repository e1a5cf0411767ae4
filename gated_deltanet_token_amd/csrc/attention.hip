// Attention over the 8-bit paged cache (gdn_paged_attention_kv8), gfx950.
//
// Scores are formed transposed, X^T = K Q^T (keys down, rows across), so that
// the exponentials P^T leave the matrix cores in the lanes and order in which
// the second product O^T = V^T P^T wants them: no value changes lanes between
// the two.  A row here is one (token, q head) pair of the q heads that share
// a kv head.
//
// K Q^T runs on e4m3 operands.  The cache's codes go into the matrix cores as
// they lie in memory, and q is split into two e4m3 parts, q = (hi + lo) / f
// with f a power of two that brings the row's largest element to [128, 256):
// hi keeps 4 significant bits, lo the other 4 of a bf16 value.  The split is
// exact for elements down to 2^-10 of the row's largest, and within 2^-18 of
// that for smaller ones.  Two products of 8-bit operands take as long as one
// of bf16, and no key is converted.
//
// V^T P^T runs on bf16: values are converted in registers (exact), weights
// rounded to bf16 with their page's value scale in them.  Scores and sums are
// fp32; the running maximum is in units of log2.
#include "fp8.h"
#include "serving_internal.h"

namespace gdn {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
constexpr int kTileKeys = 64;           // keys a wave takes at once
constexpr int kTileRows = 16;           // rows of a workgroup of the few-rows kernel

// one request's part in a call, as the kernels see it
struct Request {
    int begin, n;       // its first token, and how many
    int len;            // keys, as seq_lens says (>= 0)
    int L;              // keys within the block table's row
};

__device__ __forceinline__ Request request_of(const AttentionArgs &a, int s) {
    Request r;
    int end;
    clamp_range(a.qsl[s], a.qsl[s + 1], a.num_tokens, r.begin, end);
    r.n = end - r.begin;
    r.len = max(a.seq_lens[s], 0);
    r.L = (int)min((long long)r.len, (long long)a.max_pages * a.page);
    return r;
}

// the keys [jb, je) that token i of the request sees
__device__ __forceinline__ void key_range(const AttentionArgs &a, const Request &r, int i, int &jb, int &je) {
    const int upto = r.len - r.n + i + 1;            // its position + 1
    je = a.causal ? min(r.L, upto) : r.L;
    jb = a.window > 0 && upto > a.window ? upto - a.window : 0;
}

// Row tiles: request s owns the tile numbers from floor(query_start_loc[s] * G
// / rows) + s on, G rows per token: at least as many as it needs, found
// without a list.  Returns the last request whose first tile is at or before
// `tile` (64 candidates per step), and the tile's number within it.
__device__ __forceinline__ int find_request(const AttentionArgs &a, long long tile, int group, int rows, int &within) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.num_seqs;
    auto first = [&](int s) { return (long long)max(a.qsl[s], 0) * group / rows + s; };
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

__device__ __forceinline__ float max_over(float x, int lanes_apart) { return fmaxf(x, __shfl_xor(x, lanes_apart, 64)); }

// 16 codes -> 16 bf16 values
__device__ __forceinline__ void codes_to_bf16(const uint4 &w, bf16x8 &lo, bf16x8 &hi) {
    const uint32_t d[4] = {w.x, w.y, w.z, w.w};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d[i], 1.0f, false));
        r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d[i], 1.0f, true));
    }
    const i32x4 a = {(int)r[0], (int)r[1], (int)r[2], (int)r[3]}, b = {(int)r[4], (int)r[5], (int)r[6], (int)r[7]};
    lo = __builtin_bit_cast(bf16x8, a);
    hi = __builtin_bit_cast(bf16x8, b);
}

// per byte: 0x80 where an e4m3 code is NaN (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// The splits of a row tile's keys [lo, hi): split i takes the keys of [i C,
// (i + 1) C), the last one all that follow.
struct Splits {
    int first, last;    // those that have keys (last < first: none)
};
__device__ __forceinline__ Splits splits_of(int lo, int hi, int chunk, int n) {
    Splits s;
    s.first = min(lo / chunk, n - 1);
    s.last = hi > lo ? min((hi - 1) / chunk, n - 1) : s.first - 1;
    return s;
}

// partial results of (row, split): D sums and, behind all of them, the maximum and the sum of weights
__device__ __forceinline__ float *part_o(const AttentionArgs &a, long long row, int split, int n) {
    return a.workspace + (row * n + split) * a.d;
}
__device__ __forceinline__ float *part_ml(const AttentionArgs &a, long long row, int split, int n) {
    return a.workspace + (long long)a.num_tokens * a.num_q_heads * n * a.d + (row * n + split) * 2;
}

// ---------------------------------------------------------------------------
// Few rows: one workgroup of W waves per (16 rows of one request that share a
// kv head, split of its keys).  Bound by reading the cache: each wave takes
// every W-th tile of 64 keys straight from HBM into registers in the order of
// the matrix operands (16-byte loads, whole 64-byte sectors), with the next
// tile's keys and values on their way while it works on this one.  The waves'
// sums are joined in the LDS.
//
// Lanes: with c = lane % 16 and g = lane / 16, a lane holds row c and the keys
// 16 g .. 16 g + 15 of the tile, which lie in one page: one page number and
// one pair of scales per lane.  For that, row i of the a-th K operand is key
// 16 (i / 4) + 4 a + i % 4.
// ---------------------------------------------------------------------------
template <int D, int W>
__global__ __launch_bounds__(64 * W, W / 4) void attention_few_kernel(AttentionArgs a, int chunk, int n_splits) {
    constexpr int KS = D >= 128 ? D / 128 : 1;       // contraction steps of 128
    constexpr int KL = D / 64;                       // 16-byte loads per key operand
    constexpr int DT = D / 16;                       // operands of 16 value elements
    constexpr int DTH = DT < 8 ? DT : 8;             // of which joined at once
    __shared__ f32x4 red[W][DTH][64];
    __shared__ float red_m[W][16], red_l[W][16];
    // at D = 256 q's parts wait in the LDS: with sums, keys and values they
    // would pass a lane's 256 registers
    constexpr bool QLDS = D == 256;
    __shared__ i32x4 q_lds[QLDS ? 4 * KS : 1][64];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4, kg = c >> 2;
    const int G = a.num_q_heads / a.num_kv_heads;
    const long long unit = blockIdx.x / n_splits;
    const int split = blockIdx.x - (int)(unit * n_splits);
    const long long tile = unit / a.num_kv_heads;
    const int hk = (int)(unit - tile * a.num_kv_heads);
    int within;
    const int s = find_request(a, tile, G, kTileRows, within);
    const Request rq = request_of(a, s);
    const long long row0 = (long long)within * kTileRows, n_rows = (long long)rq.n * G;
    if (within < 0 || row0 >= n_rows) return;
    const int i_first = (int)(row0 / G), i_last = (int)(min(row0 + kTileRows, n_rows) - 1) / G;
    int lo, hi, x0, x1;                              // keys that some row sees, that every row sees
    key_range(a, rq, i_first, lo, x1);
    key_range(a, rq, i_last, x0, hi);
    const Splits sp = splits_of(lo, hi, chunk, n_splits);
    if (split != sp.first && (split < sp.first || split > sp.last)) return;
    const bool whole = sp.last <= sp.first;          // no other split: write o itself
    const int k_lo = max(lo, split * chunk);
    const int k_hi = split == n_splits - 1 ? hi : min(hi, (split + 1) * chunk);

    const long long row = row0 + c;
    const int i_row = (int)(row / G), h = hk * G + (int)(row - (long long)i_row * G);
    const bool live = row < n_rows;
    int jb = 0, je = 0;
    if (live) key_range(a, rq, i_row, jb, je);
    jb = max(jb, k_lo);
    je = min(je, k_hi);

    // q's two parts, in the order of the key loads: bytes 16 m + e of step s
    // are elements 128 s + 64 m + 16 g + e (for D = 64 the upper 16 bytes are lo)
    i32x8 qh[KS], ql[KS];
    float unscale;
    {
        const uint16_t *qp = a.q + (long long)(rq.begin + (live ? i_row : 0)) * a.q_stride + (long long)(live ? h : hk * G) * D;
        float f[KL][16];
        float m = 0.f;
#pragma unroll
        for (int l = 0; l < KL; ++l) {
            float t[8];
            unpack8(*reinterpret_cast<const uint4 *>(qp + 64 * l + 16 * g), t);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[l][e] = t[e];
            unpack8(*reinterpret_cast<const uint4 *>(qp + 64 * l + 16 * g + 8), t);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[l][8 + e] = t[e];
#pragma unroll
            for (int e = 0; e < 16; ++e) m = is_finite(f[l][e]) ? fmaxf(m, fabsf(f[l][e])) : m;
        }
        m = max_over(max_over(m, 16), 32);
        // up = 2^(7 - exponent of m), within [2^-120, 2^126]
        const int ex = max((int)(__builtin_bit_cast(uint32_t, m) >> 23), 8);
        const float up = __builtin_bit_cast(float, (uint32_t)(261 - ex) << 23);
        unscale = 1.f / up;
#pragma unroll
        for (int l = 0; l < KL; ++l) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float v[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = is_finite(f[l][4 * w + e]) ? f[l][4 * w + e] * up : __builtin_bit_cast(float, 0x7fc00000u);
                const uint32_t hw = e4m3x4(v[0], v[1], v[2], v[3]);
                e4m3_values(hw, b);
                const uint32_t lw = e4m3x4(v[0] - b[0], v[1] - b[1], v[2] - b[2], v[3] - b[3]);
                if constexpr (D == 64) {
                    qh[0][w] = (int)hw;
                    qh[0][4 + w] = (int)lw;
                } else {
                    qh[l / 2][4 * (l & 1) + w] = (int)hw;
                    ql[l / 2][4 * (l & 1) + w] = (int)lw;
                }
            }
        }
    }
    const float to_log2 = a.scale * kLog2e * unscale;
    if constexpr (QLDS) {
        if (wave == 0) {
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                q_lds[4 * st][lane] = i32x4{qh[st][0], qh[st][1], qh[st][2], qh[st][3]};
                q_lds[4 * st + 1][lane] = i32x4{qh[st][4], qh[st][5], qh[st][6], qh[st][7]};
                q_lds[4 * st + 2][lane] = i32x4{ql[st][0], ql[st][1], ql[st][2], ql[st][3]};
                q_lds[4 * st + 3][lane] = i32x4{ql[st][4], ql[st][5], ql[st][6], ql[st][7]};
            }
        }
        __syncthreads();
    }

    const int shift = __builtin_ctz(a.page), in_page = a.page - 1;
    const int32_t *bt = a.block_table + s * a.block_table_stride;
    auto page_at = [&](int j) {
        const int p = j >> shift;
        return j < k_hi && p < a.max_pages ? bt[p] : -1;
    };
    auto good = [&](int p) { return (unsigned)p < (unsigned)a.num_pages; };

    uint4 kr[4][KL], vr[DT];
    float ks = 0.f, vs = 0.f;
    auto load_k = [&](int j0, int page) {
        const int j = j0 + 16 * kg;
        const uint8_t *p = a.k_cache + (((long long)(good(page) ? page : 0) * a.num_kv_heads + hk) * a.page + (j & in_page) + (c & 3)) * D + 16 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int l = 0; l < KL; ++l) kr[t][l] = *reinterpret_cast<const uint4 *>(p + 4 * t * D + 64 * l);
    };
    auto load_v = [&](int j0, int page) {
        const int j = j0 + 16 * g;
        const long long ph = (long long)(good(page) ? page : 0) * a.num_kv_heads + hk;
        const uint8_t *p = a.v_cache + (ph * D + c) * a.page + (j & in_page);
#pragma unroll
        for (int t = 0; t < DT; ++t) vr[t] = *reinterpret_cast<const uint4 *>(p + (long long)16 * t * a.page);
        ks = a.k_scale[ph];
        vs = a.v_scale[ph];
    };

    f32x4 o[DT] = {};
    float m = kNegInf, l = 0.f;
    const int step = W * kTileKeys;
    int j0 = (k_lo & ~(kTileKeys - 1)) + wave * kTileKeys;
    int pk = page_at(j0 + 16 * kg), pv = page_at(j0 + 16 * g);
    if (j0 < k_hi) {
        load_k(j0, pk);
        load_v(j0, pv);
    }
    for (; j0 < k_hi; j0 += step) {
        const int jn = j0 + step;
        const int pk_n = page_at(jn + 16 * kg), pv_n = page_at(jn + 16 * g);
        // X^T: keys 16 g + 4 t + r of row c
        f32x4 x[4] = {};
#pragma unroll
        for (int st = 0; st < KS; ++st) {
            i32x8 hi8 = qh[st], lo8 = ql[st];
            if constexpr (QLDS) {
                const i32x4 a0 = q_lds[4 * st][lane], a1 = q_lds[4 * st + 1][lane];
                const i32x4 b0 = q_lds[4 * st + 2][lane], b1 = q_lds[4 * st + 3][lane];
                hi8 = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
                lo8 = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint4 u = kr[t][D == 64 ? 0 : 2 * st], w = kr[t][D == 64 ? 0 : 2 * st + 1];
                const i32x8 k8 = {(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)w.x, (int)w.y, (int)w.z, (int)w.w};
                x[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, hi8, x[t], 0, 0, 0, 0, 0, 0);
                if constexpr (D != 64)
                    x[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, lo8, x[t], 0, 0, 0, 0, 0, 0);
            }
        }
        if (jn < k_hi) load_k(jn, pk_n);
        asm volatile("" ::: "memory");

        const float factor = to_log2 * ks;
        const int jg = j0 + 16 * g;
        const bool seen_page = good(pv);
        const bool masked = __any(!seen_page) || j0 < max(x0, k_lo) || j0 + kTileKeys > min(x1, k_hi);
        float mx = kNegInf;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[t][r] *= factor;
                if (masked) {
                    const int j = jg + 4 * t + r;
                    if (!(seen_page && j >= jb && j < je)) x[t][r] = kNegInf;
                }
                mx = fmaxf(mx, x[t][r]);
            }
        mx = max_over(max_over(mx, 16), 32);
        if (__any(mx > m)) {
            const float m_new = fmaxf(m, mx);
            const float f = m_new == m ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
            m = m_new;
            l *= f;
#pragma unroll
            for (int t = 0; t < DT; ++t) o[t] *= f;
        }
        const float at = m == kNegInf ? 0.f : m;
        bf16x8 p[2];
        {
            uint32_t pw[8];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float e[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    e[r] = __builtin_amdgcn_exp2f(x[t][r] - at);
                    l += e[r];
                    // a masked key's scale may be anything
                    e[r] = masked && x[t][r] == kNegInf ? 0.f : e[r] * vs;
                }
                pw[2 * t] = pack_bf16x2(e[0], e[1]);
                pw[2 * t + 1] = pack_bf16x2(e[2], e[3]);
            }
            const i32x4 u = {(int)pw[0], (int)pw[1], (int)pw[2], (int)pw[3]}, w = {(int)pw[4], (int)pw[5], (int)pw[6], (int)pw[7]};
            p[0] = __builtin_bit_cast(bf16x8, u);
            p[1] = __builtin_bit_cast(bf16x8, w);
        }
        if (masked) {
            // Values that no row sees may be anything: zero.  NaN among those
            // that some rows see must reach those rows only: its codes are
            // zeroed too, and rows that see it get their NaN from a count.
            uint32_t keep[4], any_nan = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                keep[w] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int j = jg + 4 * w + b;
                    if (seen_page && j >= max(lo, k_lo) && j < k_hi) keep[w] |= 0xffu << (8 * b);
                }
            }
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                vr[t].x &= keep[0];
                vr[t].y &= keep[1];
                vr[t].z &= keep[2];
                vr[t].w &= keep[3];
                any_nan |= nan_codes(vr[t].x) | nan_codes(vr[t].y) | nan_codes(vr[t].z) | nan_codes(vr[t].w);
            }
            if (__any(any_nan != 0)) {
                bf16x8 sees[2];
                uint32_t pw[8];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; r += 2) {
                        const int j = jg + 4 * t + r;
                        pw[2 * t + r / 2] = (j >= jb && j < je ? 0x3f80u : 0u) | (j + 1 >= jb && j + 1 < je ? 0x3f800000u : 0u);
                    }
                const i32x4 u = {(int)pw[0], (int)pw[1], (int)pw[2], (int)pw[3]}, w = {(int)pw[4], (int)pw[5], (int)pw[6], (int)pw[7]};
                sees[0] = __builtin_bit_cast(bf16x8, u);
                sees[1] = __builtin_bit_cast(bf16x8, w);
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    uint32_t d[4] = {vr[t].x, vr[t].y, vr[t].z, vr[t].w}, ones[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t bad = nan_codes(d[i]) >> 7;       // 1 per NaN byte
                        d[i] &= ~(bad * 0xffu);
                        ones[i] = bad * 0x38u;                           // e4m3 1.0
                    }
                    vr[t] = make_uint4(d[0], d[1], d[2], d[3]);
                    bf16x8 lo8, hi8;
                    codes_to_bf16(make_uint4(ones[0], ones[1], ones[2], ones[3]), lo8, hi8);
                    f32x4 count = {0.f, 0.f, 0.f, 0.f};
                    count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo8, sees[0], count, 0, 0, 0);
                    count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi8, sees[1], count, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (count[r] > 0.f) o[t][r] = __builtin_bit_cast(float, 0x7fc00000u);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            bf16x8 lo8, hi8;
            codes_to_bf16(vr[t], lo8, hi8);
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo8, p[0], o[t], 0, 0, 0);
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi8, p[1], o[t], 0, 0, 0);
        }
        if (jn < k_hi) load_v(jn, pv_n);
        asm volatile("" ::: "memory");
        pv = pv_n;
    }

    // join the waves: maxima, then each wave's sums at the common maximum
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0) {
        red_m[wave][c] = m;
        red_l[wave][c] = l;
    }
    __syncthreads();
    float m_all = kNegInf, l_all = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) m_all = fmaxf(m_all, red_m[w][c]);
    const float at = m_all == kNegInf ? 0.f : m_all;
#pragma unroll
    for (int w = 0; w < W; ++w) l_all += red_l[w][c] * __builtin_amdgcn_exp2f(red_m[w][c] - at);
    const float f = __builtin_amdgcn_exp2f(m - at);
    const long long out_row = (long long)(rq.begin + i_row) * a.num_q_heads + h;
    const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
#pragma unroll
    for (int t0 = 0; t0 < DT; t0 += DTH) {
        if (t0) __syncthreads();
#pragma unroll
        for (int t = 0; t < DTH; ++t) red[wave][t][lane] = o[t0 + t] * f;
        __syncthreads();
        for (int t = wave; t < DTH; t += W) {
            f32x4 sum = red[0][t][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += red[w][t][lane];
            if (!live) continue;
            const int d = 16 * (t0 + t) + 4 * g;
            if (whole) {
                uint2 w;
                w.x = pack_bf16x2(sum.x * inv, sum.y * inv);
                w.y = pack_bf16x2(sum.z * inv, sum.w * inv);
                *reinterpret_cast<uint2 *>(a.o + (long long)(rq.begin + i_row) * a.o_stride + (long long)h * D + d) = w;
            } else {
                *reinterpret_cast<f32x4 *>(part_o(a, out_row, split, n_splits) + d) = sum;
            }
        }
    }
    if (!whole && wave == 0 && g == 0 && live) {
        float *ml = part_ml(a, out_row, split, n_splits);
        ml[0] = m_all;
        ml[1] = l_all;
    }
}

// ---------------------------------------------------------------------------
// The splits of a row joined: one wave per row, its splits' sums brought to
// the common maximum.
// ---------------------------------------------------------------------------
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a, int chunk, int n_splits) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= (long long)a.num_tokens * a.num_q_heads) return;
    const int t = (int)(row / a.num_q_heads), h = (int)(row - (long long)t * a.num_q_heads);
    // the request of token t: tiles of one row per token are its tokens
    int lo = 0, n = a.num_seqs;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const unsigned long long b = __ballot(lane * step < n && a.qsl[lo + lane * step] <= t);
        const int k = b ? 63 - __builtin_clzll(b) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    const Request rq = request_of(a, lo);
    if (t < rq.begin || t >= rq.begin + rq.n) return;
    // the keys of the row's tile decide which splits wrote
    const int G = a.num_q_heads / a.num_kv_heads;
    const long long r = (long long)(t - rq.begin) * G + h % G, r0 = r / kTileRows * kTileRows;
    const int i_first = (int)(r0 / G), i_last = (int)(min(r0 + kTileRows, (long long)rq.n * G) - 1) / G;
    int k_lo, k_hi, x;
    key_range(a, rq, i_first, k_lo, x);
    key_range(a, rq, i_last, x, k_hi);
    const Splits sp = splits_of(k_lo, k_hi, chunk, n_splits);
    if (sp.last <= sp.first) return;
    float m = kNegInf, l = 0.f, o[E] = {};
    for (int i = sp.first; i <= sp.last; ++i) m = fmaxf(m, part_ml(a, row, i, n_splits)[0]);
    const float at = m == kNegInf ? 0.f : m;
    for (int i = sp.first; i <= sp.last; ++i) {
        const float *ml = part_ml(a, row, i, n_splits), *p = part_o(a, row, i, n_splits);
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
// How a call is split.  A workgroup of the few-rows kernel holds eight waves;
// splits are made until there is a workgroup for every CU, each split at least
// one tile per wave.
// ---------------------------------------------------------------------------
constexpr int few_waves(int d) { return d == 256 ? 4 : 8; }
constexpr int kCUs = 256;
constexpr int kMinChunk = 8 * kTileKeys;

struct Plan {
    long long units;    // (row tile, kv head) pairs, upper bound
    int chunk, splits;
};

static Plan plan_of(long long num_tokens, long long num_seqs, int num_q_heads, int num_kv_heads, int max_seq_len) {
    Plan p;
    const long long group = num_q_heads / num_kv_heads;
    p.units = (num_tokens * group / kTileRows + num_seqs) * num_kv_heads;
    // tiles that hold rows, as far as the host can tell
    const long long full = num_tokens * group / kTileRows, asked = num_tokens < num_seqs ? num_tokens : num_seqs;
    const long long busy = num_kv_heads * (full > asked ? full : asked);
    long long want = busy > 0 ? (kCUs + busy - 1) / busy : 1;
    const long long most = (max_seq_len + (long long)kMinChunk - 1) / kMinChunk;
    if (want > most) want = most;
    if (want < 1) want = 1;
    long long chunk = (max_seq_len + want - 1) / want;
    chunk = (chunk + kTileKeys - 1) / kTileKeys * kTileKeys;
    p.splits = (int)((max_seq_len + chunk - 1) / chunk);
    p.chunk = (int)(p.splits == 1 ? 0x40000000 : chunk);
    return p;
}

int64_t attention_workspace_bytes(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int d, int max_seq_len) {
    const Plan p = plan_of(num_tokens, num_seqs, num_q_heads, num_kv_heads, max_seq_len);
    if (p.splits == 1) return 0;
    return (int64_t)num_tokens * num_q_heads * p.splits * (d + 2) * 4;
}

template <int D>
static hipError_t launch_d(const AttentionArgs &a, hipStream_t stream) {
    const Plan p = plan_of(a.num_tokens, a.num_seqs, a.num_q_heads, a.num_kv_heads, a.max_seq_len);
    const long long blocks = p.units * p.splits, rows = (long long)a.num_tokens * a.num_q_heads;
    if (blocks > 0x7fffffffLL || rows > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((attention_few_kernel<D, few_waves(D)>), dim3((unsigned)blocks), dim3(64 * few_waves(D)), 0, stream, a, p.chunk,
                       p.splits);
    if (p.splits > 1)
        hipLaunchKernelGGL((attention_join_kernel<D>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, p.chunk,
                           p.splits);
    return hipGetLastError();
}

hipError_t launch_attention(const AttentionArgs &a, hipStream_t stream) {
    switch (a.d) {
        case 64: return launch_d<64>(a, stream);
        case 128: return launch_d<128>(a, stream);
        case 256: return launch_d<256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
