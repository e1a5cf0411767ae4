// Attention over the 8-bit paged cache (gdn_paged_attention_kv8), gfx950.
//
// Scores are formed transposed, X^T = K Q^T (keys down, rows across), so that
// the exponentials P^T leave the matrix cores in the lanes and order in which
// the second product O^T = V^T P^T wants them: no value changes lanes between
// the two.  A row here is one (token, q head) pair of the q heads that share
// a kv head.
//
// K Q^T runs on e4m3 operands.  The cache's codes go into the matrix cores as
// they lie in memory, and q is split into two e4m3 parts, q = (hi + lo / 32) / f
// with f a power of two that brings the row's largest element to [128, 256):
// hi keeps 4 significant bits, lo the other 4 of a bf16 value, at most 8 and 32
// times that in its operand.  The split is exact for elements down to 2^-14 of
// the row's largest, where lo is 2^-9 or a multiple, and within 2^-22 of that for
// smaller ones (2^-9 and 2^-17 if lo were not taken 32-fold).  Two products of
// 8-bit operands take as long as one of bf16, and no key is converted.  The 32
// goes back out as a power of two of lo's product in waves of 32 rows, where
// that costs nothing, and by sums of lo's own, an fma per score, in waves of 16 (a
// prompt of 8,192 tokens, heads of 256: 614 us, 645 by scaled products, 600 without
// the 32; heads of 128: 572 with it and without).
//
// V^T P^T runs on bf16: values are converted in registers (exact), weights
// rounded to bf16 with their page's value scale in them: a light key beside a
// heavy one keeps its 8 bits.  (Weights in two e4m3 parts with a power of two
// per 32 keys need no conversion of values, but lose what is below 2^-20 of the
// heaviest: a prompt of 8,192 tokens with heads of 256 took 589 us so, 596 us now.)
// Scores and sums are fp32; the maximum is in units of log2.
#include "attention_split.h"
#include "fp8.h"

namespace gdn {

// 8 codes -> 8 bf16 values
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w0, uint32_t w1) {
    const i32x4 v = {__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false)),
                     __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true)),
                     __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false)),
                     __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true))};
    return __builtin_bit_cast(bf16x8, v);
}

// per byte: 0x80 where an e4m3 code is NaN (0x7f or 0xff)
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// a word's NaN codes become zero; returned: whether there were any
__device__ __forceinline__ uint32_t take_nan(uint32_t &w) {
    const uint32_t b = nan_codes(w) >> 7;
    w &= ~(b * 0xffu);
    return b;
}
// four words of values, those of no key in `keep` and NaN codes zeroed; returned:
// whether there were any of the latter
__device__ __forceinline__ uint32_t masked_values(uint4 &w, const uint32_t (&keep)[4]) {
    w.x &= keep[0];
    w.y &= keep[1];
    w.z &= keep[2];
    w.w &= keep[3];
    return take_nan(w.x) | take_nan(w.y) | take_nan(w.z) | take_nan(w.w);
}
// the bytes of a word of keys j .. j + 3 that lie in [lo, hi)
__device__ __forceinline__ uint32_t key_bytes(int j, int lo, int hi) {
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (j + b >= lo && j + b < hi) m |= 0xffu << (8 * b);
    return m;
}

// The larger of the magnitudes of two bf16 pairs, as integers in the same order
// (an infinity or NaN among a row of q: its scores are NaN at any factor).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, w & 0x7fff7fffu)));
}
__device__ __forceinline__ uint32_t larger(uint32_t m, const uint4 &w) {
    return larger(larger(larger(larger(m, w.x), w.y), w.z), w.w);
}
__device__ __forceinline__ float larger_half(uint32_t m) { return __builtin_bit_cast(float, max(m << 16, m & 0xffff0000u)); }

// The largest magnitude m of a row of q, brought to [128, 256): the power of
// two for it, within [2^-121, 2^126].
__device__ __forceinline__ float split_factor(float m) {
    const int ex = max((int)(__builtin_bit_cast(uint32_t, m) >> 23), 8);
    return __builtin_bit_cast(float, (uint32_t)(261 - ex) << 23);
}
// four elements' two parts, the second one 32-fold
constexpr float kLowTimes = 32.f;
constexpr int kWhole = 127, kLowPart = 127 - 5;         // 1 and 1 / 32 as powers of two of a scaled product
__device__ __forceinline__ void split4(const float *f, float up, int &hi, int &lo) {
    float v[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f[e] * up;           // infinities and NaN: NaN codes
    const uint32_t w = e4m3x4(v[0], v[1], v[2], v[3]);
    e4m3_values(w, b);
    hi = (int)w;
    lo = (int)e4m3x4(kLowTimes * (v[0] - b[0]), kLowTimes * (v[1] - b[1]), kLowTimes * (v[2] - b[2]), kLowTimes * (v[3] - b[3]));
}

// A lane's elements of one row, for lanes of 16 rows: 64 l + 16 g + e.
template <int D>
struct Row16 {
    uint4 w[D / 64][2];
};
template <int D>
__device__ __forceinline__ Row16<D> load_q16(const uint16_t *q, int g) {
    Row16<D> r;
#pragma unroll
    for (int l = 0; l < D / 64; ++l)
#pragma unroll
        for (int b = 0; b < 2; ++b) r.w[l][b] = *reinterpret_cast<const uint4 *>(q + 64 * l + 16 * g + 8 * b);
    return r;
}

// What brings the row to its parts' range.
template <int D>
__device__ __forceinline__ float factor_q16(const Row16<D> &q) {
    uint32_t mm = 0;
#pragma unroll
    for (int l = 0; l < D / 64; ++l) mm = larger(larger(mm, q.w[l][0]), q.w[l][1]);
    return split_factor(max_over32(max_over16(larger_half(mm))));
}

// The row's two parts, in the order of the key operands: bytes
// 16 m + e of step s are elements 128 s + 64 m + 16 g + e (for D = 64 the upper
// 16 bytes are lo).
template <int D>
__device__ __forceinline__ void split_q16(const Row16<D> &q, float up, i32x8 (&qh)[D >= 128 ? D / 128 : 1],
                                          i32x8 (&ql)[D >= 128 ? D / 128 : 1]) {
#pragma unroll
    for (int l = 0; l < D / 64; ++l)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float f[8];
            unpack8(q.w[l][b], f);
#pragma unroll
            for (int w = 2 * b; w < 2 * b + 2; ++w) {
                int hw, lw;
                split4(&f[4 * (w & 1)], up, hw, lw);
                if constexpr (D == 64) {
                    qh[0][w] = hw;
                    qh[0][4 + w] = lw;
                } else {
                    qh[l / 2][4 * (l & 1) + w] = hw;
                    ql[l / 2][4 * (l & 1) + w] = lw;
                }
            }
        }
}

// A factor for scores whose signs were turned where it is negative: not zero,
// so that it keeps a masked score at -infinity.
__device__ __forceinline__ float usable(float factor) { return factor == 0.f ? 0x1p-126f : factor < 0.f ? -factor : factor; }

// The sums are brought to a row's new maximum only where that is more than this
// above the maximum m that they are relative to (in units of log2): weights up
// to 2^8 cost bf16 and fp32 nothing, and most tiles have a new maximum for some
// row of a wave, hardly any such a one (a prompt of 8,192 tokens, heads of 128: 589
// us with none, 573).  None is let through where the values' scale is so large
// that weight times scale or their sum could pass fp32's end, nor in the first
// kLateKeys keys of a workgroup's part: of few keys the heaviest often makes up
// the sum, and its weight of 1 is exact.  (A wave that begins behind them begins
// with its first tile's maximum, too.)
__device__ __forceinline__ float slack(float vs, bool late) { return late && fabsf(vs) < 0x1p64f ? 8.f : 0.f; }

// One tile of a wave with 16 rows: the scores x (keys jg + 4 t + r of the lane's
// row) become weights, packed to bf16 pairs with the values' scale in them;
// the running maximum m, the lane's sum l and the sums o follow.
template <int NT, int DT>
__device__ __forceinline__ void weigh(f32x4 (&x)[NT], float factor, float vs, bool late, bool masked, bool seen_page, int jg, int jb,
                                      int je, float &m, float &l, f32x4 (&o)[DT], uint32_t (&pw)[2 * NT]) {
    if (masked) {
        // from the row's first and past its last key of these, none of a missing page
        const int from = seen_page ? jb - jg : 4 * NT, to = je - jg;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * t + r < from || 4 * t + r >= to) x[t][r] = kNegInf;
        // scales of a page that the row does not see may be anything
        if (max(from, 0) >= min(to, 4 * NT)) {
            vs = 0.f;
            factor = 1.f;
        }
    }
    if (__any(!(factor > 0.f))) {              // zero, below it or NaN
        if (factor < 0.f)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (x[t][r] != kNegInf) x[t][r] = -x[t][r];
        factor = usable(factor);
    }
    float mx = kNegInf;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = fmaxf(mx, x[t][r]);
    mx = max_over32(max_over16(mx * factor));
    if (__any(mx > m + slack(vs, late))) {
        const float m_new = fmaxf(m, mx);
        const float f = m_new == m ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
        m = m_new;
        l *= f;
#pragma unroll
        for (int t = 0; t < DT; ++t) o[t] *= f;
    }
    const float at = m == kNegInf ? 0.f : m;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float e[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r], factor, -at));
            l += e[r];
        }
        pw[2 * t] = pack_bf16x2(e[0] * vs, e[1] * vs);
        pw[2 * t + 1] = pack_bf16x2(e[2] * vs, e[3] * vs);
    }
}

// A tile that some of the rows see and others do not cannot pass NaN codes of
// its values through the matrix cores: they would reach all rows.  They go in
// as zeros there, and this pass, where any was met, finds the sums that they
// belong to: bit i of `bits` for the lane's sum i, element `element(i)`
// of the row that sees [jb, je).  `late(j0)`: whether the tile at j0 went in so.
template <int N, typename Late, typename Element, typename Page>
__device__ __forceinline__ void find_nan(const AttentionArgs &a, int hk, int j0, int end, int step, int tile, int jb, int je,
                                         unsigned long long (&bits)[(N + 63) / 64], Late late, Element element, Page page_at) {
#pragma unroll 1
    for (; j0 < end; j0 += step) {
        if (!late(j0)) continue;
#pragma unroll 1
        for (int j = j0; j < min(j0 + tile, end); ++j) {
            const int page = page_at(j);
            if ((unsigned)page >= (unsigned)a.num_pages || j < jb || j >= je) continue;
            const uint8_t *v = a.v_cache + ((long long)page * a.num_kv_heads + hk) * a.d * a.page + (j & (a.page - 1));
#pragma unroll 1
            for (int i = 0; i < N; ++i)
                if ((v[(long long)element(i) * a.page] & 0x7f) == 0x7f) bits[N > 64 ? i / 64 : 0] |= 1ull << (i & 63);
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows: one workgroup of W waves per (16 rows of one request that
// share a kv head, split of its keys).  Bound by reading the cache: each wave
// takes every W-th tile of TK keys straight from HBM into registers in the
// order of the matrix operands (16-byte loads, whole 64-byte sectors), with
// the next tile's keys and values on their way while it works on this one.
// The waves' sums are joined in the LDS.
//
// Lanes: with c = lane % 16 and g = lane / 16, a lane holds row c and the NK =
// TK / 4 keys from NK g on, which lie in one page: one page number and one pair
// of scales per lane.  For that, row i of the t-th K operand is key NK (i / 4) +
// 4 t + i % 4.
// TK is 64; at D = 256, 32, so that two tiles and the sums fit a lane's 256
// registers (with 64 keys and no tile ahead a decode step of 32 requests took
// 25.0 us).
// Measured: 32 requests of 1,100 tokens, 16/4 heads of 256: 20 to 22 us, half of it start
// and end; five of 40,000 to 131,000, 32/8 heads of 128: 188 us, 5.9 TB/s, and 6 us to
// join the parts.
// ---------------------------------------------------------------------------
constexpr int few_keys(int d) { return d == 256 ? 32 : 64; }

template <int D, int W>
struct FewLds {
    f32x4 red[W][D >= 128 ? 8 : D / 16][64];
    float red_m[W][16], red_l[W][16];
    // at D = 256 q's parts wait in the LDS: with sums, keys and values they
    // would pass a lane's 256 registers
    i32x4 q[D == 256 ? 8 : 1][64];
};

template <int D, int W, Take TAKE>
__device__ __forceinline__ void few_rows(const AttentionArgs &a, const Division &v, int block, FewLds<D, W> &lds) {
    constexpr int TK = few_keys(D), NK = TK / 4, NT = TK / 16, NV = TK / 16;
    constexpr int KS = D >= 128 ? D / 128 : 1;       // contraction steps of 128
    constexpr int KL = D / 64;                       // 16-byte loads per key operand
    constexpr int DT = D / 16;                       // operands of 16 value elements
    constexpr int DTH = DT < 8 ? DT : 8;             // of which joined at once
    constexpr bool QLDS = D == 256;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4, kg = c >> 2;
    const int G = a.num_q_heads / a.num_kv_heads;
    // rows and workgroups of a launch are fewer than 2^31 (launch_d): 32-bit
    // divisions, in the registers of one lane or all
    const unsigned unit = (unsigned)block / (unsigned)v.splits;
    const int split = block - (int)(unit * v.splits);
    const int tile = (int)(unit / (unsigned)a.num_kv_heads);
    const int hk = (int)(unit - tile * a.num_kv_heads);
    int within, s;
    if constexpr (TAKE == Take::kSmall) {
        // the first tiles, most of them the only ones, first (with each request's two
        // next to each other, half of the XCDs had nothing but empty ones: a mixed step
        // of 2,048 tokens took 63 us, 54 so)
        within = (unsigned)tile / (unsigned)a.num_seqs;
        s = tile - within * a.num_seqs;
    } else if (tile < a.num_seqs) {
        s = tile;                                    // every request's first tile: no search
        within = 0;
    } else {
        s = find_request(a, tile - a.num_seqs, G, kTileRows, 0, false, within);
        ++within;
    }
    const Request rq = request_of(a, s);
    const int n_rows = rq.n * G;
    if (within < 0 || (long long)within * kTileRows >= n_rows || (TAKE == Take::kSmall && n_rows > kSmallRows)) return;
    const int row0 = within * kTileRows, i_first = token_of(row0, G), i_last = token_of(last_row(row0, kTileRows, n_rows), G);
    int lo, hi, x0, x1;                              // keys that some row sees, that every row sees
    key_range(a, rq, i_first, lo, x1);
    key_range(a, rq, i_last, x0, hi);
    const Splits sp = splits_of(lo, hi, v.chunk, v.splits);
    if (split != sp.first && (split < sp.first || split > sp.last)) return;
    const bool whole = sp.last <= sp.first;          // no other split: write o itself
    const int k_lo = max(lo, split * v.chunk);
    const int k_hi = split == v.splits - 1 ? hi : min(hi, (split + 1) * v.chunk);

    const int row = row0 + c, i_row = token_of(row, G), h = hk * G + row - i_row * G;
    const bool live = row < n_rows;
    int jb = 0, je = 0;
    if (live) key_range(a, rq, i_row, jb, je);
    jb = max(jb, k_lo);
    je = min(je, k_hi);

    const Row16<D> q =
        load_q16<D>(a.q + (long long)(rq.begin + (live ? i_row : 0)) * a.q_stride + (long long)(live ? h : hk * G) * D, g);
    const int shift = __builtin_ctz(a.page), in_page = a.page - 1;
    const int32_t *bt = a.block_table + s * a.block_table_stride;
    auto page_at = [&](int j) {
        const int p = j >> shift;
        return j < k_hi && p < a.max_pages ? bt[p] : -1;
    };
    auto good = [&](int p) { return (unsigned)p < (unsigned)a.num_pages; };
    // Page numbers are loaded a tile ahead of the loads that use them, and not
    // looked at before: loads come back in order, so that looking at one that was
    // asked for behind a tile waits for the tile.
    auto entry_at = [&](int j) { return bt[min(j >> shift, a.max_pages - 1)]; };
    auto page_of = [&](int entry, int j) { return j < k_hi && good(entry) ? entry : -1; };

    uint4 kr[NT][KL];
    uint32_t vr[DT][NV];
    float ks = 0.f, vs = 0.f;
    auto load_k = [&](int j0, int page) {
        const int j = j0 + NK * kg;
        const long long ph = (long long)(good(page) ? page : 0) * a.num_kv_heads + hk;
        const uint8_t *p = a.k_cache + (ph * a.page + (j & in_page) + (c & 3)) * D + 16 * g;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int l = 0; l < KL; ++l) kr[t][l] = *reinterpret_cast<const uint4 *>(p + 4 * t * D + 64 * l);
    };
    auto load_v = [&](int j0, int page) {
        const int j = j0 + NK * g;
        const long long ph = (long long)(good(page) ? page : 0) * a.num_kv_heads + hk;
        const uint8_t *p = a.v_cache + (ph * D + c) * a.page + (j & in_page);
        ks = static_cast<const float *>(a.k_scale)[ph];              // needed before the values
        vs = static_cast<const float *>(a.v_scale)[ph];
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            if constexpr (NV == 4) {
                const uint4 w = *reinterpret_cast<const uint4 *>(p + (long long)16 * t * a.page);
                vr[t][0] = w.x;
                vr[t][1] = w.y;
                vr[t][2] = w.z;
                vr[t][3] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(p + (long long)16 * t * a.page);
                vr[t][0] = w.x;
                vr[t][1] = w.y;
            }
        }
    };

    f32x4 o[DT] = {};
    float m = kNegInf, l = 0.f;
    uint32_t met_nan = 0;
    constexpr int step = W * TK;
    int j0 = first_tile(k_lo, TK, wave);
    int ek = entry_at(j0 + NK * kg), ev = entry_at(j0 + NK * g), pv = -1;
    // the next tile's keys, and the entries behind it
    auto turn = [&](int j) {
        const int pk = page_of(ek, j + NK * kg), page = page_of(ev, j + NK * g);
        load_k(j, pk);
        ek = entry_at(j + step + NK * kg);
        ev = entry_at(j + step + NK * g);
        return page;
    };
    if (j0 < k_hi) {
        pv = turn(j0);
        asm volatile("" ::: "memory");
        load_v(j0, pv);
        asm volatile("" ::: "memory");
    }
    // q is split while the first tile is on its way
    i32x8 qh[KS], ql[KS];
    const float up = factor_q16<D>(q), to_log2 = a.scale * kLog2e * (1.f / up);
    if constexpr (!QLDS) {
        split_q16<D>(q, up, qh, ql);
    } else {
        if (wave == 0) {
            split_q16<D>(q, up, qh, ql);
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                lds.q[4 * st][lane] = i32x4{qh[st][0], qh[st][1], qh[st][2], qh[st][3]};
                lds.q[4 * st + 1][lane] = i32x4{qh[st][4], qh[st][5], qh[st][6], qh[st][7]};
                lds.q[4 * st + 2][lane] = i32x4{ql[st][0], ql[st][1], ql[st][2], ql[st][3]};
                lds.q[4 * st + 3][lane] = i32x4{ql[st][4], ql[st][5], ql[st][6], ql[st][7]};
            }
        }
        __syncthreads();
    }

    // At D = 64 one product takes both parts.  Its powers are those of 32 elements
    // in a row: the lanes of groups 0 and 1 hold those of the lower 16 bytes, groups
    // 2 and 3 those of the upper ones (measured with one-hot operands).
    [[maybe_unused]] const int both = g < 2 ? kWhole : kLowPart;

    for (; j0 < k_hi; j0 += step) {
        const int jn = j0 + step;
        int pv_n = -1;
        // X^T: keys NK g + 4 t + r of row c
        f32x4 x[NT] = {}, y[NT] = {};
#pragma unroll
        for (int st = 0; st < KS; ++st) {
            i32x8 hi8 = qh[st], lo8 = ql[st];
            if constexpr (QLDS) {
                const i32x4 a0 = lds.q[4 * st][lane], a1 = lds.q[4 * st + 1][lane];
                const i32x4 b0 = lds.q[4 * st + 2][lane], b1 = lds.q[4 * st + 3][lane];
                hi8 = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
                lo8 = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 u = kr[t][D == 64 ? 0 : 2 * st], w = kr[t][D == 64 ? 0 : 2 * st + 1];
                const i32x8 k8 = {(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)w.x, (int)w.y, (int)w.z, (int)w.w};
                if constexpr (D == 64) {
                    x[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, hi8, x[t], 0, 0, 0, kWhole, 0, both);
                } else {
                    x[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, hi8, x[t], 0, 0, 0, 0, 0, 0);
                    y[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, lo8, y[t], 0, 0, 0, 0, 0, 0);
                }
            }
        }
        if constexpr (D != 64) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[t][r] = __builtin_fmaf(y[t][r], 1.f / kLowTimes, x[t][r]);
        }
        if (jn < k_hi) pv_n = turn(jn);
        asm volatile("" ::: "memory");

        const int jg = j0 + NK * g;
        const bool seen_page = good(pv);
        const bool masked = __any(!seen_page) || j0 < max(x0, k_lo) || j0 + TK > min(x1, k_hi);
        uint32_t pw[2 * NT];
        weigh(x, to_log2 * ks, vs, j0 - k_lo >= kLateKeys, masked, seen_page, jg, jb, je, m, l, o, pw);
        if (masked) {
            // values that no row sees may be anything: zero; NaN: find_nan
#pragma unroll
            for (int w = 0; w < NV; ++w) {
                const uint32_t keep = seen_page ? key_bytes(jg + 4 * w, max(lo, k_lo), k_hi) : 0u;
#pragma unroll
                for (int t = 0; t < DT; ++t) {
                    vr[t][w] &= keep;
                    met_nan |= take_nan(vr[t][w]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < NV / 2; ++u) {
            const bf16x8 p = as_bf16x8(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]);
#pragma unroll
            for (int t = 0; t < DT; ++t)
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(vr[t][2 * u], vr[t][2 * u + 1]), p, o[t], 0, 0, 0);
        }
        if (jn < k_hi) load_v(jn, pv_n);
        asm volatile("" ::: "memory");
        pv = pv_n;
    }

    if (__any(met_nan != 0)) {
        unsigned long long bits[1] = {0};
        find_nan<4 * DT>(
            a, hk, first_tile(k_lo, TK, wave), k_hi, step, TK, jb, je, bits,
            [&](int j) { return __any(!good(page_at(j + NK * g))) || j < max(x0, k_lo) || j + TK > min(x1, k_hi); },
            [&](int i) { return 16 * (i >> 2) + 4 * g + (i & 3); }, page_at);
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (bits[0] >> (4 * t + r) & 1) o[t][r] = __builtin_bit_cast(float, 0x7fc00000u);
    }

    // join the waves: maxima, then each wave's sums at the common maximum
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (g == 0) {
        lds.red_m[wave][c] = m;
        lds.red_l[wave][c] = l;
    }
    __syncthreads();
    float m_all = kNegInf, l_all = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) m_all = fmaxf(m_all, lds.red_m[w][c]);
    const float at = m_all == kNegInf ? 0.f : m_all;
#pragma unroll
    for (int w = 0; w < W; ++w) l_all += lds.red_l[w][c] * __builtin_amdgcn_exp2f(lds.red_m[w][c] - at);
    const float f = __builtin_amdgcn_exp2f(m - at);
    const long long out_row = part_row<TAKE>(a, s, rq.begin + i_row, h, row, hk);
    const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
#pragma unroll
    for (int t0 = 0; t0 < DT; t0 += DTH) {
        if (t0) __syncthreads();
#pragma unroll
        for (int t = 0; t < DTH; ++t) lds.red[wave][t][lane] = o[t0 + t] * f;
        __syncthreads();
        for (int t = wave; t < DTH; t += W) {
            f32x4 sum = lds.red[0][t][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += lds.red[w][t][lane];
            if (!live) continue;
            const int d = 16 * (t0 + t) + 4 * g;
            if (whole) {
                uint2 w;
                w.x = pack_bf16x2(sum.x * inv, sum.y * inv);
                w.y = pack_bf16x2(sum.z * inv, sum.w * inv);
                *reinterpret_cast<uint2 *>(a.o + (long long)(rq.begin + i_row) * a.o_stride + (long long)h * D + d) = w;
            } else {
                *reinterpret_cast<f32x4 *>(part_o(v, D, out_row, split) + d) = sum;
            }
        }
    }
    if (!whole && wave == 0 && g == 0 && live) {
        float *ml = part_ml(v, out_row, split);
        ml[0] = m_all;
        ml[1] = l_all;
    }
}

// ---------------------------------------------------------------------------
// Many rows: one workgroup of four waves per (128 rows of one request that
// share a kv head, split of its keys); a wave holds 32 of the rows.  Bound by
// the matrix cores and the exponentials: tiles of 64 keys and values pass
// through the LDS once for all four waves, the next one on its way from HBM
// to registers meanwhile, with one barrier per tile between two buffers.
// Measured: a prompt of 8,192 tokens, 32/8 heads of 128: 552 to 618 us, by card,
// 996 to 890 TFLOP/s (4 D per row and key it sees).  Vector and matrix instructions hardly overlap here: an
// operation takes 2.4 cycles of a SIMD, an exponential 8, a pair of values'
// conversion 4, a matrix product 32 of which it hides 10; their sum over a tile is
// what a tile takes.  (Values converted once for the workgroup, on their way to the
// LDS: 612 us against 573 then, twice the LDS reads.)
//
// Lanes: with c = lane % 32 and h = lane / 32, a lane holds row c and the keys
// 32 h .. 32 h + 31 of the tile, x[a][r] being key 32 h + 16 a + r.  For that,
// row i of the a-th K operand is key 32 (i / 4 % 2) + 16 a + 4 (i / 8) + i % 4.
// LDS rows are cut into 16-byte pieces, piece p of a row kept at p ^ (a few
// bits of the row's number) so that the 16 lanes that are served together find
// theirs in 16 different places of the 256 bytes that the banks span.  Those are
// lanes 0-3, 12-15 and 20-27 of a half-wave, or the other 16 of it (measured: a
// read takes 4 cycles, and 5 with two of these lanes at the same banks).
// ---------------------------------------------------------------------------
constexpr int kWideThreads = 256;      // of a workgroup with 32 rows per wave
constexpr int kWideAhead = 3;

// use(i, read(i)) for i < N, each read A steps before its use and, left alone
// by the compiler, not earlier: it would read until it runs out of registers.
template <int N, int A, typename Read, typename Use>
__device__ __forceinline__ void run_ahead(Read read, Use use) {
    decltype(read(0)) w[N];          // all but A + 1 of them dead at any time
#pragma unroll
    for (int i = 0; i < (A < N ? A : N); ++i) w[i] = read(i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i + A < N) w[i + A] = read(i + A);
        asm volatile("" ::: "memory");
        use(i, w[i]);
    }
}

template <int D>
struct ManyLds {
    uint4 k[2][kTileKeys * D / 16], v[2][kTileKeys * D / 16];
    // of the tile's four granules of 16 keys: scales, and whether there is a page
    float ks[2][4], vs[2][4];
    int ok[2][4];
    int met_nan;
};

// the LDS place of piece p of element row d of a tile's values
__device__ __forceinline__ int v_piece(int d, int p) { return d * 4 + (p ^ (-(d >> 2) & 3)); }

// Staging of a workgroup of THREADS threads: the next tile's pieces are loaded
// into registers before the work on this one and put into the other LDS buffer
// after it, and the page numbers of the one behind with them.  (Loads from
// memory straight to the LDS need no registers, but the compiler waits for all
// of them before any read of the LDS: with them every tile waited out a round
// trip to memory, and a prompt of 8,192 tokens took 660 us.)  PLACE: the LDS
// place of a key's piece.
template <int D, int THREADS, int (*PLACE)(int, int)>
struct Staging {
    static constexpr int NL = 64 * D / 16 / THREADS;             // loads of a thread, of keys and of values
    static constexpr int PPK = D / 16, KEYS = THREADS / PPK;     // pieces per key; keys per load
    const AttentionArgs &a;
    ManyLds<D> &lds;
    const int32_t *bt;
    int k_hi, shift, hk, wave;
    uint32_t pitch;                // bytes of a page, all kv heads
    // a tile begins at a multiple of 64 keys, so a piece's place in its page
    // stays the same
    uint32_t k_off[NL], v_off;
    // the block table's entry for granule tid % 4 of the tile to load next, as it
    // came (looking at it here would wait for it and all loads before it)
    int entry, tile;
    uint4 kr[NL], vr[NL];
    int own;                       // the page of granule tid % 4 of these
    float s_ks, s_vs;              // its scales
    int k_lo, all0, all1;          // the first key; the keys that all rows see
    uint32_t met_nan;

    static_assert(64 / PPK <= 16, "");

    __device__ __forceinline__ Staging(const AttentionArgs &a_, ManyLds<D> &lds_, const ManyShare &w, int wave_)
        : a(a_), lds(lds_), bt(a_.block_table + w.s * a_.block_table_stride), k_hi(w.k_hi), shift(__builtin_ctz(a_.page)),
          hk(w.hk), wave(wave_), pitch((uint32_t)a_.num_kv_heads * a_.page * D), entry(-1), tile(0), own(-1), s_ks(0.f),
          s_vs(0.f), k_lo(w.k_lo), met_nan(0) {
        const WaveKeys all = wave_keys(a, w, w.row0, kManyRows);
        all0 = all.all0;
        all1 = all.all1;
        const int tid = threadIdx.x, in_page = a.page - 1;
#pragma unroll
        for (int i = 0; i < NL; ++i) k_off[i] = (hk * a.page + (i * KEYS + tid / PPK & in_page)) * D + 16 * (tid % PPK);
        v_off = (hk * D + (tid >> 2)) * a.page + (16 * (tid & 3) & in_page);
    }
    // the page of key j, -1: none
    __device__ __forceinline__ int page_at(int j) const {
        const int p = j >> shift, id = j < k_hi && p < a.max_pages ? bt[p] : -1;
        return (unsigned)id < (unsigned)a.num_pages ? id : -1;
    }
    __device__ __forceinline__ void pages(int j0) {
        tile = j0;
        entry = bt[min((j0 + 16 * (int)(threadIdx.x & 3)) >> shift, a.max_pages - 1)];
    }
    __device__ __forceinline__ void load() {
        const int j = tile + 16 * (threadIdx.x & 3);
        own = j < k_hi && (unsigned)entry < (unsigned)a.num_pages ? entry : -1;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            // a wave's keys lie in one granule: a scalar address
            const int granule = (i * KEYS + wave * (64 / PPK)) >> 4, page = __builtin_amdgcn_readlane(own, granule);
            const uint8_t *k = a.k_cache + (uint64_t)max(page, 0) * pitch;
            kr[i] = *reinterpret_cast<const uint4 *>(k + k_off[i]);
        }
        const uint8_t *v = a.v_cache + ((uint64_t)max(own, 0) * pitch + v_off);
#pragma unroll
        for (int i = 0; i < NL; ++i) vr[i] = *reinterpret_cast<const uint4 *>(v + i * (THREADS / 4) * a.page);
        if (threadIdx.x < 4) {
            const long long ph = (long long)max(own, 0) * a.num_kv_heads + hk;
            s_ks = static_cast<const float *>(a.k_scale)[ph];
            s_vs = static_cast<const float *>(a.v_scale)[ph];
        }
    }
    // Whether some rows see keys of the tile at j0 and others do not.  Zero weights
    // do not keep NaN codes of its values out of the sums: they go in as zeros, and so
    // does what no row sees and may be anything; find_nan looks for them afterwards.
    __device__ __forceinline__ bool late(int j0, int page) const {
        return j0 < all0 || j0 + kTileKeys > all1 || __any(page < 0);
    }
    __device__ __forceinline__ void put(int buf, int j0) {
        const int tid = threadIdx.x;
        if (late(j0, own)) {
            uint32_t keep[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) keep[i] = own < 0 ? 0u : key_bytes(j0 + 16 * (tid & 3) + 4 * i, k_lo, k_hi);
#pragma unroll
            for (int i = 0; i < NL; ++i) met_nan |= masked_values(vr[i], keep);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            lds.k[buf][PLACE(i * KEYS + tid / PPK, tid % PPK)] = kr[i];
            lds.v[buf][v_piece(i * (THREADS / 4) + (tid >> 2), tid & 3)] = vr[i];
        }
        if (tid < 4) {
            lds.ks[buf][tid] = s_ks;
            lds.vs[buf][tid] = s_vs;
            lds.ok[buf][tid] = own >= 0;
        }
    }
    __device__ __forceinline__ void begin(int j0) {
        pages(j0);
        load();
        pages(j0 + kTileKeys);
        put(0, j0);
        if (threadIdx.x == 0) lds.met_nan = 0;
        __syncthreads();
    }
    // before the work on the tile at j0: the next one's loads go out
    __device__ __forceinline__ void ahead(int j0) {
        if (j0 + kTileKeys < k_hi) {
            load();
            pages(j0 + 2 * kTileKeys);
        }
        asm volatile("" ::: "memory");
    }
    // after it: into the other buffer
    __device__ __forceinline__ void next(int j0, int buf) {
        asm volatile("" ::: "memory");
        if (j0 + kTileKeys < k_hi) put(buf ^ 1, j0 + kTileKeys);
        __syncthreads();
    }
    // after the last one, where there was one: whether a value was NaN and went in as zero
    __device__ __forceinline__ bool nan_left_out() {
        if (met_nan) lds.met_nan = 1;
        __syncthreads();
        return lds.met_nan != 0;
    }
};

template <int D>
__device__ __forceinline__ int k_piece(int key, int p) {
    constexpr int shift = D == 256 ? 0 : D == 128 ? 1 : 2;
    return key * (D / 16) + (p ^ (((key & 7) | (key >> 5 & 1) << 3) >> shift));
}

template <int D>
__device__ __forceinline__ void many_rows_wide(const AttentionArgs &a, const Division &v, int block, int blocks, ManyLds<D> &lds) {
    constexpr int KS = D / 64;                       // contraction steps of 64
    constexpr int DT = D / 32;                       // operands of 32 value elements

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 31, h2 = lane >> 5;
    const int G = a.num_q_heads / a.num_kv_heads;
    ManyShare w;
    if (!many_share(a, v, block, blocks, w)) return;
    const Request &rq = w.rq;
    const int hk = w.hk, k_lo = w.k_lo, k_hi = w.k_hi;

    // this wave's rows
    const int wrow = w.row0 + 32 * wave, row = wrow + c;
    const bool live = row < w.n_rows;
    const int i_row = live ? token_of(row, G) : 0, h = hk * G + (live ? row - i_row * G : 0);
    int jb = 0, je = 0;
    if (live) key_range(a, rq, i_row, jb, je);
    jb = max(jb, k_lo);
    je = min(je, k_hi);
    const WaveKeys wk = wave_keys(a, w, wrow, 32);

    // q's two parts: bytes 16 m + e of step st are elements 64 st + 32 h2 + 16 m + e
    i32x8 qh[KS], ql[KS];
    float to_log2;
    {
        const uint16_t *qp = a.q + (long long)(rq.begin + i_row) * a.q_stride + (long long)h * D + 32 * h2;
        uint32_t mm = 0;
#pragma unroll
        for (int st = 0; st < KS; ++st)
#pragma unroll
            for (int b = 0; b < 4; ++b) mm = larger(mm, *reinterpret_cast<const uint4 *>(qp + 64 * st + 8 * b));
        const float m = max_over32(larger_half(mm));
        const float up = split_factor(m);
        to_log2 = a.scale * kLog2e * (1.f / up);
#pragma unroll
        for (int st = 0; st < KS; ++st)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float f[8];
                unpack8(*reinterpret_cast<const uint4 *>(qp + 64 * st + 8 * b), f);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    int hw, lw;
                    split4(f + 4 * w, up, hw, lw);
                    qh[st][2 * b + w] = hw;
                    ql[st][2 * b + w] = lw;
                }
            }
    }

    Staging<D, kWideThreads, k_piece<D>> stage(a, lds, w, wave);
    // this lane's operand rows: the t-th K operand's is 16 t keys further on, with
    // its pieces in the same order, and so the t-th V operand's, 32 t elements
    const int key = 32 * (c >> 2 & 1) + 4 * (c >> 3) + (c & 3);
    const int k_row = key * (D / 16), k_swap = k_piece<D>(key, 2 * h2) - k_row, v_swap = v_piece(c, 2 * h2) - 4 * c;
    f32x16 o[DT] = {};
    float m = kNegInf, l = 0.f;
    int j0 = first_tile(k_lo, kTileKeys, 0), buf = 0;
    const bool any = j0 < k_hi;
    if (any) stage.begin(j0);
    for (; j0 < k_hi; j0 += kTileKeys, buf ^= 1) {
        const int jn = j0 + kTileKeys;
        stage.ahead(j0);
        if (j0 < wk.hi && jn > wk.lo) {
            const bool ok01[2] = {lds.ok[buf][2 * h2] != 0, lds.ok[buf][2 * h2 + 1] != 0};
            const bool masked = j0 < wk.all0 || jn > wk.all1 || __any(!(ok01[0] && ok01[1])), late = j0 - k_lo >= kLateKeys;
            const uint4 *kt = lds.k[buf] + k_row, *vt = lds.v[buf] + 4 * c;
            // half of the tile at a time: keys 16 t .. 16 t + 15 of each of its halves
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x16 x = {};
                run_ahead<KS, 1>(
                    [&](int st) {
                        const uint4 u = kt[16 * t * (D / 16) + (k_swap ^ 4 * st)];
                        const uint4 b = kt[16 * t * (D / 16) + (k_swap ^ (4 * st + 1))];
                        return i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
                    },
                    [&](int st, const i32x8 &k8) {
                        x = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k8, qh[st], x, 0, 0, 0, 0, 0, 0);
                        x = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k8, ql[st], x, 0, 0, 0, kWhole, 0, kLowPart);
                    });
                const bool ok = ok01[t];
                float mx = kNegInf, factor = to_log2 * lds.ks[buf][2 * h2 + t], vs = lds.vs[buf][2 * h2 + t];
                const int jg = j0 + 32 * h2 + 16 * t;
                if (masked) {
                    // from the row's first and past its last key of these 16, none of a missing page
                    const int from = ok ? jb - jg : 16, to = je - jg;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (r < from || r >= to) x[r] = kNegInf;
                    // scales of a page that the row does not see may be anything
                    if (max(from, 0) >= min(to, 16)) {
                        vs = 0.f;
                        factor = 1.f;
                    }
                }
                if (__any(!(factor > 0.f))) {              // zero, below it or NaN
                    if (factor < 0.f)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (x[r] != kNegInf) x[r] = -x[r];
                    factor = usable(factor);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) mx = fmaxf(mx, x[r]);
                mx = max_over32(mx * factor);
                if (__any(mx > m + slack(vs, late))) {
                    const float m_new = fmaxf(m, mx);
                    const float f = m_new == m ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
                    m = m_new;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < DT; ++i) o[i] *= f;
                }
                const float at = m == kNegInf ? 0.f : m;
                uint32_t pw[8];
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r], factor, -at));
                    const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r + 1], factor, -at));
                    l += e0 + e1;
                    pw[r / 2] = pack_bf16x2(e0 * vs, e1 * vs);
                }
                const bf16x8 p0 = as_bf16x8(pw[0], pw[1], pw[2], pw[3]), p1 = as_bf16x8(pw[4], pw[5], pw[6], pw[7]);
                run_ahead<DT, kWideAhead>([&](int i) { return vt[32 * 4 * i + (v_swap ^ t)]; }, [&](int i, const uint4 &w) {
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16(w.x, w.y), p0, o[i], 0, 0, 0);
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16(w.z, w.w), p1, o[i], 0, 0, 0);
                });
            }
        }
        stage.next(j0, buf);
    }

    if (any && stage.nan_left_out()) {
        unsigned long long bits[(16 * DT + 63) / 64] = {};
        find_nan<16 * DT>(
            a, hk, first_tile(k_lo, kTileKeys, 0), k_hi, kTileKeys, kTileKeys, jb, je, bits,
            [&](int j) { return stage.late(j, stage.page_at(j + 16 * (lane & 3))); },
            [&](int i) { return 32 * (i >> 4) + 8 * (i >> 2 & 3) + 4 * h2 + (i & 3); }, [&](int j) { return stage.page_at(j); });
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (bits[t / 4] >> (16 * (t & 3) + r) & 1) o[t][r] = __builtin_bit_cast(float, 0x7fc00000u);
    }
    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long out_row = (long long)(rq.begin + i_row) * a.num_q_heads + h;
    // element 32 t + 8 q + 4 h2 + r of row c is o[t][4 q + r]
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int d = 32 * t + 8 * q + 4 * h2;
            if (w.whole) {
                uint2 b;
                b.x = pack_bf16x2(o[t][4 * q] * inv, o[t][4 * q + 1] * inv);
                b.y = pack_bf16x2(o[t][4 * q + 2] * inv, o[t][4 * q + 3] * inv);
                *reinterpret_cast<uint2 *>(a.o + (long long)(rq.begin + i_row) * a.o_stride + (long long)h * D + d) = b;
            } else {
                *reinterpret_cast<f32x4 *>(part_o(v, D, out_row, w.split) + d) =
                    f32x4{o[t][4 * q], o[t][4 * q + 1], o[t][4 * q + 2], o[t][4 * q + 3]};
            }
        }
    if (!w.whole && h2 == 0) {
        float *ml = part_ml(v, out_row, w.split);
        ml[0] = m;
        ml[1] = l;
    }
}

// ---------------------------------------------------------------------------
// The same with 16 rows per wave and eight waves, for D = 256: 32 rows' sums
// and q parts leave room for one wave per SIMD only (360 registers), and a
// lone wave issues every other slot and overlaps nothing (a mixed step of
// 2,048 tokens: 71 us against 67 when it was tried; at D = 128, where both fit, a
// prompt of 8,192 tokens took 948 us with 16 rows per wave and 583 with 32).
// Lanes as in the few-rows kernel with 64 keys, operands from the LDS.
// A prompt of 8,192 tokens, 16/4 heads of 256: 598 to 615 us; a mixed step of 2,048:
// 55 to 57 us.  What bounds it are latencies within a tile, which two waves per SIMD
// do not hide: one of the eight waves alone takes three quarters of a tile's time.
// ---------------------------------------------------------------------------
constexpr int kNarrowThreads = 512;
constexpr int kNarrowAhead = 3;

// 16 lanes read the same piece of keys 16 (i / 4) + 4 t + i % 4
template <int D>
__device__ __forceinline__ int k_piece_narrow(int key, int p) {
    static_assert(D >= 128, "");
    constexpr int shift = D == 256 ? 0 : 1;
    return key * (D / 16) + (p ^ (((key & 3) | (key >> 4 & 3) << 2) >> shift));
}

template <int D>
__device__ __forceinline__ void many_rows_narrow(const AttentionArgs &a, const Division &v, int block, int blocks, ManyLds<D> &lds) {
    constexpr int KS = D / 128, DT = D / 16;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int G = a.num_q_heads / a.num_kv_heads;
    ManyShare w;
    if (!many_share(a, v, block, blocks, w)) return;
    const Request &rq = w.rq;
    const int hk = w.hk, k_lo = w.k_lo, k_hi = w.k_hi;
    const int wrow = w.row0 + 16 * wave, row = wrow + c;
    const bool live = row < w.n_rows;
    const int i_row = live ? token_of(row, G) : 0, h = hk * G + (live ? row - i_row * G : 0);
    int jb = 0, je = 0;
    if (live) key_range(a, rq, i_row, jb, je);
    jb = max(jb, k_lo);
    je = min(je, k_hi);
    const WaveKeys wk = wave_keys(a, w, wrow, 16);
    i32x8 qh[KS], ql[KS];
    const Row16<D> q = load_q16<D>(a.q + (long long)(rq.begin + i_row) * a.q_stride + (long long)h * D, g);
    const float up = factor_q16<D>(q), to_log2 = a.scale * kLog2e * (1.f / up);
    split_q16<D>(q, up, qh, ql);
    Staging<D, kNarrowThreads, k_piece_narrow<D>> stage(a, lds, w, wave);
    // this lane's operand rows: the t-th K operand's is 4 t keys further on, with its
    // pieces in the same order, and so the t-th V operand's, 16 t elements
    const int key = 16 * (c >> 2) + (c & 3);
    const int k_row = key * (D / 16), k_swap = k_piece_narrow<D>(key, g) - k_row, v_swap = v_piece(c, g) - 4 * c;

    f32x4 o[DT] = {};
    float m = kNegInf, l = 0.f;
    int j0 = first_tile(k_lo, kTileKeys, 0), buf = 0;
    const bool any = j0 < k_hi;
    if (any) stage.begin(j0);
    for (; j0 < k_hi; j0 += kTileKeys, buf ^= 1) {
        const int jn = j0 + kTileKeys;
        stage.ahead(j0);
        if (j0 < wk.hi && jn > wk.lo) {
            f32x4 x[4] = {}, y[4] = {};
            const uint4 *kt = lds.k[buf] + k_row, *vt = lds.v[buf] + 4 * c + v_swap;
            auto k_operand = [&](int i) {
                const int t = i / KS, st = i % KS;
                const uint4 u = kt[4 * t * (D / 16) + (k_swap ^ 8 * st)], b = kt[4 * t * (D / 16) + (k_swap ^ (8 * st + 4))];
                return i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
            };
            run_ahead<4 * KS, kNarrowAhead>(k_operand, [&](int i, const i32x8 &k8) {
                x[i / KS] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, qh[i % KS], x[i / KS], 0, 0, 0, 0, 0, 0);
                y[i / KS] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k8, ql[i % KS], y[i / KS], 0, 0, 0, 0, 0, 0);
            });
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[t][r] = __builtin_fmaf(y[t][r], 1.f / kLowTimes, x[t][r]);
            const int jg = j0 + 16 * g;
            const bool ok = lds.ok[buf][g] != 0;
            const bool masked = j0 < wk.all0 || jn > wk.all1 || __any(!ok);
            uint32_t pw[8];
            weigh(x, to_log2 * lds.ks[buf][g], lds.vs[buf][g], j0 - k_lo >= kLateKeys, masked, ok, jg, jb, je, m, l, o, pw);
            const bf16x8 p0 = as_bf16x8(pw[0], pw[1], pw[2], pw[3]), p1 = as_bf16x8(pw[4], pw[5], pw[6], pw[7]);
            run_ahead<DT, kNarrowAhead>([&](int t) { return vt[16 * 4 * t]; }, [&](int t, const uint4 &w) {
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(w.x, w.y), p0, o[t], 0, 0, 0);
                o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(w.z, w.w), p1, o[t], 0, 0, 0);
            });
        }
        stage.next(j0, buf);
    }

    if (any && stage.nan_left_out()) {
        unsigned long long bits[1] = {0};
        find_nan<4 * DT>(
            a, hk, first_tile(k_lo, kTileKeys, 0), k_hi, kTileKeys, kTileKeys, jb, je, bits,
            [&](int j) { return stage.late(j, stage.page_at(j + 16 * (lane & 3))); },
            [&](int i) { return 16 * (i >> 2) + 4 * g + (i & 3); }, [&](int j) { return stage.page_at(j); });
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (bits[0] >> (4 * t + r) & 1) o[t][r] = __builtin_bit_cast(float, 0x7fc00000u);
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long out_row = (long long)(rq.begin + i_row) * a.num_q_heads + h;
#pragma unroll
    for (int t = 0; t < DT; ++t) {
        const int d = 16 * t + 4 * g;
        if (w.whole) {
            uint2 b;
            b.x = pack_bf16x2(o[t].x * inv, o[t].y * inv);
            b.y = pack_bf16x2(o[t].z * inv, o[t].w * inv);
            *reinterpret_cast<uint2 *>(a.o + (long long)(rq.begin + i_row) * a.o_stride + (long long)h * D + d) = b;
        } else {
            *reinterpret_cast<f32x4 *>(part_o(v, D, out_row, w.split) + d) = o[t];
        }
    }
    if (!w.whole && g == 0) {
        float *ml = part_ml(v, out_row, w.split);
        ml[0] = m;
        ml[1] = l;
    }
}

// ---------------------------------------------------------------------------
// The kernels: a token per request at most on average (few rows alone, eight
// waves), and else both kinds of requests in one grid -- the large ones'
// workgroups first, those of the small ones (decode rows) take the CUs that
// are left and each that becomes free.
// ---------------------------------------------------------------------------
template <int D>
__global__ __launch_bounds__(512, 2) void attention_few_kernel(AttentionArgs a, Division v) {
    __shared__ FewLds<D, 8> lds;
    few_rows<D, 8, Take::kAll>(a, v, blockIdx.x, lds);
}

constexpr int mixed_threads(int d) { return d == 256 ? kNarrowThreads : kWideThreads; }

template <int D>
__global__ __launch_bounds__(mixed_threads(D), 2) void attention_mixed_kernel(AttentionArgs a, Division few, Division many,
                                                                              int many_blocks) {
    constexpr int W = mixed_threads(D) / 64;
    __shared__ union {
        FewLds<D, W> few;
        ManyLds<D> many;
    } lds;
    const int block = blockIdx.x;
    if (block >= many_blocks) few_rows<D, W, Take::kSmall>(a, few, block - many_blocks, lds.few);
    else if constexpr (D == 256) many_rows_narrow<D>(a, many, block, many_blocks, lds.many);
    else many_rows_wide<D>(a, many, block, many_blocks, lds.many);
}

// ---------------------------------------------------------------------------
// How a call is split.  With at most a token per request on average the
// few-rows kernel takes everything; else it takes the requests of up to
// kSmallRows rows, and the many-rows kernel the others (16 rows of a wave cost
// it as much as 32, and it reads a key once for 128 rows).
//
// Keys are split until there is a workgroup for every CU, two of the wide
// kernel's, which fit a CU together.  Where eight waves share a part's keys it has
// at least kMinChunk (joining costs a launch: 32 decode rows of 1,100 keys take 20.8
// us in one part and 21.6 in two, 16 of 1,500 with heads of 128 15.7 and 17.4), or
// kIdleChunk where three of four CUs had no work else (one row of 4,000 keys: 18.7
// us with 512, 25.3 with 1,024; eight of 1,100: 18.1 and 20.3; four of 2,500 with heads
// of 128: 15.1, 16.7, and 16.9 with 256; not beside prompts, whose rows take longer:
// 300 tokens and five such rows 33.6 and 29.9; five of 40,000 to 131,000 take 206 us in
// parts for 240 CUs and 321 for 120), and kManyChunk where each wave works on
// them all: 300 tokens of three prompts of up to 1,100 tokens, 16/4 heads of 256,
// take 31 us with 256, 38 with 512, 33 with 128 and 51 with 1,024; of 128, 27, 31,
// 32 and 37.  (More workgroups than fit at once, to even out lengths: a mixed
// step of 2,048 tokens took 100 us with two parts and 67 with one, as partial
// sums cost more than the long rows' wait.)
// ---------------------------------------------------------------------------
constexpr int kMinChunk = 1024, kIdleChunk = 512;
constexpr int kManyChunk = 256;

// a mixed workgroup is alone on its CU at D = 256, two of them fit else
static SplitRules rules(int d) {
    return {kMinChunk, kIdleChunk, kManyChunk, mixed_threads(d) / 64, d == 256 ? kCUs : 2 * kCUs};
}

int64_t attention_workspace_bytes(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int d, int max_seq_len) {
    const Plan p = plan_of(rules(d), num_tokens, num_seqs, num_q_heads, num_kv_heads, d, max_seq_len);
    return (p.few.floats + p.many.floats) * 4;
}

template <int D>
static hipError_t launch_d(const AttentionArgs &a, hipStream_t stream) {
    const Plan p = plan_of(rules(D), a.num_tokens, a.num_seqs, a.num_q_heads, a.num_kv_heads, D, a.max_seq_len);
    const long long few = p.few.units * p.few.splits, many = p.many.units * p.many.splits;
    if (few + many > 0x7fffffffLL || p.few.rows > 0x7fffffffLL || p.many.rows > 0x7fffffffLL)
        return hipErrorInvalidConfiguration;
    const Division vf = division(p.few, false, D, a.workspace);
    if (p.few_takes == Take::kAll) {
        hipLaunchKernelGGL((attention_few_kernel<D>), dim3((unsigned)few), dim3(512), 0, stream, a, vf);
        launch_join(Take::kAll, a, p.few, vf, kTileRows, stream);
        return hipGetLastError();
    }
    const Division vm = division(p.many, p.by_rows, D, a.workspace + p.few.floats);
    hipLaunchKernelGGL((attention_mixed_kernel<D>), dim3((unsigned)(few + many)), dim3(mixed_threads(D)), 0, stream, a, vf, vm,
                       (int)many);
    launch_join(Take::kSmall, a, p.few, vf, kTileRows, stream);
    launch_join(Take::kLarge, a, p.many, vm, kManyRows, stream);
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
