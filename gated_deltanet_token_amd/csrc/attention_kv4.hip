// Attention over the 4-bit paged cache (gdn_paged_attention_kv4), gfx950.
//
// Scores are formed transposed, X^T = K Q^T (keys down, rows across), so that
// the exponentials P^T leave the matrix cores in the lanes that the second
// product O^T = V^T P^T wants them in.  A row here is one (token, q head) pair of
// the q heads that share a kv head.
//
// K Q^T runs on the scaled products: a key's codes and the scale of each 32 of
// its elements go into the matrix cores as they lie in memory.  q goes in as
// three e2m3 parts, each with a power of two per 32 elements (split_q): they take
// 48 cycles per 16 keys of 128 elements (two e4m3 parts take 64, bf16 takes 64 and
// the keys' conversion).
//
// V^T P^T runs on bf16: codes are converted in registers (exact), a weight is
// rounded to bf16 with its token's value scale in it: a light key beside a heavy
// one keeps its 8 bits.  Codes are finite whatever they are; a key that a row
// does not see gets a weight of zero there, and so no influence.
// Scores and sums are fp32; the maximum is in units of log2.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "attention_split.h"
#include "fp4.h"

namespace gdn {

typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));
typedef float f32x32 __attribute__((ext_vector_type(32)));
typedef __bf16 bf16x32 __attribute__((ext_vector_type(32)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kE2m1 = 4, kE2m3 = 2;             // operand formats of the scaled products

// Weights are relative to a maximum that is this much (in units of log2) above
// the largest one met when it was set, in all but the first kLateKeys keys of a
// workgroup's part: most tiles have a new maximum for some row of a wave, hardly
// any one above that, and sums follow only then.  (In the first keys the heaviest
// often makes up the sum, and its weight of 1 is exact.)  A weight is never above
// 1, so that no product with a scale passes the values' own range; at the other end a
// product is rounded as a normal number of bf16 from 2^-118 times the heaviest's on.
constexpr float kHeadroom = 8.f;

__device__ __forceinline__ const uint8_t *k_scales(const AttentionArgs &a) { return static_cast<const uint8_t *>(a.k_scale); }
__device__ __forceinline__ const uint16_t *v_scales(const AttentionArgs &a) { return static_cast<const uint16_t *>(a.v_scale); }

__device__ __forceinline__ bf16x8 values8(uint32_t w) { return __builtin_bit_cast(bf16x8, e2m1_bf16(w)); }

// 32 values as e2m3 codes and back, over the power of two s.  These instructions write
// their first results before they have read their last operands.  The compiler keeps them
// apart, but for the one that takes fp32 values, of which it does not know: that one is
// written out, its result declared as early (and with the two wait states that a matrix
// instruction needs behind a vector one; with the values brought to bf16 for the first
// conversion instead a call took 0.2 us more).
__device__ __forceinline__ u32x6 e2m3_codes(const bf16x32 &x, float s) { return __builtin_amdgcn_cvt_scalef32_pk32_fp6_bf16(x, s); }
__device__ __forceinline__ u32x6 e2m3_codes(const f32x16 &even, const f32x16 &odd, float s) {
    u32x6 w;
    asm("v_cvt_scalef32_2xpk16_fp6_f32 %0, %1, %2, %3\n\ts_nop 1" : "=&v"(w) : "v"(even), "v"(odd), "v"(s));
    return w;
}
__device__ __forceinline__ f32x32 e2m3_values(const u32x6 &w, float s) { return __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(w, s); }

// 32 elements of q in three parts, x = s (hi + mid / 32 + lo / 1024), s the power
// of two that brings their largest to [2, 4).  A part has four significant bits and
// steps of 1/8 below 2: exact for elements down to 2^-7 of the largest, and
// within 2^-15 of that for smaller ones.  s is 2^-111 at least, so that lo's steps are
// normal numbers: below a largest of 2^-110 elements are held within 2^-125.  Scale
// bytes: hi's, mid's and lo's.  An infinity or NaN: scales of NaN, as the parts have none.
struct SplitQ {
    u32x6 part[3];
    uint32_t scale;
};
__device__ __forceinline__ SplitQ split_q(const uint4 (&w)[4], uint32_t flip) {
    u32x16 x;
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[4 * i + e] = u[e] ^ flip;
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, u[e] & 0x7fff7fffu));
        }
    }
    const int top = max((int)m[0], (int)m[1]) >> 7;              // the largest one's biased exponent
    const int s = max(top, 17) - 1;                              // 2^-111 at least
    const float s0 = __builtin_bit_cast(float, (uint32_t)s << 23), s1 = __builtin_bit_cast(float, (uint32_t)(s - 5) << 23);
    const float s2 = __builtin_bit_cast(float, (uint32_t)(s - 10) << 23);
    SplitQ q;
    const bf16x32 v = __builtin_bit_cast(bf16x32, x);
    q.part[0] = e2m3_codes(v, s0);
    f32x16 even, odd;
    f32x32 got = e2m3_values(q.part[0], s0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        even[i] = bf16_lo(x[i]) - got[2 * i];
        odd[i] = bf16_hi(x[i]) - got[2 * i + 1];
    }
    q.part[1] = e2m3_codes(even, odd, s1);
    got = e2m3_values(q.part[1], s1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        even[i] -= got[2 * i];
        odd[i] -= got[2 * i + 1];
    }
    q.part[2] = e2m3_codes(even, odd, s2);
    q.scale = top == 255 ? 0xffffffu : (uint32_t)(s | (s - 5) << 8 | (s - 10) << 16);
    return q;
}

__device__ __forceinline__ i32x8 operand(const u32x6 &p) {
    return i32x8{(int)p[0], (int)p[1], (int)p[2], (int)p[3], (int)p[4], (int)p[5], 0, 0};
}
__device__ __forceinline__ i32x8 operand(const uint4 &k) {
    return i32x8{(int)k.x, (int)k.y, (int)k.z, (int)k.w, 0, 0, 0, 0};
}

// A row's parts for waves of 16 rows: a lane's are those of its 32 elements, 128
// st + 32 g on, of step st.  At D = 64 one product takes two parts: groups 0 and 1
// have hi, groups 2 and 3 mid of the same elements, and then lo and zeros.
template <int D>
struct Q16 {
    static constexpr int KS = D >= 128 ? D / 128 : 1, P = D == 64 ? 2 : 3;
    u32x6 part[KS][P];
    uint32_t scale[KS];

    struct Raw {
        uint4 w[KS][4];
    };
    static __device__ __forceinline__ Raw load(const uint16_t *q, int g) {
        Raw r;
#pragma unroll
        for (int st = 0; st < KS; ++st)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.w[st][i] = *reinterpret_cast<const uint4 *>(q + (D == 64 ? 32 * (g & 1) : 128 * st + 32 * g) + 8 * i);
        return r;
    }
    __device__ __forceinline__ void split(const Raw &r, int g, uint32_t flip) {
#pragma unroll
        for (int st = 0; st < KS; ++st) {
            const SplitQ s = split_q(r.w[st], flip);
            if constexpr (D == 64) {
#pragma unroll
                for (int i = 0; i < 6; ++i) {
                    part[0][0][i] = g < 2 ? s.part[0][i] : s.part[1][i];
                    part[0][1][i] = g < 2 ? s.part[2][i] : 0u;
                }
                scale[0] = (s.scale >> (g < 2 ? 0 : 8) & 255) | (s.scale >> 16) << 8;
            } else {
#pragma unroll
                for (int p = 0; p < 3; ++p) part[st][p] = s.part[p];
                scale[st] = s.scale;
            }
        }
    }
};

// x += the products of 16 keys' codes and the row's parts; `ks` has the scales of
// four operands' keys, byte T this one's
template <int T, int D>
__device__ __forceinline__ void score16(f32x4 &x, const uint4 &k, uint32_t ks, const Q16<D> &q, int st) {
    x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(k), operand(q.part[st][0]), x, kE2m1, kE2m3, T, ks, 0, q.scale[st]);
    x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(k), operand(q.part[st][1]), x, kE2m1, kE2m3, T, ks, 1, q.scale[st]);
    if constexpr (D != 64)
        x = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(k), operand(q.part[st][2]), x, kE2m1, kE2m3, T, ks, 2, q.scale[st]);
}

// From products of q and k to scores in units of log2 (their sign is q's).  Not zero: a
// masked score stays at -infinity.  The least number there is instead: products may be
// as large as 2^126, and count for nothing at a scale of zero.
__device__ __forceinline__ float to_log2(float scale) { return fmaxf(fabsf(scale) * kLog2e, 0x1p-149f); }

// The larger of two scores, NaN if one is (the row is, then, whatever its maximum: fmaxf
// would first turn each operand into a quiet one).
__device__ __forceinline__ float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }

// A new maximum of a row and what its sums are multiplied by, where some row of the
// wave is past its own.
__device__ __forceinline__ bool new_maximum(float mx, bool late, float &m, float &f) {
    if (!__any(mx > m)) return false;
    const float m_new = mx > m ? mx + (late ? kHeadroom : 0.f) : m;
    f = m_new == m ? 1.f : __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    return true;
}

// One tile of a wave with 16 rows: the scores x (x[t][r]: key jg + 4 r + t of the
// lane's row) become weights, packed to bf16 pairs in the keys' order with the
// tokens' value scales vs in them; the running maximum m, the lane's sum l and the
// sums o follow.
template <int DT>
__device__ __forceinline__ void weigh16(f32x4 (&x)[4], float factor, float (&vs)[16], bool late, bool masked, bool seen_page, int jg,
                                        int jb, int je, float &m, float &l, f32x4 (&o)[DT], uint32_t (&pw)[8]) {
    if (masked) {
        // from the row's first and past its last key of these, none of a missing page
        const int from = seen_page ? jb - jg : 16, to = je - jg;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * r + t < from || 4 * r + t >= to) {
                    x[t][r] = kNegInf;
                    vs[4 * r + t] = 0.f;
                }
    }
    float mx = kNegInf;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = larger(mx, x[t][r]);
    mx = max_over32(max_over16(mx)) * factor;
    float f;
    if (new_maximum(mx, late, m, f)) {
        l *= f;
#pragma unroll
        for (int t = 0; t < DT; ++t) o[t] *= f;
    }
    const float at = m == kNegInf ? 0.f : m;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int t = 0; t < 4; t += 2) {
            const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][r], factor, -at));
            const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t + 1][r], factor, -at));
            l += e0 + e1;
            pw[2 * r + t / 2] = pack_bf16x2(e0 * vs[4 * r + t], e1 * vs[4 * r + t + 1]);
        }
}

// A row's o from its lane's sums of waves of 16 rows, 8 elements 32 i + 8 g on
// from each pair of them: written out, or as a part's sums.
__device__ __forceinline__ void put8(const AttentionArgs &a, const Division &v, bool whole, float inv, const f32x4 &s0, const f32x4 &s1,
                                     long long token, int h, long long part, int split, int d) {
    const float f[8] = {s0.x, s1.x, s0.y, s1.y, s0.z, s1.z, s0.w, s1.w};
    if (whole) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = f[e] * inv;
        *reinterpret_cast<uint4 *>(a.o + token * a.o_stride + (long long)h * a.d + d) = pack8(y);
    } else {
        float *p = part_o(v, a.d, part, split) + d;
        *reinterpret_cast<f32x4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
    }
}

// ---------------------------------------------------------------------------
// Few rows: one workgroup of W waves per (16 rows of one request that share a
// kv head, split of its keys).  Bound by reading the cache: each wave takes every
// W-th tile of 64 keys straight from HBM into registers in the order of the
// matrix operands (16-byte loads), with the next tile's keys and values on their
// way while it works on this one.  The waves' sums are joined in the LDS.  Of a
// decode step of 32 requests of 1,100 keys (13.6 us) 1.3 us go to the request's
// lengths, 2 to the first tile, 7 to 4.5 tiles of each wave, 1.5 to the join; 192
// requests of 4,096 keys (32/8 heads of 128) take 134 us, 6.3 TB/s.
//
// Lanes: with c = lane % 16 and g = lane / 16, a lane holds row c and the 16
// keys from 16 g on of the tile, a granule of the cache: one page number per
// lane for values, and one for the keys whose codes it loads.  Row i of the t-th K
// operand is key 16 (i / 4) + 4 t + i % 4, so that a load has whole lines of 128
// bytes; a lane's scale of each operand is a byte of another word.  At D = 256, where
// a key is a line and a load has half of it either way, it is key 16 (i / 4) + 4 (i % 4) + t: the
// four operands' scales are neighbouring bytes (64 requests of 1 to 4,000 keys: 32.4 us,
// 34.3 the other way; 100 of 1,000 to 2,000 at D = 64: 24.8, and 23.6 the other way).  Row i of
// the V operands 2 u and 2 u + 1 is element 32 u + 2 i and the one behind it: a 16-byte load has both.
// ---------------------------------------------------------------------------
// one of a kv head's tiles of 16 rows of a request
struct RowTile {
    int lo, hi;              // keys that some row sees
    int x0, x1;              // that every row sees
    int i_row, h;            // the lane's row: its token within the request and q head
    int jb, je;              // the keys that it sees
    bool live;
};
__device__ __forceinline__ RowTile row_tile(const AttentionArgs &a, const Request &rq, int hk, int row0, int c) {
    const int G = a.num_q_heads / a.num_kv_heads, n_rows = rq.n * G;
    RowTile w;
    key_range(a, rq, token_of(row0, G), w.lo, w.x1);
    key_range(a, rq, token_of(last_row(row0, kTileRows, n_rows), G), w.x0, w.hi);
    const int row = row0 + c;
    w.live = row < n_rows;
    w.i_row = w.live ? token_of(row, G) : 0;
    w.h = w.live ? hk * G + row - w.i_row * G : hk * G;
    w.jb = w.je = 0;
    if (w.live) key_range(a, rq, w.i_row, w.jb, w.je);
    return w;
}

// a lane's share of a row tile's sums, of the keys that its wave has taken
template <int D>
struct Sums {
    f32x4 o[D / 16];
    float m, l;              // l: the lane's own keys
};

// The block table's entries for a wave's tile of 64 keys at j: of the keys that the lane
// loads and of the values.
struct Entries {
    int k, v;
};
__device__ __forceinline__ Entries entries_at(const AttentionArgs &a, int s, unsigned j) {
    const int lane = threadIdx.x & 63, shift = __builtin_ctz(a.page);
    const int32_t *bt = a.block_table + s * a.block_table_stride;
    const unsigned last = a.max_pages - 1;
    return {bt[min((j + 16 * (lane >> 2 & 3)) >> shift, last)], bt[min((j + 16 * (lane >> 4)) >> shift, last)]};
}

// 16 bytes of the cache
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint8_t *p) {
    if constexpr (STREAM) return load_stream16(reinterpret_cast<const uint16_t *>(p));
    else return *reinterpret_cast<const uint4 *>(p);
}

// One wave takes the keys [k_lo, k_hi) of a row tile from `first` on, 64 at a time and
// `step` further on the next time, one tile on its way while it works on another.
// `next`: the entries of the first one.
template <int D, bool STREAM>
__device__ __forceinline__ void take_keys(const AttentionArgs &a, int s, const Request &rq, int hk, const RowTile &w, int k_lo, int k_hi,
                                          int first, int step, Entries next, Sums<D> &sum) {
    constexpr int KS = Q16<D>::KS, DT = D / 16;      // DT operands of 16 value elements
    constexpr bool kLines = D != 256;
    constexpr int kRow = kLines ? 1 : 4, kNext = kLines ? 4 : 1;                  // keys from a lane's to the next one's, and to its next
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, kg = c >> 2;
    const int jb = max(w.jb, k_lo), je = min(w.je, k_hi);
    const int in_page = a.page - 1;
    auto good = [&](int p) { return (unsigned)p < (unsigned)a.num_pages; };
    // Entries are loaded a tile ahead of the loads that use them, and not looked at
    // before: loads come back in order, so that looking at one that was asked for
    // behind a tile waits for the tile.  Keys are counted without a sign: a few tiles
    // past the last one may lie past 2^31.  Tiles past it are loaded all the same, from
    // the first page: with their loads under a condition the compiler cannot tell how
    // many are on their way, and waits for all of them before the values of the tile
    // at hand.
    const unsigned end = max(k_hi, 0);
    auto page_of = [&](int entry, unsigned j) { return j < end && good(entry) ? entry : -1; };

    uint4 kr[4][KS], vr[DT / 2], vw[2];
    using Scales = typename std::conditional<kLines, uint4, uint32_t>::type;
    Scales kw[KS];                                   // the keys' scales
    const uint32_t pick = (c & 3) | (4 + (c & 3)) << 8;
    int pv;                                          // the values' page
    // a tile begins at a multiple of 64 keys: places in a page stay the same
    const uint32_t pitch = (uint32_t)(a.num_kv_heads * a.page) * (D / 2);        // bytes of codes, all kv heads
    const uint32_t k_row = hk * a.page + (16 * kg + kRow * (c & 3) & in_page), v_row = hk * a.page + (16 * g & in_page);
    const uint8_t *k_at = a.k_cache + (k_row * (D / 2) + 16 * (D == 64 ? g & 1 : g));
    const uint8_t *ks_at = k_scales(a) + ((hk * (D / 32) + (D == 64 ? g & 1 : g)) * a.page + (16 * kg + (kLines ? 0 : 4 * (c & 3)) & in_page));
    const uint8_t *v_at = a.v_cache + (v_row * (D / 2) + 16 * c);
    const uint8_t *vs_at = reinterpret_cast<const uint8_t *>(v_scales(a) + v_row);
    auto load_k = [&](int page) {
        const uint64_t off = (uint64_t)(uint32_t)max(page, 0) * pitch;
        const uint8_t *p = k_at + off, *sc = ks_at + (off >> 4);                 // (scales: a 16th of the codes)
#pragma unroll
        for (int st = 0; st < KS; ++st) kw[st] = *reinterpret_cast<const Scales *>(sc + 4 * st * a.page);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int st = 0; st < KS; ++st) kr[t][st] = load16<STREAM && kLines>(p + kNext * t * (D / 2) + 64 * st);
    };
    auto load_v = [&]() {
        const uint64_t off = (uint64_t)(uint32_t)max(pv, 0) * pitch;
        const uint4 *sc = reinterpret_cast<const uint4 *>(vs_at + (off >> __builtin_ctz(D / 4)));        // needed before the values
        vw[0] = sc[0];
        vw[1] = sc[1];
        const uint8_t *p = v_at + off;
#pragma unroll
        for (int u = 0; u < DT / 2; ++u) vr[u] = load16<STREAM>(p + 256 * u);
        asm volatile("" ::: "memory");
    };

#pragma unroll
    for (int t = 0; t < DT; ++t) sum.o[t] = f32x4{};
    float m = kNegInf, l = 0.f;
    unsigned j0 = first;
    // a tile's keys, and the entries of the one behind it
    auto turn = [&](unsigned j) {
        const int pk = page_of(next.k, j + 16 * kg);
        pv = page_of(next.v, j + 16 * g);
        load_k(pk);
        next = entries_at(a, s, j + step);
        asm volatile("" ::: "memory");
    };
    // q is asked for before the first tile, and split while that is on its way
    const auto raw = Q16<D>::load(a.q + (long long)(rq.begin + w.i_row) * a.q_stride + (long long)w.h * D, g);
    asm volatile("" ::: "memory");
    turn(j0);
    load_v();
    __builtin_amdgcn_sched_barrier(0);
    Q16<D> q;
    q.split(raw, g, a.scale < 0.f ? 0x80008000u : 0u);
    const float factor = to_log2(a.scale);
    const int all0 = max(w.x0, k_lo), all1 = min(w.x1, k_hi) - kTileKeys;

    for (; j0 < end; j0 += step) {
        f32x4 x[4] = {};
#pragma unroll
        for (int st = 0; st < KS; ++st) {
            uint32_t ks;
            if constexpr (kLines)
                ks = __builtin_amdgcn_perm(__builtin_amdgcn_perm(kw[st].w, kw[st].z, pick),
                                           __builtin_amdgcn_perm(kw[st].y, kw[st].x, pick), 0x05040100u);
            else
                ks = kw[st];
            score16<0>(x[0], kr[0][st], ks, q, st);
            score16<1>(x[1], kr[1][st], ks, q, st);
            score16<2>(x[2], kr[2][st], ks, q, st);
            score16<3>(x[3], kr[3][st], ks, q, st);
        }
        const bool seen_page = good(pv);
        turn(j0 + step);

        const int j = (int)j0;
        const bool masked = __any(!seen_page) || j < all0 || j > all1;
        float vs[16];
        unpack8(vw[0], vs);
        unpack8(vw[1], vs + 8);
        uint32_t pw[8];
        if constexpr (kLines) {
            const f32x4 y[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = f32x4{y[0][t], y[1][t], y[2][t], y[3][t]};
        }
        weigh16(x, factor, vs, j - k_lo >= kLateKeys, masked, seen_page, j + 16 * g, jb, je, m, l, sum.o, pw);
        const bf16x8 p0 = as_bf16x8(pw[0], pw[1], pw[2], pw[3]), p1 = as_bf16x8(pw[4], pw[5], pw[6], pw[7]);
#pragma unroll
        for (int u = 0; u < DT / 2; ++u) {
            sum.o[2 * u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(vr[u].x), p0, sum.o[2 * u], 0, 0, 0);
            sum.o[2 * u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(vr[u].y), p1, sum.o[2 * u], 0, 0, 0);
            sum.o[2 * u + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(vr[u].z), p0, sum.o[2 * u + 1], 0, 0, 0);
            sum.o[2 * u + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(vr[u].w), p1, sum.o[2 * u + 1], 0, 0, 0);
        }
        load_v();
    }
    sum.m = m;
    sum.l = l;
}

// The waves' sums of a row tile, row by row.  Rows are 8 floats longer than they are, so
// that four of them do not begin at the same bank.
template <int D, int W>
struct FewLds {
    float sums[W][16][D + 8];
    float m[W][16], l[W][16];
};

// The request with the r-th most keys, in 64 classes up to max_seq_len, and in order
// within a class: found by a whole workgroup from a histogram, in every one alike.
constexpr int kOrderThreads = 256, kOrdered = 4;        // passes over the requests

struct OrderLds {
    int count[64], wave[kOrdered][kOrderThreads / 64];
    Request request;
    int found;
};
__device__ __forceinline__ int nth_longest(const AttentionArgs &a, int r, OrderLds &lds, Request &rq) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid < 64) lds.count[tid] = 0;
    __syncthreads();
    const float classes = 64.f / (float)a.max_seq_len;
    int part[kOrdered];
    Request own[kOrdered];
#pragma unroll
    for (int i = 0; i < kOrdered; ++i) {
        const int s = i * kOrderThreads + tid;
        part[i] = -1;
        if (s < a.num_seqs) {
            own[i] = request_of(a, s);
            int lo, hi, x;
            key_range(a, own[i], 0, lo, x);
            key_range(a, own[i], max(own[i].n - 1, 0), x, hi);
            const int keys = own[i].n > 0 ? max(hi - lo, 0) : 0;
            part[i] = 63 - (int)fminf(63.f, (float)keys * classes);
            atomicAdd(&lds.count[part[i]], 1);
        }
    }
    __syncthreads();
    const int n = lds.count[lane];
    int up = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int other = __shfl_up(up, d, 64);
        if (lane >= d) up += other;
    }
    const int at = __builtin_ctzll(__ballot(up > r)), left = r - __shfl(up - n, at, 64);
    unsigned long long mine[kOrdered];
#pragma unroll
    for (int i = 0; i < kOrdered; ++i) {
        mine[i] = __ballot(part[i] == at);
        if (lane == 0) lds.wave[i][wave] = __builtin_popcountll(mine[i]);
    }
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int i = 0; i < kOrdered; ++i)
#pragma unroll
        for (int w = 0; w < kOrderThreads / 64; ++w) {
            if (w == wave && part[i] == at && before + __builtin_popcountll(mine[i] & ((1ull << lane) - 1)) == left) {
                lds.request = own[i];
                lds.found = i * kOrderThreads + tid;
            }
            before += lds.wave[i][w];
        }
    __syncthreads();
    rq = lds.request;
    const int s = __builtin_amdgcn_readfirstlane(lds.found);
    __syncthreads();                     // (the LDS has another use behind this)
    return s;
}

template <int D, int W, Take TAKE, bool STREAM = false>
__device__ __forceinline__ void few_rows(const AttentionArgs &a, const Division &v, int block, FewLds<D, W> &lds, OrderLds *order = nullptr) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int G = a.num_q_heads / a.num_kv_heads;
    // rows and workgroups of a launch are fewer than 2^31 (launch_d): 32-bit divisions
    const unsigned unit = (unsigned)block / (unsigned)v.splits;
    const int split = block - (int)(unit * v.splits);
    const int tile = (int)(unit / (unsigned)a.num_kv_heads);
    const int hk = (int)(unit - tile * a.num_kv_heads);
    int within, s;
    Request rq{};
    if constexpr (TAKE == Take::kSmall) {
        // the first tiles, most of them the only ones, first
        within = (unsigned)tile / (unsigned)a.num_seqs;
        s = tile - within * a.num_seqs;
    } else if (tile < a.num_seqs) {
        s = tile;                                    // every request's first tile: no search
        within = 0;
        if (order) s = nth_longest(a, tile, *order, rq);
    } else {
        s = find_request(a, tile - a.num_seqs, G, kTileRows, 0, false, within);
        ++within;
    }
    // without a window the part's first key is known before its request is
    const int start = a.window ? 0 : split * v.chunk + wave * kTileKeys;
    Entries next = entries_at(a, s, start);
    asm volatile("" ::: "memory");
    if (!order || tile >= a.num_seqs) rq = request_of(a, s);
    const int n_rows = rq.n * G;
    if (within < 0 || (long long)within * kTileRows >= n_rows || (TAKE == Take::kSmall && n_rows > kSmallRows)) return;
    const int row0 = within * kTileRows;
    const RowTile w = row_tile(a, rq, hk, row0, c);
    const Splits sp = splits_of(w.lo, w.hi, v.chunk, v.splits);
    if (split != sp.first && (split < sp.first || split > sp.last)) return;
    const bool whole = sp.last <= sp.first;          // no other split: write o itself
    const int k_lo = max(w.lo, split * v.chunk);
    const int k_hi = split == v.splits - 1 ? w.hi : min(w.hi, (split + 1) * v.chunk);
    const int first = first_tile(k_lo, kTileKeys, wave);
    if (first != start) next = entries_at(a, s, first);
    Sums<D> sum;
    take_keys<D, STREAM>(a, s, rq, hk, w, k_lo, k_hi, first, W * kTileKeys, next, sum);

    // join the waves: maxima, then each wave's sums at the common maximum
    float l = sum.l;
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (w.live) {
        float *p = &lds.sums[wave][c][8 * g];
#pragma unroll
        for (int t = 0; t < D / 16; t += 2) {
            const f32x4 s0 = sum.o[t], s1 = sum.o[t + 1];
            *reinterpret_cast<f32x4 *>(p + 16 * t) = f32x4{s0.x, s1.x, s0.y, s1.y};
            *reinterpret_cast<f32x4 *>(p + 16 * t + 4) = f32x4{s0.z, s1.z, s0.w, s1.w};
        }
        if (g == 0) {
            lds.m[wave][c] = sum.m;
            lds.l[wave][c] = l;
        }
    }
    __syncthreads();
    const int rows = min(n_rows - row0, kTileRows), h0 = hk * G;
    for (int i = threadIdx.x; i < rows * (D / 4); i += 64 * W) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float m = kNegInf, all = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) m = fmaxf(m, lds.m[j][r]);
        const float at = m == kNegInf ? 0.f : m;
        f32x4 o = {};
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float f = __builtin_amdgcn_exp2f(lds.m[j][r] - at);
            all += lds.l[j][r] * f;
            o += *reinterpret_cast<const f32x4 *>(&lds.sums[j][r][d]) * f;
        }
        const int row = row0 + r, i_row = token_of(row, G), h = h0 + row - i_row * G;
        if (whole) {
            const float inv = all == 0.f ? 0.f : 1.f / all;
            uint2 y;
            y.x = pack_bf16x2(o.x * inv, o.y * inv);
            y.y = pack_bf16x2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2 *>(a.o + (long long)(rq.begin + i_row) * a.o_stride + (long long)h * D + d) = y;
        } else {
            const long long out_row = part_row<TAKE>(a, s, rq.begin + i_row, h, row, hk);
            *reinterpret_cast<f32x4 *>(part_o(v, D, out_row, split) + d) = o;
            if (d == 0) {
                float *ml = part_ml(v, out_row, split);
                ml[0] = m;
                ml[1] = all;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows: one workgroup of four waves per (128 rows of one request that share a kv
// head, 64 at D = 256, split of its keys).  Tiles of 64 keys and values pass through
// the LDS once for all waves, the next one on its way from HBM to registers
// meanwhile, with one barrier per tile between two buffers.
// Bound by vector arithmetic and what two or three waves per SIMD leave uncovered: of a
// prompt of 8,192 tokens (32/8 heads of 128: 516 us, 1,065 TFLOP/s; of 64: 328; 16/4 of
// 256: 517) the vector unit is busy for 77% of the time, the matrix cores for 45%.  Waves
// that feed the matrix cores go before those that form weights (s_setprio: the same prompt
// at D = 64 333 us without, 29 decode rows with 2,019 tokens at D = 256 40.0 and 37.6 with it).
// What did not help: the values turned to bf16 once, on their way to the LDS (fewer
// conversions, more traffic there: 543 us); q's parts in the LDS for a third wave (666:
// registers spill; at D = 64 341, 336 then without); a tile's scores taken with the weights
// of the tile before (655 and 374: registers).
//
// Keys lie in the LDS as rows of 16-byte pieces (32 elements), values as in
// memory, granule by granule.  The 16 lanes that a 16-byte read serves together are
// lanes 0-3, 12-15 and 20-27 of a half-wave, or the other 16 of it: PLACE puts
// the pieces that they read into 16 different places of the 256 bytes that the
// banks span.  A read of values is of 512 bytes in a row.
// ---------------------------------------------------------------------------
constexpr int kManyThreads = 256;

template <int D>
struct ManyLds {
    uint4 k[kTileKeys * D / 32], v[kTileKeys * D / 32];
    uint2 ks[kTileKeys * D / 128];         // [block of 32 elements][four keys]: their scales; the granule's page, or below 0
    f32x2 vs[kTileKeys / 2];
    uint2 none[2];                         // what no one reads
};

// Staging: D / 2 pieces of 16 bytes of a granule's keys, and as many of its values.  A
// thread has N of each (at D = 64 one of either), each of one granule: the first ones
// also four keys' scales or two values' of the same granule.  As in take_keys, loads are
// without conditions, tiles past the last one come from the first page.
template <int D, int (*PLACE)(int, int)>
struct Staging {
    static constexpr int THREADS = kManyThreads;
    static constexpr int PER = D / 2, PPK = D / 32;
    static constexpr int N = 4 * PER / THREADS > 1 ? 4 * PER / THREADS : 1;
    static constexpr bool BOTH = 4 * PER >= THREADS;
    static_assert((BOTH ? 4 * PER == N * THREADS : 8 * PER == THREADS) && THREADS % PER == 0, "");
    static constexpr int kNext = THREADS / PER;          // a thread's pieces are of every kNext-th granule
    const int32_t *bt;
    int granule, i;
    bool keys, values;
    unsigned end;
    // of a page: bytes of codes, of all kv heads; where the thread's pieces and their scales
    // are (a tile begins at a multiple of 64 keys: the same in every one)
    uint32_t pitch, at[N], sc_at[N], sc_shift, put_at[N];
    const uint8_t *sc_base;
    u32x4 kr[N], vr[N];          // what is on its way
    uint32_t sc[N];
    int entry[N], own[N];        // the block table's entries for the tile behind it, as they came; its pages

    __device__ __forceinline__ Staging(const AttentionArgs &a, const ManyShare &w)
        : bt(a.block_table + w.s * a.block_table_stride), granule((threadIdx.x % (4 * PER)) / PER), i(threadIdx.x % PER),
          keys(BOTH || threadIdx.x < 4 * PER), values(BOTH || threadIdx.x >= 4 * PER), end(max(w.k_hi, 0)),
          pitch((uint32_t)(a.num_kv_heads * a.page) * PER) {
        // key scales are a 16th of the codes, value scales 2 of a token's D / 2 bytes
        const bool of_keys = i < D / 8;
        sc_base = of_keys ? k_scales(a) : reinterpret_cast<const uint8_t *>(v_scales(a));
        sc_shift = of_keys ? 4 : __builtin_ctz(PER / 2);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t in_page = 16 * (granule + n * kNext) & (a.page - 1), row = w.hk * a.page + in_page;
            at[n] = row * PER + 16 * i;
            sc_at[n] = of_keys ? (w.hk * PPK + i / 4) * a.page + in_page + 4 * (i % 4) : 2 * row + 4 * (i % 8);
            const int gr = granule + n * kNext;
            put_at[n] = keys && of_keys           ? offsetof(ManyLds<D>, ks) + 8 * ((i / 4) * 16 + gr * 4 + i % 4)
                        : keys && i < D / 8 + 8 ? offsetof(ManyLds<D>, vs) + 8 * (8 * gr + i - D / 8)
                                                  : offsetof(ManyLds<D>, none);
        }
    }
    __device__ __forceinline__ void pages(const AttentionArgs &a, unsigned j0) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            entry[n] = bt[min((j0 + 16 * (granule + n * kNext)) >> __builtin_ctz(a.page), (unsigned)a.max_pages - 1)];
    }
    __device__ __forceinline__ void load(const AttentionArgs &a, unsigned j0) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const unsigned j = j0 + 16 * (granule + n * kNext);
            own[n] = j < end && (unsigned)entry[n] < (unsigned)a.num_pages ? entry[n] : -1;
            const uint64_t page = (uint64_t)(uint32_t)max(own[n], 0) * pitch;
            if constexpr (BOTH) {
                kr[n] = *reinterpret_cast<const u32x4 *>(a.k_cache + (page + at[n]));
                vr[n] = *reinterpret_cast<const u32x4 *>(a.v_cache + (page + at[n]));
            } else {
                kr[n] = vr[n] = *reinterpret_cast<const u32x4 *>((keys ? a.k_cache : a.v_cache) + (page + at[n]));
            }
            sc[n] = *reinterpret_cast<const uint32_t *>(sc_base + ((page >> sc_shift) + sc_at[n]));
        }
    }
    __device__ __forceinline__ void put(ManyLds<D> &lds) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int gr = granule + n * kNext;
            if (keys) *reinterpret_cast<u32x4 *>(&lds.k[PLACE(16 * gr + i / PPK, i % PPK)]) = kr[n];
            if (values) *reinterpret_cast<u32x4 *>(&lds.v[gr * PER + i]) = vr[n];
            // one store for whatever the thread's scales are, without branches
            const bool of_keys = i < D / 8;
            *reinterpret_cast<uint2 *>(reinterpret_cast<char *>(&lds) + put_at[n]) =
                make_uint2(of_keys ? sc[n] : sc[n] << 16, of_keys ? (uint32_t)own[n] : sc[n] & 0xffff0000u);
        }
    }
};

// ---------------------------------------------------------------------------
// 32 rows per wave, four waves (D = 64 and 128).
//
// Lanes: with c = lane % 32 and h = lane / 32, a lane holds row c and the keys
// 32 h .. 32 h + 31 of the tile, x[b][r] being key 32 h + 2 r + b.  For that, row i
// of the b-th K operand is key 32 (i / 4 % 2) + 8 (i / 8) + 2 (i % 4) + b: the two
// operands' scales are neighbouring bytes.  Row i of the V operands 2 u and 2 u + 1
// is element 64 u + 2 i and the one behind it.
// ---------------------------------------------------------------------------
// 32 lanes read the same piece of keys 32 (c / 4 % 2) + 8 (c / 8) + 2 (c % 4) + b
template <int D>
__device__ __forceinline__ int k_place(int key, int p) {
    // with the tile's key bits 5 .. 0 as (h a1 a0 r1 r0 b), b leads, so that the lanes'
    // rows follow each other
    const int row = (key & 1) << 5 | key >> 1;
    constexpr int shift = D == 64 ? 3 : 2, mask = D / 32 - 1;
    return row * (D / 32) + (p ^ (row >> shift & mask));
}

template <int D>
__device__ __forceinline__ void many_rows_wide(const AttentionArgs &a, const Division &v, int block, int blocks, ManyLds<D> (&lds)[2]) {
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

    // q's parts of step st: elements 64 st + 32 h2 on
    SplitQ q[KS];
    {
        const uint16_t *qp = a.q + (long long)(rq.begin + i_row) * a.q_stride + (long long)h * D + 32 * h2;
#pragma unroll
        for (int st = 0; st < KS; ++st) {
            uint4 e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = *reinterpret_cast<const uint4 *>(qp + 64 * st + 8 * i);
            q[st] = split_q(e, a.scale < 0.f ? 0x80008000u : 0u);
        }
    }
    const float factor = to_log2(a.scale);

    Staging<D, k_place<D>> stage(a, w);
    const int key = 32 * (c >> 2 & 1) + 8 * (c >> 3) + 2 * (c & 3);
    const int k_row = k_place<D>(key, 0) & ~(D / 32 - 1), k_swap = k_place<D>(key, h2) - k_row;
    f32x16 o[DT] = {};
    float m = kNegInf, l = 0.f;
    int j0 = first_tile(k_lo, kTileKeys, 0), buf = 0;
    if (j0 < k_hi) {
        stage.pages(a, j0);
        stage.load(a, j0);
        stage.pages(a, j0 + kTileKeys);
        stage.put(lds[0]);
        __syncthreads();
    }
    for (; j0 < k_hi; j0 += kTileKeys, buf ^= 1) {
        const int jn = j0 + kTileKeys;
        stage.load(a, jn);
        stage.pages(a, jn + kTileKeys);
        __builtin_amdgcn_sched_barrier(0);
        if (j0 < wk.hi && jn > wk.lo) {
            const ManyLds<D> &t = lds[buf];
            const bool ok0 = (int)t.ks[8 * h2].y >= 0, ok1 = (int)t.ks[8 * h2 + 4].y >= 0;
            const bool masked = j0 < wk.all0 || jn > wk.all1 || __any(!(ok0 && ok1)), late = j0 - k_lo >= kLateKeys;
            const uint4 *kt = t.k + k_row, *vt = t.v + h2 * D + c;
            const uint8_t *kst = reinterpret_cast<const uint8_t *>(t.ks) + 2 * (key & ~3) + (key & 3) + 128 * h2;
            f32x16 x[2] = {};
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                const int sc = *reinterpret_cast<const uint16_t *>(kst + 256 * st);
                const uint4 k0 = kt[k_swap ^ 2 * st], k1 = kt[32 * (D / 32) + (k_swap ^ 2 * st)];
                // (the products' operand selections are constants)
                x[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(k0), operand(q[st].part[0]), x[0], kE2m1, kE2m3, 0, sc, 0, q[st].scale);
                x[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(k1), operand(q[st].part[0]), x[1], kE2m1, kE2m3, 1, sc, 0, q[st].scale);
                x[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(k0), operand(q[st].part[1]), x[0], kE2m1, kE2m3, 0, sc, 1, q[st].scale);
                x[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(k1), operand(q[st].part[1]), x[1], kE2m1, kE2m3, 1, sc, 1, q[st].scale);
                x[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(k0), operand(q[st].part[2]), x[0], kE2m1, kE2m3, 0, sc, 2, q[st].scale);
                x[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(k1), operand(q[st].part[2]), x[1], kE2m1, kE2m3, 1, sc, 2, q[st].scale);
            }
            // asked for before the weights are formed: the compiler would read each just before its product
            uint4 w4[2][DT / 2];
#pragma unroll
            for (int i = 0; i < DT; ++i) w4[i / (DT / 2)][i % (DT / 2)] = vt[i / (DT / 2) * (D / 2) + 32 * (i % (DT / 2))];
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            const int jg = j0 + 32 * h2;
            if (masked) {
                // from the row's first and past its last key of these, none of a missing page
                const int from = jb - jg, to = je - jg;
#pragma unroll
                for (int r = 0; r < 16; ++r)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (2 * r + b < from || 2 * r + b >= to || !(r < 8 ? ok0 : ok1)) x[b][r] = kNegInf;
            }
            float mx = kNegInf;
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = larger(larger(mx, x[0][r]), x[1][r]);
            mx = max_over32(mx) * factor;
            float f;
            if (new_maximum(mx, late, m, f)) {
                l *= f;
#pragma unroll
                for (int i = 0; i < DT; ++i) o[i] *= f;
            }
            const float at = m == kNegInf ? 0.f : m;
            f32x4 vs[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) vs[i] = reinterpret_cast<const f32x4 *>(t.vs + 16 * h2)[i];
            if (masked)
#pragma unroll
                for (int r = 0; r < 32; ++r) vs[r / 4][r & 3] = x[r & 1][r / 2] == kNegInf ? 0.f : vs[r / 4][r & 3];
            uint32_t pw[16];
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                const f32x4 s = vs[r / 2];
                const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[0][r], factor, -at));
                const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[1][r], factor, -at));
                const float e2 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[0][r + 1], factor, -at));
                const float e3 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[1][r + 1], factor, -at));
                l += (e0 + e1) + (e2 + e3);
                pw[r] = pack_bf16x2(e0 * s.x, e1 * s.y);
                pw[r + 1] = pack_bf16x2(e2 * s.z, e3 * s.w);
            }
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const bf16x8 p0 = as_bf16x8(pw[8 * b], pw[8 * b + 1], pw[8 * b + 2], pw[8 * b + 3]);
                const bf16x8 p1 = as_bf16x8(pw[8 * b + 4], pw[8 * b + 5], pw[8 * b + 6], pw[8 * b + 7]);
#pragma unroll
                for (int u = 0; u < DT / 2; ++u) {
                    const uint4 &w = w4[b][u];
                    o[2 * u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values8(w.x), p0, o[2 * u], 0, 0, 0);
                    o[2 * u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values8(w.y), p1, o[2 * u], 0, 0, 0);
                    o[2 * u + 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values8(w.z), p0, o[2 * u + 1], 0, 0, 0);
                    o[2 * u + 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values8(w.w), p1, o[2 * u + 1], 0, 0, 0);
                }
            }
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        stage.put(lds[buf ^ 1]);
        __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long token = rq.begin + i_row, out_row = token * a.num_q_heads + h;
    // elements 64 u + 16 i + 8 h2 + 2 r and the one behind it of row c are o[2 u][4 i + r] and o[2 u + 1][4 i + r]
#pragma unroll
    for (int u = 0; u < DT / 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 s0 = {o[2 * u][4 * i], o[2 * u][4 * i + 1], o[2 * u][4 * i + 2], o[2 * u][4 * i + 3]};
            const f32x4 s1 = {o[2 * u + 1][4 * i], o[2 * u + 1][4 * i + 1], o[2 * u + 1][4 * i + 2], o[2 * u + 1][4 * i + 3]};
            put8(a, v, w.whole, inv, s0, s1, token, h, out_row, w.split, 64 * u + 16 * i + 8 * h2);
        }
    if (!w.whole && h2 == 0) {
        float *ml = part_ml(v, out_row, w.split);
        ml[0] = m;
        ml[1] = l;
    }
}

// ---------------------------------------------------------------------------
// 16 rows per wave, for D = 256: 32 rows' sums and q parts leave room for one wave per
// SIMD only (with the parts in the LDS registers spill: a prompt of 8,192, 16/4 heads, takes
// 687 us, 517 so).  Four waves: two workgroups on a CU do not wait for each other (eight
// waves of 128 rows: 555).  Lanes as in the few-rows kernel, operands from the LDS.
// ---------------------------------------------------------------------------
constexpr int kNarrowRows = 64;

// 16 lanes read the same piece of keys 16 (c / 4) + 4 (c % 4) + t
template <int D>
__device__ __forceinline__ int k_place_narrow(int key, int p) {
    static_assert(D == 256, "");
    // key bit 2 leads within eight keys, so that the lanes' rows are even and odd
    const int row = (key & ~7) | (key & 3) << 1 | (key >> 2 & 1);
    return row * 8 + (p ^ ((key >> 5 & 1) << 1 | (key >> 3 & 1) << 2));
}

template <int D>
__device__ __forceinline__ void many_rows_narrow(const AttentionArgs &a, const Division &v, int block, int blocks, ManyLds<D> (&lds)[2]) {
    constexpr int KS = D / 128, DT = D / 16;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int G = a.num_q_heads / a.num_kv_heads;
    ManyShare w;
    if (!many_share<kNarrowRows>(a, v, block, blocks, w)) return;
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
    Q16<D> q;
    q.split(Q16<D>::load(a.q + (long long)(rq.begin + i_row) * a.q_stride + (long long)h * D, g), g, a.scale < 0.f ? 0x80008000u : 0u);
    const float factor = to_log2(a.scale);

    Staging<D, k_place_narrow<D>> stage(a, w);
    const int key = 16 * (c >> 2) + 4 * (c & 3);
    const int k_row = k_place_narrow<D>(key, 0) & ~7, k_swap = k_place_narrow<D>(key, g) & 7;
    f32x4 o[DT] = {};
    float m = kNegInf, l = 0.f;
    int j0 = first_tile(k_lo, kTileKeys, 0), buf = 0;
    if (j0 < k_hi) {
        stage.pages(a, j0);
        stage.load(a, j0);
        stage.pages(a, j0 + kTileKeys);
        stage.put(lds[0]);
        __syncthreads();
    }
    for (; j0 < k_hi; j0 += kTileKeys, buf ^= 1) {
        const int jn = j0 + kTileKeys;
        stage.load(a, jn);
        stage.pages(a, jn + kTileKeys);
        __builtin_amdgcn_sched_barrier(0);
        if (j0 < wk.hi && jn > wk.lo) {
            const ManyLds<D> &tile = lds[buf];
            const bool ok = (int)tile.ks[4 * g].y >= 0;
            const bool masked = j0 < wk.all0 || jn > wk.all1 || __any(!ok);
            const uint4 *kt = tile.k + k_row, *vt = tile.v + g * (D / 2) + c;
            f32x4 x[4] = {};
            __builtin_amdgcn_s_setprio(1);
            uint4 kr[KS][4];
            uint32_t ks[KS];
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                ks[st] = tile.ks[16 * (4 * st + g) + key / 4].x;
#pragma unroll
                for (int t = 0; t < 4; ++t) kr[st][t] = kt[2 * t * 8 + (k_swap ^ 4 * st)];       // (key t is row 2 t of these eight)
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int st = 0; st < KS; ++st) {
                score16<0>(x[0], kr[st][0], ks[st], q, st);
                score16<1>(x[1], kr[st][1], ks[st], q, st);
                score16<2>(x[2], kr[st][2], ks[st], q, st);
                score16<3>(x[3], kr[st][3], ks[st], q, st);
            }
            // asked for before the weights are formed: the compiler would read each just before its product
            uint4 w4[DT / 2];
#pragma unroll
            for (int u = 0; u < DT / 2; ++u) w4[u] = vt[16 * u];
            float vs[16];
            const f32x4 *vst = reinterpret_cast<const f32x4 *>(tile.vs + 8 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 s = vst[i];
                vs[4 * i] = s.x;
                vs[4 * i + 1] = s.y;
                vs[4 * i + 2] = s.z;
                vs[4 * i + 3] = s.w;
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(0);
            uint32_t pw[8];
            weigh16(x, factor, vs, j0 - k_lo >= kLateKeys, masked, ok, j0 + 16 * g, jb, je, m, l, o, pw);
            __builtin_amdgcn_s_setprio(1);
            const bf16x8 p0 = as_bf16x8(pw[0], pw[1], pw[2], pw[3]), p1 = as_bf16x8(pw[4], pw[5], pw[6], pw[7]);
#pragma unroll
            for (int u = 0; u < DT / 2; ++u) {
                const uint4 &w = w4[u];
                o[2 * u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(w.x), p0, o[2 * u], 0, 0, 0);
                o[2 * u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(w.y), p1, o[2 * u], 0, 0, 0);
                o[2 * u + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(w.z), p0, o[2 * u + 1], 0, 0, 0);
                o[2 * u + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values8(w.w), p1, o[2 * u + 1], 0, 0, 0);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        stage.put(lds[buf ^ 1]);
        __syncthreads();
    }

    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long token = rq.begin + i_row, out_row = token * a.num_q_heads + h;
#pragma unroll
    for (int t = 0; t < DT; t += 2) put8(a, v, w.whole, inv, o[t], o[t + 1], token, h, out_row, w.split, 16 * t + 8 * g);
    if (!w.whole && g == 0) {
        float *ml = part_ml(v, out_row, w.split);
        ml[0] = m;
        ml[1] = l;
    }
}

// ---------------------------------------------------------------------------
// The kernels: a token per request at most on average (few rows alone), and else
// both kinds of requests in one grid.  The workgroups of the kind of which there is more
// go first, the others take the CUs that are left and each that becomes free.
// ---------------------------------------------------------------------------
template <int D, int W, bool STREAM>
__global__ __launch_bounds__(64 * W, 2) void attention_few_kv4_kernel(AttentionArgs a, Division v, bool ordered) {
    __shared__ union {
        FewLds<D, W> few;
        OrderLds order;
    } lds;
    few_rows<D, W, Take::kAll, STREAM>(a, v, blockIdx.x, lds.few, ordered ? &lds.order : nullptr);
}

constexpr int many_rows(int d) { return d == 256 ? kNarrowRows : kManyRows; }

template <int D, bool STREAM>
__global__ __launch_bounds__(kManyThreads, 2) void attention_mixed_kv4_kernel(AttentionArgs a, Division few, Division many,
                                                                              int few_blocks, int many_blocks, bool few_first) {
    constexpr int W = kManyThreads / 64;
    __shared__ union {
        FewLds<D, W> few;
        ManyLds<D> many[2];
    } lds;
    const int block = (int)blockIdx.x - (few_first ? few_blocks : 0), few_block = block + (few_first ? few_blocks : -many_blocks);
    if (few_first ? block < 0 : block >= many_blocks) few_rows<D, W, Take::kSmall, STREAM>(a, few, few_block, lds.few);
    else if constexpr (D == 256) many_rows_narrow<D>(a, many, block, many_blocks, lds.many);
    else many_rows_wide<D>(a, many, block, many_blocks, lds.many);
}

// A decode call's keys are split until there is a workgroup for every CU, into
// parts of 1,024 keys or more, or of 512 where three of four CUs are idle (one
// request of 4,000 keys, 16/4 heads of 256: 14.5 us, 10 and 5 to join the parts).
constexpr int kMinChunk = 1024, kIdleChunk = 512, kManyChunk = 256;
static SplitRules rules(int d) {
    return {kMinChunk, kIdleChunk, kManyChunk, kManyThreads / 64, 2 * kCUs, many_rows(d)};
}

// Workgroups of four waves: two of them on a CU, one of which streams while the other begins or
// ends (200 requests of 1 to 8,000 keys, 32/8 heads of 128: 150 us, 158 with eight waves; 32
// of 1,100, 16/4 of 256: 13.5, 14.4).  Of eight where parts are long and there is one for
// a CU at most (five of 40,000 to 131,000: 96 us, 137 with four; eight of up to
// 30,000: 36.5 and 50).
constexpr int kLongPart = 2048;
// Longest requests first where there are two rounds of workgroups and more: the last ones
// then end together (200 requests of 1 to 8,000 keys, 32/8 heads of 128: 150 us, 165 in
// order; 192 of 4,096 each: 137 and 133).  Finding its request costs a workgroup 1.9 us (100
// requests of 1,000 to 2,000, 32/8 of 64, in one round: 27.8 us, 24.7 in order).
constexpr int kManyUnits = 4 * kCUs;

int64_t attention_kv4_workspace_bytes(int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int d, int max_seq_len) {
    const Plan p = plan_of(rules(d), num_tokens, num_seqs, num_q_heads, num_kv_heads, d, max_seq_len);
    return (p.few.floats + p.many.floats) * 4;
}

// Streaming loads of few rows' keys and values where a call may read more of the cache
// than this: what is kept is of no use, and is kept at the expense of what is still to be
// read (200 requests of 1 to 8,000 keys, 32/8 heads of 128, 953 MB: 151 us, 170 with ordinary
// loads; five of 40,000 to 131,000, 577 MB: 96 and 107; 150 of 4,000 to 8,000 beside a chunk
// of 512: 186 and 203).  Smaller caches are still there in the next step (32 requests of
// 1,100, 16/4 of 256, 38 MB each, three sets of inputs in turn: 16.1 us, 13.5 with ordinary ones).
constexpr double kStreamed = 1 << 27;

template <int D, bool STREAM>
static void launch_few(const AttentionArgs &a, const Launch &few, const Division &v, hipStream_t stream) {
    const dim3 grid((unsigned)(few.units * few.splits));
    if (few.splits > 1 && few.chunk >= kLongPart)
        hipLaunchKernelGGL((attention_few_kv4_kernel<D, 8, STREAM>), grid, dim3(512), 0, stream, a, v, false);
    else
        hipLaunchKernelGGL((attention_few_kv4_kernel<D, 4, STREAM>), grid, dim3(kOrderThreads), 0, stream, a, v,
                           (long long)a.num_tokens * a.num_kv_heads > kManyUnits && a.num_seqs <= kOrdered * kOrderThreads);
}

template <int D>
static hipError_t launch_d(const AttentionArgs &a, hipStream_t stream) {
    const Plan p = plan_of(rules(D), a.num_tokens, a.num_seqs, a.num_q_heads, a.num_kv_heads, D, a.max_seq_len, a.window);
    const long long few = p.few.units * p.few.splits, many = p.many.units * p.many.splits;
    if (few + many > 0x7fffffffLL || p.few.rows > 0x7fffffffLL || p.many.rows > 0x7fffffffLL)
        return hipErrorInvalidConfiguration;
    const Division vf = division(p.few, false, D, a.workspace);
    // the most that the call can see: the requests' keys, or every page
    const double keys = a.window > 0 && a.window < a.max_seq_len ? a.window : a.max_seq_len;
    const double seen = std::min(a.num_seqs * keys, (double)a.num_pages * a.page) * a.num_kv_heads * (D + D / 32 + 2);
    if (p.few_takes == Take::kAll) {
        if (seen > kStreamed) launch_few<D, true>(a, p.few, vf, stream);
        else launch_few<D, false>(a, p.few, vf, stream);
        launch_join(Take::kAll, a, p.few, vf, kTileRows, stream);
        return hipGetLastError();
    }
    const Division vm = division(p.many, p.by_rows, D, a.workspace + p.few.floats);
    const dim3 grid((unsigned)(few + many)), block(kManyThreads);
    // small requests first where they are more than the large ones' row tiles: 150 of 4,000 to
    // 8,000 keys and a chunk of 512, 32/8 heads of 128: 177 us, 185 the other way; 29 of 1,100 and 300
    // tokens, 16/4 of 256: 23.9 and 26.3; but 20 of 1,100 and 1,800 tokens, 32/8 of 128: 33.2, 29.5 so
    const bool few_first = (long long)a.num_tokens * (a.num_q_heads / a.num_kv_heads) / many_rows(D) < a.num_seqs;
    const auto kernel = seen > kStreamed ? attention_mixed_kv4_kernel<D, true> : attention_mixed_kv4_kernel<D, false>;
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, vf, vm, (int)few, (int)many, few_first);
    launch_join(Take::kSmall, a, p.few, vf, kTileRows, stream);
    launch_join(Take::kLarge, a, p.many, vm, many_rows(D), stream);
    return hipGetLastError();
}

hipError_t launch_attention_kv4(const AttentionArgs &a, hipStream_t stream) {
    switch (a.d) {
        case 64: return launch_d<64>(a, stream);
        case 128: return launch_d<128>(a, stream);
        case 256: return launch_d<256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
