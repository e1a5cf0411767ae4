// Rotary positions on q and k, and the new k and v written into the 8-bit
// paged cache (gdn_rope_append_kv8), gfx950.
//
// Rotation: (a, b) -> m (a cos t - b sin t, b cos t + a sin t), t = position *
// frequency, in 64 bits.  The angle is taken in turns, so that only its
// fraction reaches sincospi.  Sines and cosines are formed once per token and
// pair in the LDS and used by every head that the workgroup rotates.
//
// Cache: the scale of a (page, kv head) covers all of its tokens, so one wave
// owns a page's new tokens of one head, k or v: it finds their largest
// magnitude, settles the scale, rounds the older codes again if the scale
// grew, and writes.  No two waves share a page and head, so there are no
// atomics, and results do not depend on order.
//
// The first of a page's new tokens stands for them: every window of tokens has
// its workgroups, which look for such tokens in it and end where there are
// none.  That needs no list of pages and no request boundaries.
//
// Bound by HBM for prompts (q in and out, k and v in, codes out) and by the
// 64-bit sines, by latency for decode rows.  Measured: 32 decode rows, 16/4 heads
// of 256 with 64 elements rotated: 7.3 us; 2,048 tokens, of prompts and decode
// rows: 19.1 us, 2.4 TB/s; 16,384 tokens, 32/8 heads of 128, all rotated: 101 us, 3.7
// TB/s.
#include "fp8.h"
#include "rope.h"

namespace gdn {

constexpr int kAppendThreads = 256;
constexpr int kAppendWaves = kAppendThreads / 64;
constexpr int kGranule = 16;            // a page's tokens that are one 16-byte store of an element of v

// a pair's cosine and sine, times the rope scale
struct CosSin {
    double c, s;
};

// those of tokens [t0, t0 + n), n <= 16, into cs[n][half]
__device__ __forceinline__ void fill_cos_sin(const RopeAppendArgs &a, CosSin *cs, long long t0, int n) {
    const int half = a.rot / 2, across = half > 32 ? 64 : 32;       // lanes per token
    if (half == 0) return;
    // one load brings every token's position; the loop's lanes take theirs from there
    const int pos = a.positions[t0 + min((int)(threadIdx.x & 15), n - 1)];
    for (int p = threadIdx.x & (across - 1); p - (int)(threadIdx.x & (across - 1)) < half; p += across) {
        const double f = a.freq[min(p, half - 1)];
#pragma unroll 1
        for (int t = threadIdx.x / across; t < n; t += kAppendThreads / across) {
            double s, c;
            sin_cos_turns((double)__shfl(pos, t, 64) * f * 0.15915494309189533577, s, c);
            if (p < half) cs[t * half + pair_at(a, p)] = {a.rope_scale * c, a.rope_scale * s};
        }
    }
}

// the eight elements (e0 < rot), rotated; `cs` of their token
__device__ __forceinline__ void rotated(const RopeAppendArgs &a, const Raw &r, int e0, const CosSin *cs, float (&f)[8]) {
    unpack8(r.own, f);
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i == 2) asm volatile("" ::: "memory");     // the second half's sines are read after the first is done with
            const CosSin w = cs[i * (a.rot / 8) + e0 / 8];
            const double x = f[2 * i], y = f[2 * i + 1];
            f[2 * i] = (float)(x * w.c - y * w.s);
            f[2 * i + 1] = (float)(y * w.c + x * w.s);
        }
    } else {
        const int half = a.rot / 2;
        const bool first = e0 < half;
        const int p0 = first ? e0 : e0 - half;
        const uint32_t turn = first ? 0x80008000u : 0u;
        float g[8];
        unpack8(make_uint4(r.other.x ^ turn, r.other.y ^ turn, r.other.z ^ turn, r.other.w ^ turn), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i % 4 == 0) asm volatile("" ::: "memory");
            const CosSin w = cs[i * (half / 8) + p0 / 8];
            const double x = f[i], y = g[i];          // the first of a pair meets -b
            f[i] = (float)(x * w.c + y * w.s);
        }
    }
}

// Largest finite magnitudes.  The bits of a magnitude order as integers, and
// with one more in the exponent infinities and NaN become negative ones: a
// signed maximum passes over them.  Kept in that form until the end.
constexpr int kNoMagnitude = 0x00800000;                       // of a zero
__device__ __forceinline__ int magnitude_max(int m, float x) {
    return max(m, (int)((__builtin_bit_cast(uint32_t, x) & 0x7fffffffu) + 0x00800000u));
}
__device__ __forceinline__ float magnitude(int m) { return __builtin_bit_cast(float, m - 0x00800000); }

// the same of bf16 pairs, in the two halves
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ i16x2 magnitude_max(i16x2 m, uint32_t w) {
    const u16x2 y = __builtin_bit_cast(u16x2, w & 0x7fff7fffu) + u16x2{0x0080, 0x0080};
    return __builtin_elementwise_max(m, __builtin_bit_cast(i16x2, y));
}
__device__ __forceinline__ i16x2 magnitude_max(i16x2 m, const uint4 &w) {
    return magnitude_max(magnitude_max(magnitude_max(magnitude_max(m, w.x), w.y), w.z), w.w);
}
__device__ __forceinline__ int magnitude_max(int m, i16x2 x) { return max(m, (int)max(x[0], x[1]) << 16); }
constexpr i16x2 kNoMagnitudes = {0x0080, 0x0080};

__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = max(x, __shfl_xor(x, d, 64));
    return x;
}

// The scale for a page whose new elements reach `amax` and begin at offset
// `off`, `old` the one it has; stores it, and returns what older codes are to
// be multiplied by (1: nothing to do) and its inverse.
__device__ __forceinline__ float settle_scale(float *scale, float old, float amax, int off, float &inv) {
    const float fit = e4m3_block_scale(amax);
    float now = fit, ratio = 1.f;
    if (off > 0) {
        now = fmaxf(old, fit);
        if (now != old) ratio = old / now;
    }
    if ((threadIdx.x & 63) == 0) *scale = now;
    inv = 1.f / now;               // exact: a power of two
    return ratio;
}

// One wave's share of a page: its new tokens of one k head, 16 at a time.  The
// elements that turn go through the wave's part of the LDS, where a token has
// `rot` words: first its bf16 elements, then in their place the rotated ones in
// fp32.  Lanes go over them without gaps (`across` lanes of eight elements per
// token, a power of two), so that a head of which a quarter turns costs a
// quarter; a token's lanes read it before any of them writes.  The other
// elements stay in registers.  Loops are not unrolled: a wave comes by once or
// twice, and what it runs has to be fetched first.
template <int D>
struct KeyPart {
    static constexpr int LPT = D / 8, TPI = 64 / LPT, ITER = kGranule / TPI;
    float *turned;                 // [16][rot]
    int across;
    uint4 w[ITER];

    // tokens i0 .. i0 + 15 of the run (zeros past its last one)
    __device__ __forceinline__ void load(const Rows &src, int i0) {
        const int lane = threadIdx.x & 63, e0 = (lane % LPT) * 8, sub = lane / LPT;
#pragma unroll
        for (int it = 0; it < ITER; ++it) w[it] = src.load16(i0 + it * TPI + sub, e0);
    }
    // the n of them, rotated; their largest finite magnitude, or m
    __device__ __forceinline__ int turn(const RopeAppendArgs &a, const CosSin *cs, int n, int m) const {
        const int lane = threadIdx.x & 63, e0 = (lane % LPT) * 8, sub = lane / LPT, half = a.rot / 2;
        if (e0 < a.rot) {
#pragma unroll
            for (int it = 0; it < ITER; ++it)
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(turned + (it * TPI + sub) * a.rot) + e0) = w[it];
        } else {
            i16x2 x = kNoMagnitudes;
#pragma unroll
            for (int it = 0; it < ITER; ++it) x = magnitude_max(x, w[it]);
            m = magnitude_max(m, x);
        }
        wave_sync();
        const int r0 = (lane & (across - 1)) * 8;
        if (r0 < a.rot)
#pragma unroll 1
            for (int i = lane / across; i < n; i += 64 / across) {
                float *t = turned + i * a.rot, f[8];
                const Raw r = load_raw(a, reinterpret_cast<const uint16_t *>(t), r0);
                wave_sync();
                rotated(a, r, r0, cs + i * half, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) m = magnitude_max(m, f[e]);
                *reinterpret_cast<f32x4 *>(t + r0) = f32x4{f[0], f[1], f[2], f[3]};
                *reinterpret_cast<f32x4 *>(t + r0 + 4) = f32x4{f[4], f[5], f[6], f[7]};
            }
        wave_sync();
        return m;
    }
    // their codes to dst
    __device__ __forceinline__ void store(const RopeAppendArgs &a, uint8_t *dst, int n, float inv) const {
        const int lane = threadIdx.x & 63, e0 = (lane % LPT) * 8, sub = lane / LPT;
        auto put = [&](int i, const float (&f)[8]) {
            uint2 c;
            c.x = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            c.y = e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
            *reinterpret_cast<uint2 *>(dst + i * D + e0) = c;
        };
        if (e0 < a.rot) {
#pragma unroll 1
            for (int i = sub; i < n; i += TPI) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(turned + i * a.rot + e0);
                const f32x4 y = *reinterpret_cast<const f32x4 *>(turned + i * a.rot + e0 + 4);
                const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                put(i, f);
            }
        } else {
#pragma unroll
            for (int it = 0; it < ITER; ++it) {
                float f[8];
                unpack8(w[it], f);
                if (it * TPI + sub < n) put(it * TPI + sub, f);
            }
        }
        wave_sync();
    }
};

// the first `bytes` codes at `dst` (a multiple of 64), at a larger scale
__device__ __forceinline__ void rescale_codes(uint8_t *dst, int bytes, float ratio) {
#pragma unroll 1
    for (int i = (threadIdx.x & 63) * 16; i < bytes; i += 64 * 16) {
        uint4 w = *reinterpret_cast<const uint4 *>(dst + i);
        w.x = e4m3_rescaled(w.x, ratio);
        w.y = e4m3_rescaled(w.y, ratio);
        w.z = e4m3_rescaled(w.z, ratio);
        w.w = e4m3_rescaled(w.w, ratio);
        *reinterpret_cast<uint4 *>(dst + i) = w;
    }
}

// The same of one v head, 16 tokens of the page at a time.  A lane takes eight
// elements of four tokens, codes them, and puts each element's four codes
// into the wave's part of the LDS, where an element's 16 codes come together
// for one 16-byte store.
template <int D>
struct ValuePart {
    static constexpr int LPT = D / 8, TG = 64 / LPT < 4 ? 64 / LPT : 4, ITER = 4 / TG;
    uint32_t *tile;                // [D][4] words of four codes
    uint4 raw[ITER][4];

    // granule g of the page (zeros where the run has no token)
    __device__ __forceinline__ void load(const Rows &src, int g, int off) {
        const int lane = threadIdx.x & 63, e0 = (lane % LPT) * 8, tg = lane / LPT % TG;
#pragma unroll
        for (int it = 0; it < ITER; ++it)
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[it][i] = src.load16(g * kGranule + 4 * (it * TG + tg) + i - off, e0);
    }
    __device__ __forceinline__ int amax(int m) const {
        i16x2 x = kNoMagnitudes;
#pragma unroll
        for (int it = 0; it < ITER; ++it)
#pragma unroll
            for (int i = 0; i < 4; ++i) x = magnitude_max(x, raw[it][i]);
        return magnitude_max(m, x);
    }
    // granule g: its new codes, older ones at the new scale, the rest as it is
    __device__ __forceinline__ void store(uint8_t *head, int page, int off, int g, int n, float inv, float ratio) const {
        const int lane = threadIdx.x & 63, e0 = (lane % LPT) * 8, tg = lane / LPT % TG;
        const int lo = off - g * kGranule, hi = lo + n;     // the granule's new tokens: [lo, hi)
        if (lane < LPT * TG)
#pragma unroll
            for (int it = 0; it < ITER; ++it) {
                float f[4][8];
#pragma unroll
                for (int i = 0; i < 4; ++i) unpack8(raw[it][i], f[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    tile[(e0 + e) * 4 + it * TG + tg] = e4m3x4(f[0][e] * inv, f[1][e] * inv, f[2][e] * inv, f[3][e] * inv);
            }
        wave_sync();
#pragma unroll 1
        for (int d = lane; d < D; d += 64) {
            uint4 w = *reinterpret_cast<const uint4 *>(tile + d * 4);
            uint4 *dst = reinterpret_cast<uint4 *>(head + d * page + g * kGranule);
            if (lo > 0 || hi < kGranule) {
                const uint4 o = *dst;
                w.x = merged(w.x, o.x, lo, hi, ratio);
                w.y = merged(w.y, o.y, lo - 4, hi - 4, ratio);
                w.z = merged(w.z, o.z, lo - 8, hi - 8, ratio);
                w.w = merged(w.w, o.w, lo - 12, hi - 12, ratio);
            }
            *dst = w;
        }
        wave_sync();
    }
    // a word's bytes [lo, hi) from `fresh`; of `old` the others, those below lo at the new scale
    static __device__ __forceinline__ uint32_t merged(uint32_t fresh, uint32_t old, int lo, int hi, float ratio) {
        const uint32_t older = below(lo), mine = below(hi) & ~older;
        if (ratio != 1.f) old = (e4m3_rescaled(old, ratio) & older) | (old & ~older);
        return (fresh & mine) | (old & ~mine);
    }
    // the lowest n bytes of a word
    static __device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 4 ? ~0u : (1u << (8 * n)) - 1u; }
};

template <int D>
__global__ __launch_bounds__(kAppendThreads, D == 256 ? 3 : 4) void rope_append_kernel(RopeAppendArgs a, int append_blocks, int ranks,
                                                                        int groups, int q_tokens) {
    extern __shared__ CosSin cs[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // (scalar addresses)
    const int half = a.rot / 2;
    int across = 1;                                   // lanes per token over the rotated elements
    while (across * 8 < a.rot) across *= 2;

    if ((int)blockIdx.x >= append_blocks) {
        // q of q_tokens tokens: a lane per eight elements that turn, two heads
        // in hand and the next two on their way; then the others, copied
        constexpr int LPT = D / 8, TPI = 64 / LPT, UNROLL = 2;
        const long long t0 = (long long)(blockIdx.x - append_blocks) * q_tokens;
        const int n = (int)min((long long)q_tokens, a.num_tokens - t0), rows = n * a.num_q_heads;
        const int e0 = (lane & (across - 1)) * 8, step = kAppendThreads / across;
        const bool turns = e0 < a.rot;
        auto load = [&](int i0, Raw (&r)[UNROLL]) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int i = min(i0 + u * step, rows - 1), t = (unsigned)i / (unsigned)a.num_q_heads, h = i - t * a.num_q_heads;
                r[u] = load_raw(a, a.q + (t0 + t) * a.q_stride + (long long)h * D, e0);
            }
        };
        int i0 = threadIdx.x / across;
        Raw now[UNROLL], next[UNROLL];
        if (turns) load(i0, now);
        fill_cos_sin(a, cs, t0, n);
        __syncthreads();
        if (turns)
            for (; i0 < rows; i0 += UNROLL * step) {
                if (i0 + UNROLL * step < rows) load(i0 + UNROLL * step, next);
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    const int i = i0 + u * step;
                    if (i >= rows) continue;
                    const int t = (unsigned)i / (unsigned)a.num_q_heads, h = i - t * a.num_q_heads;
                    float f[8];
                    rotated(a, now[u], e0, cs + t * half, f);
                    *reinterpret_cast<uint4 *>(a.q_out + (t0 + t) * a.q_out_stride + (long long)h * D + e0) = pack8(f);
                    now[u] = next[u];
                }
            }
        const int c0 = (lane % LPT) * 8;
        if (a.q != a.q_out && c0 >= a.rot)
#pragma unroll 4
            for (int i = wave * TPI + lane / LPT; i < rows; i += kAppendWaves * TPI) {
                const int t = (unsigned)i / (unsigned)a.num_q_heads, h = i - t * a.num_q_heads;
                *reinterpret_cast<uint4 *>(a.q_out + (t0 + t) * a.q_out_stride + (long long)h * D + c0) =
                    *reinterpret_cast<const uint4 *>(a.q + (t0 + t) * a.q_stride + (long long)h * D + c0);
            }
        return;
    }

    // a window is as many tokens as a page holds; the block takes the rank-th,
    // (rank + ranks)-th ... of the window's tokens that stand for their page,
    // the first of its new ones.  Rank 0 of all windows comes first, v's heads
    // before k's, and ranks are shifted against each other, so that the blocks with
    // work are spread over the XCDs and CUs whatever their spacing.  (The heads of a
    // window next to each other give an XCD nothing but k, or v: 16,384 tokens took
    // 103.5 us and 4,000 decode rows 109, 100.6 and 99 so.)
    const int shift = __builtin_ctz(a.page);
    const unsigned windows = ((unsigned)a.num_tokens + a.page - 1) >> shift, parts = 2 * groups;
    const unsigned unit = blockIdx.x / windows;
    const int rank = (int)(unit / parts), part = (int)(parts - 1 - (unit - rank * parts));
    const int w0 = (int)((blockIdx.x + 5 * rank) % windows);
    const long long slots = (long long)a.num_pages * a.page;
    const int first = w0 * a.page;
    // the slots of the window's tokens and of as many behind them (a page's run
    // may reach there), and which of them continue their predecessor's
    auto slot_at = [&](int t) { return t >= 0 && t < a.num_tokens ? a.slots[t] : -2; };
    const long long mine = slot_at(first + lane), behind = slot_at(first + 64 + lane);
    const bool on = mine == slot_at(first + lane - 1) + 1;
    const unsigned long long on0 = __ballot(on), on1 = __ballot(behind == slot_at(first + 63 + lane) + 1);
    const bool leads = lane < a.page && mine >= 0 && mine < slots && (!on || (mine & (a.page - 1)) == 0);
    unsigned long long todo = __ballot(leads);
    const bool is_k = part < groups;
    const int item = (is_k ? part : part - groups) * kAppendWaves + wave;
    const bool live = item < a.num_kv_heads;
    const int head = live ? item : 0;
    // the next page of the block: its new tokens t .. t + n, from offset off on
    int skip = rank, t, n, off;
    long long ph;
    auto next_page = [&]() {
        for (; skip > 0 && todo; --skip) todo &= todo - 1;
        if (!todo) return false;
        const int at = __builtin_ctzll(todo);
        skip = ranks;
        t = first + at;
        const long long slot = (long long)(unsigned)__builtin_amdgcn_readlane((int)mine, at) |
                               (long long)__builtin_amdgcn_readlane((int)(mine >> 32), at) << 32;
        off = (int)slot & (a.page - 1);
        ph = (slot >> shift) * a.num_kv_heads + head;
        const unsigned long long ones = at == 63 ? on1 : on0 >> (at + 1) | on1 << (63 - at);
        n = min(a.page - off, ones == ~0ull ? 64 : 1 + __builtin_ctzll(~ones));
        return true;
    };

    if (is_k) {
        while (next_page()) {
            float *scale = static_cast<float *>(a.k_scale) + ph;
            const float old = *scale;
            int m = kNoMagnitude;
            KeyPart<D> p;
            p.turned = reinterpret_cast<float *>(cs + kGranule * half) + wave * kGranule * a.rot;
            p.across = across;
            const Rows src(a.k + (long long)t * a.k_stride + (long long)head * D, a.k_stride, n, D);
            uint8_t *dst = a.k_cache + ph * a.page * D;
            // 16 tokens: their rows, and for the block's heads their sines
            auto take = [&](int i0) {
                if (live) p.load(src, i0);
                const int count = min(kGranule, n - i0);
                __syncthreads();
                fill_cos_sin(a, cs, (long long)t + i0, count);
                __syncthreads();
                if (live) m = p.turn(a, cs, count, m);
            };
            // forth to find the scale, and back: the last 16 are still there
            // then, those before are taken again
            float inv = 0.f;
            int step = kGranule;
            for (int i0 = 0; i0 >= 0; i0 += step) {
                if (step > 0 || i0 + kGranule < (n + kGranule - 1) / kGranule * kGranule) take(i0);
                if (step > 0 && i0 + kGranule >= n) {
                    step = -kGranule;
                    if (live) {
                        const float ratio = settle_scale(scale, old, magnitude(wave_max(m)), off, inv);
                        if (ratio != 1.f) rescale_codes(dst, off * D, ratio);
                    }
                }
                if (step < 0 && live) p.store(a, dst + (off + i0) * D, min(kGranule, n - i0), inv);
            }
        }
        return;
    }
    if (!live) return;
    while (next_page()) {
        float *scale = static_cast<float *>(a.v_scale) + ph, inv;
        const float old = *scale;
        int m = kNoMagnitude;
        ValuePart<D> p;
        p.tile = reinterpret_cast<uint32_t *>(cs) + wave * D * 4;
        const Rows src(a.v + (long long)t * a.v_stride + (long long)head * D, a.v_stride, n, D);
        uint8_t *dst = a.v_cache + ph * a.page * D;
        const int g0 = off / kGranule, g1 = (off + n - 1) / kGranule;
        for (int g = g0; g <= g1; ++g) {
            p.load(src, g, off);
            m = p.amax(m);
        }
        const float ratio = settle_scale(scale, old, magnitude(wave_max(m)), off, inv);
        for (int g = ratio != 1.f ? 0 : g0; g <= g1; ++g) {
            if (g0 != g1 && g >= g0) p.load(src, g, off);
            p.store(dst, a.page, off, g, n, inv, ratio);
        }
    }
}

// How many blocks share a window: one for every token of it in a small call, so
// that decode rows run side by side, down to two in a large one: a block costs
// its start, and most tokens of a prompt continue a page (2,048 tokens: 25 us with
// four, 19 with eight, 23 with 16; a prompt of 16,384: 95 us with one and 100 with
// two, but 8,000 tokens and 500 decode rows, which then go one after the other, 98
// and 70).  A q block takes one token while they are few, up to eight as they become
// many.  (q's blocks first, or between: 23 to 24 us for 2,048 tokens, as the cache's
// part is the longer chain.)
template <int D>
static hipError_t launch_append_d(const RopeAppendArgs &a, hipStream_t stream) {
    const int ranks = a.num_tokens <= 512 ? a.page : a.num_tokens <= 4096 ? 8 : 2, q_tokens = min(max(a.num_tokens / 512, 1), 8);
    const int groups = (a.num_kv_heads + kAppendWaves - 1) / kAppendWaves;    // of k heads, and as many of v heads
    const long long append_blocks = ((long long)a.num_tokens + a.page - 1) / a.page * ranks * 2 * groups;
    const long long q_blocks = a.q ? ((long long)a.num_tokens + q_tokens - 1) / q_tokens : 0;
    if (append_blocks + q_blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    // sines of 16 tokens and the waves' rotated elements, or the waves' codes of v (at most 96 KB)
    const size_t lds = max((size_t)kGranule * (a.rot / 2) * sizeof(CosSin) +
                               (size_t)kAppendWaves * kGranule * a.rot * sizeof(float),
                           (size_t)kAppendWaves * kGranule * D);
    hipLaunchKernelGGL((rope_append_kernel<D>), dim3((unsigned)(append_blocks + q_blocks)), dim3(kAppendThreads), lds,
                       stream, a, (int)append_blocks, ranks, groups, q_tokens);
    return hipGetLastError();
}

hipError_t launch_rope_append(const RopeAppendArgs &a, hipStream_t stream) {
    switch (a.d) {
        case 64: return launch_append_d<64>(a, stream);
        case 128: return launch_append_d<128>(a, stream);
        case 256: return launch_append_d<256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
