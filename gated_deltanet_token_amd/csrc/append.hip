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
// The first of a page's new tokens stands for them: every token has its
// workgroups, and those of a token that continues its predecessor's slot end
// after one load.  That needs no list of pages and no request boundaries.
//
// Bound by HBM for prompts (q in and out, k and v in, codes out), by latency
// for decode rows.
#include "fp8.h"
#include "serving_internal.h"

namespace gdn {

constexpr int kAppendThreads = 256;
constexpr int kAppendWaves = kAppendThreads / 64;
constexpr int kGranule = 16;            // tokens whose values a wave holds at once

struct CosSin {
    double c, s;
};

// cos and sin, times the rope scale, of tokens [t0, t0 + n) into cs[n][half]
__device__ __forceinline__ void fill_cos_sin(const RopeAppendArgs &a, CosSin *cs, long long t0, int n) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < n * half; i += kAppendThreads) {
        const int t = i / half;
        const double turns = (double)a.positions[t0 + t] * a.freq[i - t * half] * 0.15915494309189533577;
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        cs[i] = {a.rope_scale * c, a.rope_scale * s};
    }
}

// eight elements [e0, e0 + 8) of one head at `row`, rotated; `cs` of its token
__device__ __forceinline__ void load_rotated(const RopeAppendArgs &a, const uint16_t *row, int e0, const CosSin *cs,
                                             float (&f)[8]) {
    unpack8(*reinterpret_cast<const uint4 *>(row + e0), f);
    if (e0 >= a.rot) return;
    const int half = a.rot / 2;
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const CosSin w = cs[e0 / 2 + i];
            const double x = f[2 * i], y = f[2 * i + 1];
            f[2 * i] = (float)(x * w.c - y * w.s);
            f[2 * i + 1] = (float)(y * w.c + x * w.s);
        }
    } else {
        const bool first = e0 < half;                 // rot is a multiple of 16: all eight on one side
        const int p0 = first ? e0 : e0 - half;
        float g[8];
        unpack8(*reinterpret_cast<const uint4 *>(row + (first ? e0 + half : p0)), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const CosSin w = cs[p0 + i];
            const double x = f[i], y = g[i];
            f[i] = (float)(first ? x * w.c - y * w.s : x * w.c + y * w.s);
        }
    }
}

__device__ __forceinline__ float finite_max(float m, float x) { return is_finite(x) ? fmaxf(m, fabsf(x)) : m; }

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
    return x;
}

// x / scale as a value to code: infinities and NaN become NaN
__device__ __forceinline__ float to_code(float x, float inv) {
    return is_finite(x) ? x * inv : __builtin_bit_cast(float, 0x7fc00000u);
}

// The scale for a page whose new elements reach `amax` and begin at offset
// `off`; stores it, and returns its inverse and what older codes are to be
// multiplied by (1: nothing to do).
__device__ __forceinline__ float settle_scale(float *scale, float amax, int off, float &inv) {
    const float fit = e4m3_block_scale(amax);
    float now = fit, ratio = 1.f;
    if (off > 0) {
        const float old = *scale;
        now = fmaxf(old, fit);
        if (now != old) ratio = old / now;
    }
    if ((threadIdx.x & 63) == 0) *scale = now;
    inv = 1.f / now;               // exact: a power of two
    return ratio;
}

template <int D>
__global__ __launch_bounds__(kAppendThreads) void rope_append_kernel(RopeAppendArgs a, int q_blocks, int q_tokens,
                                                                     int groups) {
    extern __shared__ CosSin cs[];
    constexpr int LPT = D / 8, TPI = 64 / LPT;        // lanes per token of 8 elements; tokens a wave takes at once
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int half = a.rot / 2;

    if ((int)blockIdx.x < q_blocks) {
        const long long t0 = (long long)blockIdx.x * q_tokens;
        const int n = (int)min((long long)q_tokens, a.num_tokens - t0);
        fill_cos_sin(a, cs, t0, n);
        __syncthreads();
        // in place only the rotated elements change
        const bool in_place = a.q == a.q_out;
        const int e0 = (lane % LPT) * 8;
        for (int i = wave * TPI + lane / LPT; i < n * a.num_q_heads; i += kAppendWaves * TPI) {
            const int t = i / a.num_q_heads, h = i - t * a.num_q_heads;
            if (in_place && e0 >= a.rot) continue;
            float f[8];
            load_rotated(a, a.q + (t0 + t) * a.q_stride + (long long)h * D, e0, cs + t * half, f);
            *reinterpret_cast<uint4 *>(a.q_out + (t0 + t) * a.q_out_stride + (long long)h * D + e0) = pack8(f);
        }
        return;
    }

    const int b = (int)blockIdx.x - q_blocks;
    const int t = b / (2 * groups), part = b - t * 2 * groups;
    const long long slots = (long long)a.num_pages * a.page;
    const long long slot = a.slots[t];
    if (slot < 0 || slot >= slots) return;
    const long long page = slot / a.page;
    const int off = (int)(slot - page * a.page);
    if (off > 0 && t > 0 && a.slots[t - 1] == slot - 1) return;      // its page's first new token stands for it
    // the page's new tokens: t .. t + n
    const int room = (int)min((long long)(a.page - off), (long long)a.num_tokens - t);
    const bool next = lane < room && a.slots[t + lane] == slot + lane;
    const unsigned long long run = __ballot(next);
    const int n = run == ~0ull ? 64 : __builtin_ctzll(~run);

    const bool is_k = part < groups;
    const int head = (is_k ? part : part - groups) * kAppendWaves + wave;
    const bool live = head < a.num_kv_heads;
    const long long ph = page * a.num_kv_heads + (live ? head : 0);

    if (is_k) {
        constexpr int ITER = kGranule / TPI;
        const uint16_t *src = a.k + (long long)t * a.k_stride + (long long)(live ? head : 0) * D;
        uint8_t *dst = a.k_cache + ph * a.page * D;
        const int e0 = (lane % LPT) * 8, sub = lane / LPT;
        const int granules = (n + kGranule - 1) / kGranule;
        float f[ITER][8];
        auto load = [&](int g) {
            __syncthreads();
            fill_cos_sin(a, cs, (long long)t + g * kGranule, min(kGranule, n - g * kGranule));
            __syncthreads();
            if (!live) return;
#pragma unroll
            for (int it = 0; it < ITER; ++it) {
                const int i = g * kGranule + it * TPI + sub;
                if (i < n) load_rotated(a, src + i * a.k_stride, e0, cs + (it * TPI + sub) * half, f[it]);
            }
        };
        float m = 0.f;
        for (int g = 0; g < granules; ++g) {
            load(g);
#pragma unroll
            for (int it = 0; it < ITER; ++it)
                if (g * kGranule + it * TPI + sub < n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = finite_max(m, f[it][e]);
        }
        float inv = 0.f;
        if (live) {
            const float ratio = settle_scale(a.k_scale + ph, wave_max(m), off, inv);
            if (ratio != 1.f)
                for (int i = lane * 16; i < off * D; i += 64 * 16) {
                    uint4 w = *reinterpret_cast<const uint4 *>(dst + i);
                    w.x = e4m3_rescaled(w.x, ratio);
                    w.y = e4m3_rescaled(w.y, ratio);
                    w.z = e4m3_rescaled(w.z, ratio);
                    w.w = e4m3_rescaled(w.w, ratio);
                    *reinterpret_cast<uint4 *>(dst + i) = w;
                }
        }
        for (int g = 0; g < granules; ++g) {
            if (granules > 1) load(g);
            if (!live) continue;
#pragma unroll
            for (int it = 0; it < ITER; ++it) {
                const int i = g * kGranule + it * TPI + sub;
                if (i >= n) continue;
                uint2 w;
                w.x = e4m3x4(to_code(f[it][0], inv), to_code(f[it][1], inv), to_code(f[it][2], inv), to_code(f[it][3], inv));
                w.y = e4m3x4(to_code(f[it][4], inv), to_code(f[it][5], inv), to_code(f[it][6], inv), to_code(f[it][7], inv));
                *reinterpret_cast<uint2 *>(dst + (off + i) * D + e0) = w;
            }
        }
        return;
    }

    // v: a lane holds E neighbouring elements of 16 tokens at once, so that a
    // page's 16 tokens of an element are one 16-byte store
    if (!live) return;
    constexpr int E = D / 64;
    const uint16_t *src = a.v + (long long)t * a.v_stride + (long long)head * D + lane * E;
    uint8_t *dst = a.v_cache + (ph * D + lane * E) * a.page;
    const int g0 = off / kGranule, g1 = (off + n - 1) / kGranule;
    float f[kGranule][E];
    auto load = [&](int g) {
#pragma unroll
        for (int i = 0; i < kGranule; ++i) {
            const int j = g * kGranule + i - off;           // token of the run
#pragma unroll
            for (int e = 0; e < E; ++e) f[i][e] = 0.f;
            if (j >= 0 && j < n) {
                const uint16_t *p = src + j * a.v_stride;
                if constexpr (E == 4) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(p);
                    f[i][0] = bf16_lo(w.x);
                    f[i][1] = bf16_hi(w.x);
                    f[i][2] = bf16_lo(w.y);
                    f[i][3] = bf16_hi(w.y);
                } else if constexpr (E == 2) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
                    f[i][0] = bf16_lo(w);
                    f[i][1] = bf16_hi(w);
                } else {
                    f[i][0] = bf16_to_f32(*p);
                }
            }
        }
    };
    float m = 0.f;
    for (int g = g0; g <= g1; ++g) {
        load(g);
#pragma unroll
        for (int i = 0; i < kGranule; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) m = finite_max(m, f[i][e]);
    }
    float inv;
    const float ratio = settle_scale(a.v_scale + ph, wave_max(m), off, inv);
    for (int g = ratio != 1.f ? 0 : g0; g <= g1; ++g) {
        if (g0 != g1 && g >= g0) load(g);
        const int lo = off - g * kGranule, hi = lo + n;     // the granule's new tokens: [lo, hi)
#pragma unroll
        for (int e = 0; e < E; ++e) {
            uint4 *row = reinterpret_cast<uint4 *>(dst + e * a.page + g * kGranule);
            uint32_t w[4] = {0, 0, 0, 0};
            if (lo > 0 || hi < kGranule) {                  // some codes stay
                const uint4 o = *row;
                w[0] = o.x;
                w[1] = o.y;
                w[2] = o.z;
                w[3] = o.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t older = 0, fresh = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (4 * j + i < lo) older |= 0xffu << (8 * i);
                    else if (4 * j + i < hi) fresh |= 0xffu << (8 * i);
                }
                if (ratio != 1.f && older) w[j] = (e4m3_rescaled(w[j], ratio) & older) | (w[j] & ~older);
                if (fresh) {
                    const uint32_t x = e4m3x4(to_code(f[4 * j][e], inv), to_code(f[4 * j + 1][e], inv),
                                              to_code(f[4 * j + 2][e], inv), to_code(f[4 * j + 3][e], inv));
                    w[j] = (x & fresh) | (w[j] & ~fresh);
                }
            }
            *row = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// A q block takes one token when there are few tokens (as many blocks as
// possible), else four (their sines in one round of the workgroup).
constexpr int kQTokensFew = 1, kQTokensMany = 4, kManyTokens = 1024;

template <int D>
static hipError_t launch_append_d(const RopeAppendArgs &a, hipStream_t stream) {
    const int q_tokens = a.num_tokens >= kManyTokens ? kQTokensMany : kQTokensFew;
    const long long q_blocks = a.q ? (a.num_tokens + q_tokens - 1) / q_tokens : 0;
    const int groups = (a.num_kv_heads + kAppendWaves - 1) / kAppendWaves;
    const long long blocks = q_blocks + (long long)a.num_tokens * 2 * groups;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)kGranule * (a.rot / 2) * sizeof(CosSin);
    hipLaunchKernelGGL((rope_append_kernel<D>), dim3((unsigned)blocks), dim3(kAppendThreads), lds, stream, a,
                       (int)q_blocks, q_tokens, groups);
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
