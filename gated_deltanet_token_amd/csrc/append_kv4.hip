// Rotary positions on q and k, and the new k and v written into the 4-bit
// paged cache (gdn_rope_append_kv4), gfx950.
//
// Rotation: (a, b) -> m (a cos t - b sin t, b cos t + a sin t), t = position *
// frequency.  Angles, and their sines and cosines, are formed in 64 bits, once per
// token and pair in the LDS for all heads of q and k; k's products are in 64 bits too.
//
// Keys: a scale belongs to 32 elements of one token, four lanes' eights.  Tokens
// are independent of each other.
// Values: a scale belongs to a token's head; the codes of 16 neighbouring tokens (a
// granule) of an element share eight bytes.  One wave owns a granule's new
// tokens of a head: it turns their codes in the LDS and, where the granule is not
// all new, puts them between the old ones.  The first of a granule's new tokens
// stands for them: every window of 64 tokens has its workgroups, whose waves take
// the (granule, head) pairs that begin in it in turns.  That needs no list of
// granules and no request boundaries, and no atomics.
// Bound by q's way there and back for many tokens (16,384 of 32 + 8 heads of 128: 73
// us, 354 MB; v alone 16.6, which waits for one thing after another: its workgroups
// are spread among the others, 3 us more with all of them first), by latency for few (32
// tokens: 5.3 us).  q leaves by streaming stores (with ordinary ones 7 us more).  A row
// at a time per group of lanes: with two, fewer waves fit (4 us more).
#include "fp4.h"
#include "rope.h"

namespace gdn {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kWindow = 64;             // tokens

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float fma_of(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return __builtin_fma(a, b, c); }

// a pair's cosine and sine, times the rope scale
template <class T>
struct CosSin {
    T c, s;
};

// those of `tokens` tokens, token by token, for k in 64 bits and for q
struct Turns {
    CosSin<double> *k;
    CosSin<float> *q;
    __device__ Turns(void *lds, int pairs) : k(static_cast<CosSin<double> *>(lds)), q(reinterpret_cast<CosSin<float> *>(k + pairs)) {}
};
constexpr size_t kTurnBytes = sizeof(CosSin<double>) + sizeof(CosSin<float>);

// those of tokens [t0, t0 + n), n <= 16
__device__ __forceinline__ void fill_cos_sin(const RopeAppendArgs &a, const Turns &turns, long long t0, int n) {
    const int half = a.rot / 2, across = half > 32 ? 64 : 32;       // lanes per token
    if (half == 0) return;
    // one load brings every token's position; the loop's lanes take theirs from there
    const int pos = a.positions[t0 + min((int)(threadIdx.x & 15), n - 1)];
    for (int p = threadIdx.x & (across - 1); p - (int)(threadIdx.x & (across - 1)) < half; p += across) {
        const double f = a.freq[min(p, half - 1)];
#pragma unroll 1
        for (int t = threadIdx.x / across; t < n; t += kThreads / across) {
            double s, c;
            sin_cos_turns((double)__shfl(pos, t, 64) * f * 0.15915494309189533577, s, c);
            c *= a.rope_scale, s *= a.rope_scale;
            if (p < half) {
                turns.k[t * half + pair_at(a, p)] = {c, s};
                turns.q[t * half + pair_at(a, p)] = {(float)c, (float)s};
            }
        }
    }
}

// eight elements (e0 < rot), rotated; `cs` of their token.  q's products are in fp32,
// as it is rounded to bf16; k's in 64 bits: what fp32 leaves out (2^-23 of a pair) would turn
// codes of elements between two of them, a few in ten million, into their neighbours.
template <class T>
__device__ __forceinline__ void rotated(const RopeAppendArgs &a, const Raw &r, int e0, const CosSin<T> *cs, float (&f)[8]) {
    unpack8(r.own, f);
    if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const CosSin<T> w = cs[i * (a.rot / 8) + e0 / 8];
            const T x = f[2 * i], y = f[2 * i + 1];
            f[2 * i] = (float)fma_of(x, w.c, -(y * w.s));
            f[2 * i + 1] = (float)fma_of(y, w.c, x * w.s);
        }
    } else {
        const int half = a.rot / 2;
        const bool first = e0 < half;
        const int p0 = first ? e0 : e0 - half;
        const uint32_t turn = first ? 0x80008000u : 0u;             // the first of a pair meets -b
        float g[8];
        unpack8(make_uint4(r.other.x ^ turn, r.other.y ^ turn, r.other.z ^ turn, r.other.w ^ turn), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const CosSin<T> w = cs[i * (half / 8) + p0 / 8];
            f[i] = (float)fma_of((T)f[i], w.c, (T)g[i] * w.s);
        }
    }
}

// the largest of four neighbouring lanes' values
__device__ __forceinline__ uint32_t max4(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor1, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor2, 0xF, 0xF, false));
}

// Eight elements of a key, a quarter of a block with its neighbours': their codes
// and, by the first of the four lanes, the block's scale to head `ph`'s offset
// `off`.
template <int D>
__device__ __forceinline__ void store_key(const RopeAppendArgs &a, const float (&f)[8], long long ph, int off, int e0, bool on) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __builtin_bit_cast(uint32_t, f[e]) & 0x7fffffffu);
    m = max4(m);
    const int ex = e2m1_block_exponent(__builtin_bit_cast(float, m));
    const float inv = __builtin_bit_cast(float, (uint32_t)(127 - ex) << 23);         // exact: a power of two
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f[e] * inv;
    if (!on) return;
    *reinterpret_cast<uint32_t *>(a.k_cache + (ph * a.page + off) * (D / 2) + e0 / 2) = e2m1x8(x);
    if (e0 % kScaleBlock == 0)
        static_cast<uint8_t *>(a.k_scale)[(ph * (D / kScaleBlock) + e0 / kScaleBlock) * a.page + off] =
            (uint8_t)(m >= 0x7f800000u ? 255 : ex + 127);
}

// One wave's share: the n new tokens from `t` on of a granule's v head, from offset
// `off` of the granule on.  A lane has eight elements of ITER neighbouring tokens.
template <int D>
__device__ __forceinline__ void append_values(const RopeAppendArgs &a, uint8_t *tile, long long t, int n, long long slot, int head) {
    constexpr int LPT = D / 8, TPI = 64 / LPT, ITER = kGranule / TPI;
    constexpr int PIECES = D / 128 > 0 ? D / 128 : 1;               // 16-byte pieces of a granule per lane
    const int lane = threadIdx.x & 63, e0 = (lane % LPT) * 8, sub = lane / LPT;
    const int shift = __builtin_ctz(a.page), off = (int)slot & (kGranule - 1);
    const long long at = ((slot >> shift) * a.num_kv_heads + head) * a.page + ((int)slot & (a.page - 1) & ~(kGranule - 1));
    uint4 *dst = reinterpret_cast<uint4 *>(a.v_cache + at * (D / 2));
    const bool part = n < kGranule;
    uint4 old[PIECES];
    if (part)
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            if (D >= 128 || lane < 32) old[i] = dst[lane + 64 * i];
    const Rows src(a.v + t * a.v_stride + (long long)head * D, a.v_stride, n, D);
    uint4 w[ITER];
#pragma unroll
    for (int it = 0; it < ITER; ++it) w[it] = src.load16(sub * ITER + it - off, e0);      // (zeros where the run has no token)
    // the tokens' largest magnitudes, two to a word
    float inv[ITER], scale[ITER];
#pragma unroll
    for (int i = 0; i < ITER; i += 2) {
        u16x2 m = {0, 0};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint4 &u = w[i + b];
            u16x2 x = __builtin_bit_cast(u16x2, u.x & 0x7fff7fffu);
            x = __builtin_elementwise_max(x, __builtin_bit_cast(u16x2, u.y & 0x7fff7fffu));
            x = __builtin_elementwise_max(x, __builtin_bit_cast(u16x2, u.z & 0x7fff7fffu));
            x = __builtin_elementwise_max(x, __builtin_bit_cast(u16x2, u.w & 0x7fff7fffu));
            m[b] = max(x[0], x[1]);
        }
#pragma unroll
        for (int d = 1; d < LPT; d <<= 1)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, __shfl_xor(__builtin_bit_cast(int, m), d, 64)));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            // a sixth of it as bf16: a third of eight bits is never close to the middle of two such values
            const float s = fmaxf(bf16_to_f32(f32_to_bf16(bf16_to_f32(m[b]) * (1.f / 6.f))), kLeastScale);
            scale[i + b] = m[b] >= 0x7f80 ? __builtin_nanf("") : s;
            inv[i + b] = __builtin_amdgcn_rcpf(s);
        }
    }
    // their codes, an element's of neighbouring tokens side by side
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x[8] = {};
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
            const uint32_t u = e < 2 ? w[it].x : e < 4 ? w[it].y : e < 6 ? w[it].z : w[it].w;
            const float f = e & 1 ? bf16_hi(u) : bf16_lo(u), y = f * inv[it];
            // the quotient: exact where it is a tie of two codes (a zero's sign would be lost)
            x[it] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-y, scale[it], f), inv[it], y), f);
        }
        const uint32_t codes = e2m1x8(x);
        uint8_t *p = tile + (e0 + e) * 8 + sub * (ITER / 2);
        if constexpr (ITER == 8) *reinterpret_cast<uint32_t *>(p) = codes;
        else if constexpr (ITER == 4) *reinterpret_cast<uint16_t *>(p) = (uint16_t)codes;
        else *p = (uint8_t)codes;
    }
    if (lane % LPT == 0)
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
            const int i = sub * ITER + it;
            if (i >= off && i < off + n) static_cast<uint16_t *>(a.v_scale)[at + i] = f32_to_bf16(scale[it]);
        }
    wave_sync();
    const uint64_t mine = (n == kGranule ? ~0ull : (1ull << (4 * n)) - 1) << (4 * off);
    const uint32_t m0 = (uint32_t)mine, m1 = (uint32_t)(mine >> 32);
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        if (D >= 128 || lane < 32) {
            uint4 x = *reinterpret_cast<const uint4 *>(tile + (lane + 64 * i) * 16);
            if (part) {
                x.x = (x.x & m0) | (old[i].x & ~m0);
                x.y = (x.y & m1) | (old[i].y & ~m1);
                x.z = (x.z & m0) | (old[i].z & ~m0);
                x.w = (x.w & m1) | (old[i].w & ~m1);
            }
            dst[lane + 64 * i] = x;
        }
    wave_sync();
}

template <int D>
__global__ __launch_bounds__(kThreads) void rope_append_kv4_kernel(RopeAppendArgs a, int value_blocks, int per, int ranks, int tokens) {
    extern __shared__ double2 shared[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const long long slots = (long long)a.num_pages * a.page;

    // a block of values, then per - 1 of rows; the rows that are left behind them
    const unsigned block = blockIdx.x, turn = block / (unsigned)per;
    if (turn >= (unsigned)value_blocks || block != turn * per) {
        // q and k of `tokens` tokens, a head per LPT lanes of eight elements
        constexpr int LPT = D / 8, TPI = 64 / LPT, STEP = kWaves * TPI;
        const int half = a.rot / 2, heads = a.num_q_heads + a.num_kv_heads, shift = __builtin_ctz(a.page);
        const long long t0 = (long long)(block - min(turn + 1, (unsigned)value_blocks)) * tokens;
        const int n = (int)min((long long)tokens, a.num_tokens - t0), rows = n * heads;
        const int e0 = (lane % LPT) * 8;
        const bool turned = e0 < a.rot;
        auto load = [&](int i) {
            i = min(i, rows - 1);
            const int t = (unsigned)i / (unsigned)heads, h = i - t * heads;
            const uint16_t *row = h < a.num_q_heads ? a.q + (t0 + t) * a.q_stride + (long long)h * D
                                                    : a.k + (t0 + t) * a.k_stride + (long long)(h - a.num_q_heads) * D;
            return load_raw(a, row, e0);
        };
        int i = wave * TPI + lane / LPT;
        Raw now = load(i), next = now;
        const Turns turns(shared, tokens * half);
        fill_cos_sin(a, turns, t0, n);
        __syncthreads();
        // (every lane of a wave takes as many turns: keys' lanes look at each other)
        for (int w0 = wave * TPI; w0 < rows; w0 += STEP, i += STEP) {
            if (w0 + STEP < rows) next = load(i + STEP);
            const bool live = i < rows;
            const int at = live ? i : rows - 1, t = (unsigned)at / (unsigned)heads, h = at - t * heads;
            float f[8];
            if (!turned) unpack8(now.own, f);
            else if (h < a.num_q_heads) rotated(a, now, e0, turns.q + t * half, f);
            else rotated(a, now, e0, turns.k + t * half, f);
            if (h < a.num_q_heads) {
                if (live && (turned || a.q != a.q_out))
                    store_stream16(a.q_out + (t0 + t) * a.q_out_stride + (long long)h * D + e0, pack8(f));
            } else {
                const long long slot = a.slots[t0 + t];
                const bool on = live && slot >= 0 && slot < slots;
                store_key<D>(a, f, (slot >> shift) * a.num_kv_heads + h - a.num_q_heads, (int)slot & (a.page - 1), e0, on);
            }
            now = next;
        }
        return;
    }

    // the slots of the window's tokens and of as many behind them (a granule's run
    // may reach there), and which of them continue their predecessor's granule
    const int first = (int)(turn / (unsigned)ranks) * kWindow, rank = (int)(turn % (unsigned)ranks);
    auto slot_at = [&](long long t) { return t >= 0 && t < a.num_tokens ? a.slots[t] : -2; };
    const long long mine = slot_at((long long)first + lane), behind = slot_at((long long)first + kWindow + lane);
    const bool on = mine == slot_at((long long)first + lane - 1) + 1 && (mine & (kGranule - 1)) != 0;
    const unsigned long long on0 = __ballot(on);
    const unsigned long long on1 =
        __ballot(behind == slot_at((long long)first + kWindow - 1 + lane) + 1 && (behind & (kGranule - 1)) != 0);
    unsigned long long todo = __ballot(mine >= 0 && mine < slots && !on);
    const int items = __builtin_popcountll(todo) * a.num_kv_heads;
    int leader = 0;
    uint8_t *tile = reinterpret_cast<uint8_t *>(shared) + wave * D * 8;
    for (int i = rank * kWaves + wave; i < items; i += ranks * kWaves) {
        const int l = (unsigned)i / (unsigned)a.num_kv_heads;
        for (; leader < l; ++leader) todo &= todo - 1;
        const int b = __builtin_ctzll(todo);
        const unsigned long long ones = b == 63 ? on1 : on0 >> (b + 1) | on1 << (63 - b);
        const long long slot = (long long)(unsigned)__builtin_amdgcn_readlane((int)mine, b) |
                               (long long)__builtin_amdgcn_readlane((int)(mine >> 32), b) << 32;
        append_values<D>(a, tile, (long long)first + b, 1 + __builtin_ctzll(~ones), slot, i - l * a.num_kv_heads);
    }
}

template <int D>
static hipError_t launch_d(const RopeAppendArgs &a, hipStream_t stream) {
    // two tokens per workgroup of rows where there are many (16,384 of 32 + 8 heads of 128: 73 us, 97
    // with four, 83 with one)
    const int tokens = a.num_tokens >= 1024 ? 2 : 1;
    const long long windows = ((long long)a.num_tokens + kWindow - 1) / kWindow;
    // a small call: a wave per (token, head), should each be a granule's first
    const int begin = a.num_tokens <= 512 ? min(a.num_tokens, kWindow) : 8;
    const int ranks = (begin * a.num_kv_heads + kWaves - 1) / kWaves;
    const long long value_blocks = windows * ranks, row_blocks = ((long long)a.num_tokens + tokens - 1) / tokens;
    if (value_blocks + row_blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    // sines of the tokens, or the waves' codes of v
    const size_t lds = max((size_t)tokens * (a.rot / 2) * kTurnBytes, (size_t)kWaves * D * 8);
    hipLaunchKernelGGL((rope_append_kv4_kernel<D>), dim3((unsigned)(value_blocks + row_blocks)), dim3(kThreads), lds, stream, a,
                       (int)value_blocks, (int)(row_blocks / value_blocks) + 1, ranks, tokens);
    return hipGetLastError();
}

hipError_t launch_rope_append_kv4(const RopeAppendArgs &a, hipStream_t stream) {
    switch (a.d) {
        case 64: return launch_d<64>(a, stream);
        case 128: return launch_d<128>(a, stream);
        case 256: return launch_d<256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
