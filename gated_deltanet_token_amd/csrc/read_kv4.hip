// Keys and values read back out of the 4-bit paged cache (gdn_paged_read_kv4),
// gfx950.
//
// Requests' ranges are cut where the cache's granules of 16 tokens are.  A wave
// takes a granule of keys, or of values, of as many heads as 64 lanes hold: D / 8
// lanes per head, each with eight elements.  A key's eight codes are four bytes; the
// eight elements' codes of a value lie in 64 bytes, for all 16 tokens.  A store is 16
// bytes per lane, whole heads.
// Bound by the stores, 32 bits for every 8.3 read: streaming ones, that leave the
// caches to what is still to be read (30,000 rows of 4 heads of 256: 26.4 us; 131,071 of
// 8 of 128: 124, 5.5 TB/s of both directions; with ordinary ones 9 and 7 us more).
// Streaming loads would lose the halves of a line that another load takes (6 and 9 us
// more).  All keys before all values: granule by granule 1.3 us more each.
#include "attention_split.h"
#include "fp4.h"

namespace gdn {

constexpr int kReadThreads = 256;

// the eight elements' values of token t (0 to 15) of a granule, scaled
__device__ __forceinline__ uint4 value_row(const uint2 (&w)[8], int t, float scale) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t u = t < 8 ? w[e].x : w[e].y;
        const auto two = t % 8 < 2   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 0)
                         : t % 8 < 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 1)
                         : t % 8 < 6 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 2)
                                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 3);
        f[e] = (t & 1 ? two[1] : two[0]) * scale;
    }
    return pack8(f);
}

template <int D>
__global__ __launch_bounds__(kReadThreads) void paged_read_kv4_kernel(PagedReadArgs a, int groups, long long waves) {
    constexpr int LPH = D / 8, HEADS = 64 / LPH;     // lanes per head; heads of a wave
    const int lane = threadIdx.x & 63;
    const long long unit = (long long)blockIdx.x * (kReadThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (unit >= waves) return;
    // all keys, then all values
    const bool is_k = unit < waves / 2;
    const long long of = is_k ? unit : unit - waves / 2;
    const int tile = (int)(of / groups), head = (int)(of - (long long)tile * groups) * HEADS + lane / LPH, e0 = (lane % LPH) * 8;
    if (is_k ? !a.k_out : !a.v_out) return;
    // request s owns the tile numbers from floor(out_start_loc[s] / 16) + 2 s on: as
    // many as its granules or more
    AttentionArgs q{};
    q.num_seqs = a.num_seqs;
    q.qsl = a.out_start_loc;
    int within;
    const int s = find_request(q, tile, 1, kGranule, 2, false, within);
    int begin, end;
    clamp_range(a.out_start_loc[s], a.out_start_loc[s + 1], a.num_rows, begin, end);
    const int start = a.key_starts ? max(a.key_starts[s], 0) : 0;
    const long long j0 = ((long long)(start / kGranule) + within) * kGranule;        // the granule's first key
    const long long lo = max((long long)start, j0), hi = min((long long)start + (end - begin), j0 + kGranule);
    if (within < 0 || lo >= hi) return;
    const long long at_page = j0 / a.page;
    if (at_page >= a.max_pages) return;
    const int page = a.block_table[s * a.block_table_stride + at_page];
    if ((unsigned)page >= (unsigned)a.num_pages || head >= a.num_kv_heads) return;
    const long long ph = (long long)page * a.num_kv_heads + head, at = ph * a.page + (int)(j0 & (a.page - 1));
    const long long row0 = begin + (j0 - start);     // the output row of the granule's first key
    const int t0 = (int)(lo - j0), t1 = (int)(hi - j0);
    if (is_k) {
        const uint8_t *p = a.k_cache + at * (D / 2) + e0 / 2;
        const uint8_t *sc = a.k_scale + (ph * (D / kScaleBlock) + e0 / kScaleBlock) * a.page + (int)(j0 & (a.page - 1));
        const uint4 scales = *reinterpret_cast<const uint4 *>(sc);
        uint32_t w[kGranule];
#pragma unroll
        for (int t = 0; t < kGranule; ++t) w[t] = *reinterpret_cast<const uint32_t *>(p + t * (D / 2));
        uint16_t *out = a.k_out + row0 * a.k_out_stride + (long long)head * D + e0;
#pragma unroll
        for (int t = 0; t < kGranule; ++t) {
            const uint32_t u = t < 4 ? scales.x : t < 8 ? scales.y : t < 12 ? scales.z : scales.w, e = u >> 8 * (t % 4) & 255;
            // a power of two; 255: NaN
            const float scale = __builtin_bit_cast(float, e == 255 ? 0x7fc00000u : e == 0 ? 0x00400000u : e << 23);
            const uint4 v = e2m1_bf16(w[t]);
            float f[8];
            unpack8(v, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= scale;
            if (t >= t0 && t < t1) store_stream16(out + t * a.k_out_stride, pack8(f));
        }
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(a.v_cache + at * (D / 2) + e0 * 8);
        uint2 w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = p[i];
            w[2 * i] = make_uint2(u.x, u.y);
            w[2 * i + 1] = make_uint2(u.z, u.w);
        }
        const uint4 *sc = reinterpret_cast<const uint4 *>(a.v_scale + at);
        float scale[kGranule];
        unpack8(sc[0], scale);
        unpack8(sc[1], scale + 8);
        uint16_t *out = a.v_out + row0 * a.v_out_stride + (long long)head * D + e0;
#pragma unroll
        for (int t = 0; t < kGranule; ++t)
            if (t >= t0 && t < t1) store_stream16(out + t * a.v_out_stride, value_row(w, t, scale[t]));
    }
}

template <int D>
static hipError_t launch_d(const PagedReadArgs &a, hipStream_t stream) {
    constexpr int HEADS = 64 / (D / 8);
    const int groups = (a.num_kv_heads + HEADS - 1) / HEADS;
    const long long waves = (a.num_rows / kGranule + 2LL * a.num_seqs) * 2 * groups;
    const long long blocks = (waves + kReadThreads / 64 - 1) / (kReadThreads / 64);
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((paged_read_kv4_kernel<D>), dim3((unsigned)blocks), dim3(kReadThreads), 0, stream, a, groups, waves);
    return hipGetLastError();
}

hipError_t launch_paged_read_kv4(const PagedReadArgs &a, hipStream_t stream) {
    switch (a.d) {
        case 64: return launch_d<64>(a, stream);
        case 128: return launch_d<128>(a, stream);
        case 256: return launch_d<256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
