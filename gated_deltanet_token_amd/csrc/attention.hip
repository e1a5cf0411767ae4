// Attention over the 8-bit paged cache (gdn_paged_attention_kv8), gfx950.
//
// One wave per (token, q head): 64 keys at a time, a lane per key for the
// scores, then a lane per element for the values, with the running maximum
// and sum of the softmax.
#include "fp8.h"
#include "serving_internal.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ __launch_bounds__(64) void attention_rows_kernel(AttentionArgs a) {
    constexpr int E = D / 64;
    __shared__ float qs[D];
    __shared__ float ps[64];
    __shared__ long long pg[4];
    const int lane = threadIdx.x;
    const int t = blockIdx.x / a.num_q_heads, h = blockIdx.x - t * a.num_q_heads;
    const int hk = h / (a.num_q_heads / a.num_kv_heads);

    // the request of token t: the last one that begins at or before it
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.qsl[mid] <= t) lo = mid;
        else hi = mid;
    }
    int begin, end;
    clamp_range(a.qsl[lo], a.qsl[lo + 1], a.num_tokens, begin, end);
    if (t < begin || t >= end) return;
    const long long L = min((long long)max(a.seq_lens[lo], 0), (long long)a.max_pages * a.page);
    const long long pos = (long long)max(a.seq_lens[lo], 0) - (end - begin) + (t - begin);
    const long long j_end = a.causal ? min(L, pos + 1) : L;
    const long long j_begin = a.window > 0 ? max(0LL, pos + 1 - a.window) : 0;

    for (int e = lane; e < D; e += 64) qs[e] = bf16_to_f32(a.q[(long long)t * a.q_stride + (long long)h * D + e]);
    __syncthreads();
    float m = -__builtin_inff(), l = 0.f, o[E] = {};
    for (long long j0 = j_begin & ~63LL; j0 < j_end; j0 += 64) {
        if (lane < 4) {
            const long long jg = j0 + lane * 16, pi = jg / a.page;
            pg[lane] = pi < a.max_pages ? a.block_table[lo * a.block_table_stride + pi] : -1;
        }
        __syncthreads();
        const long long j = j0 + lane, page = pg[lane >> 4];
        const bool seen = j >= j_begin && j < j_end && page >= 0 && page < a.num_pages;
        float x = -__builtin_inff(), vs = 0.f;
        if (seen) {
            const long long ph = page * a.num_kv_heads + hk;
            const uint8_t *kp = a.k_cache + (ph * a.page + j % a.page) * D;
            float s = 0.f;
            for (int e = 0; e < D; e += 16) {
                const uint4 w = *reinterpret_cast<const uint4 *>(kp + e);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[4];
                    e4m3_values(ws[i], f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) s = __builtin_fmaf(f[c], qs[e + 4 * i + c], s);
                }
            }
            x = s * (a.k_scale[ph] * a.scale * kLog2e);
            vs = a.v_scale[ph];
        }
        float mx = x;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const float y = __shfl_xor(mx, d, 64);
            mx = mx > y || mx != mx ? mx : y;             // keeps a NaN
        }
        const float m_new = m > mx || m != m ? m : mx;
        const float old = m == m_new ? 1.f : exp2f(m - m_new);
        const float p = seen ? exp2f(x - m_new) : 0.f;
        float sum = p;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
        m = m_new;
        l = l * old + sum;
        ps[lane] = p * vs;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            o[e] *= old;
            for (int g = 0; g < 4; ++g) {
                const long long page_g = pg[g];
                if (page_g < 0 || page_g >= a.num_pages) continue;
                const long long jg = j0 + g * 16;
                const uint8_t *vp = a.v_cache + ((page_g * a.num_kv_heads + hk) * D + lane + 64 * e) * a.page + jg % a.page;
                const uint4 w = *reinterpret_cast<const uint4 *>(vp);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[4];
                    e4m3_values(ws[i], f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const long long jj = jg + 4 * i + c;
                        if (jj >= j_begin && jj < j_end) o[e] = __builtin_fmaf(ps[g * 16 + 4 * i + c], f[c], o[e]);
                    }
                }
            }
        }
        __syncthreads();
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.o[(long long)t * a.o_stride + (long long)h * D + lane + 64 * e] = f32_to_bf16(o[e] * inv);
}

int64_t attention_workspace_bytes(int, int, int, int, int, int) { return 0; }

template <int D>
static hipError_t launch_rows(const AttentionArgs &a, hipStream_t stream) {
    const long long blocks = (long long)a.num_tokens * a.num_q_heads;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((attention_rows_kernel<D>), dim3((unsigned)blocks), dim3(64), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_attention(const AttentionArgs &a, hipStream_t stream) {
    switch (a.d) {
        case 64: return launch_rows<64>(a, stream);
        case 128: return launch_rows<128>(a, stream);
        case 256: return launch_rows<256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
