// Norms between blocks, gfx950: gdn_gated_rms_norm (each head, with its
// output gate) and gdn_residual_rms_norm (norm after a block, gate, residual
// scale and sum, norm before the next block).
//
// Both move every operand once and do a few operations per element: bound by
// HBM.  A row stays in registers between its passes (sum of squares, then
// scaling), in 16-byte vectors of 8 elements; sums are fp32.
//
// Measured: 2,048 tokens x 32 heads of 128 with their gate: 11.0 us, 4.6 TB/s;
// between blocks, 16,384 rows of 4,096 with both norms and the gate: 119 us, 5.6 TB/s
// (a streaming copy with one access per lane reaches 6.65, with four 5.96); 32 rows
// of 2,560: 3.5 us, a launch.
#include "gdn_device.h"
#include "serving_internal.h"

namespace gdn {

// sum over aligned groups of G lanes (a power of two up to 64), the same in every lane
template <int G>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
    return x;
}

__device__ __forceinline__ float sum_squares(const float (&f)[8]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(f[e], f[e], s);
    return s;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + __expf(-z)); }

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// One head is a group of G lanes, 8 elements each (G >= head_dim / 8).
template <int G>
__global__ __launch_bounds__(256) void head_norm_kernel(HeadNormArgs a) {
    const int e0 = (threadIdx.x % G) * 8;
    const bool live = e0 < a.d;
    const long long n = (long long)a.num_tokens * a.num_heads;
    const long long row = (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
    if (row >= n) return;
    // (64-bit divisions take a hundred instructions: for more than 2^32 rows only)
    const long long t = n <= 0xffffffffLL ? (unsigned)row / (unsigned)a.num_heads : row / a.num_heads, h = row - t * a.num_heads;
    float f[8] = {}, w[8] = {}, z[8] = {};
    if (live) {
        unpack8(load16(a.x + t * a.x_stride + h * a.d + e0), f);
        unpack8(load16(a.weight + e0), w);
        if (a.gate) unpack8(load16(a.gate + t * a.gate_stride + h * a.d + e0), z);
    }
    const float r = rsqrtf(lanes_sum<G>(sum_squares(f)) / (float)a.d + a.eps);
    if (!live) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        f[e] = f[e] * r * (a.offset + w[e]);
        if (a.gate) f[e] *= z[e] * sigmoid(z[e]);
    }
    *reinterpret_cast<uint4 *>(a.y + t * a.y_stride + h * a.d + e0) = pack8(f);
}

// One row is a workgroup of W waves; a thread holds V vectors of it, vector v
// at element (v * 64 W + thread) * 8.
template <int W, int V>
__global__ __launch_bounds__(64 * W) void residual_norm_kernel(ResidualNormArgs a) {
    const long long row = blockIdx.x;
    const int tid = threadIdx.x;
    __shared__ float part[2][W];
    auto row_sum = [&](float x, int which) {
        x = lanes_sum<64>(x);
        if constexpr (W > 1) {
            if ((tid & 63) == 0) part[which][tid >> 6] = x;
            __syncthreads();
            x = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) x += part[which][w];
        }
        return x;
    };
    float u[V][8] = {}, res[V][8] = {};
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = (v * 64 * W + tid) * 8;
        if (e < a.hidden) {
            unpack8(load16(a.x + row * a.x_stride + e), u[v]);
            unpack8(load16(a.residual + row * a.residual_stride + e), res[v]);
        }
        s += sum_squares(u[v]);
    }
    float r = 0.f;
    if (a.post_weight) r = rsqrtf(row_sum(s, 0) / (float)a.hidden + a.eps);
    s = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = (v * 64 * W + tid) * 8;
        if (e < a.hidden) {
            if (a.post_weight) {
                float w[8];
                unpack8(load16(a.post_weight + e), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[v][i] = u[v][i] * r * (a.offset + w[i]);
            }
            if (a.gate) {
                float z[8];
                unpack8(load16(a.gate + row * a.gate_stride + e), z);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[v][i] *= sigmoid(z[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) u[v][i] = __builtin_fmaf(a.residual_scale, u[v][i], res[v][i]);
            *reinterpret_cast<uint4 *>(a.new_residual + row * a.new_residual_stride + e) = pack8(u[v]);
        }
        s += sum_squares(u[v]);
    }
    r = rsqrtf(row_sum(s, 1) / (float)a.hidden + a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = (v * 64 * W + tid) * 8;
        if (e < a.hidden) {
            float w[8];
            unpack8(load16(a.weight + e), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[v][i] = u[v][i] * r * (a.offset + w[i]);
            *reinterpret_cast<uint4 *>(a.y + row * a.y_stride + e) = pack8(u[v]);
        }
    }
}

template <int G>
static void launch_head(const HeadNormArgs &a, unsigned blocks, hipStream_t stream) {
    hipLaunchKernelGGL((head_norm_kernel<G>), dim3(blocks), dim3(256), 0, stream, a);
}

hipError_t launch_head_norm(const HeadNormArgs &a, hipStream_t stream) {
    int g = 1;
    while (g * 8 < a.d) g *= 2;
    const long long rows = (long long)a.num_tokens * a.num_heads, blocks = (rows * g + 255) / 256;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    switch (g) {
        case 1: launch_head<1>(a, blocks, stream); break;
        case 2: launch_head<2>(a, blocks, stream); break;
        case 4: launch_head<4>(a, blocks, stream); break;
        case 8: launch_head<8>(a, blocks, stream); break;
        case 16: launch_head<16>(a, blocks, stream); break;
        case 32: launch_head<32>(a, blocks, stream); break;
        default: launch_head<64>(a, blocks, stream); break;
    }
    return hipGetLastError();
}

template <int W, int V>
static void launch_residual(const ResidualNormArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL((residual_norm_kernel<W, V>), dim3(a.rows), dim3(64 * W), 0, stream, a);
}

hipError_t launch_residual_norm(const ResidualNormArgs &a, hipStream_t stream) {
    // As many waves as a row has vectors for, one each (rows of 2,560, 32 of them:
    // 3.5 us with eight waves, 3.8 with two vectors in each of four; 16,384: 59.1 and
    // 60.3; rows of 2,048 with four vectors in one wave: 51.6, in four waves 46.4).
    const int vectors = a.hidden / 8;
    if (vectors <= 64) launch_residual<1, 1>(a, stream);
    else if (vectors <= 256) launch_residual<4, 1>(a, stream);
    else if (vectors <= 512) launch_residual<8, 1>(a, stream);
    else if (vectors <= 1024) launch_residual<16, 1>(a, stream);
    else launch_residual<16, 2>(a, stream);
    return hipGetLastError();
}

}  // namespace gdn
