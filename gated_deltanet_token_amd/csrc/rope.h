// What the appends to a paged cache share, whatever its format (gfx950): sines of
// positions in 64 bits, the places of rotated pairs, rows of tokens.
#pragma once

#include "gdn_device.h"
#include "serving_internal.h"

namespace gdn {

// Sine and cosine of `turns` whole turns, to about 2^-52: the fraction, then
// the quarter of a turn nearest to it, then the Taylor series of what is left
// (at most an eighth of a turn: the terms left out are below 2^-54).  The
// coefficients are read as scalars; as literals they would hold 30 registers
// of every lane.
__constant__ double kSinSeries[7] = {-1.0 / 6.0, 1.0 / 120.0, -1.0 / 5040.0, 1.0 / 362880.0, -1.0 / 39916800.0,
                                     1.0 / 6227020800.0, -1.0 / 1307674368000.0};
__constant__ double kCosSeries[8] = {-0.5, 1.0 / 24.0, -1.0 / 720.0, 1.0 / 40320.0, -1.0 / 3628800.0,
                                     1.0 / 479001600.0, -1.0 / 87178291200.0, 1.0 / 20922789888000.0};

__device__ __forceinline__ void sin_cos_turns(double turns, double &s, double &c) {
    const double r = turns - rint(turns), quarter = rint(4.0 * r);
    const double x = __builtin_fma(-0.25, quarter, r) * 6.283185307179586476925286766559, z = x * x;
    double p = kSinSeries[6], q = kCosSeries[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) {
        q = __builtin_fma(q, z, kCosSeries[i]);
        if (i < 6) p = __builtin_fma(p, z, kSinSeries[i]);
    }
    const double sx = __builtin_fma(x * z, p, x), cx = __builtin_fma(q, z, 1.0);
    const int k = (int)quarter;
    s = k & 1 ? cx : sx;
    c = k & 1 ? sx : cx;
    if (k & 2) s = -s;
    if ((k + 1) & 2) c = -c;
}

// Where a pair's lie within its token's: lanes that rotate neighbouring eights
// of elements (four neighbouring pairs, or eight in the half layout) read
// neighbouring entries, which no two lanes of a read take from one LDS bank.
__device__ __forceinline__ int pair_at(const RopeAppendArgs &a, int p) {
    const int half = a.rot / 2;
    return a.interleaved ? (p & 3) * (half / 4) + (p >> 2) : (p & 7) * (half / 8) + (p >> 3);
}

// Eight elements [e0, e0 + 8) of one head, and the eight that they are paired
// with in the half layout (rot is a multiple of 16: all eight lie on one side
// of the pairing).
struct Raw {
    uint4 own, other;
};
__device__ __forceinline__ int paired(const RopeAppendArgs &a, int e0) {
    const int half = a.rot / 2;
    return a.interleaved || e0 >= a.rot ? e0 : (e0 < half ? e0 + half : e0 - half);
}
__device__ __forceinline__ Raw load_raw(const RopeAppendArgs &a, const uint16_t *row, int e0) {
    return {*reinterpret_cast<const uint4 *>(row + e0), *reinterpret_cast<const uint4 *>(row + paired(a, e0))};
}

// The rows of a run's tokens, one head of each.  A token past the run reads as
// zeros: its offset lies past the buffer's range.  (Offsets are 32-bit: token
// strides are below 2^24 elements.)
struct Rows {
    __amdgpu_buffer_rsrc_t rsrc;
    int stride;                    // bytes

    __device__ __forceinline__ Rows(const uint16_t *first, int64_t stride_, int n, int d)
        : rsrc(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(first), (short)0,
                                                 (n - 1) * (int)stride_ * 2 + 2 * d, kBufferFlags)),
          stride((int)stride_ * 2) {}
    __device__ __forceinline__ uint4 load16(int i, int e) const {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, i * stride + 2 * e, 0, 0));
    }
};

// what one lane wrote to the wave's part of the LDS is there for the others
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace gdn
