// Shared parts of the map operators (RMS norm over channels, dropout): the
// shape they run on, stored-type conversions, and the counter-based mask.
//
// A map is B x C x H x W.  Its rows are the B*H*W pixels, n = b*H*W + p; the
// C values of a row are `cs` elements apart (NHWC: 1, NCHW: H*W).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wtconv.h"

namespace wtc {

struct MapShape {
    long long rows;  // B * H * W
    int C, HW;
    int nhwc;        // 1: the C values of a row are adjacent
};

// Dropout of one call.  Nothing is dropped when `on` is 0.
struct MapDrop {
    uint32_t thresh;                // dropped where the random word is below this
    float grown;                    // factor of what stays: the float next to 1 / (1 - p)
    uint32_t k0, k1;                // Philox key: the seed
    uint32_t offset;
    const long long* offset_dev;    // added to offset if not NULL (read by the kernel: a replayed graph sees its value)
    int mode;                       // wtconv_drop_mode_t
    int on;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): four random words from a 128-bit counter and a
// 64-bit key.
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint32_t drop_offset(const MapDrop& d) {
    return d.offset + (d.offset_dev ? (uint32_t)*d.offset_dev : 0u);
}

// The mask's row: the pixel (element), or the sample (channel, sample).
__device__ __forceinline__ long long drop_row(const MapDrop& d, const MapShape& m, long long n) {
    return d.mode == WTCONV_DROP_ELEMENT ? n : n / m.HW;
}

// Keep bits (bit j: channel 4 * quad + j) of one mask row.
__device__ __forceinline__ uint32_t keep_quad(const MapDrop& d, uint32_t offset, long long row, uint32_t quad) {
    const uint4 u = philox(quad, (uint32_t)row, (uint32_t)((unsigned long long)row >> 32), offset, d.k0, d.k1);
    if (d.mode == WTCONV_DROP_SAMPLE) return u.x >= d.thresh ? 15u : 0u;
    return (u.x >= d.thresh ? 1u : 0u) | (u.y >= d.thresh ? 2u : 0u) | (u.z >= d.thresh ? 4u : 0u) |
           (u.w >= d.thresh ? 8u : 0u);
}

}  // namespace wtc
