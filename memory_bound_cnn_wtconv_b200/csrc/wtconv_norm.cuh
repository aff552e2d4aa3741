// What the two layouts' RMS norm kernels share (the formulas: wtconv_norm.cu).
#pragma once

#include <cuda_fp8.h>

#include <algorithm>

#include "wtconv_map_launch.h"

namespace wtc {

// CTAs of a kernel that an SM holds.
template <typename K>
int norm_resident(K kernel, int threads, size_t smem) {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) == cudaSuccess && n > 0 ? n : 1;
}

// How JOIN reads h: x itself, residual + x, or residual + dropout of x.
enum { kPlain = 0, kResidual = 1, kDropped = 2 };

// The scale of a group whose largest |v| has these bits (one rounding more than
// the quotient), and what its values are multiplied with: the reciprocal to one
// unit in the last place, so that q is v / scale with two roundings more, far
// within its own rounding to 8 bits.
__device__ __forceinline__ float q8_scale(uint32_t bits, int q8) {
    const float s = __uint_as_float(bits) * (q8 == WTCONV_E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f);
    return s < 1.17549435e-38f ? 1.17549435e-38f : s;  // a NaN stays
}
__device__ __forceinline__ float q8_inverse(float scale) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(scale));
    return r;
}

// c >> this is the group of channel c: groups are a power of two of channels, or all of them one.
__device__ __forceinline__ int group_shift(int group, int groups) { return groups == 1 ? 31 : 31 - __clz(group); }

// A whole number; |v| is 127 and a few units in the last place at most, and a
// NaN is 0 by the conversion's definition.
__device__ __forceinline__ uint32_t q8_whole(float v) { return (uint32_t)__float2int_rn(v) & 255; }

// Four values to four bytes.
__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d, int q8) {
    if (q8 == WTCONV_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
    return q8_whole(a) | q8_whole(b) << 8 | q8_whole(c) << 16 | q8_whole(d) << 24;
}

__device__ __forceinline__ uint8_t q8_one(float v, int q8) {
    if (q8 == WTCONV_E4M3) return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    return (uint8_t)q8_whole(v);
}

// |v| as bits that are ordered like |v|, NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

cudaError_t launch_norm_rows_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);
cudaError_t launch_norm_rows_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s);
cudaError_t launch_norm_planes_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);
cudaError_t launch_norm_planes_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s);

}  // namespace wtc
