// What the RMS norm kernels of maps whose pixels are adjacent (NCHW) share.
#pragma once

#include "wtconv_norm.cuh"

namespace wtc {

// 4 * VP keep bits: bit j * VP + v is channel 4 * quad + j of pixel v.
template <int VP>
__device__ __forceinline__ uint32_t keep_tile(const MapDrop& d, uint32_t offset, long long row, long long b, int quad) {
    uint32_t bits = 0;
    if (d.mode == WTCONV_DROP_ELEMENT) {
#pragma unroll
        for (int v = 0; v < VP; ++v) {
            const uint4 u = drop_words(d, offset, row + v, quad);
            bits |= (u.x >= d.thresh ? 1u << v : 0u) | (u.y >= d.thresh ? 1u << (VP + v) : 0u) |
                    (u.z >= d.thresh ? 1u << (2 * VP + v) : 0u) | (u.w >= d.thresh ? 1u << (3 * VP + v) : 0u);
        }
    } else {
        const uint32_t k = keep_bits(d, drop_words(d, offset, b, quad));
#pragma unroll
        for (int j = 0; j < 4; ++j) bits |= k >> j & 1 ? ((1u << VP) - 1) << (j * VP) : 0u;
    }
    return bits;
}

// One sum for each pixel of the tile over all owners of channels, through
// `finish(pixel of the tile, sum)`, which runs once a pixel; every owner gets
// its result.  smem: [warps + 1][lp * VP] floats.
template <int VP, typename F>
__device__ __forceinline__ void lane_tile_sum(float (&v)[VP], int lp, float* smem, F finish) {
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32, pl = lane & (lp - 1), px = lp * VP;
    for (int o = lp; o < 32; o *= 2) {
#pragma unroll
        for (int e = 0; e < VP; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    }
    if (lane < lp) {
#pragma unroll
        for (int e = 0; e < VP; ++e) smem[(threadIdx.x / 32) * px + pl * VP + e] = v[e];
    }
    __syncthreads();
    for (int p = threadIdx.x; p < px; p += blockDim.x) {
        float s = smem[p];
        for (int k = 1; k < warps; ++k) s += smem[k * px + p];
        smem[warps * px + p] = finish(p, s);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VP; ++e) v[e] = smem[warps * px + pl * VP + e];
}

// Eight-bit values of VP pixels to o.
template <int VP>
__device__ __forceinline__ void q8_store(uint8_t* o, const float (&f)[VP], int q8) {
    if constexpr (VP == 1) {
        *o = q8_one(f[0], q8);
    } else if constexpr (VP == 2) {
        *reinterpret_cast<uint16_t*>(o) = (uint16_t)q8_pack4(f[0], f[1], 0.0f, 0.0f, q8);
    } else if constexpr (VP == 4) {
        *reinterpret_cast<uint32_t*>(o) = q8_pack4(f[0], f[1], f[2], f[3], q8);
    } else {
        *reinterpret_cast<uint2*>(o) = make_uint2(q8_pack4(f[0], f[1], f[2], f[3], q8), q8_pack4(f[4], f[5], f[6], f[7], q8));
    }
}

cudaError_t launch_norm_planes_long_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);
cudaError_t launch_norm_planes_long_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);

}  // namespace wtc
