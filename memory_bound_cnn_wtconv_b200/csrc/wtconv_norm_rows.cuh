// What the RMS norm kernels of maps whose channels are adjacent (NHWC, rows)
// share.
//
// A row belongs to a team of `tpr` threads: a part of a warp, a warp, or, for
// long rows, a CTA.  Thread t of it owns slots t, t + tpr, ... of every row the
// team meets, NV of them, in registers between the sum of squares and the
// output: h is read from memory once.  A slot is a 16-byte chunk of channels
// (V = 16 / sizeof(T)) where rows are whole chunks, else one channel (V = 1;
// neighbouring lanes then still read neighbouring values).  NV = 0 is for rows
// longer than a CTA's registers: the slots are read again.
#pragma once

#include <type_traits>

#include "wtconv_norm.cuh"

namespace wtc {

// Whether a kernel is for teams within a warp only (CTA-wide ones have four
// chunks or any number of single channels a thread), so for kTeamThreads.
template <int V, int NV, int TPR>
constexpr bool kWithinWarp = NV != 0 && (V > 1 ? NV != 4 : TPR != 0);

// go(nv, tpr) with the geometry's numbers as constants (tpr 0: a runtime one).
// WARP: with the teams that only whole warps need.
template <int V, bool WARP, typename F>
void rows_dispatch(const RowsGeom& g, F go) {
    using std::integral_constant;
    constexpr integral_constant<int, 0> any{};
    if constexpr (V > 1) {
        switch (g.nv) {
            case 1: return go(integral_constant<int, 1>{}, any);
            case 2: return go(integral_constant<int, 2>{}, any);
            case 3: return go(integral_constant<int, 3>{}, any);
            case 4: return go(integral_constant<int, 4>{}, any);
        }
    } else {
        if (g.nv == 4 && g.tpr == 4) return go(integral_constant<int, 4>{}, integral_constant<int, 4>{});
        if (g.nv == 4 && g.tpr == 8) return go(integral_constant<int, 4>{}, integral_constant<int, 8>{});
        if (g.nv == 8 && g.tpr == 8) return go(integral_constant<int, 8>{}, integral_constant<int, 8>{});
        if (g.nv == 8 && g.tpr == 16) return go(integral_constant<int, 8>{}, integral_constant<int, 16>{});
        if constexpr (WARP) {
            if (g.nv == 2 && g.tpr == 32) return go(integral_constant<int, 2>{}, integral_constant<int, 32>{});
            if (g.nv == 4 && g.tpr == 32) return go(integral_constant<int, 4>{}, integral_constant<int, 32>{});
        }
        if (g.nv == 8 && g.tpr == 32) return go(integral_constant<int, 8>{}, integral_constant<int, 32>{});
        if (g.nv == 16 && g.tpr == 32) return go(integral_constant<int, 16>{}, integral_constant<int, 32>{});
        if (g.nv == 8) return go(integral_constant<int, 8>{}, any);
        if (g.nv == 16) return go(integral_constant<int, 16>{}, any);
    }
    go(any, any);
}

// Sum (or largest bits) over a team; `red` holds one value a warp.
__device__ __forceinline__ float team_sum(float v, int tpr, float* red) {
    for (int o = min(tpr, 32) / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr > 32) {
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.0f;
        for (int k = 0; k < tpr / 32; ++k) v += red[k];
        __syncthreads();
    }
    return v;
}
__device__ __forceinline__ uint32_t team_max(uint32_t v, int tpr, float* red) {
    for (int o = min(tpr, 32) / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr > 32) {
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = __uint_as_float(v);
        __syncthreads();
        v = 0;
        for (int k = 0; k < tpr / 32; ++k) v = max(v, __float_as_uint(red[k]));
        __syncthreads();
    }
    return v;
}

// The weights of a slot.
template <int V>
__device__ __forceinline__ void load_weight(const float* w, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = *w;
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(w + e);
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    }
}

// r + d * f of N slots i0, i0 + 1, ... of a thread, into r.  Chunks draw their
// own quads.  Four single channels of a lane lie in four quads that it shares
// with three neighbours: each of the four draws one, then they exchange words
// (a transpose of 4 x 4 in two steps of two shuffles).
template <int V, int N>
__device__ __forceinline__ void drop_add_slots(const MapDrop& d, uint32_t offset, long long drow, int i0, int tpr, int t,
                                               const float (&f)[N][V], float (&r)[N][V]) {
    if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int e = 0; e < V; e += 4)
                drop_add4(d, drop_words(d, offset, drow, (((i0 + i) * tpr + t) * V + e) >> 2), f[i] + e, r[i] + e);
        }
    } else {
        static_assert(N % 4 == 0);
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            uint4 u = drop_words(d, offset, drow, ((i0 + i + (t & 3)) * tpr + (t & ~3)) >> 2);
            const bool odd = t & 1, high = t & 2;
            uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? u.x : u.y, 1);
            uint32_t b = __shfl_xor_sync(0xffffffffu, odd ? u.z : u.w, 1);
            // lanes 0, 2: words 0 and 2 of this pair of lanes; lanes 1, 3: words 1 and 3
            const uint32_t p0 = odd ? a : u.x, p1 = odd ? u.y : a, q0 = odd ? b : u.z, q1 = odd ? u.w : b;
            a = __shfl_xor_sync(0xffffffffu, high ? p0 : q0, 2);
            b = __shfl_xor_sync(0xffffffffu, high ? p1 : q1, 2);
            u = make_uint4(high ? a : p0, high ? b : p1, high ? q0 : a, high ? q1 : b);
            if (u.x >= d.thresh) r[i][0] = __fmaf_rn(f[i][0], d.grown, r[i][0]);
            if (u.y >= d.thresh) r[i + 1][0] = __fmaf_rn(f[i + 1][0], d.grown, r[i + 1][0]);
            if (u.z >= d.thresh) r[i + 2][0] = __fmaf_rn(f[i + 2][0], d.grown, r[i + 2][0]);
            if (u.w >= d.thresh) r[i + 3][0] = __fmaf_rn(f[i + 3][0], d.grown, r[i + 3][0]);
        }
    }
}

inline bool aligned_to(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

}  // namespace wtc
