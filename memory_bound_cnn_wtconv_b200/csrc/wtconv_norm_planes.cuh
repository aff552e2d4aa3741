// RMS norm of maps whose pixels are adjacent (NCHW).
//
// A CTA walks tiles of lp * VP neighbouring pixels of one sample with all their
// channels.  lp lanes of a warp lie along the pixels, VP of them each; the other
// lanes and the warps share out the channels in quads of four, since a random
// word quad covers four channels: owner o has the quads o, o + owners, ...
//
// The inputs of the next tile come into shared memory (cp.async, 16 bytes)
// while this one is computed.  VP = 16 bytes of pixels where planes are whole
// 16-byte chunks, 8 where they are whole halves: each thread copies the chunks
// that it owns itself, so nothing but its own copies has to arrive.  Where they
// are neither (RAG, "ragged"), each channel's pixels come as the aligned chunks
// that cover them, shifted by the plane's own distance from a 16-byte boundary,
// and are read value by value: a thread then has the pixels pl, pl + lp, ...,
// four of them.
//
// Bound by memory.  Without the copies ahead a CTA loads, waits, sums and
// stores in turn, and too few CTAs fit an SM to hide it: 388 us for the
// backward of 32 x 512 x 64 x 64 fp32 with the gradient of h.
//
// The squares are summed over an owner's channels, the lanes, then the warps
// (tile_sum).  The weight gradient's sums of a thread's own channels stay in
// its registers for all its tiles.
#pragma once

#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "wtconv_norm.cuh"

namespace wtc {

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

__device__ __forceinline__ void copy16(void* to, const void* from, int bytes) {  // the rest of the 16 bytes as zeros
    const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(to));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(void* to, const void* from, int bytes) {
    const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(to));
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(s), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// Where a thread is: its tile, and its channels' places in it.
template <typename T, int VP, int RAG>
struct Tile {
    using R = typename Chunk<T, VP>::type;

    const MapShape& m;
    const PlanesGeom& geom;
    char* smem;
    int pl, owner;
    uint32_t own;       // this thread's first pixel of its first channel, from the tile's first element on
    long long b;
    int p0;             // first pixel of the tile
    int live;           // how many of this thread's pixels are the map's
    long long origin;   // the tile's first element

    __device__ __forceinline__ int lp() const { return RAG > 1 ? RAG : geom.lp; }
    __device__ __forceinline__ Tile(const MapShape& shape, const PlanesGeom& g, char* s) : m(shape), geom(g), smem(s) {
        const int lane = threadIdx.x % 32;
        pl = lane & (lp() - 1);
        owner = (threadIdx.x / 32) * (32 / lp()) + lane / lp();
        own = 4u * owner * m.HW + pixel(0);
    }
    // The tile's pixel that is this thread's e-th.
    __device__ __forceinline__ int pixel(int e) const { return RAG ? pl + e * lp() : pl * VP + e; }
    __device__ __forceinline__ void at(long long tile) {
        b = geom.by_tiles(tile);
        p0 = (int)(tile - b * geom.tiles) * lp() * VP;
        origin = b * m.C * m.HW + p0;
        const int left = m.HW - p0 - pixel(0);  // chunks: HW is a multiple of VP
        live = !RAG ? (left > 0 ? VP : 0) : left <= 0 ? 0 : min(VP, (left - 1) / lp() + 1);
    }
    // This thread's pixels of one value for each of the tile's.
    __device__ __forceinline__ void get(const float* p, float (&v)[VP]) const {
        if constexpr (RAG) {
#pragma unroll
            for (int e = 0; e < VP; ++e) v[e] = p[pixel(e)];
        } else if constexpr (VP == 2) {
            const float2 q = *reinterpret_cast<const float2*>(p + pixel(0));
            v[0] = q.x, v[1] = q.y;
        } else {
#pragma unroll
            for (int e = 0; e < VP; e += 4) {
                const float4 q = *reinterpret_cast<const float4*>(p + pixel(e));
                v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
            }
        }
    }
    __device__ __forceinline__ bool has(int e) const { return RAG ? e < live : true; }
    __device__ __forceinline__ long long row() const { return b * m.HW + p0 + pixel(0); }
    __device__ __forceinline__ int channel(int g, int j) const { return 4 * (g * geom.owners + owner) + j; }
    __device__ __forceinline__ bool in(int g, int j) const { return live && channel(g, j) < m.C; }
    // This thread's first pixel of channel(g, j), from the tile's first element on.
    __device__ __forceinline__ uint32_t offset(int g, int j) const { return own + (uint32_t)(4 * g * geom.owners + j) * m.HW; }

    __device__ __forceinline__ R raw(int stage, int tensors, int k, int g, int j) const {
        return reinterpret_cast<const R*>(smem + (stage * tensors + k) * geom.tensor)[(4 * g + j) * blockDim.x + threadIdx.x];
    }
    // This thread's pixels of channel(g, j) of tensor k of a stage, as floats;
    // ragged: anything for those that it does not have.
    __device__ __forceinline__ void load(int stage, int tensors, int k, int g, int j, float (&f)[VP]) const {
        if constexpr (RAG) {
            const char* s = smem + (stage * tensors + k) * geom.tensor;
            const int c = channel(g, j);
            const uint32_t first = ((uint32_t)origin + (uint32_t)c * m.HW) * (uint32_t)sizeof(T);  // modulo 2^32
            const T* p = reinterpret_cast<const T*>(s + c * geom.row + (first & 15)) + pl;
#pragma unroll
            for (int e = 0; e < VP; ++e) f[e] = to_f(p[e * lp()]);
        } else {
            unpack(raw(stage, tensors, k, g, j), f);
        }
    }
    // The same from a map in global memory.
    __device__ __forceinline__ void load(const void* from, int g, int j, float (&f)[VP]) const {
        const T* p = static_cast<const T*>(from) + origin + offset(g, j);
        if constexpr (RAG) {
#pragma unroll
            for (int e = 0; e < VP; ++e) f[e] = e < live ? to_f(p[e * lp()]) : 0.0f;
        } else {
            unpack(*reinterpret_cast<const R*>(p), f);
        }
    }
    // To a map in global memory, rounded to its type.
    __device__ __forceinline__ void store(void* to, int g, int j, const float (&f)[VP]) const {
        T* p = static_cast<T*>(to) + origin + offset(g, j);
        if constexpr (RAG) {
#pragma unroll
            for (int e = 0; e < VP; ++e)
                if (e < live) p[e * lp()] = from_f<T>(f[e]);
        } else {
            *reinterpret_cast<R*>(p) = Chunk<T, VP>::from(f);
        }
    }
    // r + dropout of f of quad g, into r.
    __device__ __forceinline__ void drop(const MapDrop& d, uint32_t off, int g, const float (&f)[4][VP], float (&r)[4][VP]) const {
        const int quad = channel(g, 0) / 4;
        if (!RAG || d.mode != WTCONV_DROP_ELEMENT) {
            drop_add_tile<VP>(d, off, row(), b, quad, f, r);
        } else {
#pragma unroll
            for (int e = 0; e < VP; ++e) {
                const uint4 u = drop_words(d, off, row() + e * lp(), quad);
                if (u.x >= d.thresh) r[0][e] = __fmaf_rn(f[0][e], d.grown, r[0][e]);
                if (u.y >= d.thresh) r[1][e] = __fmaf_rn(f[1][e], d.grown, r[1][e]);
                if (u.z >= d.thresh) r[2][e] = __fmaf_rn(f[2][e], d.grown, r[2][e]);
                if (u.w >= d.thresh) r[3][e] = __fmaf_rn(f[3][e], d.grown, r[3][e]);
            }
        }
    }

    // Starts the copies of this tile's tensors; with skip, zeros for the first.
    template <int G, int NT>
    __device__ __forceinline__ void fetch(int stage, const void* const (&from)[NT], int tensors, bool skip) const {
        char* s = smem + stage * tensors * geom.tensor;
        if constexpr (RAG) {
            const long long bytes = m.rows * m.C * (long long)sizeof(T);
            const int pixels = min(lp() * VP, m.HW - p0), chunks = geom.row / 16;
            const int n = m.C * chunks;
            for (int i = threadIdx.x; i < n; i += blockDim.x) {
                const int c = (int)((__umulhi((uint32_t)i, geom.by_chunks.mul) + (uint32_t)i) >> geom.by_chunks.shift);
                const int q = i - c * chunks;
                const long long first = (origin + (uint32_t)c * m.HW) * (long long)sizeof(T);
                const int span = (int)(first & 15) + pixels * (int)sizeof(T);  // from the chunk boundary on
                if (16 * q >= span) continue;
                const long long at = (first & ~15LL) + 16 * q;
                const int count = (int)min(16LL, bytes - at);
                char* to = s + c * geom.row + 16 * q;
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    if (k < tensors) copy16(to + k * geom.tensor, static_cast<const char*>(from[k]) + at, k == 0 && skip ? 0 : count);
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool ok = in(g, j);
                    const long long at = origin + (ok ? offset(g, j) : 0u);
                    char* to = s + ((4 * g + j) * blockDim.x + threadIdx.x) * sizeof(R);
#pragma unroll
                    for (int k = 0; k < NT; ++k) {
                        if (k >= tensors) continue;
                        const int bytes = ok && !(k == 0 && skip) ? (int)sizeof(R) : 0;
                        if constexpr (sizeof(R) == 16) copy16(to + k * geom.tensor, static_cast<const T*>(from[k]) + at, bytes);
                        else copy8(to + k * geom.tensor, static_cast<const T*>(from[k]) + at, bytes);
                    }
                }
            }
        }
    }
    // A stage has arrived (and, where threads read what others copied, for all
    // of them; their reads of the other stage are over).
    __device__ __forceinline__ void arrive() const {
        copies_wait<0>();
        if constexpr (RAG) __syncthreads();
    }
};

// One sum for each pixel of the tile over all owners of channels, through
// `finish(pixel of the tile, sum)`, which runs once a pixel; every owner gets
// its result.  smem: [warps + 1][lp * VP] floats.
template <int VP, typename Tl, typename F>
__device__ __forceinline__ void tile_sum(const Tl& tile, float (&v)[VP], float* smem, F finish) {
    const int lp = tile.lp(), warps = blockDim.x / 32, lane = threadIdx.x % 32, px = lp * VP;
    for (int o = lp; o < 32; o *= 2) {
#pragma unroll
        for (int e = 0; e < VP; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    }
    if (lane < lp) {
#pragma unroll
        for (int e = 0; e < VP; ++e) smem[(threadIdx.x / 32) * px + tile.pixel(e)] = v[e];
    }
    __syncthreads();
    for (int p = threadIdx.x; p < px; p += blockDim.x) {
        float s = smem[p];
        for (int k = 1; k < warps; ++k) s += smem[k * px + p];
        smem[warps * px + p] = finish(p, s);
    }
    __syncthreads();
    tile.get(smem + warps * px, v);
}

// go(RAG, G) with the geometry's numbers as constants (RAG 1: a runtime lp).
template <int RAG, typename F>
int planes_dispatch(const PlanesGeom& g, F go) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one{};
    constexpr integral_constant<int, 2> two{};
    if constexpr (RAG != 0) {
        if (g.lp != RAG) return g.iters == 1 ? go(one, one) : go(one, two);
    }
    constexpr integral_constant<int, RAG> rag{};
    return g.iters == 1 ? go(rag, one) : go(rag, two);
}

// Lets a kernel have the shared memory that any call asks for, once per kernel
// and device.  The limit belongs to the kernel, not to a call: set to each
// call's own size it would fall below what a call on another host thread is
// about to launch with.  Threads that meet in the first call set the same value.
template <auto kernel>
cudaError_t opt_in_smem() {
    static std::atomic<bool> done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (e != cudaSuccess || (known && done[dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
    if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_release);
    return e;
}

// Launches a kernel on at most `most` CTAs, as many as the SMs hold at once.
// An error is left for the caller's cudaGetLastError().
template <auto kernel, typename A>
int launch(const MapShape& m, const A& a, const MapDrop& d, const PlanesGeom& g, size_t smem, long long most, int sms, cudaStream_t s) {
    const int threads = g.warps * 32;
    long long ctas = std::min(m.rows / m.HW * g.tiles, most);
    if (smem > 48 * 1024 && opt_in_smem<kernel>() != cudaSuccess) return 1;
    if (ctas > sms) ctas = std::min(ctas, (long long)norm_resident(kernel, threads, smem) * sms);
    kernel<<<(unsigned)ctas, threads, smem, s>>>(m, a, d, g);
    return (int)ctas;
}

inline bool all_aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if ((uintptr_t)p % 16) return false;
    return true;
}

cudaError_t launch_norm_planes_long_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);
cudaError_t launch_norm_planes_long_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);

}  // namespace wtc
