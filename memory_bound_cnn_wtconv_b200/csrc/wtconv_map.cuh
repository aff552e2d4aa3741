// Shared parts of the map operators (RMS norm over channels, dropout): the
// shape they run on, stored-type conversions, and the counter-based mask.
//
// A map is B x C x H x W.  Its rows are the B*H*W pixels, n = b*H*W + p.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wtconv.h"
#include "wtconv_map_geom.h"

namespace wtc {

// Dropout of one call.  Nothing is dropped when `on` is 0.
struct MapDrop {
    uint32_t thresh;                // dropped where the random word is below this
    float grown;                    // factor of what stays: the float next to 1 / (1 - p)
    uint32_t key[20];               // Philox's round keys, two a round (kernel parameters: free operands)
    uint32_t offset;
    const long long* offset_dev;    // added to offset if not NULL (read by the kernel: a replayed graph sees its value)
    int mode;                       // wtconv_drop_mode_t
    int on;
    Divide by_hw;                   // a row's sample
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Sixteen stored bytes and the V = 16 / sizeof(T) floats they hold.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y), f[2] = __uint_as_float(r.z), f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Half a chunk: eight stored bytes.
__device__ __forceinline__ void unpack(const uint2& r, float (&f)[2]) { f[0] = __uint_as_float(r.x), f[1] = __uint_as_float(r.y); }
__device__ __forceinline__ void unpack(const uint2& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x << 16), f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16), f[3] = __uint_as_float(r.y & 0xffff0000u);
}

// One stored value (rows or planes that are not whole chunks).
__device__ __forceinline__ void unpack(float r, float (&f)[1]) { f[0] = r; }
__device__ __forceinline__ void unpack(__nv_bfloat16 r, float (&f)[1]) { f[0] = __bfloat162float(r); }

// N stored values as one register group: uint4 for a chunk, uint2 for half a one, T for one value.
template <typename T, int N>
struct Chunk {
    using type = uint4;
    static __device__ __forceinline__ uint4 zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ uint4 from(const float (&f)[N]) { return pack(f); }
};
template <>
struct Chunk<float, 2> {
    using type = uint2;
    static __device__ __forceinline__ uint2 zero() { return make_uint2(0, 0); }
    static __device__ __forceinline__ uint2 from(const float (&f)[2]) { return make_uint2(__float_as_uint(f[0]), __float_as_uint(f[1])); }
};
template <>
struct Chunk<__nv_bfloat16, 4> {
    using type = uint2;
    static __device__ __forceinline__ uint2 zero() { return make_uint2(0, 0); }
    static __device__ __forceinline__ uint2 from(const float (&f)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};
__device__ __forceinline__ uint32_t& word_of(uint4& r, int k) { return k == 0 ? r.x : k == 1 ? r.y : k == 2 ? r.z : r.w; }
__device__ __forceinline__ uint32_t& word_of(uint2& r, int k) { return k == 0 ? r.x : r.y; }
template <typename T>
struct Chunk<T, 1> {
    using type = T;
    static __device__ __forceinline__ T zero() { return from_f<T>(0.0f); }
    static __device__ __forceinline__ T from(const float (&f)[1]) { return from_f<T>(f[0]); }
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011): four random words from a 128-bit counter and a
// 64-bit key, whose ten round keys come ready made.
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, const uint32_t (&key)[20]) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ key[2 * r];
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ key[2 * r + 1];
        c3 = (uint32_t)a;
    }
    return make_uint4(c0, c1, c2, c3);
}
inline void philox_keys(unsigned long long seed, uint32_t (&key)[20]) {
    for (uint32_t r = 0; r < 10; ++r) {
        key[2 * r] = (uint32_t)seed + r * 0x9E3779B9u;
        key[2 * r + 1] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
    }
}

__device__ __forceinline__ uint32_t drop_offset(const MapDrop& d) {
    return d.offset + (d.offset_dev ? (uint32_t)*d.offset_dev : 0u);
}

// The mask's row: the pixel (element), or the sample (channel, sample).
__device__ __forceinline__ long long drop_row(const MapDrop& d, long long n) {
    return d.mode == WTCONV_DROP_ELEMENT ? n : d.by_hw(n);
}

// The random words of channels 4 * quad .. 4 * quad + 3 of mask row (hi, lo).
// Written so that rows which share quad and hi share the multiplications that
// the first three rounds owe to them alone.
__device__ __forceinline__ uint4 drop_words(const MapDrop& d, uint32_t offset, uint32_t lo, uint32_t hi, uint32_t quad) {
    return philox(quad, lo, hi, offset, d.key);
}
__device__ __forceinline__ uint4 drop_words(const MapDrop& d, uint32_t offset, long long row, uint32_t quad) {
    return philox(quad, (uint32_t)row, (uint32_t)((unsigned long long)row >> 32), offset, d.key);
}
// A sample's one decision.
__device__ __forceinline__ bool keep_sample(const MapDrop& d, uint32_t offset, long long b) {
    return drop_words(d, offset, b, 0).x >= d.thresh;
}
// Four keep bits.
__device__ __forceinline__ uint32_t keep_bits(const MapDrop& d, const uint4& u) {
    return (u.x >= d.thresh ? 1u : 0u) | (u.y >= d.thresh ? 2u : 0u) | (u.z >= d.thresh ? 4u : 0u) |
           (u.w >= d.thresh ? 8u : 0u);
}
// r + d * f of four channels, into r.
__device__ __forceinline__ void drop_add4(const MapDrop& d, const uint4& u, const float* f, float* r) {
    if (u.x >= d.thresh) r[0] = __fmaf_rn(f[0], d.grown, r[0]);
    if (u.y >= d.thresh) r[1] = __fmaf_rn(f[1], d.grown, r[1]);
    if (u.z >= d.thresh) r[2] = __fmaf_rn(f[2], d.grown, r[2]);
    if (u.w >= d.thresh) r[3] = __fmaf_rn(f[3], d.grown, r[3]);
}

// T(r + d * x) of a chunk (or half a one) of pixels of four channels, into r, word
// by word, so that few values are held as floats at once.
template <typename T>
__device__ __forceinline__ void drop_add_words(const MapDrop& d, const uint4 (&u)[sizeof(uint32_t) / sizeof(T)], uint32_t x, uint32_t& r, int j) {
    auto word = [&](int v) { return j == 0 ? u[v].x : j == 1 ? u[v].y : j == 2 ? u[v].z : u[v].w; };
    if constexpr (sizeof(T) == 4) {
        if (word(0) >= d.thresh) r = __float_as_uint(__fmaf_rn(__uint_as_float(x), d.grown, __uint_as_float(r)));
    } else {
        float lo = __uint_as_float(r << 16), hi = __uint_as_float(r & 0xffff0000u);
        if (word(0) >= d.thresh) lo = __fmaf_rn(__uint_as_float(x << 16), d.grown, lo);
        if (word(1) >= d.thresh) hi = __fmaf_rn(__uint_as_float(x & 0xffff0000u), d.grown, hi);
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        r = *reinterpret_cast<const uint32_t*>(&p);
    }
}
template <typename T, typename R>
__device__ __forceinline__ void drop_add_chunks(const MapDrop& d, uint32_t offset, long long row, long long b, int quad,
                                                R (&x)[4], R (&r)[4]) {
    constexpr int N = sizeof(uint32_t) / sizeof(T);  // pixels of a word
    const uint32_t lo = (uint32_t)row, hi = (uint32_t)((unsigned long long)row >> 32);
    uint4 u[N];
    const bool element = d.mode == WTCONV_DROP_ELEMENT;
    if (!element) {
        u[0] = drop_words(d, offset, b, d.mode == WTCONV_DROP_SAMPLE ? 0 : quad);
        if (d.mode == WTCONV_DROP_SAMPLE) u[0].y = u[0].z = u[0].w = u[0].x;
        u[N - 1] = u[0];
    }
#pragma unroll
    for (int k = 0; k < (int)sizeof(R) / 4; ++k) {
        if (element) {
#pragma unroll
            for (int v = 0; v < N; ++v) u[v] = drop_words(d, offset, lo + k * N + v, hi, quad);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) drop_add_words<T>(d, u, word_of(x[j], k), word_of(r[j], k), j);
    }
}

// r + d * f of N pixels of four channels, into r; row: the first pixel's (all of
// them share its upper word); b: the sample.
template <int N>
__device__ __forceinline__ void drop_add_tile(const MapDrop& d, uint32_t offset, long long row, long long b, int quad,
                                              const float (&f)[4][N], float (&r)[4][N]) {
    if (d.mode == WTCONV_DROP_ELEMENT) {
        const uint32_t lo = (uint32_t)row, hi = (uint32_t)((unsigned long long)row >> 32);
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const uint4 u = drop_words(d, offset, lo + v, hi, quad);
            if (u.x >= d.thresh) r[0][v] = __fmaf_rn(f[0][v], d.grown, r[0][v]);
            if (u.y >= d.thresh) r[1][v] = __fmaf_rn(f[1][v], d.grown, r[1][v]);
            if (u.z >= d.thresh) r[2][v] = __fmaf_rn(f[2][v], d.grown, r[2][v]);
            if (u.w >= d.thresh) r[3][v] = __fmaf_rn(f[3][v], d.grown, r[3][v]);
        }
    } else {
        const bool sample = d.mode == WTCONV_DROP_SAMPLE;
        uint4 u = drop_words(d, offset, b, sample ? 0 : quad);
        if (sample) u.y = u.z = u.w = u.x;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            if (u.x >= d.thresh) r[0][v] = __fmaf_rn(f[0][v], d.grown, r[0][v]);
            if (u.y >= d.thresh) r[1][v] = __fmaf_rn(f[1][v], d.grown, r[1][v]);
            if (u.z >= d.thresh) r[2][v] = __fmaf_rn(f[2][v], d.grown, r[2][v]);
            if (u.w >= d.thresh) r[3][v] = __fmaf_rn(f[3][v], d.grown, r[3][v]);
        }
    }
}

// a * b + c, a * b and a + b of N floats, two at an instruction where N is even.
template <int N>
__device__ __forceinline__ void fma_n(const float (&a)[N], const float (&b)[N], float (&c)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 t = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]));
            c[e] = t.x, c[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) c[e] = __fmaf_rn(a[e], b[e], c[e]);
    }
}
template <int N>
__device__ __forceinline__ void fma_n(const float (&a)[N], float b, float (&c)[N]) {
    float t[N];
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = b;
    fma_n(a, t, c);
}
template <int N>
__device__ __forceinline__ void mul_n(float (&a)[N], const float (&b)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 t = __fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
            a[e] = t.x, a[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = __fmul_rn(a[e], b[e]);
    }
}
template <int N>
__device__ __forceinline__ void mul_n(float (&a)[N], float b) {
    float t[N];
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = b;
    mul_n(a, t);
}
template <int N>
__device__ __forceinline__ void add_n(float (&a)[N], const float (&b)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const float2 t = __fadd2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
            a[e] = t.x, a[e + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) a[e] = __fadd_rn(a[e], b[e]);
    }
}

}  // namespace wtc
