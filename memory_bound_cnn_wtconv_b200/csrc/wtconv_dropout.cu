// Counter-based dropout of a map: y = residual + d * x, d = 0 or the float
// next to 1 / (1 - p).  The mask is a function of (seed, offset, row,
// channel) alone, so it is never stored: the backward is the same kernel on dy.
//
// Bound by memory: x (and the residual) read once, y written once.  A random
// quad covers four channels of a pixel, and each kernel gives a thread all of
// what it draws:
//   rows    channels adjacent: a 16-byte chunk of channels (one or two quads);
//   planes  pixels adjacent: a 16-byte chunk of pixels of four channels (one
//           quad a pixel), or single pixels where planes are not whole chunks;
//   spans   whole stretches of memory under one decision (samples in either
//           layout, channels of NCHW): x is not read where it is dropped.
#include <algorithm>

#include "wtconv_map_launch.h"

namespace wtc {

namespace {

constexpr int kThreads = 256;
// Shorter stretches under one decision go to the rows and planes kernels.
constexpr long long kLeastSpan = 2048;

template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) wtconv_dropout_rows_kernel(MapShape m, DropArgs a, MapDrop d, Divide by_slots, Divide by_hw, int vec) {
    constexpr int V = kVec<T>;
    const int slots = (int)by_slots.d;
    const long long n = m.rows * slots, step = (long long)gridDim.x * kThreads;
    const uint32_t offset = drop_offset(d);
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        const long long row = by_slots(i);
        const int c = (int)(i - row * slots) * V;
        const long long base = row * m.C;
        const uint4 x = load_channels(static_cast<const T*>(a.x) + base, c, m.C, vec);
        uint4 res = make_uint4(0, 0, 0, 0);
        if (RES) res = load_channels(static_cast<const T*>(a.residual) + base, c, m.C, vec);
        const long long drow = d.mode == WTCONV_DROP_ELEMENT ? row : by_hw(row);
        float f[V], r[V];
        unpack(x, f);
        unpack(res, r);
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            uint4 u = drop_words(d, offset, drow, d.mode == WTCONV_DROP_SAMPLE ? 0 : (c + e) >> 2);
            if (d.mode == WTCONV_DROP_SAMPLE) u = make_uint4(u.x, u.x, u.x, u.x);
            drop_add4(d, u, f + e, r + e);
        }
        store_channels(static_cast<T*>(a.y) + base, c, m.C, vec, pack(r));
    }
}

template <typename T, int VP, bool RES>
__global__ void __launch_bounds__(kThreads) wtconv_dropout_planes_kernel(MapShape m, DropArgs a, MapDrop d, Divide by_chunks, Divide by_quads) {
    using R = typename Chunk<T, VP>::type;
    const int quads = (int)by_quads.d, chunks = (int)by_chunks.d;
    const long long n = m.rows / VP * quads, step = (long long)gridDim.x * kThreads;
    const uint32_t offset = drop_offset(d);
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        const long long bq = by_chunks(i), b = by_quads(bq);
        const int p = (int)(i - bq * chunks) * VP, quad = (int)(bq - b * quads);
        const long long base = (b * m.C + 4 * quad) * m.HW + p;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        R rx[4], rr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * quad + j < m.C) {
                rx[j] = *reinterpret_cast<const R*>(x + (long long)j * m.HW);
                if (RES) rr[j] = *reinterpret_cast<const R*>(res + (long long)j * m.HW);
            }
        uint32_t keep[4] = {};  // bit v: pixel v
        if (d.mode == WTCONV_DROP_ELEMENT) {
#pragma unroll
            for (int v = 0; v < VP; ++v) {
                const uint4 u = drop_words(d, offset, b * m.HW + p + v, quad);
                keep[0] |= u.x >= d.thresh ? 1u << v : 0u;
                keep[1] |= u.y >= d.thresh ? 1u << v : 0u;
                keep[2] |= u.z >= d.thresh ? 1u << v : 0u;
                keep[3] |= u.w >= d.thresh ? 1u << v : 0u;
            }
        } else {
            const bool sample = d.mode == WTCONV_DROP_SAMPLE;
            const uint4 u = drop_words(d, offset, b, sample ? 0 : quad);
            keep[0] = u.x >= d.thresh ? ~0u : 0u;
            keep[1] = (sample ? u.x : u.y) >= d.thresh ? ~0u : 0u;
            keep[2] = (sample ? u.x : u.z) >= d.thresh ? ~0u : 0u;
            keep[3] = (sample ? u.x : u.w) >= d.thresh ? ~0u : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * quad + j < m.C) {
                float f[VP], r[VP] = {};
                unpack(rx[j], f);
                if (RES) unpack(rr[j], r);
#pragma unroll
                for (int e = 0; e < VP; ++e)
                    if (keep[j] >> e & 1) r[e] = __fmaf_rn(f[e], d.grown, r[e]);
                *reinterpret_cast<R*>(static_cast<T*>(a.y) + base + (long long)j * m.HW) = Chunk<T, VP>::from(r);
            }
    }
}

// Spans of `len` adjacent elements, each under one decision; blockIdx.y walks
// the spans and blockIdx.x shares one out.  All three pointers are equally far
// from a 16-byte boundary where vec is set.
template <typename T, bool RES>
__global__ void __launch_bounds__(kThreads) wtconv_dropout_spans_kernel(MapShape m, DropArgs a, MapDrop d, long long spans, long long len, int vec) {
    constexpr int V = kVec<T>;
    const uint32_t offset = drop_offset(d);
    for (long long k = blockIdx.y; k < spans; k += gridDim.y) {
        bool keep;
        if (d.mode == WTCONV_DROP_SAMPLE || !d.on) {
            keep = keep_sample(d, offset, k);
        } else {
            const long long b = k / m.C;
            const int c = (int)(k - b * m.C);
            keep = keep_bits(d, drop_words(d, offset, b, c >> 2)) >> (c & 3) & 1;
        }
        const T* x = static_cast<const T*>(a.x) + k * len;
        const T* res = static_cast<const T*>(a.residual) + k * len;
        T* y = static_cast<T*>(a.y) + k * len;
        auto one = [&](long long i) {
            const float r = RES ? to_f(res[i]) : 0.0f;
            y[i] = from_f<T>(keep ? __fmaf_rn(to_f(x[i]), d.grown, r) : r);
        };
        const long long head = vec ? min(len, (long long)((16 - (uintptr_t)y % 16) % 16 / sizeof(T))) : len;
        const long long body = (len - head) / V, first = (long long)blockIdx.x * kThreads + threadIdx.x;
        const long long step = (long long)gridDim.x * kThreads;
        const uint4* xv = reinterpret_cast<const uint4*>(x + head);
        const uint4* rv = reinterpret_cast<const uint4*>(res + head);
        uint4* yv = reinterpret_cast<uint4*>(y + head);
        if (keep) {
#pragma unroll 4
            for (long long i = first; i < body; i += step) {
                float f[V], r[V] = {};
                unpack(xv[i], f);
                if (RES) unpack(rv[i], r);
#pragma unroll
                for (int e = 0; e < V; ++e) r[e] = __fmaf_rn(f[e], d.grown, r[e]);
                yv[i] = pack(r);
            }
        } else {
#pragma unroll 4
            for (long long i = first; i < body; i += step) yv[i] = RES ? rv[i] : make_uint4(0, 0, 0, 0);
        }
        for (long long i = first; i < head; i += step) one(i);
        for (long long i = head + body * V + first; i < len; i += step) one(i);
    }
}

template <typename T, bool RES>
void run(const MapShape& m, const DropArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const uintptr_t ax = (uintptr_t)a.x % 16, ar = (uintptr_t)a.residual % 16, ay = (uintptr_t)a.y % 16;
    const bool whole = !ax && !ar && !ay;
    auto ctas = [&](long long threads) { return (unsigned)std::min((threads + kThreads - 1) / kThreads, 64LL * sms); };
    // Nothing dropped: one span, kept by any decision (the threshold is 0).
    const bool sample = d.mode == WTCONV_DROP_SAMPLE;
    const long long samples = m.rows / m.HW, spans = !d.on ? 1 : samples * (sample ? 1 : m.C), len = m.rows * m.C / spans;
    const bool stretches = !d.on || sample || (d.mode == WTCONV_DROP_CHANNEL && !m.nhwc);
    if (stretches && len >= kLeastSpan) {
        const bool vec = ax == ay && (!RES || ar == ay);
        const unsigned across = (unsigned)std::min((len / V + kThreads) / kThreads, std::max(1LL, 32LL * sms / spans));
        const dim3 grid(across, (unsigned)std::min(spans, std::max(1LL, 32LL * sms / across)));
        wtconv_dropout_spans_kernel<T, RES><<<grid, kThreads, 0, s>>>(m, a, d, spans, len, vec);
    } else if (m.nhwc) {
        const bool vec = m.C % V == 0 && whole;
        const int slots = (m.C + V - 1) / V;
        wtconv_dropout_rows_kernel<T, RES><<<ctas(m.rows * slots), kThreads, 0, s>>>(
            m, a, d, divide_by(slots, m.rows * slots), divide_by(m.HW, m.rows), vec);
    } else {
        const int quads = (m.C + 3) / 4;
        const Divide by_quads = divide_by(quads, samples * quads);
        if (m.HW % V == 0 && whole)
            wtconv_dropout_planes_kernel<T, V, RES><<<ctas(m.rows / V * quads), kThreads, 0, s>>>(
                m, a, d, divide_by(m.HW / V, m.rows / V * quads), by_quads);
        else
            wtconv_dropout_planes_kernel<T, 1, RES><<<ctas(m.rows * quads), kThreads, 0, s>>>(
                m, a, d, divide_by(m.HW, m.rows * quads), by_quads);
    }
}

}  // namespace

cudaError_t launch_dropout(const MapShape& m, int dtype, const DropArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) a.residual ? run<float, true>(m, a, d, sms, s) : run<float, false>(m, a, d, sms, s);
    else a.residual ? run<__nv_bfloat16, true>(m, a, d, sms, s) : run<__nv_bfloat16, false>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
