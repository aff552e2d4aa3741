// Counter-based dropout of a map: y = residual + d * x, d = 0 or the float
// next to 1 / (1 - p).  The mask is a function of (seed, offset, row,
// channel) alone, so it is never stored: the backward is the same kernel on dy.
//
// Bound by memory (x and the residual read once, y written once), but element
// dropout in bf16, where few warps load and draw in turn: 64 x 96 x 56 x 56 at
// 63% of the copy rate, with the ALU pipe at 56 to 61%.  A random quad covers
// four channels of a pixel, and each kernel gives a thread all of what it draws:
//   rows    channels adjacent: a 16-byte chunk of channels (one or two quads);
//   planes  pixels adjacent: a 16-byte chunk of pixels of four channels (one
//           quad a pixel);
//   ragged  the same where planes are not whole chunks, pixel by pixel;
//   spans   whole stretches of memory under one decision (samples in either
//           layout, channels of NCHW): x is not read where it is dropped.
#include <algorithm>

#include "wtconv_map_launch.h"

namespace wtc {

namespace {

constexpr int kThreads = 256;
// Shorter stretches under one decision go to the rows and planes kernels.
constexpr long long kLeastSpan = 2048;

// N channels of a row a thread, the same ones in all its rows: a 16-byte chunk
// (VEC), or four single values (a warp's four loads then meet in two to four
// lines).
template <typename T, bool VEC, bool RES>
__global__ void __launch_bounds__(kThreads) wtconv_dropout_rows_kernel(MapShape m, DropArgs a, MapDrop d, int slots) {
    constexpr int N = VEC ? kVec<T> : 4;
    const uint32_t offset = drop_offset(d);
    const int across = min(slots, kThreads), down = kThreads / across;
    const int k = blockIdx.y * kThreads + threadIdx.x % across, c = k * N, y = threadIdx.x / across;
    if (k >= slots || y >= down) return;
    const bool sample = d.mode == WTCONV_DROP_SAMPLE;
    const long long step = (long long)gridDim.x * down;
#pragma unroll 2
    for (long long row = (long long)blockIdx.x * down + y; row < m.rows; row += step) {
        const long long base = row * m.C + c;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        T* out = static_cast<T*>(a.y) + base;
        float f[N], r[N] = {};
        if constexpr (VEC) {
            unpack(*reinterpret_cast<const uint4*>(x), f);
            if (RES) unpack(*reinterpret_cast<const uint4*>(res), r);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                f[e] = c + e < m.C ? to_f(x[e]) : 0.0f;
                if (RES) r[e] = c + e < m.C ? to_f(res[e]) : 0.0f;
            }
        }
        const long long drow = drop_row(d, row);
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            uint4 u = drop_words(d, offset, drow, sample ? 0 : (c + e) >> 2);
            if (sample) u.y = u.z = u.w = u.x;
            drop_add4(d, u, f + e, r + e);
        }
        if constexpr (VEC) {
            *reinterpret_cast<uint4*>(out) = pack(r);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (c + e < m.C) out[e] = from_f<T>(r[e]);
        }
    }
}

// V: the pixels of a chunk, or of half a one where planes are whole halves only.
template <typename T, int V, bool RES>
__global__ void __launch_bounds__(kThreads) wtconv_dropout_planes_kernel(MapShape m, DropArgs a, MapDrop d, Divide by_chunks, Divide by_quads) {
    using R = typename Chunk<T, V>::type;
    const int quads = (int)by_quads.d, chunks = (int)by_chunks.d;
    const long long n = m.rows / V * quads, step = (long long)gridDim.x * kThreads;
    const uint32_t offset = drop_offset(d);
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
        const long long bq = by_chunks(i), b = by_quads(bq);
        const int p = (int)(i - bq * chunks) * V, quad = (int)(bq - b * quads);
        const long long base = (b * m.C + 4 * quad) * m.HW + p;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        R rx[4], rr[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = 4 * quad + j < m.C;
            rx[j] = in ? *reinterpret_cast<const R*>(x + (long long)j * m.HW) : Chunk<T, V>::zero();
            rr[j] = RES && in ? *reinterpret_cast<const R*>(res + (long long)j * m.HW) : Chunk<T, V>::zero();
        }
        drop_add_chunks<T>(d, offset, b * m.HW + p, b, quad, rx, rr);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * quad + j < m.C) *reinterpret_cast<R*>(static_cast<T*>(a.y) + base + (long long)j * m.HW) = rr[j];
    }
}

// Planes that are not whole chunks: four channels of E pixels a thread.  E = 2:
// a warp has 64 neighbouring pixels, a lane two of them, 32 apart.  E = 1, for
// small planes: the threads lie along the pixels of all planes, and none idles.
template <typename T, int E, bool RES>
__global__ void __launch_bounds__(kThreads) wtconv_dropout_ragged_kernel(MapShape m, DropArgs a, MapDrop d, Divide by_chunks, Divide by_quads) {
    constexpr int kLanes = E == 1 ? 1 : 32;  // threads of a chunk
    const int quads = (int)by_quads.d, chunks = (int)by_chunks.d;
    const long long n = m.rows / m.HW * quads * chunks, step = (long long)gridDim.x * (kThreads / kLanes);
    const uint32_t offset = drop_offset(d);
    for (long long i = (long long)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; i < n; i += step) {
        const long long bq = by_chunks(i), b = by_quads(bq);
        const int p = (int)(i - bq * chunks) * kLanes * E + threadIdx.x % kLanes, quad = (int)(bq - b * quads);
        const long long base = (b * m.C + 4 * quad) * m.HW + p;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        T rx[4][E], rr[4][E];  // all loads first
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in = 4 * quad + j < m.C && (E == 1 || p + 32 * e < m.HW);
                rx[j][e] = in ? x[(long long)j * m.HW + 32 * e] : from_f<T>(0.0f);
                rr[j][e] = RES && in ? res[(long long)j * m.HW + 32 * e] : from_f<T>(0.0f);
            }
        }
        float f[4][E], r[4][E];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < E; ++e) f[j][e] = to_f(rx[j][e]), r[j][e] = to_f(rr[j][e]);
        }
        const bool element = d.mode == WTCONV_DROP_ELEMENT, sample = d.mode == WTCONV_DROP_SAMPLE;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (!element) {
            u = drop_words(d, offset, b, sample ? 0 : quad);
            if (sample) u.y = u.z = u.w = u.x;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (element) u = drop_words(d, offset, b * m.HW + p + 32 * e, quad);
            if (u.x >= d.thresh) r[0][e] = __fmaf_rn(f[0][e], d.grown, r[0][e]);
            if (u.y >= d.thresh) r[1][e] = __fmaf_rn(f[1][e], d.grown, r[1][e]);
            if (u.z >= d.thresh) r[2][e] = __fmaf_rn(f[2][e], d.grown, r[2][e]);
            if (u.w >= d.thresh) r[3][e] = __fmaf_rn(f[3][e], d.grown, r[3][e]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            T* y = static_cast<T*>(a.y) + base + (long long)j * m.HW;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (4 * quad + j < m.C && (E == 1 || p + 32 * e < m.HW)) y[32 * e] = from_f<T>(r[j][e]);
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
        // Four chunks a thread (the decision is drawn once for them) where that leaves two CTAs for every SM.
        const long long chunks = len / V + 1, fours = (chunks + 4 * kThreads - 1) / (4 * kThreads);
        const long long want = fours * spans >= 2LL * sms ? fours : (chunks + kThreads - 1) / kThreads;
        const unsigned across = (unsigned)std::min(want, std::max(1LL, 32LL * sms / spans));
        const dim3 grid(across, (unsigned)std::min(spans, std::max(1LL, 32LL * sms / across)));
        wtconv_dropout_spans_kernel<T, RES><<<grid, kThreads, 0, s>>>(m, a, d, spans, len, vec);
    } else if (m.nhwc) {
        const bool vec = m.C % V == 0 && whole;
        const int slots = (m.C + (vec ? V : 4) - 1) / (vec ? V : 4), down = kThreads / std::min(slots, kThreads);
        const unsigned columns = (slots + kThreads - 1) / kThreads;
        const dim3 grid((unsigned)std::min((m.rows + down - 1) / down, std::max(1LL, 16LL * sms / columns)), columns);
        if (vec) wtconv_dropout_rows_kernel<T, true, RES><<<grid, kThreads, 0, s>>>(m, a, d, slots);
        else wtconv_dropout_rows_kernel<T, false, RES><<<grid, kThreads, 0, s>>>(m, a, d, slots);
    } else {
        const int quads = (m.C + 3) / 4;
        const Divide by_quads = divide_by(quads, samples * quads);
        auto planes = [&](auto kernel, int chunk) {
            const long long n = m.rows / chunk * quads;
            kernel<<<ctas(n), kThreads, 0, s>>>(m, a, d, divide_by(m.HW / chunk, n), by_quads);
        };
        if (m.HW % V == 0 && whole) {
            planes(wtconv_dropout_planes_kernel<T, V, RES>, V);
        } else if (m.HW % (V / 2) == 0 && ax % 8 == 0 && ar % 8 == 0 && ay % 8 == 0) {
            planes(wtconv_dropout_planes_kernel<T, V / 2, RES>, V / 2);
        } else {
            // Two pixels a lane where a plane has several chunks of 64 (64 x 101 x 57 x 57: bf16 43 us, 47 with one; fp32 41
            // and 47; four hold too many registers with a residual, fp32 72 us and 51 with two).
            const int E = m.HW > 256 ? 2 : 1, chunks = E == 1 ? m.HW : (m.HW + 63) / 64;
            const Divide by_chunks = divide_by(chunks, samples * quads * chunks);
            const unsigned grid = ctas(samples * quads * chunks * (E == 1 ? 1 : 32));
            if (E == 2) wtconv_dropout_ragged_kernel<T, 2, RES><<<grid, kThreads, 0, s>>>(m, a, d, by_chunks, by_quads);
            else wtconv_dropout_ragged_kernel<T, 1, RES><<<grid, kThreads, 0, s>>>(m, a, d, by_chunks, by_quads);
        }
    }
}

}  // namespace

cudaError_t launch_dropout(const MapShape& m, int dtype, const DropArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) a.residual ? run<float, true>(m, a, d, sms, s) : run<float, false>(m, a, d, sms, s);
    else a.residual ? run<__nv_bfloat16, true>(m, a, d, sms, s) : run<__nv_bfloat16, false>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
