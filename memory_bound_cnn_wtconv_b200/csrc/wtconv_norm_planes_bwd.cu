// Backward of the RMS norm of maps whose pixels are adjacent (tiles, owners and
// stages: wtconv_norm_planes.cuh).  Bound by memory: h, dy (and dh) read once,
// the gradients written once.  The weight gradient's sums of a thread's own
// channels stay in its registers for all its tiles; each CTA then writes one
// vector of C partial sums.
#include "wtconv_norm_planes.cuh"

namespace wtc {

namespace {

// The gradient that reaches h itself: none, staged, or read where it is used
// (tiles that it would make too narrow).
enum { kNone = 0, kStaged = 1, kDirect = 2 };

template <typename T, int VP, int RAG, int G, bool DROP, int DH>
__global__ void __launch_bounds__(kMaxWarps * 32) wtconv_norm_planes_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d, PlanesGeom geom) {
    extern __shared__ __align__(16) char smem[];
    float* sums = reinterpret_cast<float*>(smem + geom.head);
    constexpr int NT = DH == kStaged ? 3 : 2;
    const uint32_t offset = DROP ? drop_offset(d) : 0;
    const long long total = m.rows / m.HW * geom.tiles;
    const bool outputs = a.dres || (DROP && a.dx);
    Tile<T, VP, RAG> now(m, geom, smem), next(m, geom, smem);
    auto fetch = [&](const Tile<T, VP, RAG>& t, int stage) {
        const void* const from[3] = {a.h, a.dy, a.dh};
        t.template fetch<G>(stage, from, NT, false);
        copies_commit();
    };
    float w[G][4], acc[G][4] = {};
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[g][j] = now.channel(g, j) < m.C ? a.weight[now.channel(g, j)] : 0.0f;
    }
    next.at(blockIdx.x);
    fetch(next, 0);
    int stage = 0;
    for (long long tile = blockIdx.x; tile < total; tile += gridDim.x, stage ^= 1) {
        now.at(tile);
        float r[VP] = {}, gh[VP] = {};
        if (now.live) {
#pragma unroll
            for (int e = 0; e < VP; ++e)
                if (now.has(e)) r[e] = a.rstd[now.b * m.HW + now.p0 + now.pixel(e)];
        }
        now.arrive();
        if (tile + gridDim.x < total) next.at(tile + gridDim.x), fetch(next, stage ^ 1);
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (RAG && !now.in(g, j)) continue;  // chunks: zeros past the map's end
                float fh[VP], fg[VP], own[VP] = {};
                now.load(stage, NT, 0, g, j, fh);
                now.load(stage, NT, 1, g, j, fg);
                mul_n(fg, fh);
                if (RAG) {  // what lies past a plane's end is another plane's, or nothing
#pragma unroll
                    for (int e = 0; e < VP; ++e) fg[e] = now.has(e) ? fg[e] : 0.0f;
                }
                fma_n(fg, w[g][j], gh);
                fma_n(fg, r, own);
#pragma unroll
                for (int e = 0; e < VP; ++e) acc[g][j] += own[e];
            }
        }
        if (!outputs) continue;
        tile_sum<VP>(now, gh, sums, [&](int, float s) { return s * geom.per_channel; });
        bool whole = true;
        if (DROP && d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, now.b);
        // dres = dh + r * (w * dy - (r^2 mean(g * h)) * h), factor by factor: r^3 is no float32 number for r above 7e12
        // or, with all its bits, below 2e-13
#pragma unroll
        for (int e = 0; e < VP; ++e) gh[e] = -(gh[e] * r[e]) * r[e];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float fe[4][VP] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (RAG && !now.in(g, j)) continue;
                float fh[VP], fg[VP];
                now.load(stage, NT, 0, g, j, fh);
                now.load(stage, NT, 1, g, j, fg);
                if (DH == kStaged) now.load(stage, NT, 2, g, j, fe[j]);
                if (DH == kDirect && now.in(g, j)) now.load(a.dh, g, j, fe[j]);
                mul_n(fh, gh);
                fma_n(fg, w[g][j], fh);
                fma_n(fh, r, fe[j]);
                if (a.dres && now.in(g, j)) now.store(a.dres, g, j, fe[j]);
            }
            if (DROP && a.dx) {
                float dx[4][VP] = {};
                if (d.mode != WTCONV_DROP_SAMPLE) {
                    if (now.in(g, 0)) now.drop(d, offset, g, fe, dx);
                } else if (whole) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) fma_n(fe[j], d.grown, dx[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (now.in(g, j)) now.store(a.dx, g, j, dx[j]);
            }
        }
    }
    if (a.dweight) {
        float* part = a.part + (size_t)blockIdx.x * m.C;
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v = acc[g][j];
                for (int o = 1; o < now.lp(); o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                const int c = now.channel(g, j);
                if (now.pl == 0 && c < m.C) part[c] = v;
            }
        }
    }
}

template <typename T, int VP, int RAG, bool DROP>
int run_bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    PlanesGeom g;
    // dh is staged unless that takes a tile below 64 bytes of a plane (768 channels, 128 x 7 x 7 fp32: 142 us with it, 79
    // without).
    int dh = !a.dh ? kNone : kStaged;
    if (!a.dh || !planes_geom(m, VP, RAG, sizeof(T), 3, &g) || g.lp * VP * (int)sizeof(T) < std::min(64, m.HW * (int)sizeof(T))) {
        if (!planes_geom(m, VP, RAG, sizeof(T), 2, &g)) return 0;
        dh = !a.dh ? kNone : kDirect;
    }
    const size_t smem = g.head + (size_t)planes_sums(g, VP, 0) * 4;
    const long long most = norm_parts(m, sms);
    return planes_dispatch<RAG>(g, [&](auto rag, auto quads) {
        if (dh == kNone) return launch<wtconv_norm_planes_bwd_kernel<T, VP, rag, quads, DROP, kNone>>(m, a, d, g, smem, most, sms, s);
        if (dh == kStaged) return launch<wtconv_norm_planes_bwd_kernel<T, VP, rag, quads, DROP, kStaged>>(m, a, d, g, smem, most, sms, s);
        return launch<wtconv_norm_planes_bwd_kernel<T, VP, rag, quads, DROP, kDirect>>(m, a, d, g, smem, most, sms, s);
    });
}

// The number of partial vectors, or 0 if the map is not one for these kernels.
template <typename T>
int bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (!all_aligned({a.h, a.dy, a.dh})) return 0;
    if (all_aligned({a.dres, a.dx})) {
        if (m.HW % V == 0) return a.dx ? run_bwd<T, V, 0, true>(m, a, d, sms, s) : run_bwd<T, V, 0, false>(m, a, d, sms, s);
        if (m.HW % (V / 2) == 0) return a.dx ? run_bwd<T, V / 2, 0, true>(m, a, d, sms, s) : run_bwd<T, V / 2, 0, false>(m, a, d, sms, s);
    }
    return a.dx ? run_bwd<T, kRagged, kRaggedLanes, true>(m, a, d, sms, s) : run_bwd<T, kRagged, kRaggedLanes, false>(m, a, d, sms, s);
}

}  // namespace

cudaError_t launch_norm_planes_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s) {
    *parts = dtype == WTCONV_F32 ? bwd<float>(m, a, d, sms, s) : bwd<__nv_bfloat16>(m, a, d, sms, s);
    if (*parts) return cudaGetLastError();
    return a.dres || a.dx ? launch_norm_planes_long_bwd(m, dtype, a, d, sms, s) : cudaSuccess;
}

}  // namespace wtc
