// RMS norm of maps whose pixels are adjacent (NCHW), for what
// wtconv_norm_planes.cu does not take: more channels than a CTA's shared memory
// holds, and buffers that are not 16-byte aligned.
//
// The same tiles and owners (there), one pixel a lane, nothing kept: the
// channels are read once for each pass over them.
#include "wtconv_norm_planes.cuh"

namespace wtc {

namespace {

constexpr int kWarps = kLongWarps;

// The sum over all owners of channels for each of the tile's lp pixels, through
// `finish(pixel, sum)`, which runs once a pixel; every owner gets its result.
// smem: [kWarps + 1][lp] floats.
template <typename F>
__device__ __forceinline__ float lane_sum(float v, int lp, float* smem, F finish) {
    const int lane = threadIdx.x % 32, pl = lane & (lp - 1);
    for (int o = lp; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane < lp) smem[(threadIdx.x / 32) * lp + pl] = v;
    __syncthreads();
    if (threadIdx.x < lp) {
        float s = smem[threadIdx.x];
        for (int k = 1; k < kWarps; ++k) s += smem[k * lp + threadIdx.x];
        smem[kWarps * lp + threadIdx.x] = finish(threadIdx.x, s);
    }
    __syncthreads();
    return smem[kWarps * lp + pl];
}

// Keep bits of a pixel's quad.
__device__ __forceinline__ uint32_t keep_pixel(const MapDrop& d, uint32_t offset, long long row, long long b, int quad) {
    return keep_bits(d, drop_words(d, offset, d.mode == WTCONV_DROP_ELEMENT ? row : b, quad));
}

template <typename T, int JOIN, bool Q8>
__global__ void __launch_bounds__(kWarps * 32) wtconv_norm_planes_long_kernel(MapShape m, NormFwdArgs a, MapDrop d, LongGeom geom) {
    const int lp = geom.lp, tiles = geom.tiles;
    extern __shared__ float smem[];  // tile_sum's, then (Q8) the groups' largest bits
    const int lane = threadIdx.x % 32, lanes = 32 / lp, owners = kWarps * lanes;
    const int pl = lane & (lp - 1), owner = (threadIdx.x / 32) * lanes + lane / lp;
    const int iters = (m.C + 4 * owners - 1) / (4 * owners);
    const uint32_t offset = JOIN == kDropped ? drop_offset(d) : 0;
    const long long total = m.rows / m.HW * tiles;
    for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const long long b = tile / tiles;
        const int p0 = (int)(tile - b * tiles) * lp, p = p0 + pl;
        const bool live = p < m.HW;
        const long long base = b * m.C * m.HW + p, row = b * m.HW + p;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        T* h = static_cast<T*>(a.h) + base;
        bool whole = true;
        if (JOIN == kDropped && d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, b);
        float ss = 0.0f;
        for (int g = 0; g < iters; ++g) {
            const int quad = g * owners + owner;
            uint32_t keep = whole ? 15u : 0u;
            if (JOIN == kDropped && d.mode != WTCONV_DROP_SAMPLE) keep = keep_pixel(d, offset, row, b, quad);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * quad + j;
                if (!live || c >= m.C) continue;
                const long long at = (long long)c * m.HW;
                float f = keep >> j & 1 || JOIN != kDropped ? to_f(x[at]) : 0.0f;
                if (JOIN != kPlain) {
                    const float r = to_f(res[at]);
                    if (JOIN == kResidual) f += r;
                    else f = keep >> j & 1 ? __fmaf_rn(f, d.grown, r) : r;
                    const T v = from_f<T>(f);
                    h[at] = v;
                    f = to_f(v);  // the norm is of h as it is stored
                }
                ss += f * f;
            }
        }
        ss = lane_sum(ss, lp, smem, [&](int q, float s) {
            const float r = rsqrtf(s / m.C + a.eps);
            if (a.rstd && p0 + q < m.HW) a.rstd[b * m.HW + p0 + q] = r;
            return r;
        });
        const T* hs = JOIN == kPlain ? x : h;  // what this thread wrote itself
        auto value = [&](int c) { return to_f(hs[(long long)c * m.HW]) * ss * a.weight[c]; };
        if (!Q8) {
            for (int g = 0; g < iters; ++g) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = 4 * (g * owners + owner) + j;
                    if (live && c < m.C) static_cast<T*>(a.y)[base + (long long)c * m.HW] = from_f<T>(value(c));
                }
            }
            continue;
        }
        // Rounds of whole groups (a round is 4 * owners channels, a multiple of 128), or the whole row as one.
        uint32_t* top = reinterpret_cast<uint32_t*>(smem + (kWarps + 1) * lp);
        const int groups = (m.C + a.group - 1) / a.group, n = geom.round;
        const int span = groups == 1 ? iters : 1;
        for (int g0 = 0; g0 < iters; g0 += span) {
            const int first = groups == 1 ? 0 : g0 * n;
            for (int q = threadIdx.x; q < n * lp; q += blockDim.x) top[q] = 0;
            __syncthreads();
            for (int g = g0; g < g0 + span; ++g) {
                const int c0 = 4 * (g * owners + owner);
                uint32_t bits = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (live && c0 + j < m.C) bits = max(bits, abs_bits(value(c0 + j)));
                if (live && c0 < m.C) atomicMax(&top[(c0 / a.group - first) * lp + pl], bits);
            }
            __syncthreads();
            for (int q = threadIdx.x; q < n * lp; q += blockDim.x) {
                const float s = q8_scale(top[q], a.q8);
                top[q] = __float_as_uint(q8_inverse(s));
                const int gr = first + q / lp, pixel = p0 + q % lp;
                if (gr < groups && pixel < m.HW) a.scale[(b * groups + gr) * m.HW + pixel] = s;
            }
            __syncthreads();
            for (int g = g0; g < g0 + span; ++g) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = 4 * (g * owners + owner) + j;
                    if (!live || c >= m.C) continue;
                    const float f[1] = {value(c) * __uint_as_float(top[(c / a.group - first) * lp + pl])};
                    q8_store<1>(static_cast<uint8_t*>(a.y) + base + (long long)c * m.HW, f, a.q8);
                }
            }
            __syncthreads();  // before `top` is cleared again
        }
    }
}

template <typename T, bool DROP>
__global__ void __launch_bounds__(kWarps * 32) wtconv_norm_planes_long_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d, LongGeom geom) {
    const int lp = geom.lp, tiles = geom.tiles;
    extern __shared__ float smem[];
    const int lane = threadIdx.x % 32, lanes = 32 / lp, owners = kWarps * lanes;
    const int pl = lane & (lp - 1), owner = (threadIdx.x / 32) * lanes + lane / lp;
    const int iters = (m.C + 4 * owners - 1) / (4 * owners);
    const uint32_t offset = DROP ? drop_offset(d) : 0;
    const long long total = m.rows / m.HW * tiles;
    for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const long long b = tile / tiles;
        const int p = (int)(tile - b * tiles) * lp + pl;
        const bool live = p < m.HW;
        const long long base = b * m.C * m.HW + p, row = b * m.HW + p;
        const T* h = static_cast<const T*>(a.h) + base;
        const T* dy = static_cast<const T*>(a.dy) + base;
        bool whole = true;
        if (DROP && d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, b);
        const float r = live ? a.rstd[row] : 0.0f;
        float gh = 0.0f;
        for (int g = 0; g < iters; ++g) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * (g * owners + owner) + j;
                if (live && c < m.C) gh += to_f(dy[(long long)c * m.HW]) * to_f(h[(long long)c * m.HW]) * a.weight[c];
            }
        }
        gh = lane_sum(gh, lp, smem, [&](int, float s) { return s / m.C; });
        const float s = gh * r * r;
        for (int g = 0; g < iters; ++g) {
            const int quad = g * owners + owner;
            uint32_t keep = whole ? 15u : 0u;
            if (DROP && d.mode != WTCONV_DROP_SAMPLE) keep = keep_pixel(d, offset, row, b, quad);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * quad + j;
                if (!live || c >= m.C) continue;
                const long long at = (long long)c * m.HW;
                float v = r * (to_f(dy[at]) * a.weight[c] - to_f(h[at]) * s);
                if (a.dh) v += to_f(static_cast<const T*>(a.dh)[base + at]);
                if (a.dres) static_cast<T*>(a.dres)[base + at] = from_f<T>(v);
                if (DROP) static_cast<T*>(a.dx)[base + at] = from_f<T>(keep >> j & 1 ? v * d.grown : 0.0f);
            }
        }
    }
}

template <typename T, int JOIN, bool Q8>
void run_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    const LongGeom g = long_geom(m, sms, Q8, a.group);
    const unsigned grid = (unsigned)std::min(m.rows / m.HW * g.tiles, 64LL * sms);
    const size_t smem = (size_t)(kWarps + 1 + g.round) * g.lp * 4;
    wtconv_norm_planes_long_kernel<T, JOIN, Q8><<<grid, kWarps * 32, smem, s>>>(m, a, d, g);
}

template <typename T>
void fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (a.q8 >= 0) a.residual ? run_fwd<T, kResidual, true>(m, a, d, sms, s) : run_fwd<T, kPlain, true>(m, a, d, sms, s);
    else if (!a.residual) run_fwd<T, kPlain, false>(m, a, d, sms, s);
    else if (!d.on) run_fwd<T, kResidual, false>(m, a, d, sms, s);
    else run_fwd<T, kDropped, false>(m, a, d, sms, s);
}

template <typename T>
void bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    const LongGeom g = long_geom(m, sms, false, 0);
    const unsigned grid = (unsigned)std::min(m.rows / m.HW * g.tiles, 64LL * sms);
    const size_t smem = (size_t)(kWarps + 1) * g.lp * 4;
    if (a.dx) wtconv_norm_planes_long_bwd_kernel<T, true><<<grid, kWarps * 32, smem, s>>>(m, a, d, g);
    else wtconv_norm_planes_long_bwd_kernel<T, false><<<grid, kWarps * 32, smem, s>>>(m, a, d, g);
}

}  // namespace

cudaError_t launch_norm_planes_long_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) fwd<float>(m, a, d, sms, s);
    else fwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

cudaError_t launch_norm_planes_long_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) bwd<float>(m, a, d, sms, s);
    else bwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
