// Backward of the RMS norm of maps whose channels are adjacent (teams and
// slots: wtconv_norm_rows.cuh).  Bound by memory: h, dy (and dh) read once, the
// gradients written once.  CTAs walk the rows, so that the weight gradient's
// sums of a thread's own channels stay in its registers until the end; each CTA
// then writes one vector of C partial sums.
#include "wtconv_norm_rows.cuh"

namespace wtc {

namespace {

// Kernels held to the registers (80) that let an SM hold three CTAs: those that
// would take more and lose little by it (512 bf16 channels, 32 x 64 x 64, with dh
// 93 us, and 101 with two CTAs; three bf16 chunks would spill: 96 channels 54 and
// 38 us).
template <int V, int NV, int TPR>
constexpr bool kThree = kWithinWarp<V, NV, TPR> && (V == 8 ? NV == 2 : V == 4 ? NV == 3 : NV == 8);

template <typename T, int V, int NV, int TPR, bool DROP>
__global__ void __launch_bounds__(kThree<V, NV, TPR> ? kTeamThreads : kMaxTeam, kThree<V, NV, TPR> ? 3 : 0)
    wtconv_norm_rows_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d, int team, float per_channel) {
    const int tpr = TPR ? TPR : team;
    using R = typename Chunk<T, V>::type;
    constexpr int NR = NV ? NV : V == 1 ? 4 : 1;
    // Slots past a row's end hold zeros, and are passed over by a branch or
    // computed all the same.  No branch lets all loads start first, at the price
    // of registers: 96 fp32 channels 36 us without, 40 with it (32 x 56 x 56, with
    // dh), but 512 bf16 ones 116 and 103 us, and 512 fp32 with dropout 230 and 212.
    constexpr bool kSkip = !NV || V == 8 || (V == 4 && DROP);
    // The weights of a thread's channels stay in registers, but for four bf16 chunks, which then spill: 131072 rows of
    // 1024 with dh and element dropout 273 us with them, 249 without.
    constexpr bool kHold = NV && !(V == 8 && NV == 4);
    __shared__ float red[kMaxTeam / 32];
    extern __shared__ float sums[];  // [warps][C] at the end, for teams within a warp
    const int t = threadIdx.x % tpr, step = blockDim.x / tpr, slots = (m.C + V - 1) / V;
    const int iters = NV ? NV : (slots + tpr - 1) / tpr;
    const uint32_t offset = DROP ? drop_offset(d) : 0;
    float acc[NR][V] = {}, w[NR][V] = {};  // of this thread's channels, for all its rows
    if (kHold) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (i * tpr + t < slots) load_weight<V>(a.weight + (i * tpr + t) * V, w[i]);
        }
    }
    for (long long row0 = (long long)blockIdx.x * step; row0 < m.rows; row0 += (long long)gridDim.x * step) {
        const long long row = row0 + threadIdx.x / tpr;
        const bool live = row < m.rows;
        const long long base = row * m.C;
        const T* h = static_cast<const T*>(a.h) + base;
        const T* dy = static_cast<const T*>(a.dy) + base;
        const T* dh = static_cast<const T*>(a.dh) + base;
        const float r = live ? a.rstd[row] : 0.0f;
        long long drow = 0;
        bool whole = true;
        if (DROP) {
            drow = drop_row(d, row);
            if (d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, drow);
        }
        auto in = [&](int i) { return live && i * tpr + t < slots; };
        R hr[NR], gr[NR], er[NR];
        float gh = 0.0f;
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int c = ((i0 + i) * tpr + t) * V;
                hr[i] = in(i0 + i) ? *reinterpret_cast<const R*>(h + c) : Chunk<T, V>::zero();
                gr[i] = in(i0 + i) ? *reinterpret_cast<const R*>(dy + c) : Chunk<T, V>::zero();
            }
        };
        auto load_dh = [&](int i0) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                er[i] = a.dh && in(i0 + i) ? *reinterpret_cast<const R*>(dh + ((i0 + i) * tpr + t) * V) : Chunk<T, V>::zero();
        };
        auto dot = [&](int i0) {
            float sum[V] = {};
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if (kSkip && !in(i0 + i)) continue;
                float fh[V], fg[V];
                unpack(hr[i], fh);
                unpack(gr[i], fg);
                if (!kHold) load_weight<V>(a.weight + ((i0 + i) * tpr + t) * V, w[i]);
                mul_n(fg, fh);
                fma_n(fg, w[i], sum);
                if (NV) fma_n(fg, r, acc[i]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) gh += sum[e];
        };
        if (NV) {
            load(0);
            load_dh(0);
            dot(0);
        } else {
            for (int i0 = 0; i0 < iters; i0 += NR) load(i0), dot(i0);
        }
        if (!a.dres && !(DROP && a.dx)) continue;
        gh = team_sum(gh, tpr, red);
        // dres = dh + r * (w * dy + s * h): r^3 mean(g * h) may leave float32 where the gradient does not
        const float s = -(gh * per_channel) * r * r;
        auto out = [&](int i0) {
            if (!NV) load(i0), load_dh(i0);
            float fe[NR][V];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int c = ((i0 + i) * tpr + t) * V;
                unpack(er[i], fe[i]);
                if (kSkip && !in(i0 + i)) continue;
                float fh[V], fg[V];
                unpack(hr[i], fh);
                unpack(gr[i], fg);
                if (!kHold) load_weight<V>(a.weight + c, w[i]);
                mul_n(fg, w[i]);
                fma_n(fh, s, fg);
                fma_n(fg, r, fe[i]);
                if (a.dres && in(i0 + i)) *reinterpret_cast<R*>(static_cast<T*>(a.dres) + base + c) = Chunk<T, V>::from(fe[i]);
            }
            if (DROP && a.dx) {
                float g[NR][V] = {};
                if (d.mode != WTCONV_DROP_SAMPLE) {
                    drop_add_slots<V, NR>(d, offset, drow, i0, tpr, t, fe, g);
                } else if (whole) {
#pragma unroll
                    for (int i = 0; i < NR; ++i) fma_n(fe[i], d.grown, g[i]);
                }
#pragma unroll
                for (int i = 0; i < NR; ++i)
                    if (in(i0 + i)) *reinterpret_cast<R*>(static_cast<T*>(a.dx) + base + ((i0 + i) * tpr + t) * V) = Chunk<T, V>::from(g[i]);
            }
        };
        if (NV) {
            out(0);
        } else {
            for (int i0 = 0; i0 < iters; i0 += NR) out(i0);
        }
    }
    if (NV && a.dweight) {
        // The CTA's teams' sums of each channel, in a fixed order: the teams of a warp, then the warps.
        float* part = a.part + (size_t)blockIdx.x * m.C;
        const int warps = blockDim.x / 32;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int c = (i * tpr + t) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float v = acc[i][e];
                for (int o = tpr; o < 32; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (c + e >= m.C) continue;
                if (tpr > 32 || warps == 1) {
                    if (tpr >= 32 || threadIdx.x < tpr) part[c + e] = v;
                } else if (threadIdx.x % 32 < tpr) {
                    sums[(threadIdx.x / 32) * m.C + c + e] = v;
                }
            }
        }
        if (tpr <= 32 && warps > 1) {
            __syncthreads();
            for (int c = threadIdx.x; c < m.C; c += blockDim.x) {
                float v = sums[c];
                for (int k = 1; k < warps; ++k) v += sums[k * m.C + c];
                part[c] = v;
            }
        }
    }
}

// The number of partial vectors, or 0 if there are none (NV = 0).
template <typename T, int V, bool DROP>
int run(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    const RowsGeom g = rows_geom(m, V, 0, false, false, sms);
    const long long ctas = std::min((m.rows + g.step - 1) / g.step, norm_parts(m, sms));
    const size_t smem = g.nv && g.tpr <= 32 && g.threads > 32 && a.dweight ? (size_t)(g.threads / 32) * m.C * 4 : 0;
    int parts = 0;
    rows_dispatch<V, false>(g, [&](auto nv, auto tpr) {
        if (nv == 0 && !a.dres && !a.dx) return;
        auto kernel = wtconv_norm_rows_bwd_kernel<T, V, nv, tpr, DROP>;
        const unsigned grid = (unsigned)std::min(ctas, ctas <= 2LL * sms ? ctas : (long long)norm_resident(kernel, g.threads, smem) * sms);
        kernel<<<grid, g.threads, smem, s>>>(m, a, d, g.tpr, 1.0f / m.C);
        if (nv) parts = (int)grid;
    });
    return parts;
}

template <typename T>
int bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (m.C % V == 0 && aligned_to(a.h, 16) && aligned_to(a.dy, 16) && aligned_to(a.dh, 16) && aligned_to(a.weight, 16) &&
        aligned_to(a.dres, 16) && aligned_to(a.dx, 16))
        return a.dx ? run<T, V, true>(m, a, d, sms, s) : run<T, V, false>(m, a, d, sms, s);
    return a.dx ? run<T, 1, true>(m, a, d, sms, s) : run<T, 1, false>(m, a, d, sms, s);
}

}  // namespace

cudaError_t launch_norm_rows_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s) {
    *parts = dtype == WTCONV_F32 ? bwd<float>(m, a, d, sms, s) : bwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
