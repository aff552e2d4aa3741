// Forward of the RMS norm of maps whose pixels are adjacent (tiles, owners and
// stages: wtconv_norm_planes.cuh).  Bound by memory: x (and the residual) read
// once, y (and h) written once; h stays in registers between the sum of squares
// and the output.
#include "wtconv_norm_planes.cuh"

namespace wtc {

namespace {

// h between the sum and the output: as stored, or as the floats that it stands for.
template <typename T, int VP>
struct HeldChunk {
    typename Chunk<T, VP>::type v;
    __device__ __forceinline__ void put(float (&f)[VP]) { v = Chunk<T, VP>::from(f), unpack(v, f); }
    __device__ __forceinline__ void get(float (&f)[VP]) const { unpack(v, f); }
};
template <typename T, int VP>
struct HeldFloats {
    float v[VP];
    __device__ __forceinline__ void put(float (&f)[VP]) {
#pragma unroll
        for (int e = 0; e < VP; ++e) v[e] = f[e] = to_f(from_f<T>(f[e]));
    }
    __device__ __forceinline__ void get(float (&f)[VP]) const {
#pragma unroll
        for (int e = 0; e < VP; ++e) f[e] = v[e];
    }
};

template <typename T, int VP, int RAG>
using Held = std::conditional_t<RAG != 0, HeldFloats<T, VP>, HeldChunk<T, VP>>;

// G: quads of an owner (geom.iters), at compile time for what stays in registers.
template <typename T, int VP, int RAG, int G, int JOIN, bool Q8>
__global__ void __launch_bounds__(kMaxWarps * 32) wtconv_norm_planes_kernel(MapShape m, NormFwdArgs a, MapDrop d, PlanesGeom geom) {
    constexpr int NT = JOIN == kPlain ? 1 : 2;
    extern __shared__ __align__(16) char smem[];  // two stages; tile_sum's; (Q8) the groups' largest bits: [groups][px]
    float* sums = reinterpret_cast<float*>(smem + geom.head);
    Tile<T, VP, RAG> now(m, geom, smem), next(m, geom, smem);
    const int px = now.lp() * VP, warps = blockDim.x / 32;
    const uint32_t offset = JOIN == kDropped ? drop_offset(d) : 0;
    const long long total = m.rows / m.HW * geom.tiles;
    auto fetch = [&](const Tile<T, VP, RAG>& t, int stage) {
        bool skip = false;
        if (JOIN == kDropped && d.mode == WTCONV_DROP_SAMPLE) skip = !keep_sample(d, offset, t.b);
        const void* const from[2] = {a.x, a.residual};
        t.template fetch<G>(stage, from, NT, skip);
        copies_commit();
    };
    float w[G][4];
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[g][j] = now.channel(g, j) < m.C ? a.weight[now.channel(g, j)] : 0.0f;
    }
    const int groups = Q8 ? (m.C + a.group - 1) / a.group : 0, gs = Q8 ? group_shift(a.group, groups) : 0;
    next.at(blockIdx.x);
    fetch(next, 0);
    int stage = 0;
    for (long long tile = blockIdx.x; tile < total; tile += gridDim.x, stage ^= 1) {
        now.at(tile);
        now.arrive();
        if (tile + gridDim.x < total) next.at(tile + gridDim.x), fetch(next, stage ^ 1);
        Held<T, VP, RAG> h[G][4];
        float ss[VP] = {};
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float f[4][VP] = {};
            if constexpr (JOIN == kDropped && !RAG) {
                typename Chunk<T, VP>::type x[4], r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = now.raw(stage, NT, 0, g, j);  // zeros past the map's end
                    r[j] = now.raw(stage, NT, 1, g, j);
                }
                drop_add_chunks<T>(d, offset, now.row(), now.b, now.channel(g, 0) / 4, x, r);
#pragma unroll
                for (int j = 0; j < 4; ++j) unpack(r[j], f[j]);
            } else if (JOIN == kDropped) {
                float x[4][VP] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!now.in(g, j)) continue;
                    now.load(stage, NT, 0, g, j, x[j]);
                    now.load(stage, NT, 1, g, j, f[j]);
                }
                if (now.in(g, 0)) now.drop(d, offset, g, x, f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (JOIN != kDropped && (!RAG || now.in(g, j))) {  // chunks: zeros past the map's end
                    now.load(stage, NT, 0, g, j, f[j]);
                    if (JOIN == kResidual) {
                        float r[VP];
                        now.load(stage, NT, 1, g, j, r);
                        add_n(f[j], r);
                    }
                }
                h[g][j].put(f[j]);  // the norm is of h as it is stored
                if (JOIN != kPlain && now.in(g, j)) now.store(a.h, g, j, f[j]);
                fma_n(f[j], f[j], ss);
            }
        }
        tile_sum<VP>(now, ss, sums, [&](int q, float s) {
            const float r = rsqrtf(s * geom.per_channel + a.eps);
            if (a.rstd && now.p0 + q < m.HW) a.rstd[now.b * m.HW + now.p0 + q] = r;
            return r;
        });
        // v = h * r * w
        auto value = [&](int g, int j, float (&f)[VP]) {
            h[g][j].get(f);
            mul_n(f, ss);
            mul_n(f, w[g][j]);
        };
        if (!Q8) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f[VP];
                    value(g, j, f);
                    if (now.in(g, j)) now.store(a.y, g, j, f);
                }
            }
        } else {
            uint32_t* top = reinterpret_cast<uint32_t*>(sums + (warps + 1) * px);
            for (int q = threadIdx.x; q < groups * px; q += blockDim.x) top[q] = 0;
            __syncthreads();
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint32_t bits[VP] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f[VP];
                    value(g, j, f);  // 0 past the last channel
#pragma unroll
                    for (int e = 0; e < VP; ++e) bits[e] = max(bits[e], abs_bits(f[e]));
                }
                // The lanes of a group first, then one of them to shared memory.
                int o = now.lp();
                for (; o < 32 && o / now.lp() * 4 < a.group; o *= 2) {
#pragma unroll
                    for (int e = 0; e < VP; ++e) bits[e] = max(bits[e], __shfl_xor_sync(0xffffffffu, bits[e], o));
                }
                if (now.in(g, 0) && (threadIdx.x & (o - 1) & ~(now.lp() - 1)) == 0) {
#pragma unroll
                    for (int e = 0; e < VP; ++e)
                        if (now.has(e)) atomicMax(&top[(now.channel(g, 0) >> gs) * px + now.pixel(e)], bits[e]);
                }
            }
            __syncthreads();
            for (int q = threadIdx.x; q < groups * px; q += blockDim.x) {
                const float s = q8_scale(top[q], a.q8);
                top[q] = __float_as_uint(q8_inverse(s));
                const int gr = q / px, pixel = now.p0 + q - gr * px;
                if (pixel < m.HW) a.scale[(now.b * groups + gr) * m.HW + pixel] = s;
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (!now.in(g, 0)) continue;
                float inv[VP];
                now.get(reinterpret_cast<const float*>(top) + (now.channel(g, 0) >> gs) * px, inv);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!now.in(g, j)) continue;
                    float f[VP];
                    value(g, j, f);
                    mul_n(f, inv);
                    uint8_t* q = static_cast<uint8_t*>(a.y) + now.origin + now.offset(g, j);
                    if constexpr (RAG) {
#pragma unroll
                        for (int e = 0; e < VP; ++e)
                            if (now.has(e)) q[e * now.lp()] = q8_one(f[e], a.q8);
                    } else {
                        q8_store<VP>(q, f, a.q8);
                    }
                }
            }
            __syncthreads();  // before the next tile clears `top`
        }
    }
}

template <typename T, int VP, int RAG, int JOIN, bool Q8>
bool run_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    PlanesGeom g;
    if (!planes_geom(m, VP, RAG, sizeof(T), JOIN == kPlain ? 1 : 2, &g)) return false;
    const int groups = Q8 ? (m.C + a.group - 1) / a.group : 0;
    const size_t smem = g.head + (size_t)planes_sums(g, VP, groups) * 4;
    if (smem > kMostSmem) return false;
    planes_dispatch<RAG>(g, [&](auto rag, auto quads) {
        return launch<wtconv_norm_planes_kernel<T, VP, rag, quads, JOIN, Q8>>(m, a, d, g, smem, 1LL << 30, sms, s);
    });
    return true;
}

template <typename T, int VP, int RAG>
bool pick_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (a.q8 >= 0)
        return a.residual ? run_fwd<T, VP, RAG, kResidual, true>(m, a, d, sms, s) : run_fwd<T, VP, RAG, kPlain, true>(m, a, d, sms, s);
    if (!a.residual) return run_fwd<T, VP, RAG, kPlain, false>(m, a, d, sms, s);
    if (!d.on) return run_fwd<T, VP, RAG, kResidual, false>(m, a, d, sms, s);
    return run_fwd<T, VP, RAG, kDropped, false>(m, a, d, sms, s);
}

template <typename T>
bool fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (!all_aligned({a.x, a.residual})) return false;
    if (all_aligned({a.h}) && (uintptr_t)a.y % (a.q8 >= 0 ? V : 16) == 0) {
        if (m.HW % V == 0) return pick_fwd<T, V, 0>(m, a, d, sms, s);
        if (m.HW % (V / 2) == 0) return pick_fwd<T, V / 2, 0>(m, a, d, sms, s);
    }
    return pick_fwd<T, kRagged, kRaggedLanes>(m, a, d, sms, s);
}

}  // namespace

cudaError_t launch_norm_planes_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32 ? fwd<float>(m, a, d, sms, s) : fwd<__nv_bfloat16>(m, a, d, sms, s)) return cudaGetLastError();
    return launch_norm_planes_long_fwd(m, dtype, a, d, sms, s);
}

}  // namespace wtc
