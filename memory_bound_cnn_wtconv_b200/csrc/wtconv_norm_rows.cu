// RMS norm of maps whose channels are adjacent (NHWC, rows).
//
// A row belongs to a team of `tpr` threads: a part of a warp, a warp, or, for
// long rows, a CTA.  Thread t of it owns the 16-byte slots t, t + tpr, ... of
// every row the team meets, NV of them, which it keeps in registers between the
// sum of squares and the output: h is read from memory once.  NV = 0 is for
// rows longer than a CTA's registers: the slots are read again.
//
// Bound by memory: forward reads x (and the residual) and writes y (and h).
// The backward's CTAs walk the rows, so that the weight gradient's sums of a
// thread's own channels stay in registers until the end; each CTA writes one
// vector of C partial sums.
#include "wtconv_norm.cuh"

namespace wtc {

namespace {

constexpr int kMaxTeam = 512;   // threads of a CTA-wide team
constexpr int kTeamThreads = 256;  // threads of a CTA of smaller teams

struct RowsGeom {
    int tpr, nv, threads, vec, step;  // step: rows a CTA holds at once
};

// The smallest team (at least `least` threads) whose threads hold a row in at
// most four slots each; full slots count more than short reductions.
RowsGeom rows_geom(const MapShape& m, int V, bool vec, int least) {
    const int slots = (m.C + V - 1) / V;
    RowsGeom g{};
    g.vec = vec;
    int tpr = least;
    while (tpr < 32 && (slots + tpr - 1) / tpr > 4) tpr *= 2;
    if ((slots + tpr - 1) / tpr > 4) {
        tpr = std::min(kMaxTeam, ((slots + 3) / 4 + 31) / 32 * 32);
        g.nv = (slots + tpr - 1) / tpr > 4 ? 0 : (slots + tpr - 1) / tpr;
        g.threads = tpr;
    } else {
        g.nv = (slots + tpr - 1) / tpr;
        g.threads = kTeamThreads;
        while (g.threads > 32 && (g.threads / 2 / tpr) * 148LL >= m.rows) g.threads /= 2;  // few rows: spread them
    }
    g.tpr = tpr;
    g.step = g.threads / tpr;
    return g;
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

// The weights of channels c .. c + V - 1.
template <int V>
__device__ __forceinline__ void load_weight(const float* w, int c, int C, bool vec, float (&f)[V]) {
    if (vec) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(w + c + e);
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = c + e < C ? w[c + e] : 0.0f;
    }
}

template <typename T, int NV, int JOIN, bool Q8>
__global__ void __launch_bounds__(kMaxTeam) wtconv_norm_rows_kernel(MapShape m, NormFwdArgs a, MapDrop d, int tpr, int vec) {
    constexpr int V = kVec<T>;
    constexpr int NR = NV ? NV : 1;
    __shared__ float red[kMaxTeam / 32];
    const int t = threadIdx.x % tpr, step = blockDim.x / tpr, slots = (m.C + V - 1) / V;
    const int iters = NV ? NV : (slots + tpr - 1) / tpr;
    const uint32_t offset = JOIN == kDropped ? drop_offset(d) : 0;
    float wr[NR][V];  // the weights of this thread's channels, for all its rows
    if (NV) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (i * tpr + t < slots) load_weight<V>(a.weight, (i * tpr + t) * V, m.C, vec, wr[i]);
        }
    }
    // Every thread of a CTA makes the same number of rounds.
    for (long long row0 = (long long)blockIdx.x * step; row0 < m.rows; row0 += (long long)gridDim.x * step) {
        const long long row = row0 + threadIdx.x / tpr;
        const bool live = row < m.rows;
        const long long base = row * m.C;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        T* h = static_cast<T*>(a.h) + base;
        long long drow = 0;
        bool whole = true;  // a sample's decision
        if (JOIN == kDropped) {
            drow = drop_row(d, m, row);
            if (d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, drow);
        }
        uint4 raw[NR], rr[NR];
        float ss = 0.0f;
        auto load = [&](int i, uint4& rx, uint4& rres) {
            const int k = i * tpr + t;
            const bool in = live && k < slots;
            rx = in && whole ? load_channels(x, k * V, m.C, vec) : make_uint4(0, 0, 0, 0);
            if (JOIN != kPlain) rres = in ? load_channels(res, k * V, m.C, vec) : make_uint4(0, 0, 0, 0);
        };
        // h of one slot, stored, and its squares
        auto join = [&](int i, uint4& rx, const uint4& rres) {
            const int k = i * tpr + t;
            float f[V];
            unpack(rx, f);
            if (JOIN != kPlain) {
                float r[V];
                unpack(rres, r);
                if (JOIN == kDropped && d.mode != WTCONV_DROP_SAMPLE) {
#pragma unroll
                    for (int e = 0; e < V; e += 4) drop_add4(d, drop_words(d, offset, drow, (k * V + e) >> 2), f + e, r + e);
                } else if (JOIN == kDropped) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < V; ++e) r[e] = __fmaf_rn(f[e], d.grown, r[e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) r[e] += f[e];
                }
                rx = pack(r);
                if (live && k < slots) store_channels(h, k * V, m.C, vec, rx);
                unpack(rx, f);  // the norm is of h as it is stored
            }
#pragma unroll
            for (int e = 0; e < V; ++e) ss += f[e] * f[e];
        };
        if (NV) {
#pragma unroll
            for (int i = 0; i < NR; ++i) load(i, raw[i], rr[i]);
#pragma unroll
            for (int i = 0; i < NR; ++i) join(i, raw[i], rr[i]);
        } else {
            for (int i = 0; i < iters; ++i) load(i, raw[0], rr[0]), join(i, raw[0], rr[0]);
        }
        ss = team_sum(ss, tpr, red);
        const float r = rsqrtf(ss / m.C + a.eps);
        if (a.rstd && live && t == 0) a.rstd[row] = r;
        // v = h * r * w of slot i; false where there is none
        auto value = [&](int i, uint4 hraw, float (&f)[V]) {
            const int k = i * tpr + t;
            if (!live || k >= slots) return false;
            if (!NV) {
                hraw = load_channels(JOIN == kPlain ? x : h, k * V, m.C, vec);  // this thread's own
                load_weight<V>(a.weight, k * V, m.C, vec, wr[0]);
            }
            unpack(hraw, f);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = f[e] * r * wr[NV ? i : 0][e];
            return true;
        };
        if (!Q8) {
            auto out = [&](int i, const uint4& hraw) {
                float f[V];
                if (value(i, hraw, f)) store_channels(static_cast<T*>(a.y) + base, (i * tpr + t) * V, m.C, vec, pack(f));
            };
            if (NV) {
#pragma unroll
                for (int i = 0; i < NR; ++i) out(i, raw[i]);
            } else {
                for (int i = 0; i < iters; ++i) out(i, raw[0]);
            }
        } else {
            const int groups = (m.C + a.group - 1) / a.group;
            auto largest = [&](int i, const uint4& hraw) {
                float f[V];
                uint32_t bits = 0;
                if (value(i, hraw, f)) {
#pragma unroll
                    for (int e = 0; e < V; ++e) bits = max(bits, abs_bits(f[e]));
                }
                return bits;
            };
            float scale = 0.0f;
            if (groups == 1) {
                uint32_t bits = 0;
                if (NV) {
#pragma unroll
                    for (int i = 0; i < NR; ++i) bits = max(bits, largest(i, raw[i]));
                } else {
                    for (int i = 0; i < iters; ++i) bits = max(bits, largest(i, raw[0]));
                }
                scale = q8_scale(team_max(bits, tpr, red), a.q8);
                if (live && t == 0) a.scale[row] = scale;
            }
            auto out = [&](int i, const uint4& hraw) {
                const int k = i * tpr + t;
                if (groups > 1) {
                    // A group is group / V neighbouring slots of this round: a power of two of neighbouring lanes.
                    uint32_t bits = largest(i, hraw);
                    for (int o = a.group / V / 2; o; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
                    scale = q8_scale(bits, a.q8);
                    if (live && k < slots && k * V % a.group == 0) a.scale[row * groups + k * V / a.group] = scale;
                }
                float f[V];
                if (!value(i, hraw, f)) return;
                const float inv = 1.0f / scale;  // one rounding more than v / scale, within the rounding to 8 bits
                uint32_t b[V / 4];
#pragma unroll
                for (int e = 0; e < V; e += 4)
                    b[e / 4] = q8_pack4(f[e] * inv, f[e + 1] * inv, f[e + 2] * inv, f[e + 3] * inv, a.q8);
                uint8_t* q = static_cast<uint8_t*>(a.y) + base;
                const int c = k * V;
                if (vec) {
                    if (V == 4) *reinterpret_cast<uint32_t*>(q + c) = b[0];
                    else *reinterpret_cast<uint2*>(q + c) = make_uint2(b[0], b[V / 4 - 1]);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (c + e < m.C) q[c + e] = (uint8_t)(b[e / 4] >> (8 * (e % 4)));
                }
            };
            if (NV) {
#pragma unroll
                for (int i = 0; i < NR; ++i) out(i, raw[i]);
            } else {
                for (int i = 0; i < iters; ++i) out(i, raw[0]);
            }
        }
    }
}

template <typename T, int NV, bool DROP>
__global__ void __launch_bounds__(kMaxTeam) wtconv_norm_rows_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d, int tpr, int vec) {
    constexpr int V = kVec<T>;
    constexpr int NR = NV ? NV : 1;
    __shared__ float red[kMaxTeam / 32];
    extern __shared__ float sums[];  // [warps][C] at the end, for teams within a warp
    const int t = threadIdx.x % tpr, step = blockDim.x / tpr, slots = (m.C + V - 1) / V;
    const int iters = NV ? NV : (slots + tpr - 1) / tpr;
    const uint32_t offset = DROP ? drop_offset(d) : 0;
    float acc[NR][V] = {}, wr[NR][V];  // of this thread's channels, for all its rows
    if (NV) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (i * tpr + t < slots) load_weight<V>(a.weight, (i * tpr + t) * V, m.C, vec, wr[i]);
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
            drow = drop_row(d, m, row);
            if (d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, drow);
        }
        uint4 hr[NR], gr[NR], er[NR];
        float gh = 0.0f;
        auto load = [&](int i, uint4& rh, uint4& rg) {
            const int k = i * tpr + t;
            const bool in = live && k < slots;
            rh = in ? load_channels(h, k * V, m.C, vec) : make_uint4(0, 0, 0, 0);
            rg = in ? load_channels(dy, k * V, m.C, vec) : make_uint4(0, 0, 0, 0);
        };
        auto load_dh = [&](int i) {
            const int k = i * tpr + t;
            return a.dh && live && k < slots ? load_channels(dh, k * V, m.C, vec) : make_uint4(0, 0, 0, 0);
        };
        auto dot = [&](int i, const uint4& rh, const uint4& rg, float (&sum)[V]) {
            const int k = i * tpr + t;
            if (k >= slots) return;
            float fh[V], fg[V];
            float (&w)[V] = wr[NV ? i : 0];
            unpack(rh, fh);
            unpack(rg, fg);
            if (!NV) load_weight<V>(a.weight, k * V, m.C, vec, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float p = fg[e] * fh[e];
                gh += p * w[e];
                sum[e] += p * r;
            }
        };
        if (NV) {
#pragma unroll
            for (int i = 0; i < NR; ++i) load(i, hr[i], gr[i]);
#pragma unroll
            for (int i = 0; i < NR; ++i) er[i] = load_dh(i);
#pragma unroll
            for (int i = 0; i < NR; ++i) dot(i, hr[i], gr[i], acc[i]);
        } else {
            for (int i = 0; i < iters; ++i) load(i, hr[0], gr[0]), dot(i, hr[0], gr[0], acc[0]);
        }
        if (!a.dres && !(DROP && a.dx)) continue;
        gh = team_sum(gh, tpr, red);
        const float s = gh / m.C * r * r;
        auto out = [&](int i, uint4 rh, uint4 rg, uint4 re) {
            const int k = i * tpr + t, c = k * V;
            if (!live || k >= slots) return;
            if (!NV) load(i, rh, rg), re = load_dh(i);
            float fh[V], fg[V], fe[V];
            float (&w)[V] = wr[NV ? i : 0];
            unpack(rh, fh);
            unpack(rg, fg);
            unpack(re, fe);
            if (!NV) load_weight<V>(a.weight, c, m.C, vec, w);
#pragma unroll
            for (int e = 0; e < V; ++e) fe[e] += r * (fg[e] * w[e] - fh[e] * s);
            if (a.dres) store_channels(static_cast<T*>(a.dres) + base, c, m.C, vec, pack(fe));
            if (DROP && a.dx) {
                float g[V] = {};
                if (d.mode != WTCONV_DROP_SAMPLE) {
#pragma unroll
                    for (int e = 0; e < V; e += 4) drop_add4(d, drop_words(d, offset, drow, (c + e) >> 2), fe + e, g + e);
                } else if (whole) {
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] = fe[e] * d.grown;
                }
                store_channels(static_cast<T*>(a.dx) + base, c, m.C, vec, pack(g));
            }
        };
        if (NV) {
#pragma unroll
            for (int i = 0; i < NR; ++i) out(i, hr[i], gr[i], er[i]);
        } else {
            for (int i = 0; i < iters; ++i) out(i, hr[0], gr[0], er[0]);
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

bool aligned_to(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

template <typename T, int JOIN, bool Q8>
void run_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const bool vec = m.C % V == 0 && aligned_to(a.x, 16) && aligned_to(a.residual, 16) && aligned_to(a.h, 16) &&
                     aligned_to(a.weight, 16) && aligned_to(a.y, Q8 ? V : 16);
    // At least four threads (64 adjacent bytes); with groups, as many as make one round of slots whole groups.
    const int least = Q8 && a.group < m.C ? std::max(4, a.group / V) : 4;
    const RowsGeom g = rows_geom(m, V, vec, least);
    const long long ctas = (m.rows + g.step - 1) / g.step;
    auto go = [&](auto kernel) {
        const unsigned grid = (unsigned)std::min(ctas, ctas <= 4LL * sms ? ctas : (long long)norm_resident(kernel, g.threads, 0) * sms);
        kernel<<<grid, g.threads, 0, s>>>(m, a, d, g.tpr, vec);
    };
    switch (g.nv) {
        case 1: go(wtconv_norm_rows_kernel<T, 1, JOIN, Q8>); break;
        case 2: go(wtconv_norm_rows_kernel<T, 2, JOIN, Q8>); break;
        case 3: go(wtconv_norm_rows_kernel<T, 3, JOIN, Q8>); break;
        case 4: go(wtconv_norm_rows_kernel<T, 4, JOIN, Q8>); break;
        default: go(wtconv_norm_rows_kernel<T, 0, JOIN, Q8>); break;
    }
}

template <typename T>
void pick_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (a.q8 >= 0)
        a.residual ? run_fwd<T, kResidual, true>(m, a, d, sms, s) : run_fwd<T, kPlain, true>(m, a, d, sms, s);
    else if (!a.residual) run_fwd<T, kPlain, false>(m, a, d, sms, s);
    else if (!d.on) run_fwd<T, kResidual, false>(m, a, d, sms, s);
    else run_fwd<T, kDropped, false>(m, a, d, sms, s);
}

template <typename T, bool DROP>
int run_bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const bool vec = m.C % V == 0 && aligned_to(a.h, 16) && aligned_to(a.dy, 16) && aligned_to(a.dh, 16) &&
                     aligned_to(a.weight, 16) && aligned_to(a.dres, 16) && aligned_to(a.dx, 16);
    const RowsGeom g = rows_geom(m, V, vec, 4);
    const long long ctas = (m.rows + g.step - 1) / g.step;
    const size_t smem = g.tpr <= 32 && g.threads > 32 && a.dweight ? (size_t)(g.threads / 32) * m.C * 4 : 0;
    const long long most = norm_parts(m, sms);
    auto go = [&](auto kernel, size_t bytes) {
        const unsigned grid = (unsigned)std::min(std::min(ctas, most), ctas <= 2LL * sms ? ctas : (long long)norm_resident(kernel, g.threads, bytes) * sms);
        kernel<<<grid, g.threads, bytes, s>>>(m, a, d, g.tpr, vec);
        return (int)grid;
    };
    switch (g.nv) {
        case 1: return go(wtconv_norm_rows_bwd_kernel<T, 1, DROP>, smem);
        case 2: return go(wtconv_norm_rows_bwd_kernel<T, 2, DROP>, smem);
        case 3: return go(wtconv_norm_rows_bwd_kernel<T, 3, DROP>, smem);
        case 4: return go(wtconv_norm_rows_bwd_kernel<T, 4, DROP>, smem);
        default:
            if (a.dres || a.dx) go(wtconv_norm_rows_bwd_kernel<T, 0, DROP>, 0);
            return 0;  // no partial sums
    }
}

}  // namespace

cudaError_t launch_norm_rows_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) pick_fwd<float>(m, a, d, sms, s);
    else pick_fwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

cudaError_t launch_norm_rows_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s) {
    if (dtype == WTCONV_F32) *parts = a.dx ? run_bwd<float, true>(m, a, d, sms, s) : run_bwd<float, false>(m, a, d, sms, s);
    else *parts = a.dx ? run_bwd<__nv_bfloat16, true>(m, a, d, sms, s) : run_bwd<__nv_bfloat16, false>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
