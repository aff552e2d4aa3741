// RMS norm of maps whose pixels are adjacent (NCHW).
//
// A CTA holds a tile of LP * VP neighbouring pixels of one sample with all
// their channels.  LP lanes of a warp lie along the pixels, VP of them each (a
// 16-byte chunk, or one value where planes are not whole chunks); the other
// lanes and the warps share out the channels in quads of four, since a random
// word quad covers four channels: owner o has the quads o, o + owners, ..., G
// of them, in registers between the sum of squares and the output.  G = 0 is
// for more channels than a CTA's registers hold: they are read again.
//
// Bound by memory, like the kernels of adjacent channels.  The squares are
// summed over an owner's channels, the lanes, then the warps (through shared
// memory: one sum a pixel and warp).  The backward's CTAs walk the tiles with
// the weight gradient's sums of their own channels in registers.
#include "wtconv_norm.cuh"

namespace wtc {

namespace {

struct PlanesGeom {
    int lp, g, warps;
    int tiles;  // of a plane
    int owners;
};

constexpr int kMaxWarps = 16;

// Pixel lanes: 8 (with 16-byte chunks 128 adjacent bytes) unless the channels
// are few (more pixels, so that no owner is idle) or many (fewer, so that a
// CTA's registers hold them); single values want more lanes for the same bytes.
PlanesGeom planes_geom(const MapShape& m, int VP, const int* gs, int ngs) {
    const int quads = (m.C + 3) / 4;
    PlanesGeom g{};
    int lp = VP == 1 ? 32 : 8;
    while (lp < 32 && quads * lp <= 16) lp *= 2;
    while (lp > 1 && lp / 2 * VP >= m.HW) lp /= 2;
    for (;; lp /= 2) {
        const int lanes = 32 / lp;
        for (int i = 0; i < ngs; ++i) {
            const int warps = (quads + lanes * gs[i] - 1) / (lanes * gs[i]);
            if (warps <= (i + 1 < ngs ? kMaxWarps / 2 : kMaxWarps)) {
                g.lp = lp, g.g = gs[i], g.warps = warps;
                break;
            }
        }
        if (g.lp || lp == 1) break;
    }
    if (!g.lp) g.lp = 8, g.g = 0, g.warps = kMaxWarps;
    g.owners = g.warps * (32 / g.lp);
    g.tiles = (m.HW + g.lp * VP - 1) / (g.lp * VP);
    return g;
}

template <typename T, int VP>
using Raw = typename Chunk<T, VP>::type;

// 4 * VP keep bits: bit j * VP + v is channel 4 * quad + j of pixel v.
template <int VP>
__device__ __forceinline__ uint32_t keep_tile(const MapDrop& d, uint32_t offset, long long row, long long b, int quad) {
    uint32_t bits = 0;
    if (d.mode == WTCONV_DROP_ELEMENT) {
#pragma unroll
        for (int v = 0; v < VP; ++v) {
            const uint32_t k = keep_bits(d, drop_words(d, offset, row + v, quad));
#pragma unroll
            for (int j = 0; j < 4; ++j) bits |= (k >> j & 1) << (j * VP + v);
        }
    } else {
        const uint32_t k = keep_bits(d, drop_words(d, offset, b, quad));
#pragma unroll
        for (int j = 0; j < 4; ++j) bits |= k >> j & 1 ? ((1u << VP) - 1) << (j * VP) : 0u;
    }
    return bits;
}

// One sum for each pixel of the tile over all owners, or a function of it:
// `finish(pixel of the tile, sum)` runs once a pixel, its results are handed to
// every owner.  smem: [warps + 1][LP * VP] floats.
template <int VP, typename F>
__device__ __forceinline__ void tile_sum(float (&v)[VP], int lp, float* smem, F finish) {
    const int warps = blockDim.x / 32, lane = threadIdx.x % 32, pl = lane & (lp - 1), px = lp * VP;
    for (int o = lp; o < 32; o *= 2) {
#pragma unroll
        for (int e = 0; e < VP; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    }
    if (lane < lp) {
#pragma unroll
        for (int e = 0; e < VP; ++e) smem[(threadIdx.x / 32) * px + pl * VP + e] = v[e];
    }
    __syncthreads();
    for (int p = threadIdx.x; p < px; p += blockDim.x) {
        float s = smem[p];
        for (int k = 1; k < warps; ++k) s += smem[k * px + p];
        smem[warps * px + p] = finish(p, s);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VP; ++e) v[e] = smem[warps * px + pl * VP + e];
}

template <typename T, int VP, int G, int JOIN, bool Q8>
__global__ void __launch_bounds__(kMaxWarps * 32) wtconv_norm_planes_kernel(MapShape m, NormFwdArgs a, MapDrop d, PlanesGeom geom) {
    constexpr int GR = G ? G : 1;
    using R = Raw<T, VP>;
    using C4 = Chunk<T, VP>;
    extern __shared__ float smem[];  // tile_sum's, then (Q8) the groups' largest bits: [groups][LP * VP]
    const int lp = geom.lp, px = lp * VP, warps = blockDim.x / 32, lane = threadIdx.x % 32;
    const int pl = lane & (lp - 1), owner = (threadIdx.x / 32) * (32 / lp) + lane / lp;
    const int iters = G ? G : (m.C + 4 * geom.owners - 1) / (4 * geom.owners);
    const uint32_t offset = JOIN == kDropped ? drop_offset(d) : 0;
    const long long total = m.rows / m.HW * geom.tiles;
    for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const long long b = tile / geom.tiles;
        const int p0 = (int)(tile - b * geom.tiles) * px, p = p0 + pl * VP;
        const bool live = p < m.HW;  // with chunks, HW is a multiple of VP
        const long long base = b * m.C * m.HW + p, row = b * m.HW + p;
        const T* x = static_cast<const T*>(a.x) + base;
        const T* res = static_cast<const T*>(a.residual) + base;
        T* h = static_cast<T*>(a.h) + base;
        bool whole = true;
        if (JOIN == kDropped && d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, b);
        R raw[GR][4], rr[GR][4];
        float ss[VP] = {};
        auto load = [&](int g, R (&rx)[4], R (&rres)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * (g * geom.owners + owner) + j;
                const bool in = live && c < m.C;
                const long long at = (long long)c * m.HW;
                rx[j] = in && whole ? *reinterpret_cast<const R*>(x + at) : C4::zero();
                if (JOIN != kPlain) rres[j] = in ? *reinterpret_cast<const R*>(res + at) : C4::zero();
            }
        };
        auto join = [&](int g, R (&rx)[4], const R (&rres)[4]) {
            const int quad = g * geom.owners + owner;
            uint32_t keep = whole ? 0xffffffffu : 0u;
            if (JOIN == kDropped && d.mode != WTCONV_DROP_SAMPLE && 4 * quad < m.C)
                keep = keep_tile<VP>(d, offset, row, b, quad);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[VP];
                unpack(rx[j], f);
                if (JOIN != kPlain) {
                    float r[VP];
                    unpack(rres[j], r);
#pragma unroll
                    for (int e = 0; e < VP; ++e) {
                        if (JOIN == kDropped) f[e] = keep >> (j * VP + e) & 1 ? __fmaf_rn(f[e], d.grown, r[e]) : r[e];
                        else f[e] += r[e];
                    }
                    rx[j] = C4::from(f);
                    if (live && 4 * quad + j < m.C) *reinterpret_cast<R*>(h + (long long)(4 * quad + j) * m.HW) = rx[j];
                    unpack(rx[j], f);  // the norm is of h as it is stored
                }
#pragma unroll
                for (int e = 0; e < VP; ++e) ss[e] += f[e] * f[e];
            }
        };
        if (G) {
#pragma unroll
            for (int g = 0; g < GR; ++g) load(g, raw[g], rr[g]);
#pragma unroll
            for (int g = 0; g < GR; ++g) join(g, raw[g], rr[g]);
        } else {
            for (int g = 0; g < iters; ++g) load(g, raw[0], rr[0]), join(g, raw[0], rr[0]);
        }
        tile_sum<VP>(ss, lp, smem, [&](int q, float s) {
            const float r = rsqrtf(s / m.C + a.eps);
            if (a.rstd && p0 + q < m.HW) a.rstd[b * m.HW + p0 + q] = r;
            return r;
        });
        // v = h * r * w of channel j of round g; false where there is none
        auto value = [&](int g, int j, R hraw, float (&f)[VP]) {
            const int c = 4 * (g * geom.owners + owner) + j;
            if (!live || c >= m.C) return false;
            if (!G) hraw = *reinterpret_cast<const R*>((JOIN == kPlain ? x : h) + (long long)c * m.HW);  // this thread's own
            const float w = a.weight[c];
            unpack(hraw, f);
#pragma unroll
            for (int e = 0; e < VP; ++e) f[e] = f[e] * ss[e] * w;
            return true;
        };
        if (!Q8) {
            auto out = [&](int g, const R (&hraw)[4]) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f[VP];
                    if (value(g, j, hraw[j], f))
                        *reinterpret_cast<R*>(static_cast<T*>(a.y) + base + (long long)(4 * (g * geom.owners + owner) + j) * m.HW) = C4::from(f);
                }
            };
            if (G) {
#pragma unroll
                for (int g = 0; g < GR; ++g) out(g, raw[g]);
            } else {
                for (int g = 0; g < iters; ++g) out(g, raw[0]);
            }
        } else {
            uint32_t* top = reinterpret_cast<uint32_t*>(smem + (warps + 1) * px);
            const int groups = (m.C + a.group - 1) / a.group;
            // Largest |v| of the quad's group among this thread's channels, for each of its pixels.
            auto largest = [&](int g, const R (&hraw)[4], uint32_t (&bits)[VP]) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f[VP];
                    if (value(g, j, hraw[j], f)) {
#pragma unroll
                        for (int e = 0; e < VP; ++e) bits[e] = max(bits[e], abs_bits(f[e]));
                    }
                }
            };
            // The groups of channels c0 .. c0 + n * group - 1 in `top`, then their scales in its place.
            auto clear = [&](int n) {
                for (int q = threadIdx.x; q < n * px; q += blockDim.x) top[q] = 0;
                __syncthreads();
            };
            auto give = [&](int first, int n) {
                __syncthreads();
                for (int q = threadIdx.x; q < n * px; q += blockDim.x) {
                    const float s = q8_scale(top[q], a.q8);
                    top[q] = __float_as_uint(s);
                    const int gr = first + q / px, pp = p0 + q % px;
                    if (gr < groups && pp < m.HW) a.scale[(b * groups + gr) * m.HW + pp] = s;
                }
                __syncthreads();
            };
            auto note = [&](int at, const uint32_t (&bits)[VP]) {
                if (!live) return;
#pragma unroll
                for (int e = 0; e < VP; ++e) atomicMax(&top[at * px + pl * VP + e], bits[e]);
            };
            auto out = [&](int g, int first, const R (&hraw)[4]) {
                uint8_t* q = static_cast<uint8_t*>(a.y) + base;
                const int c0 = 4 * (g * geom.owners + owner);
                const int at = c0 / a.group - first;
                float s[VP];
                if (c0 < m.C) {
#pragma unroll
                    for (int e = 0; e < VP; ++e) s[e] = 1.0f / __uint_as_float(top[at * px + pl * VP + e]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float f[VP];
                    if (!value(g, j, hraw[j], f)) continue;
#pragma unroll
                    for (int e = 0; e < VP; ++e) f[e] *= s[e];  // one rounding more than v / scale
                    uint8_t* o = q + (long long)(c0 + j) * m.HW;
                    if constexpr (VP == 1) {
                        *o = (uint8_t)q8_pack4(f[0], 0.0f, 0.0f, 0.0f, a.q8);
                    } else if constexpr (VP == 4) {
                        *reinterpret_cast<uint32_t*>(o) = q8_pack4(f[0], f[1], f[2], f[3], a.q8);
                    } else {
                        *reinterpret_cast<uint2*>(o) = make_uint2(q8_pack4(f[0], f[1], f[2], f[3], a.q8),
                                                                  q8_pack4(f[4], f[5], f[6], f[7], a.q8));
                    }
                }
            };
            // All groups at once where the registers hold the row, or the row is one group; else round by round (a
            // round is 4 * owners channels, a multiple of 128: whole groups).
            if (G || groups == 1) {
                clear(groups);
                if (G) {
#pragma unroll
                    for (int g = 0; g < GR; ++g) {
                        const int c0 = 4 * (g * geom.owners + owner);
                        uint32_t bits[VP] = {};
                        largest(g, raw[g], bits);
                        if (c0 < m.C) note(c0 / a.group, bits);
                    }
                } else {
                    uint32_t bits[VP] = {};
                    for (int g = 0; g < iters; ++g) largest(g, raw[0], bits);
                    note(0, bits);
                }
                give(0, groups);
                if (G) {
#pragma unroll
                    for (int g = 0; g < GR; ++g) out(g, 0, raw[g]);
                } else {
                    for (int g = 0; g < iters; ++g) out(g, 0, raw[0]);
                }
                __syncthreads();  // before the next tile's clear
            } else {
                const int n = 4 * geom.owners / a.group;
                for (int g = 0; g < iters; ++g) {
                    clear(n);
                    uint32_t bits[VP] = {};
                    const int c0 = 4 * (g * geom.owners + owner);
                    largest(g, raw[0], bits);
                    if (c0 < m.C) note(c0 / a.group - g * n, bits);
                    give(g * n, n);
                    out(g, g * n, raw[0]);
                    __syncthreads();
                }
            }
        }
    }
}

template <typename T, int VP, int G, bool DROP>
__global__ void __launch_bounds__(kMaxWarps * 32) wtconv_norm_planes_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d, PlanesGeom geom) {
    constexpr int GR = G ? G : 1;
    using R = Raw<T, VP>;
    using C4 = Chunk<T, VP>;
    extern __shared__ float smem[];
    const int lp = geom.lp, px = lp * VP, lane = threadIdx.x % 32;
    const int pl = lane & (lp - 1), owner = (threadIdx.x / 32) * (32 / lp) + lane / lp;
    const int iters = G ? G : (m.C + 4 * geom.owners - 1) / (4 * geom.owners);
    const uint32_t offset = DROP ? drop_offset(d) : 0;
    const long long total = m.rows / m.HW * geom.tiles;
    float acc[GR][4] = {};
    for (long long tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const long long b = tile / geom.tiles;
        const int p = (int)(tile - b * geom.tiles) * px + pl * VP;
        const bool live = p < m.HW;
        const long long base = b * m.C * m.HW + p, row = b * m.HW + p;
        const T* h = static_cast<const T*>(a.h) + base;
        const T* dy = static_cast<const T*>(a.dy) + base;
        const T* dh = static_cast<const T*>(a.dh) + base;
        bool whole = true;
        if (DROP && d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, b);
        float r[VP] = {};
        if (live) {
#pragma unroll
            for (int e = 0; e < VP; ++e) r[e] = a.rstd[row + e];
        }
        R hr[GR][4], gr[GR][4];
        float gh[VP] = {};
        auto load = [&](int g, R (&rh)[4], R (&rg)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * (g * geom.owners + owner) + j;
                const bool in = live && c < m.C;
                rh[j] = in ? *reinterpret_cast<const R*>(h + (long long)c * m.HW) : C4::zero();
                rg[j] = in ? *reinterpret_cast<const R*>(dy + (long long)c * m.HW) : C4::zero();
            }
        };
        auto dot = [&](int g, const R (&rh)[4], const R (&rg)[4], float (&sum)[4]) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * (g * geom.owners + owner) + j;
                if (c >= m.C) continue;
                const float w = a.weight[c];
                float fh[VP], fg[VP];
                unpack(rh[j], fh);
                unpack(rg[j], fg);
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    const float q = fg[e] * fh[e];
                    gh[e] += q * w;
                    sum[j] += q * r[e];
                }
            }
        };
        if (G) {
#pragma unroll
            for (int g = 0; g < GR; ++g) load(g, hr[g], gr[g]);
#pragma unroll
            for (int g = 0; g < GR; ++g) dot(g, hr[g], gr[g], acc[g]);
        } else {
            for (int g = 0; g < iters; ++g) load(g, hr[0], gr[0]), dot(g, hr[0], gr[0], acc[0]);
        }
        if (!a.dres && !(DROP && a.dx)) continue;
        tile_sum<VP>(gh, lp, smem, [&](int, float s) { return s / m.C; });
        auto out = [&](int g, R (&rh)[4], R (&rg)[4]) {
            const int quad = g * geom.owners + owner;
            uint32_t keep = whole ? 0xffffffffu : 0u;
            if (DROP && a.dx && d.mode != WTCONV_DROP_SAMPLE && 4 * quad < m.C)
                keep = keep_tile<VP>(d, offset, row, b, quad);
            if (!G) load(g, rh, rg);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 4 * quad + j;
                if (!live || c >= m.C) continue;
                const long long at = (long long)c * m.HW;
                const float w = a.weight[c];
                float fh[VP], fg[VP], fe[VP] = {};
                unpack(rh[j], fh);
                unpack(rg[j], fg);
                if (a.dh) unpack(*reinterpret_cast<const R*>(dh + at), fe);
#pragma unroll
                for (int e = 0; e < VP; ++e) fe[e] += r[e] * (fg[e] * w - fh[e] * (gh[e] * r[e] * r[e]));
                if (a.dres) *reinterpret_cast<R*>(static_cast<T*>(a.dres) + base + at) = C4::from(fe);
                if (DROP && a.dx) {
#pragma unroll
                    for (int e = 0; e < VP; ++e) fe[e] = keep >> (j * VP + e) & 1 ? fe[e] * d.grown : 0.0f;
                    *reinterpret_cast<R*>(static_cast<T*>(a.dx) + base + at) = C4::from(fe);
                }
            }
        };
        if (G) {
#pragma unroll
            for (int g = 0; g < GR; ++g) out(g, hr[g], gr[g]);
        } else {
            for (int g = 0; g < iters; ++g) out(g, hr[0], gr[0]);
        }
    }
    if (G && a.dweight) {
        float* part = a.part + (size_t)blockIdx.x * m.C;
#pragma unroll
        for (int g = 0; g < GR; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v = acc[g][j];
                for (int o = 1; o < lp; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
                const int c = 4 * (g * geom.owners + owner) + j;
                if (pl == 0 && c < m.C) part[c] = v;
            }
    }
}

bool chunked(const MapShape& m, int V, std::initializer_list<const void*> ps, const void* y = nullptr, int ybytes = 1) {
    if (m.HW % V) return false;
    for (const void* p : ps)
        if ((uintptr_t)p % 16) return false;
    return (uintptr_t)y % ybytes == 0;
}

template <typename T, int VP, int JOIN, bool Q8>
void run_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    const int wide[2] = {1, 2}, narrow[2] = {1, 4};
    const PlanesGeom g = planes_geom(m, VP, VP == 1 ? narrow : wide, 2);
    const long long total = m.rows / m.HW * g.tiles;
    const unsigned grid = (unsigned)std::min(total, 64LL * sms);
    const int threads = g.warps * 32, px = g.lp * VP;
    const int groups = !Q8 ? 0 : g.g || a.group >= m.C ? (m.C + a.group - 1) / a.group : 4 * g.owners / a.group;
    const size_t smem = (size_t)(g.warps + 1 + groups) * px * 4;
    switch (g.g) {
        case 1: wtconv_norm_planes_kernel<T, VP, 1, JOIN, Q8><<<grid, threads, smem, s>>>(m, a, d, g); break;
        case 2: if constexpr (VP != 1) wtconv_norm_planes_kernel<T, VP, 2, JOIN, Q8><<<grid, threads, smem, s>>>(m, a, d, g); break;
        case 4: if constexpr (VP == 1) wtconv_norm_planes_kernel<T, VP, 4, JOIN, Q8><<<grid, threads, smem, s>>>(m, a, d, g); break;
        default: wtconv_norm_planes_kernel<T, VP, 0, JOIN, Q8><<<grid, threads, smem, s>>>(m, a, d, g); break;
    }
}

template <typename T, int VP>
void pick_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (a.q8 >= 0)
        a.residual ? run_fwd<T, VP, kResidual, true>(m, a, d, sms, s) : run_fwd<T, VP, kPlain, true>(m, a, d, sms, s);
    else if (!a.residual) run_fwd<T, VP, kPlain, false>(m, a, d, sms, s);
    else if (!d.on) run_fwd<T, VP, kResidual, false>(m, a, d, sms, s);
    else run_fwd<T, VP, kDropped, false>(m, a, d, sms, s);
}

template <typename T>
void fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (chunked(m, V, {a.x, a.residual, a.h}, a.y, a.q8 >= 0 ? V : 16)) pick_fwd<T, V>(m, a, d, sms, s);
    else pick_fwd<T, 1>(m, a, d, sms, s);
}

template <typename T, int VP, bool DROP>
int run_bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    const int wide[2] = {1, 2}, narrow[2] = {1, 4};
    const PlanesGeom g = planes_geom(m, VP, VP == 1 ? narrow : wide, 2);
    const long long total = m.rows / m.HW * g.tiles;
    const unsigned grid = (unsigned)std::min(total, norm_parts(m, sms));
    const int threads = g.warps * 32;
    const size_t smem = (size_t)(g.warps + 1) * g.lp * VP * 4;
    switch (g.g) {
        case 1: wtconv_norm_planes_bwd_kernel<T, VP, 1, DROP><<<grid, threads, smem, s>>>(m, a, d, g); break;
        case 2: if constexpr (VP != 1) wtconv_norm_planes_bwd_kernel<T, VP, 2, DROP><<<grid, threads, smem, s>>>(m, a, d, g); break;
        case 4: if constexpr (VP == 1) wtconv_norm_planes_bwd_kernel<T, VP, 4, DROP><<<grid, threads, smem, s>>>(m, a, d, g); break;
        default:
            if (a.dres || a.dx) wtconv_norm_planes_bwd_kernel<T, VP, 0, DROP><<<grid, threads, smem, s>>>(m, a, d, g);
            return 0;  // no partial sums
    }
    return (int)grid;
}

template <typename T>
int bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (chunked(m, V, {a.h, a.dy, a.dh, a.dres, a.dx}))
        return a.dx ? run_bwd<T, V, true>(m, a, d, sms, s) : run_bwd<T, V, false>(m, a, d, sms, s);
    return a.dx ? run_bwd<T, 1, true>(m, a, d, sms, s) : run_bwd<T, 1, false>(m, a, d, sms, s);
}

}  // namespace

cudaError_t launch_norm_planes_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) fwd<float>(m, a, d, sms, s);
    else fwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

cudaError_t launch_norm_planes_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s) {
    *parts = dtype == WTCONV_F32 ? bwd<float>(m, a, d, sms, s) : bwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
