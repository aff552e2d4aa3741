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
// are neither (RAG, "ragged"), each
// channel's pixels come as the aligned chunks that cover them, shifted by the
// plane's own distance from a 16-byte boundary, and are read value by value: a
// thread then has the pixels pl, pl + lp, ..., four of them.
//
// Bound by memory.  Without the copies ahead a CTA loads, waits, sums and
// stores in turn, and too few CTAs fit an SM to hide it: 388 us for the
// backward of 32 x 512 x 64 x 64 fp32 with the gradient of h.
//
// The squares are summed over an owner's channels, the lanes, then the warps
// (tile_sum).  The weight gradient's sums of a thread's own channels stay in
// its registers for all its tiles.
#include <type_traits>

#include "wtconv_norm_planes.cuh"

namespace wtc {

namespace {

constexpr int kMaxWarps = 16;
constexpr int kSmem = 200 * 1024;      // of the 227 KB a CTA may have
constexpr int kSmemTwo = 104 * 1024;   // two CTAs an SM, with their sums

constexpr int kRagged = 4;       // pixels of a thread where planes are ragged
constexpr int kRaggedLanes = 16;  // lanes along them, at compile time (constant offsets), unless that does not fit

struct PlanesGeom {
    int lp, warps, owners, iters;  // iters: quads of an owner
    int tiles;                     // of a plane
    int row;                       // ragged: bytes of a channel's pixels in a stage
    int tensor;                    // bytes of one tensor in a stage
    int head;                      // bytes of both stages
    FastDiv by_chunks;             // ragged: row / 16
    Divide by_tiles;
    float per_channel;             // 1 / C
};

// Tiles of 128 bytes of a plane (64 pixels where it is ragged), less where two stages of `tensors` tensors do not
// leave room for two CTAs on an SM, down to 64 bytes, and then what fits at
// all.  False if nothing does.
bool planes_geom(const MapShape& m, int VP, bool ragged, int esize, int tensors, PlanesGeom* out) {
    if ((long long)m.C * m.HW >= 1LL << 31) return false;  // offsets within a sample are 32-bit
    const int quads = (m.C + 3) / 4;
    int lp = ragged ? kRaggedLanes : 128 / (VP * esize);
    while (!ragged && lp < 32 && quads * lp <= 16) lp *= 2;
    while (lp > 1 && lp / 2 * VP >= m.HW) lp /= 2;
    for (; lp >= 1; lp /= 2) {
        PlanesGeom g{};
        const int lanes = 32 / lp;
        g.lp = lp;
        // Two quads an owner where one needs too many warps (ragged: where that leaves four, for less work around a tile).
        g.iters = ragged && quads >= 2 * 4 * lanes ? 2 : 1;
        while (g.iters < 2 && (quads + lanes * g.iters - 1) / (lanes * g.iters) > kMaxWarps) g.iters *= 2;
        g.warps = (quads + lanes * g.iters - 1) / (lanes * g.iters);
        if (g.warps > kMaxWarps) continue;
        g.owners = g.warps * lanes;
        g.tiles = (m.HW + lp * VP - 1) / (lp * VP);
        g.row = (lp * VP * esize + 15) / 16 * 16 + 16;
        const long long tensor = ragged ? (long long)g.row * m.C : 4LL * VP * esize * g.iters * g.warps * 32;
        if (2 * tensors * tensor > kSmem) continue;
        if (2 * tensors * tensor + (g.warps + 1) * lp * VP * 4 > kSmemTwo && lp * VP * esize > 64) continue;
        g.tensor = (int)tensor;
        g.head = (int)(2 * tensors * tensor);
        g.by_chunks = make_fastdiv(g.row / 16);
        g.by_tiles = divide_by(g.tiles, m.rows);
        g.per_channel = 1.0f / m.C;
        *out = g;
        return true;
    }
    return false;
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
            const int groups = (m.C + a.group - 1) / a.group;
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
                        if (now.has(e)) atomicMax(&top[now.channel(g, 0) / a.group * px + now.pixel(e)], bits[e]);
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
                now.get(reinterpret_cast<const float*>(top) + now.channel(g, 0) / a.group * px, inv);
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

template <typename T, int VP, int RAG, int G, bool DROP>
__global__ void __launch_bounds__(kMaxWarps * 32) wtconv_norm_planes_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d, PlanesGeom geom) {
    extern __shared__ __align__(16) char smem[];
    float* sums = reinterpret_cast<float*>(smem + geom.head);
    const int NT = a.dh ? 3 : 2;
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
        // dres = dh + (r * w) * dy - (r^3 mean(g * h)) * h
#pragma unroll
        for (int e = 0; e < VP; ++e) gh[e] *= -(r[e] * r[e] * r[e]);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float fe[4][VP] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (RAG && !now.in(g, j)) continue;
                float fh[VP], fg[VP];
                now.load(stage, NT, 0, g, j, fh);
                now.load(stage, NT, 1, g, j, fg);
                if (a.dh) now.load(stage, NT, 2, g, j, fe[j]);
                mul_n(fg, w[g][j]);
                fma_n(fg, r, fe[j]);
                fma_n(fh, gh, fe[j]);
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

// Launches a kernel on at most `most` CTAs, as many as the SMs hold at once.
template <typename K, typename A>
int launch(K kernel, const MapShape& m, const A& a, const MapDrop& d, const PlanesGeom& g, size_t smem, long long most, int sms, cudaStream_t s) {
    const int threads = g.warps * 32;
    long long ctas = std::min(m.rows / m.HW * g.tiles, most);
    if (smem > 48 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (ctas > sms) ctas = std::min(ctas, (long long)norm_resident(kernel, threads, smem) * sms);
    kernel<<<(unsigned)ctas, threads, smem, s>>>(m, a, d, g);
    return (int)ctas;
}

template <typename T, int VP, int RAG, int JOIN, bool Q8>
bool run_fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    PlanesGeom g;
    if (!planes_geom(m, VP, RAG, sizeof(T), JOIN == kPlain ? 1 : 2, &g)) return false;
    const int groups = Q8 ? (m.C + a.group - 1) / a.group : 0;
    const size_t smem = g.head + (size_t)(g.warps + 1 + groups) * g.lp * VP * 4;
    if (smem > 225 * 1024) return false;
    planes_dispatch<RAG>(g, [&](auto rag, auto quads) {
        return launch(wtconv_norm_planes_kernel<T, VP, rag, quads, JOIN, Q8>, m, a, d, g, smem, 1LL << 30, sms, s);
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

bool aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if ((uintptr_t)p % 16) return false;
    return true;
}

template <typename T>
bool fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (!aligned({a.x, a.residual})) return false;
    if (aligned({a.h}) && (uintptr_t)a.y % (a.q8 >= 0 ? V : 16) == 0) {
        if (m.HW % V == 0) return pick_fwd<T, V, 0>(m, a, d, sms, s);
        if (m.HW % (V / 2) == 0) return pick_fwd<T, V / 2, 0>(m, a, d, sms, s);
    }
    return pick_fwd<T, kRagged, kRaggedLanes>(m, a, d, sms, s);
}

template <typename T, int VP, int RAG, bool DROP>
int run_bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    PlanesGeom g;
    if (!planes_geom(m, VP, RAG, sizeof(T), a.dh ? 3 : 2, &g)) return 0;
    const size_t smem = g.head + (size_t)(g.warps + 1) * g.lp * VP * 4;
    const long long most = norm_parts(m, sms);
    return planes_dispatch<RAG>(g, [&](auto rag, auto quads) {
        return launch(wtconv_norm_planes_bwd_kernel<T, VP, rag, quads, DROP>, m, a, d, g, smem, most, sms, s);
    });
}

// The number of partial vectors, or 0 if the map is not one for these kernels.
template <typename T>
int bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (!aligned({a.h, a.dy, a.dh})) return 0;
    if (aligned({a.dres, a.dx})) {
        if (m.HW % V == 0) return a.dx ? run_bwd<T, V, 0, true>(m, a, d, sms, s) : run_bwd<T, V, 0, false>(m, a, d, sms, s);
        if (m.HW % (V / 2) == 0) return a.dx ? run_bwd<T, V / 2, 0, true>(m, a, d, sms, s) : run_bwd<T, V / 2, 0, false>(m, a, d, sms, s);
    }
    return a.dx ? run_bwd<T, kRagged, kRaggedLanes, true>(m, a, d, sms, s) : run_bwd<T, kRagged, kRaggedLanes, false>(m, a, d, sms, s);
}

}  // namespace

cudaError_t launch_norm_planes_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32 ? fwd<float>(m, a, d, sms, s) : fwd<__nv_bfloat16>(m, a, d, sms, s)) return cudaGetLastError();
    return launch_norm_planes_long_fwd(m, dtype, a, d, sms, s);
}

cudaError_t launch_norm_planes_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, int* parts, cudaStream_t s) {
    *parts = dtype == WTCONV_F32 ? bwd<float>(m, a, d, sms, s) : bwd<__nv_bfloat16>(m, a, d, sms, s);
    if (*parts) return cudaGetLastError();
    return a.dres || a.dx ? launch_norm_planes_long_bwd(m, dtype, a, d, sms, s) : cudaSuccess;
}

}  // namespace wtc
