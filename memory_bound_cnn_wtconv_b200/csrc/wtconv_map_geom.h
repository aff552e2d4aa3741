// How the map operators' kernels share out a map: shapes, teams, tiles and the
// sizes of their buffers.  Host code, kept apart from the kernels so that it can
// be checked on the CPU.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "wtconv_plan.h"

#ifdef __CUDACC__
#define WTC_BOTH __host__ __device__ __forceinline__
#else
#define WTC_BOTH inline
#endif

namespace wtc {

struct MapShape {
    long long rows;  // B * H * W
    int C, HW;
    int nhwc;        // 1: the C values of a row are adjacent
};

// n / d of a count: a multiply and a shift below 2^31, else a division.
struct Divide {
    FastDiv f;
    long long d;
    int small;  // every n is below 2^31
    WTC_BOTH long long operator()(long long n) const {
        return small ? (long long)(((uint32_t)(((uint64_t)(uint32_t)n * f.mul) >> 32) + (uint32_t)n) >> f.shift) : n / d;
    }
};
inline Divide divide_by(long long d, long long most) {
    Divide v{};
    v.d = d;
    v.small = most < (1LL << 31) && d < (1LL << 31);
    if (v.small) v.f = make_fastdiv((uint32_t)d);
    return v;
}

// CTAs of the backward whose partial sums of the weight gradient the workspace
// holds, one vector of C floats for each: eight for every SM, fewer where that
// is over 32 MB, but 64.
inline long long norm_parts(const MapShape& m, int sms) {
    return std::min(m.rows, std::max(64LL, std::min(8LL * sms, (1LL << 23) / m.C)));
}

// Channels adjacent (wtconv_norm_rows.cuh).
constexpr int kMaxTeam = 512;      // threads of a CTA-wide team
constexpr int kTeamThreads = 256;  // threads of a CTA of smaller teams

struct RowsGeom {
    int tpr, nv, threads, step;  // step: rows a CTA holds at once
};

// Teams of single channels, for which kernels exist with the width at compile
// time (the offsets of a thread's slots are then constants): the narrowest that
// holds a row, since the work for each row weighs more than that for a slot (11
// bf16 channels, 64 x 128 x 128, with a residual 29 us by {4, 4}, 39 by {4, 8}).
// {2, 32} and {4, 32} are left for what needs whole warps (groups of an 8-bit
// output); the last two are CTAs of any width.
struct SingleTeam {
    int nv, tpr;
};
constexpr SingleTeam kSingles[] = {{4, 4}, {4, 8}, {8, 8}, {8, 16}, {2, 32}, {4, 32}, {8, 32}, {16, 32}, {8, 0}, {16, 0}};

// Chunks: one or two threads for rows of one or two chunks (8 bf16 channels, 64
// x 128 x 128, with a residual 18 us, 33 with teams of four); else the part of a
// warp (at least `least` threads, and four: 64 adjacent bytes) that leaves the
// fewest slots empty, and of those the widest, which holds the fewest
// registers: 24 slots are 8 x 3, 64 are 32 x 2.  pairs: but two slots a thread
// rather than one, for the work around each row (256 bf16 channels, 131072 rows,
// residual: e4m3 45 us, 53 with 32 x 1, element dropout 55 and 61; but the
// backward of 128 fp32 54 and 52).  Longer rows take a CTA.  warp: no team wider than a warp.
inline RowsGeom rows_geom(const MapShape& m, int V, int least, bool warp, bool pairs, int sms) {
    const int slots = (m.C + V - 1) / V;
    RowsGeom g{};
    if (V == 1) {
        for (const SingleTeam& s : kSingles) {
            const int tpr = s.tpr ? s.tpr : std::min(kMaxTeam, ((slots + s.nv - 1) / s.nv + 31) / 32 * 32);
            if (tpr < least || (warp && tpr > 32) || tpr * s.nv < slots) continue;
            g.tpr = tpr, g.nv = s.nv;
            break;
        }
        if (!g.tpr) g.tpr = warp ? 32 : kMaxTeam;
    } else {
        int best = 0;
        for (int tpr = std::max(slots <= 2 ? slots : 4, least); tpr <= 32; tpr *= 2) {
            const int nv = (slots + tpr - 1) / tpr;
            if (nv > 4 || (best && tpr * nv > best) || (pairs && tpr * nv == best && g.nv <= 2)) continue;
            best = tpr * nv, g.tpr = tpr, g.nv = nv;
        }
        if (!best) {
            g.tpr = std::min(kMaxTeam, ((slots + 3) / 4 + 31) / 32 * 32);
            g.nv = g.tpr * 4 >= slots ? 4 : 0;
        }
    }
    g.threads = g.tpr;
    if (g.tpr <= 32) {
        g.threads = kTeamThreads;
        while (g.threads > 32 && (long long)(g.threads / 2 / g.tpr) * sms >= m.rows) g.threads /= 2;  // few rows: spread them
    }
    g.step = g.threads / g.tpr;
    return g;
}

// Pixels adjacent (wtconv_norm_planes.cuh).
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

// Tiles of 128 bytes of a plane (64 pixels where it is ragged), less where two
// stages of `tensors` tensors do not leave room for two CTAs on an SM, down to
// 64 bytes, and then what fits at all (wider tiles weigh more than a second
// CTA there: 768 ragged channels, 128 x 7 x 7 bf16, 43 us at 32 bytes, 59 at 16).
// False if nothing does.
inline bool planes_geom(const MapShape& m, int VP, bool ragged, int esize, int tensors, PlanesGeom* out) {
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
        g.iters = (ragged && quads >= 2 * 4 * lanes) || (quads + lanes - 1) / lanes > kMaxWarps ? 2 : 1;
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

// Floats of the sums over a tile (tile_sum), and of `groups` groups' largest
// values behind them.
inline long long planes_sums(const PlanesGeom& g, int VP, int groups) { return (long long)(g.warps + 1 + groups) * g.lp * VP; }
constexpr long long kMostSmem = 225 * 1024;

// Pixels adjacent, channels read again for each pass (wtconv_norm_planes_long.cu).
constexpr int kLongWarps = 16;

struct LongGeom {
    int lp, tiles;   // tiles: of a plane
    int round;       // groups of channels at once (1: all channels are one)
};

// Pixel lanes: all, unless there are few pixels to share out (the weight
// gradient's sums are taken apart, by columns).  Groups of channels want a
// round, 4 * kLongWarps * 32 / lp channels, to be whole ones: at most 16 lanes.
inline LongGeom long_geom(const MapShape& m, int sms, bool q8, int group) {
    LongGeom g{};
    g.lp = q8 ? 16 : 32;
    static_assert(4 * kLongWarps * 32 / 16 % 128 == 0);
    while (g.lp > 4 && (g.lp / 2 >= m.HW || m.rows / g.lp < sms)) g.lp /= 2;
    g.tiles = (m.HW + g.lp - 1) / g.lp;
    g.round = !q8 ? 0 : group >= m.C ? 1 : 4 * kLongWarps * (32 / g.lp) / group;
    return g;
}

}  // namespace wtc
