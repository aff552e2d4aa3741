// Host replay of how the map operators' kernels share out a map, against the
// library's own geometry (wtconv_map_geom.h).
//
//   map_geom_check B C H W     (148 SMs; both layouts, both types, every group)
//
// For each kernel that such a map can reach: every channel (and pixel) has
// exactly one owner; slots, stages, sums and groups stay inside their buffers;
// groups of channels are whole within what is reduced at once; a ragged tile's
// copies stay inside the tensor and its row; the multiply-shift divisions are
// exact.  Prints OK, or the first violation.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../memory_bound_cnn_wtconv_b200/csrc/wtconv_map_geom.h"

using namespace wtc;

static int sms = 148;
#define CHECK(cond)                                                                                     \
    do {                                                                                                \
        if (!(cond)) {                                                                                  \
            std::printf("line %d: %s (C %d, HW %d, rows %lld)\n", __LINE__, #cond, m.C, m.HW, m.rows); \
            std::exit(1);                                                                               \
        }                                                                                               \
    } while (0)

static void check_divide(const MapShape& m, long long d, long long most) {
    const Divide v = divide_by(d, most);
    for (long long n : {0LL, d - 1, d, 2 * d - 1, most / 3, most - 1, most})
        if (n >= 0 && n <= most) CHECK(v(n) == n / d);
}

static void check_rows(const MapShape& m, int esize, int V, int group, bool pairs) {  // group 0: no 8-bit output or one group
    const bool grouped = group > 0 && group < m.C;
    const RowsGeom g = rows_geom(m, V, !grouped ? 0 : V == 1 ? 32 : group / V, grouped && V == 1, pairs, sms);
    const int slots = (m.C + V - 1) / V;
    CHECK(g.threads >= 32 && g.threads % 32 == 0 && g.threads <= (g.tpr <= 32 ? kTeamThreads : kMaxTeam));
    CHECK(g.tpr <= 32 ? (g.tpr & (g.tpr - 1)) == 0 && g.tpr >= (V == 1 ? 4 : std::min(slots, 4)) : g.tpr % 32 == 0 && g.threads == g.tpr);
    CHECK(g.step * g.tpr == g.threads && g.step >= 1);
    if (g.nv) {
        CHECK(g.nv * g.tpr >= slots);
        CHECK(V > 1 ? g.nv <= 4 && (g.tpr <= 32 || g.nv == 4) : g.nv == 4 || g.nv == 8 || g.nv == 16 || (grouped && g.nv == 2));
        if (V == 1 && g.tpr <= 32) {  // a kernel of that width exists
            bool found = false;
            for (const SingleTeam& s : kSingles) found |= s.nv == g.nv && s.tpr == g.tpr;
            CHECK(found);
        }
        if (g.tpr <= 32) CHECK((long long)g.threads / 32 * m.C * 4 <= 48 * 1024);  // the weight gradient's sums
    }
    if (grouped) {
        if (V > 1) {
            CHECK(group % V == 0 && g.tpr * V % group == 0 && group / V <= 32);  // a round is whole groups, a group lies in a warp
        } else {
            CHECK(g.tpr == 32 && group % 32 == 0 && group / 32 <= 4);            // a group is 1, 2 or 4 rounds
            CHECK((g.nv ? g.nv : 4) % (group / 32) == 0);
        }
    }
    if (m.C <= 4096) {  // every channel once
        std::vector<int> owner(m.C, 0);
        const int iters = g.nv ? g.nv : (slots + g.tpr - 1) / g.tpr;
        for (int i = 0; i < iters; ++i)
            for (int t = 0; t < g.tpr; ++t)
                if (i * g.tpr + t < slots)
                    for (int e = 0; e < V; ++e)
                        if ((i * g.tpr + t) * V + e < m.C) ++owner[(i * g.tpr + t) * V + e];
        for (int c = 0; c < m.C; ++c) CHECK(owner[c] == 1);
    }
}

static void check_planes(const MapShape& m, int esize, int VP, bool ragged, int tensors, int group) {
    PlanesGeom g;
    if (!planes_geom(m, VP, ragged, esize, tensors, &g)) return;
    const int groups = group ? (m.C + group - 1) / group : 0, px = g.lp * VP, lanes = 32 / g.lp;
    const long long smem = g.head + planes_sums(g, VP, groups) * 4;
    if (smem > kMostSmem && group) return;  // the kernels that read again take it
    CHECK(smem <= kMostSmem);
    CHECK(g.lp >= 1 && g.lp * lanes == 32 && g.warps >= 1 && g.warps <= kMaxWarps && g.owners == g.warps * lanes);
    CHECK(g.iters == 1 || g.iters == 2);
    CHECK(4LL * g.owners * g.iters >= m.C);
    CHECK((long long)g.tiles * px >= m.HW && (long long)(g.tiles - 1) * px < m.HW);
    CHECK(g.head == 2 * tensors * g.tensor && g.tensor % 16 == 0);
    CHECK((g.warps * px) % (VP >= 4 ? 4 : 2) == 0);  // the sums' vector reads
    check_divide(m, g.tiles, m.rows);
    if (!ragged) {
        CHECK(m.HW % VP == 0);
        CHECK(((4 * (g.iters - 1) + 3) * (g.warps * 32) + g.warps * 32 - 1 + 1) * VP * esize <= g.tensor);
    } else {
        CHECK((long long)g.row * m.C <= g.tensor);
        const long long bytes = m.rows * m.C * esize, B = m.rows / m.HW;
        const int chunks = g.row / 16;
        for (long long b : {0LL, B - 1})
            for (int tile : {0, g.tiles / 2, g.tiles - 1})
                for (int c : {0, 1, m.C / 2, m.C - 1}) {
                    if (c >= m.C) continue;
                    const int p0 = tile * px, pixels = std::min(px, m.HW - p0);
                    const long long first = ((b * m.C + c) * m.HW + p0) * esize;
                    const int span = (int)(first & 15) + pixels * esize;
                    CHECK((first & 15) + px * esize <= g.row);   // where the values are read
                    CHECK(16 * chunks >= span && span <= g.row);
                    const uint32_t low = ((uint32_t)((b * m.C) * m.HW + p0) + (uint32_t)c * m.HW) * (uint32_t)esize;
                    CHECK((low & 15) == (first & 15));
                    for (int q = 0; q < chunks; ++q) {
                        if (16 * q >= span) continue;
                        const long long at = (first & ~15LL) + 16 * q;
                        CHECK(at >= 0 && at < bytes);
                    }
                }
        for (long long n : {0LL, (long long)chunks - 1, (long long)chunks, (long long)m.C * chunks - 1})
            CHECK((long long)fastdiv_host((uint32_t)n, g.by_chunks) == n / chunks);
    }
    if (m.C <= 4096) {
        std::vector<int> owner(m.C, 0);
        for (int o = 0; o < g.owners; ++o)
            for (int i = 0; i < g.iters; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int c = 4 * (i * g.owners + o) + j;
                    if (c < m.C) ++owner[c];
                    if (group && c < m.C) {
                        CHECK(c / group < groups);
                        CHECK(c / group == (c - j) / group);  // a quad lies in one group
                    }
                }
        for (int c = 0; c < m.C; ++c) CHECK(owner[c] == 1);
        if (group && group < m.C) {
            // Lanes reduced together (o < 32, o / lp * 4 < group) are quads of one group.
            int o = g.lp;
            for (; o < 32 && o / g.lp * 4 < group; o *= 2) {}
            const int span = o / g.lp * 4;  // channels of them, from a multiple of itself on
            CHECK(group % span == 0 && 4 * g.owners % span == 0 && 4 * lanes % span == 0);
        }
    }
}

static void check_long(const MapShape& m, int group) {
    const LongGeom g = long_geom(m, sms, group > 0, group);
    const int lanes = 32 / g.lp, owners = kLongWarps * lanes, iters = (m.C + 4 * owners - 1) / (4 * owners);
    CHECK(g.lp >= 4 && g.lp * lanes == 32 && (long long)g.tiles * g.lp >= m.HW);
    CHECK((kLongWarps + 1 + g.round) * g.lp * 4 <= 48 * 1024);
    if (!group) return;
    const int groups = (m.C + group - 1) / group, span = groups == 1 ? iters : 1;
    CHECK(g.round >= 1);
    for (int g0 = 0; g0 < iters; g0 += span) {
        const int first = groups == 1 ? 0 : g0 * g.round;
        for (int i = g0; i < g0 + span; ++i)
            for (int o : {0, 1, owners / 2, owners - 1}) {
                const int c = 4 * (i * owners + o);
                if (c < m.C) CHECK(c / group - first >= 0 && c / group - first < g.round);
            }
        if (iters > 4096 && g0 > 8) break;
    }
}

int main(int argc, char** argv) {
    if (argc != 5) return 2;
    const long long B = std::atoll(argv[1]);
    const int C = std::atoi(argv[2]), H = std::atoi(argv[3]), W = std::atoi(argv[4]);
    MapShape m{B * H * W, C, H * W, 0};
    CHECK(norm_parts(m, sms) >= 1 && norm_parts(m, sms) <= m.rows);
    check_divide(m, m.HW, m.rows);
    for (int esize : {4, 2}) {
        const int V = 16 / esize;
        for (int group : {0, 32, 64, 128}) {
            for (bool pairs : {false, true}) {
                if (C % V == 0) check_rows(m, esize, V, group, pairs);
                check_rows(m, esize, 1, group, pairs);
            }
            for (int tensors = 1; tensors <= 3; ++tensors) {
                const int clipped = group == 0 || group > C ? C : group;  // as the calls do
                for (int q : {0, clipped}) {
                    if (m.HW % V == 0) check_planes(m, esize, V, false, tensors, q);
                    if (m.HW % (V / 2) == 0) check_planes(m, esize, V / 2, false, tensors, q);
                    check_planes(m, esize, kRagged, true, tensors, q);
                }
                check_long(m, 0);
                check_long(m, clipped);
            }
        }
    }
    std::printf("OK\n");
    return 0;
}
