// Forward of the RMS norm of maps whose channels are adjacent (teams and slots:
// wtconv_norm_rows.cuh).  Bound by memory: x (and the residual) read once, y
// (and h) written once.  CTAs walk the rows, as many as the SMs hold, so that a
// thread reads the weights of its channels once.
#include "wtconv_norm_rows.cuh"

namespace wtc {

namespace {

// Kernels held to the registers (80) that let an SM hold three CTAs: those that
// would take more and lose little by it (512 bf16 channels, 32 x 64 x 64, with
// element dropout 104 us, and 118 with two CTAs).
template <int V, int NV, int TPR, int JOIN, bool Q8>
constexpr bool kThree = kWithinWarp<V, NV, TPR> && (V == 8   ? (NV == 2 && JOIN == kDropped) || (NV == 3 && Q8)
                                                    : V == 4 ? NV == 3 && JOIN == kDropped
                                                             : NV == 8);

template <typename T, int V, int NV, int TPR, int JOIN, bool Q8>
__global__ void __launch_bounds__(kThree<V, NV, TPR, JOIN, Q8> ? kTeamThreads : kMaxTeam, kThree<V, NV, TPR, JOIN, Q8> ? 3 : 0)
    wtconv_norm_rows_kernel(MapShape m, NormFwdArgs a, MapDrop d, int team, float per_channel) {
    const int tpr = TPR ? TPR : team;
    using R = typename Chunk<T, V>::type;
    // Slots at once: all of them, or for NV = 0 one (four, where quads are exchanged).
    constexpr int NR = NV ? NV : V == 1 ? 4 : 1;
    __shared__ float red[kMaxTeam / 32];
    const int t = threadIdx.x % tpr, step = blockDim.x / tpr, slots = (m.C + V - 1) / V;
    const int iters = NV ? NV : (slots + tpr - 1) / tpr;
    const uint32_t offset = JOIN == kDropped ? drop_offset(d) : 0;
    float w[NR][V] = {};  // the weights of this thread's channels, for all its rows
    if (NV) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (i * tpr + t < slots) load_weight<V>(a.weight + (i * tpr + t) * V, w[i]);
        }
    }
    const int groups = Q8 ? (m.C + a.group - 1) / a.group : 0, gs = Q8 ? group_shift(a.group, groups) : 0;
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
            drow = drop_row(d, row);
            if (d.mode == WTCONV_DROP_SAMPLE) whole = keep_sample(d, offset, drow);
        }
        auto in = [&](int i) { return live && i * tpr + t < slots; };
        R raw[NR];
        float ss = 0.0f;
        // h of slots i0 .. i0 + NR - 1, stored, and its squares
        auto join = [&](int i0) {
            R rr[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int c = ((i0 + i) * tpr + t) * V;
                raw[i] = in(i0 + i) && whole ? *reinterpret_cast<const R*>(x + c) : Chunk<T, V>::zero();
                if (JOIN != kPlain) rr[i] = in(i0 + i) ? *reinterpret_cast<const R*>(res + c) : Chunk<T, V>::zero();
            }
            if constexpr (JOIN == kDropped) {
                float f[NR][V], r[NR][V];
#pragma unroll
                for (int i = 0; i < NR; ++i) unpack(raw[i], f[i]), unpack(rr[i], r[i]);
                if (d.mode != WTCONV_DROP_SAMPLE) {
                    drop_add_slots<V, NR>(d, offset, drow, i0, tpr, t, f, r);
                } else if (whole) {
#pragma unroll
                    for (int i = 0; i < NR; ++i) fma_n(f[i], d.grown, r[i]);
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) raw[i] = Chunk<T, V>::from(r[i]);
            } else if constexpr (JOIN == kResidual) {
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    float f[V], r[V];
                    unpack(raw[i], f);
                    unpack(rr[i], r);
                    add_n(f, r);
                    raw[i] = Chunk<T, V>::from(f);
                }
            }
            float sq[V] = {};
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if (JOIN != kPlain && in(i0 + i)) *reinterpret_cast<R*>(h + ((i0 + i) * tpr + t) * V) = raw[i];
                float f[V];
                unpack(raw[i], f);  // the norm is of h as it is stored
                fma_n(f, f, sq);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) ss += sq[e];
        };
        if (NV) {
            join(0);
        } else {
            for (int i0 = 0; i0 < iters; i0 += NR) join(i0);
        }
        ss = team_sum(ss, tpr, red);
        const float r = rsqrtf(ss * per_channel + a.eps);
        if (a.rstd && live && t == 0) a.rstd[row] = r;
        // v = h * r * w of slot i0 + i (0 past the row's end)
        auto value = [&](int i0, int i, float (&f)[V]) {
            const int c = ((i0 + i) * tpr + t) * V;
            if (!NV && !in(i0 + i)) {
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = 0.0f;
                return;
            }
            if (!NV) {
                raw[i] = *reinterpret_cast<const R*>((JOIN == kPlain ? x : h) + c);  // this thread's own
                load_weight<V>(a.weight + c, w[i]);
            }
            unpack(raw[i], f);
            mul_n(f, r);
            mul_n(f, w[i]);
        };
        if (!Q8) {
            auto out = [&](int i0) {
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    float f[V];
                    value(i0, i, f);
                    if (in(i0 + i)) *reinterpret_cast<R*>(static_cast<T*>(a.y) + base + ((i0 + i) * tpr + t) * V) = Chunk<T, V>::from(f);
                }
            };
            if (NV) {
                out(0);
            } else {
                for (int i0 = 0; i0 < iters; i0 += NR) out(i0);
            }
        } else {
            float* scales = a.scale + row * groups;
            float v[NR][V];
            auto values = [&](int i0) {
#pragma unroll
                for (int i = 0; i < NR; ++i) value(i0, i, v[i]);
            };
            auto largest = [&](int i) {
                uint32_t bits = 0;
#pragma unroll
                for (int e = 0; e < V; ++e) bits = max(bits, abs_bits(v[i][e]));
                return bits;
            };
            float scale = 0.0f;
            if (NV) values(0);
            if (groups == 1) {
                uint32_t bits = 0;
                for (int i0 = 0; i0 < iters; i0 += NR) {
                    if (!NV) values(i0);
#pragma unroll
                    for (int i = 0; i < NR; ++i) bits = max(bits, largest(i));
                }
                scale = q8_scale(team_max(bits, tpr, red), a.q8);
                if (live && t == 0) *scales = scale;
            }
            auto out = [&](int i0) {
                if (!NV) values(i0);
                uint32_t bits[NR];
                if (groups > 1) {
                    // A group is group / V neighbouring slots of a round, a power of two of neighbouring lanes; of single
                    // channels (teams of one warp) one, two or four whole rounds, each reduced by one instruction
                    // (118840 rows of 109 bf16 with a residual, groups of 32: 41 us; by five shuffles, in a kernel for
                    // 256 channels and with a division for each group's address, 113).
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        bits[i] = largest(i);
                        if constexpr (V == 1) {
                            bits[i] = __reduce_max_sync(0xffffffffu, bits[i]);
                        } else {
                            for (int o = a.group / V / 2; o; o >>= 1) bits[i] = max(bits[i], __shfl_xor_sync(0xffffffffu, bits[i], o));
                        }
                    }
                    if constexpr (V == 1) {
                        if (a.group > 32) {
#pragma unroll
                            for (int i = 0; i < NR; i += 2) bits[i] = bits[i + 1] = max(bits[i], bits[i + 1]);
                        }
                        if constexpr (NR % 4 == 0) {  // two rounds are at most 64 channels, so one group of more
                            if (a.group > 64) {
#pragma unroll
                                for (int i = 0; i < NR; i += 4)
                                    bits[i] = bits[i + 1] = bits[i + 2] = bits[i + 3] = max(bits[i], bits[i + 2]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int c = ((i0 + i) * tpr + t) * V;
                    if (groups > 1) {
                        scale = q8_scale(bits[i], a.q8);
                        if (in(i0 + i) && (c & (a.group - 1)) == 0) scales[c >> gs] = scale;
                    }
                    if (!in(i0 + i)) continue;
                    float (&f)[V] = v[i];
                    mul_n(f, q8_inverse(scale));
                    uint8_t* q = static_cast<uint8_t*>(a.y) + base + c;
                    if constexpr (V == 1) {
                        *q = q8_one(f[0], a.q8);
                    } else if constexpr (V == 4) {
                        *reinterpret_cast<uint32_t*>(q) = q8_pack4(f[0], f[1], f[2], f[3], a.q8);
                    } else {
                        *reinterpret_cast<uint2*>(q) = make_uint2(q8_pack4(f[0], f[1], f[2], f[3], a.q8),
                                                                  q8_pack4(f[4], f[5], f[6], f[7], a.q8));
                    }
                }
            };
            if (NV) {
                out(0);
            } else {
                for (int i0 = 0; i0 < iters; i0 += NR) out(i0);
            }
        }
    }
}

template <typename T, int V, int JOIN, bool Q8>
void run(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    // With groups, what makes a round of slots whole groups (single channels: a warp, to which a group is whole rounds
    // or a part of one).
    const bool grouped = Q8 && a.group < m.C;
    const RowsGeom g = rows_geom(m, V, !grouped ? 0 : V == 1 ? 32 : a.group / V, grouped && V == 1, true, sms);
    const long long ctas = (m.rows + g.step - 1) / g.step;
    // Several CTAs one after another to each place on an SM, so that their loads and stores overlap other CTAs', unless
    // what a thread computes weighs more than the memory (512 channels, 32 x 64 x 64, one, two and eight: fp32 with a
    // residual 182, 178 and 166 us, bf16 94, 92 and 86; but with element dropout bf16 117, 117 and 121).
    const int each = JOIN == kDropped || Q8 ? 2 : 8;
    auto go = [&](auto kernel) {
        const unsigned grid = (unsigned)std::min(ctas, ctas <= 2LL * sms ? ctas : (long long)norm_resident(kernel, g.threads, 0) * sms * each);
        kernel<<<grid, g.threads, 0, s>>>(m, a, d, g.tpr, 1.0f / m.C);
    };
    rows_dispatch<V, Q8>(g, [&](auto nv, auto tpr) { go(wtconv_norm_rows_kernel<T, V, nv, tpr, JOIN, Q8>); });
}

template <typename T, int V>
void pick(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (a.q8 >= 0)
        a.residual ? run<T, V, kResidual, true>(m, a, d, sms, s) : run<T, V, kPlain, true>(m, a, d, sms, s);
    else if (!a.residual) run<T, V, kPlain, false>(m, a, d, sms, s);
    else if (!d.on) run<T, V, kResidual, false>(m, a, d, sms, s);
    else run<T, V, kDropped, false>(m, a, d, sms, s);
}

template <typename T>
void fwd(const MapShape& m, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    constexpr int V = kVec<T>;
    if (m.C % V == 0 && aligned_to(a.x, 16) && aligned_to(a.residual, 16) && aligned_to(a.h, 16) &&
        aligned_to(a.weight, 16) && aligned_to(a.y, a.q8 >= 0 ? V : 16))
        pick<T, V>(m, a, d, sms, s);
    else
        pick<T, 1>(m, a, d, sms, s);
}

}  // namespace

cudaError_t launch_norm_rows_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    if (dtype == WTCONV_F32) fwd<float>(m, a, d, sms, s);
    else fwd<__nv_bfloat16>(m, a, d, sms, s);
    return cudaGetLastError();
}

}  // namespace wtc
