// C ABI of the map operators (RMS norm over channels, dropout): argument
// validation and dispatch.  Declarations and contracts: include/wtconv.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "../../include/wtconv.h"
#include "wtconv_launch.h"
#include "wtconv_map_launch.h"

namespace wtc {

namespace {

// planning_sm_count() of each device, asked once (0: not yet).  A count is
// written whole and never changes, so calls on several threads agree.
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return planning_sm_count();
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) known[dev].store(n = planning_sm_count(), std::memory_order_relaxed);
    return n;
}

wtconv_status_t map_shape(const wtconv_map_desc_t* d, MapShape* m) {
    if (!d) return WTCONV_ERR_NULLPTR;
    if (d->dtype != WTCONV_F32 && d->dtype != WTCONV_BF16) return WTCONV_ERR_DTYPE;
    if (d->layout != WTCONV_NCHW && d->layout != WTCONV_NHWC) return WTCONV_ERR_LAYOUT;
    if (d->B < 0 || d->C <= 0 || d->H <= 0 || d->W <= 0) return WTCONV_ERR_BAD_SHAPE;
    const long long hw = (long long)d->H * d->W;
    if (hw > (1LL << 30) || d->C > (1 << 24)) return WTCONV_ERR_BAD_SHAPE;
    m->rows = d->B * hw;                                                // below 2^61
    if (m->rows > (1LL << 47) / d->C) return WTCONV_ERR_BAD_SHAPE;      // no device holds more
    m->C = d->C;
    m->HW = (int)hw;
    m->nhwc = d->layout == WTCONV_NHWC || hw == 1;                      // one pixel: both layouts are the same
    return WTCONV_OK;
}

wtconv_status_t map_drop(const wtconv_drop_t* p, const MapShape& m, MapDrop* d) {
    memset(d, 0, sizeof(*d));
    d->grown = 1.0f;
    if (!p) return WTCONV_OK;
    if (!(p->p >= 0.0 && p->p < 1.0)) return WTCONV_ERR_ARGUMENT;
    if (p->mode < WTCONV_DROP_ELEMENT || p->mode > WTCONV_DROP_SAMPLE) return WTCONV_ERR_ARGUMENT;
    if ((uintptr_t)p->offset_dev % 8) return WTCONV_ERR_MISALIGNED;
    d->thresh = (uint32_t)floor(p->p * 4294967296.0);  // p < 1: at most 2^32 - 1
    d->grown = (float)(1.0 / (1.0 - p->p));
    philox_keys(p->seed, d->key);
    d->offset = (uint32_t)p->offset;
    d->offset_dev = (const long long*)p->offset_dev;
    d->mode = p->mode;
    d->by_hw = divide_by(m.HW, m.rows);
    d->on = d->thresh != 0;
    return WTCONV_OK;
}

// One buffer of a call, for the checks of alignment and overlap.
struct Span {
    const void* p;
    size_t bytes;
    size_t align;
    bool out;
};

wtconv_status_t check_spans(const Span* s, int n) {
    for (int i = 0; i < n; ++i)
        if (s[i].p && (uintptr_t)s[i].p % s[i].align) return WTCONV_ERR_MISALIGNED;
    for (int i = 0; i < n; ++i) {
        if (!s[i].p || !s[i].out) continue;
        const uintptr_t a = (uintptr_t)s[i].p;
        for (int j = 0; j < n; ++j) {
            if (j == i || !s[j].p) continue;
            const uintptr_t b = (uintptr_t)s[j].p;
            if (a < b + s[j].bytes && b < a + s[i].bytes) return WTCONV_ERR_ARGUMENT;
        }
    }
    return WTCONV_OK;
}

size_t esize_of(const wtconv_map_desc_t* d) { return d->dtype == WTCONV_BF16 ? 2 : 4; }

wtconv_status_t norm_forward(const wtconv_map_desc_t* d, float eps, const void* x, const void* residual,
                             const wtconv_drop_t* drop, const float* weight, int q8, int group, void* y, float* scale,
                             void* h, float* rstd, wtconv_stream_t stream) {
    MapShape m;
    wtconv_status_t st = map_shape(d, &m);
    if (st != WTCONV_OK) return st;
    if (!(eps > 0.0f) || isinf(eps)) return WTCONV_ERR_ARGUMENT;
    MapDrop md;
    st = map_drop(drop, m, &md);
    if (st != WTCONV_OK) return st;
    if (m.rows == 0) return WTCONV_OK;  // nothing to do, whatever the (empty) buffers' addresses
    if (drop && !residual) return WTCONV_ERR_ARGUMENT;
    if (!x || !weight || !y || (residual && !h)) return WTCONV_ERR_NULLPTR;
    if (!residual && h) return WTCONV_ERR_ARGUMENT;
    const size_t es = esize_of(d), n = (size_t)m.rows * m.C;
    const size_t groups = q8 >= 0 ? (m.C + group - 1) / group : 0;
    const Span sp[] = {{x, n * es, es, false},           {residual, n * es, es, false},
                       {weight, (size_t)m.C * 4, 4, false}, {y, q8 >= 0 ? n : n * es, q8 >= 0 ? 1 : es, true},
                       {scale, (size_t)m.rows * groups * 4, 4, true}, {h, n * es, es, true},
                       {rstd, (size_t)m.rows * 4, 4, true}};
    st = check_spans(sp, 7);
    if (st != WTCONV_OK) return st;
    const NormFwdArgs a{x, residual, weight, y, h, rstd, scale, eps, q8, group};
    return launch_norm_fwd(m, d->dtype, a, md, sm_count(), (cudaStream_t)stream) == cudaSuccess ? WTCONV_OK
                                                                                                    : WTCONV_ERR_CUDA;
}

}  // namespace

}  // namespace wtc

using namespace wtc;

extern "C" {

wtconv_status_t wtconv_dropout(const wtconv_map_desc_t* d, const wtconv_drop_t* drop, const void* x,
                               const void* residual, void* y, wtconv_stream_t stream) {
    MapShape m;
    wtconv_status_t st = map_shape(d, &m);
    if (st != WTCONV_OK) return st;
    if (!drop) return WTCONV_ERR_NULLPTR;
    MapDrop md;
    st = map_drop(drop, m, &md);
    if (st != WTCONV_OK) return st;
    if (m.rows == 0) return WTCONV_OK;
    if (!x || !y) return WTCONV_ERR_NULLPTR;
    const size_t es = esize_of(d), n = (size_t)m.rows * m.C;
    const Span sp[] = {{x, n * es, es, false}, {residual, n * es, es, false}, {y, n * es, es, true}};
    st = check_spans(sp, 3);
    if (st != WTCONV_OK) return st;
    const DropArgs a{x, residual, y};
    return launch_dropout(m, d->dtype, a, md, sm_count(), (cudaStream_t)stream) == cudaSuccess ? WTCONV_OK
                                                                                                   : WTCONV_ERR_CUDA;
}

wtconv_status_t wtconv_rms_norm_forward(const wtconv_map_desc_t* d, float eps, const void* x, const void* residual,
                                        const wtconv_drop_t* drop, const float* weight, void* y, void* h, float* rstd,
                                        wtconv_stream_t stream) {
    return norm_forward(d, eps, x, residual, drop, weight, -1, 1, y, nullptr, h, rstd, stream);
}

wtconv_status_t wtconv_rms_norm_q8(const wtconv_map_desc_t* d, float eps, const void* x, const void* residual,
                                   const float* weight, int q8, int group, void* q, float* scale, void* h,
                                   wtconv_stream_t stream) {
    if (!d) return WTCONV_ERR_NULLPTR;
    if (q8 != WTCONV_E4M3 && q8 != WTCONV_I8) return WTCONV_ERR_ARGUMENT;
    if (group != 0 && group != 32 && group != 64 && group != 128) return WTCONV_ERR_ARGUMENT;
    if (!scale && d->B != 0) return WTCONV_ERR_NULLPTR;
    return norm_forward(d, eps, x, residual, nullptr, weight, q8, group == 0 || group > d->C ? (d->C > 0 ? d->C : 1) : group,
                        q, scale, h, nullptr, stream);
}

size_t wtconv_rms_norm_workspace_bytes(const wtconv_map_desc_t* d) {
    MapShape m;
    if (map_shape(d, &m) != WTCONV_OK || m.rows == 0) return 0;
    return norm_workspace_floats(m, d->dtype, sm_count()) * sizeof(float);
}

wtconv_status_t wtconv_rms_norm_backward(const wtconv_map_desc_t* d, const void* h, const void* dy, const void* dh,
                                         const wtconv_drop_t* drop, const float* weight, const float* rstd, void* dres,
                                         void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                                         wtconv_stream_t stream) {
    MapShape m;
    wtconv_status_t st = map_shape(d, &m);
    if (st != WTCONV_OK) return st;
    MapDrop md;
    st = map_drop(drop, m, &md);
    if (st != WTCONV_OK) return st;
    if (dx && !drop) return WTCONV_ERR_ARGUMENT;
    if (m.rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)m.C * 4, (cudaStream_t)stream) != cudaSuccess)
            return WTCONV_ERR_CUDA;
        return WTCONV_OK;
    }
    if (!h || !dy || !weight || !rstd || (!dres && !dx && !dweight)) return WTCONV_ERR_NULLPTR;
    const int sms = sm_count();
    const size_t need = dweight ? norm_workspace_floats(m, d->dtype, sms) * sizeof(float) : 0;
    if (need && (!workspace || workspace_bytes < need)) return WTCONV_ERR_WORKSPACE;
    const size_t es = esize_of(d), n = (size_t)m.rows * m.C;
    const Span sp[] = {{h, n * es, es, false},     {dy, n * es, es, false},
                       {dh, n * es, es, false},    {weight, (size_t)m.C * 4, 4, false},
                       {rstd, (size_t)m.rows * 4, 4, false}, {dres, n * es, es, true},
                       {dx, n * es, es, true},     {dweight, (size_t)m.C * 4, 4, true},
                       {need ? workspace : nullptr, need, 16, true}};
    st = check_spans(sp, 9);
    if (st != WTCONV_OK) return st;
    const NormBwdArgs a{h, dy, dh, weight, rstd, dres, dx, dweight, static_cast<float*>(workspace)};
    return launch_norm_bwd(m, d->dtype, a, md, sms, (cudaStream_t)stream) == cudaSuccess ? WTCONV_OK : WTCONV_ERR_CUDA;
}

}  // extern "C"
