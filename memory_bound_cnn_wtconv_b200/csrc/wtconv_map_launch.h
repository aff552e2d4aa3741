// Arguments and launchers of the map operators, defined in wtconv_norm.cu and
// wtconv_dropout.cu and called by the C ABI in wtconv_map_api.cu after
// validation.
#pragma once

#include <cuda_runtime.h>

#include "wtconv_map.cuh"

namespace wtc {

struct NormFwdArgs {
    const void *x, *residual;
    const float* weight;
    void *y, *h;      // y: stored type, or 8 bits with q8 >= 0
    float *rstd, *scale;
    float eps;
    int q8, group;    // q8: -1 or a wtconv_q8_t; group: channels a scale covers
};

struct NormBwdArgs {
    const void *h, *dy, *dh;
    const float *weight, *rstd;
    void *dres, *dx;
    float *dweight, *part;
};

struct DropArgs {
    const void *x, *residual;
    void* y;
};

size_t norm_workspace_floats(const MapShape& m, int dtype, int sms);
cudaError_t launch_norm_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);
cudaError_t launch_norm_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s);
cudaError_t launch_dropout(const MapShape& m, int dtype, const DropArgs& a, const MapDrop& d, int sms, cudaStream_t s);

}  // namespace wtc
