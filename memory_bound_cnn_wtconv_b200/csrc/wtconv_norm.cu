// RMS norm over the channels of a map, with the residual's addition.
//
//   h = T(residual + d * x)   (h = x without a residual)
//   r = 1 / sqrt(mean_c h^2 + eps)
//   y = T(h * r * w)          or 8 bits with a scale for each group of channels
//
// The norm is taken of h as it is stored, so that the backward, which reads
// the stored h, differentiates exactly what ran.  Backward, with g = dy * w:
//   dres = T(r * (g - h * r^2 * mean_c(g * h)) + dh),  dx = T(d * the same)
//   dw   = sum over rows of dy * h * r
//
// The kernels: wtconv_norm_rows.cu (channels adjacent), wtconv_norm_planes.cu
// (pixels adjacent).  Here: the dispatch and the weight gradient's last sum.
#include "wtconv_norm.cuh"

namespace wtc {

namespace {

// The partial vectors' sum: 8 channels a CTA, 128 threads to a channel, each
// with every 128th vector (a few loads in flight at once), then the 128 in a
// fixed order.  Launched to start while the kernel before it ends.
__global__ void __launch_bounds__(1024) wtconv_norm_finish_kernel(int C, int parts, const float* part, float* dweight) {
    __shared__ float sums[8][129];
    const int x = threadIdx.x % 8, y = threadIdx.x / 8, c = blockIdx.x * 8 + x;
    cudaGridDependencySynchronize();
    float v = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int k = y; k < parts; k += 128) v += part[(size_t)k * C + c];
    }
    sums[x][y] = v;
    __syncthreads();
    if (threadIdx.x >= 256) return;
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    v = sums[w][lane] + sums[w][lane + 32] + sums[w][lane + 64] + sums[w][lane + 96];
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 8 + w < C) dweight[blockIdx.x * 8 + w] = v;
}

// Partial sums where a CTA's registers do not hold a row (so there are many
// channels): a chunk of the rows and a channel a thread (NHWC), or a channel a
// warp (NCHW).
template <typename T>
__global__ void __launch_bounds__(256) wtconv_norm_columns_kernel(MapShape m, NormBwdArgs a) {
    const T* h = static_cast<const T*>(a.h);
    const T* dy = static_cast<const T*>(a.dy);
    float sum = 0.0f;
    const long long rows = (m.rows + gridDim.y - 1) / gridDim.y, r0 = rows * blockIdx.y, r1 = min(m.rows, r0 + rows);
    if (m.nhwc) {
        const int c = blockIdx.x * 256 + threadIdx.x;
        if (c >= m.C) return;
        for (long long r = r0; r < r1; ++r) sum += to_f(dy[r * m.C + c]) * to_f(h[r * m.C + c]) * a.rstd[r];
        a.part[(size_t)blockIdx.y * m.C + c] = sum;
    } else {
        const int c = blockIdx.x * 8 + threadIdx.x / 32;
        if (c >= m.C) return;
        for (long long r = r0 + threadIdx.x % 32; r < r1; r += 32) {
            const long long b = r / m.HW, i = (b * m.C + c) * m.HW + (r - b * m.HW);
            sum += to_f(dy[i]) * to_f(h[i]) * a.rstd[r];
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x % 32 == 0) a.part[(size_t)blockIdx.y * m.C + c] = sum;
    }
}

}  // namespace

size_t norm_workspace_floats(const MapShape& m, int, int sms) { return (size_t)norm_parts(m, sms) * m.C; }

cudaError_t launch_norm_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    return m.nhwc ? launch_norm_rows_fwd(m, dtype, a, d, sms, s) : launch_norm_planes_fwd(m, dtype, a, d, sms, s);
}

cudaError_t launch_norm_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    int parts = 0;
    cudaError_t e = m.nhwc ? launch_norm_rows_bwd(m, dtype, a, d, sms, &parts, s)
                           : launch_norm_planes_bwd(m, dtype, a, d, sms, &parts, s);
    if (e != cudaSuccess || !a.dweight) return e;
    if (!parts) {
        parts = (int)std::min(norm_parts(m, sms), 64LL);
        const dim3 grid((m.C + (m.nhwc ? 255 : 7)) / (m.nhwc ? 256 : 8), parts);
        if (dtype == WTCONV_F32) wtconv_norm_columns_kernel<float><<<grid, 256, 0, s>>>(m, a);
        else wtconv_norm_columns_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(m, a);
    }
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((m.C + 7) / 8);
    config.blockDim = dim3(1024);
    config.stream = s;
    config.attrs = &early;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, wtconv_norm_finish_kernel, m.C, parts, (const float*)a.part, a.dweight);
}

}  // namespace wtc
