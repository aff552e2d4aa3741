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
#include <cuda_fp8.h>

#include "wtconv_map_launch.h"

namespace wtc {

namespace {

constexpr int kThreads = 256;
constexpr int kWChunks = 64;  // row chunks of the weight gradient's first sum

template <int TPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = TPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The TPR threads of a row: 32 where the channels are adjacent, 1 where the
// pixels are (neighbouring threads then read neighbouring pixels).
template <typename T, int TPR>
__global__ void norm_fwd_kernel(MapShape m, NormFwdArgs a, MapDrop d) {
    const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) / TPR;
    const int lane = threadIdx.x % TPR;
    const bool live = row < m.rows;
    const long long cs = TPR == 1 ? m.HW : 1;
    const long long b = live ? row / m.HW : 0;
    const long long base = TPR == 1 ? b * m.C * m.HW + (live ? row - b * m.HW : 0) : (live ? row : 0) * m.C;
    const T* x = static_cast<const T*>(a.x) + base;
    const T* res = static_cast<const T*>(a.residual) + base;
    T* h = static_cast<T*>(a.h) + base;
    const uint32_t offset = d.on ? drop_offset(d) : 0;
    const long long drow = drop_row(d, m, row);
    auto joined = [&](int c) {
        float v = to_f(x[c * cs]);
        if (a.residual) {
            bool keep = true;
            if (d.on) keep = keep_quad(d, offset, drow, d.mode == WTCONV_DROP_SAMPLE ? 0 : c >> 2) >> (c & 3) & 1;
            const float r = to_f(res[c * cs]);
            v = to_f(from_f<T>(keep ? __fmaf_rn(v, d.grown, r) : r));
        }
        return v;
    };
    float ss = 0.0f;
    if (live)
        for (int c = lane; c < m.C; c += TPR) {
            const float v = joined(c);
            if (a.residual) h[c * cs] = from_f<T>(v);
            ss += v * v;
        }
    ss = row_sum<TPR>(ss);
    const float r = rsqrtf(ss / m.C + a.eps);
    if (!live) return;
    if (a.rstd && lane == 0) a.rstd[row] = r;
    if (a.q8 < 0) {
        for (int c = lane; c < m.C; c += TPR) static_cast<T*>(a.y)[base + c * cs] = from_f<T>(joined(c) * r * a.weight[c]);
        return;
    }
    const float top = a.q8 == WTCONV_E4M3 ? 448.0f : 127.0f;
    const int groups = (m.C + a.group - 1) / a.group;
    for (int g = 0; g < groups; ++g) {
        const int c1 = min(m.C, (g + 1) * a.group);
        uint32_t bits = 0;  // the bits of |v| are ordered like |v|, NaN above infinity
        for (int c = g * a.group + lane; c < c1; c += TPR)
            bits = max(bits, __float_as_uint(fabsf(joined(c) * r * a.weight[c])));
#pragma unroll
        for (int o = TPR / 2; o; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
        float scale = __uint_as_float(bits) / top;
        if (scale < 1.17549435e-38f) scale = 1.17549435e-38f;
        if (lane == 0) a.scale[TPR == 1 ? (b * groups + g) * m.HW + (row - b * m.HW) : row * groups + g] = scale;
        for (int c = g * a.group + lane; c < c1; c += TPR) {
            const float q = joined(c) * r * a.weight[c] / scale;
            const long long i = base + c * cs;
            if (a.q8 == WTCONV_E4M3)
                static_cast<uint8_t*>(a.y)[i] = __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
            else
                static_cast<int8_t*>(a.y)[i] = (int8_t)(isnan(q) ? 0 : max(-127, min(127, __float2int_rn(q))));
        }
    }
}

template <typename T, int TPR>
__global__ void norm_bwd_kernel(MapShape m, NormBwdArgs a, MapDrop d) {
    const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) / TPR;
    const int lane = threadIdx.x % TPR;
    const bool live = row < m.rows;
    const long long cs = TPR == 1 ? m.HW : 1;
    const long long b = live ? row / m.HW : 0;
    const long long base = TPR == 1 ? b * m.C * m.HW + (live ? row - b * m.HW : 0) : (live ? row : 0) * m.C;
    const T* h = static_cast<const T*>(a.h) + base;
    const T* dy = static_cast<const T*>(a.dy) + base;
    float gh = 0.0f;
    if (live)
        for (int c = lane; c < m.C; c += TPR) gh += to_f(dy[c * cs]) * a.weight[c] * to_f(h[c * cs]);
    gh = row_sum<TPR>(gh);
    if (!live) return;
    const uint32_t offset = d.on ? drop_offset(d) : 0;
    const long long drow = drop_row(d, m, row);
    const float r = a.rstd[row], s = gh / m.C * r * r;
    for (int c = lane; c < m.C; c += TPR) {
        float v = r * (to_f(dy[c * cs]) * a.weight[c] - to_f(h[c * cs]) * s);
        if (a.dh) v += to_f(static_cast<const T*>(a.dh)[base + c * cs]);
        if (a.dres) static_cast<T*>(a.dres)[base + c * cs] = from_f<T>(v);
        if (a.dx) {
            const bool keep = keep_quad(d, offset, drow, d.mode == WTCONV_DROP_SAMPLE ? 0 : c >> 2) >> (c & 3) & 1;
            static_cast<T*>(a.dx)[base + c * cs] = from_f<T>(keep ? v * d.grown : 0.0f);
        }
    }
}

// One channel's sum over a chunk of the rows, then over the chunks in order.
template <typename T>
__global__ void norm_dw_kernel(MapShape m, NormBwdArgs a) {
    const int c = blockIdx.x;
    float sum = 0.0f;
    for (long long row = (long long)blockIdx.y * kThreads + threadIdx.x; row < m.rows; row += (long long)kWChunks * kThreads) {
        const long long b = row / m.HW;
        const long long i = m.nhwc ? row * m.C + c : (b * m.C + c) * m.HW + (row - b * m.HW);
        sum += to_f(static_cast<const T*>(a.dy)[i]) * to_f(static_cast<const T*>(a.h)[i]) * a.rstd[row];
    }
    sum = row_sum<32>(sum);
    __shared__ float part[kThreads / 32];
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int k = 1; k < kThreads / 32; ++k) sum += part[k];
        a.part[(size_t)blockIdx.y * m.C + c] = sum;
    }
}
__global__ void norm_dw_finish_kernel(int C, const float* part, float* dweight) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float sum = 0.0f;
    for (int k = 0; k < kWChunks; ++k) sum += part[(size_t)k * C + c];
    dweight[c] = sum;
}

template <typename T, int TPR>
void run_bwd(const MapShape& m, const NormBwdArgs& a, const MapDrop& d, cudaStream_t s) {
    if (a.dres || a.dx) norm_bwd_kernel<T, TPR><<<(unsigned)((m.rows * TPR + kThreads - 1) / kThreads), kThreads, 0, s>>>(m, a, d);
    if (a.dweight) {
        norm_dw_kernel<T><<<dim3(m.C, kWChunks), kThreads, 0, s>>>(m, a);
        norm_dw_finish_kernel<<<(m.C + kThreads - 1) / kThreads, kThreads, 0, s>>>(m.C, a.part, a.dweight);
    }
}

}  // namespace

size_t norm_workspace_floats(const MapShape& m, int, int) { return (size_t)kWChunks * m.C; }

cudaError_t launch_norm_fwd(const MapShape& m, int dtype, const NormFwdArgs& a, const MapDrop& d, int, cudaStream_t s) {
    const unsigned grid = (unsigned)((m.rows * (m.nhwc ? 32 : 1) + kThreads - 1) / kThreads);
    if (dtype == WTCONV_F32 && m.nhwc) norm_fwd_kernel<float, 32><<<grid, kThreads, 0, s>>>(m, a, d);
    else if (dtype == WTCONV_F32) norm_fwd_kernel<float, 1><<<grid, kThreads, 0, s>>>(m, a, d);
    else if (m.nhwc) norm_fwd_kernel<__nv_bfloat16, 32><<<grid, kThreads, 0, s>>>(m, a, d);
    else norm_fwd_kernel<__nv_bfloat16, 1><<<grid, kThreads, 0, s>>>(m, a, d);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const MapShape& m, int dtype, const NormBwdArgs& a, const MapDrop& d, int, cudaStream_t s) {
    if (dtype == WTCONV_F32 && m.nhwc) run_bwd<float, 32>(m, a, d, s);
    else if (dtype == WTCONV_F32) run_bwd<float, 1>(m, a, d, s);
    else if (m.nhwc) run_bwd<__nv_bfloat16, 32>(m, a, d, s);
    else run_bwd<__nv_bfloat16, 1>(m, a, d, s);
    return cudaGetLastError();
}

}  // namespace wtc
