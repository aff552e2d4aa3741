// Counter-based dropout of a map: y = residual + d * x, d = 0 or the float
// next to 1 / (1 - p).  The mask is a function of (seed, offset, row,
// channel) alone, so it is never stored: the backward is the same kernel on dy.
#include "wtconv_map_launch.h"

namespace wtc {

template <typename T>
__global__ void wtconv_dropout_kernel(MapShape m, DropArgs a, MapDrop d) {
    const long long n = m.rows * m.C, step = (long long)gridDim.x * blockDim.x;
    const uint32_t offset = drop_offset(d);
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        long long row;
        int c;
        if (m.nhwc) {
            row = i / m.C;
            c = (int)(i - row * m.C);
        } else {
            const long long plane = i / m.HW, b = plane / m.C;
            c = (int)(plane - b * m.C);
            row = b * m.HW + (i - plane * m.HW);
        }
        const bool keep = keep_quad(d, offset, drop_row(d, m, row), d.mode == WTCONV_DROP_SAMPLE ? 0 : c >> 2) >> (c & 3) & 1;
        const float r = a.residual ? to_f(static_cast<const T*>(a.residual)[i]) : 0.0f;
        const float v = to_f(static_cast<const T*>(a.x)[i]);
        static_cast<T*>(a.y)[i] = from_f<T>(keep ? __fmaf_rn(v, d.grown, r) : r);
    }
}

cudaError_t launch_dropout(const MapShape& m, int dtype, const DropArgs& a, const MapDrop& d, int sms, cudaStream_t s) {
    const int threads = 256;
    const long long blocks = (m.rows * m.C + threads - 1) / threads;
    const unsigned grid = (unsigned)(blocks < 16LL * sms ? blocks : 16LL * sms);
    if (dtype == WTCONV_F32)
        wtconv_dropout_kernel<float><<<grid, threads, 0, s>>>(m, a, d);
    else
        wtconv_dropout_kernel<__nv_bfloat16><<<grid, threads, 0, s>>>(m, a, d);
    return cudaGetLastError();
}

}  // namespace wtc
