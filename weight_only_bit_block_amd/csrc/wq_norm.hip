// wq_norm.hip -- the norms before and after a block, its gate and residual.
//
//   t = y * rsqrt(mean(y^2) + eps) * post,  h' = h + alpha * gate * t,
//   x = h' * rsqrt(mean(h'^2) + eps) * pre
#include "wq_internal.h"
#include "wq_device.h"

namespace wq {
namespace {

__device__ __forceinline__ double block_sum(double v, double *red)
{
    for (int x = 32; x; x >>= 1) v += __shfl_xor(v, x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += red[i];
    return s;
}

// One workgroup per row, values read again for every pass.
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a)
{
    __shared__ double red[4];
    const int64_t m = blockIdx.x;
    const float *h = a.h + m * a.N, *y = a.y ? a.y + m * a.N : nullptr, *gate = a.gate ? a.gate + m * a.gate_stride : nullptr;
    float ry = 1.0f;
    if (a.post) {
        double s = 0.0;
        for (int64_t i = threadIdx.x; i < a.N; i += 256) s += (double)(y[i] * y[i]);
        ry = 1.0f / sqrtf((float)(block_sum(s, red) / (double)a.N) + a.eps);
    }
    auto residual = [&](int64_t i) {
        float t = y ? y[i] : 0.0f;
        if (a.post) t = t * ry * a.post[i];
        if (gate) t *= gate[i];
        return y ? fmaf(a.alpha, t, h[i]) : h[i];
    };
    float rh = 0.0f;
    if (a.x_out) {
        double s = 0.0;
        for (int64_t i = threadIdx.x; i < a.N; i += 256) {
            const float v = residual(i);
            s += (double)(v * v);
        }
        rh = 1.0f / sqrtf((float)(block_sum(s, red) / (double)a.N) + a.eps);
    }
    for (int64_t i = threadIdx.x; i < a.N; i += 256) {
        const float v = residual(i);
        if (a.h_out) a.h_out[m * a.N + i] = v;
        if (a.x_out) a.x_out[m * a.N + i] = a.pre ? v * rh * a.pre[i] : v * rh;
    }
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, hipStream_t stream)
{
    norm_kernel<<<(unsigned)a.M, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace wq
