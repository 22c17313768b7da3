// wq_norm.hip -- the norms before and after a block, its gate and residual.
//
//   t = y * rsqrt(mean(y^2) + eps) * post,  h' = h + alpha * gate * t,
//   x = h' * rsqrt(mean(h'^2) + eps) * pre
//
// HBM-bound: 12 to 20 bytes a value, one pass. A row is held in registers (4
// consecutive values a load) from its first read to its last write, by as many
// threads as it has groups of 4 values up to 1024 threads, which hold up to 8
// groups each (rows of 32768); longer rows are read once per sum. Many threads
// with one group each beat few with many, both where rows are few (one row of
// 1024: 2.6 us against 3.9 us for one wavefront) and where they fill the card
// (4096 x 1024: 14 against 18 us, 4.7 TB/s). Loads and stores of 4 values ask for
// 4-byte alignment only, so odd widths and offset storage take the same path;
// the last values of an odd row go one by one.
#include "wq_internal.h"
#include "wq_device.h"

namespace wq {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over a row's T threads; every thread gets it.
template <int T>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = wave_sum(v);
    if constexpr (T > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v += red[w];
    }
    return v;
}

// 4 values from i on, zeros past the row's end.
__device__ __forceinline__ f4 load4(const float *p, int64_t i, int64_t N)
{
    if (i + 4 <= N) return *reinterpret_cast<const f4u *>(p + i);
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < N) v[j] = p[i + j];
    return v;
}

__device__ __forceinline__ void store4(float *p, int64_t i, int64_t N, f4 v)
{
    if (i + 4 <= N) {
        *reinterpret_cast<f4u *>(p + i) = v;
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (i + j < N) p[i + j] = v[j];
    }
}

__device__ __forceinline__ float squares(f4 v) { return fmaf(v.x, v.x, v.y * v.y) + fmaf(v.z, v.z, v.w * v.w); }
__device__ __forceinline__ float inverse_rms(float sum, int64_t N, float eps) { return 1.0f / sqrtf(sum / (float)N + eps); }

__device__ __forceinline__ f4 residual(const NormArgs &a, f4 h, f4 y, f4 post, f4 gate, float ry)
{
    f4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float t = y[j];
        if (a.post) t = t * ry * post[j];
        if (a.gate) t *= gate[j];
        r[j] = fmaf(a.alpha, t, h[j]);
    }
    return r;
}

// T threads a row, V groups of 4 values a thread; workgroups of one row, or of
// 4 where a row is a wavefront's.
template <int T, int V>
__global__ __launch_bounds__(T == 64 ? 256 : T) void norm_kernel(NormArgs a)
{
    constexpr int kRows = T == 64 ? 4 : 1;
    __shared__ float red[T / 64];
    const int tid = threadIdx.x % T;
    for (int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / T; m < a.M; m += (int64_t)gridDim.x * kRows) {
        const float *hp = a.h + m * a.N, *yp = a.y ? a.y + m * a.N : nullptr, *gp = a.gate ? a.gate + m * a.gate_stride : nullptr;
        f4 h[V], y[V], gate[V], post[V], pre[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t i = 4 * (tid + T * v);
            h[v] = load4(hp, i, a.N);
            if (yp) y[v] = load4(yp, i, a.N);
            if (gp) gate[v] = load4(gp, i, a.N);
            if (a.post) post[v] = load4(a.post, i, a.N);
            if (a.pre && a.x_out) pre[v] = load4(a.pre, i, a.N);
        }
        if (yp) {
            float ry = 1.0f;
            if (a.post) {
                float s = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) s += squares(y[v]);
                ry = inverse_rms(row_sum<T>(s, red), a.N, a.eps);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = residual(a, h[v], y[v], post[v], gate[v], ry);
        }
        if (a.h_out) {
#pragma unroll
            for (int v = 0; v < V; ++v) store4(a.h_out + m * a.N, 4 * (tid + T * v), a.N, h[v]);
        }
        if (a.x_out) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) s += squares(h[v]);
            const float rh = inverse_rms(row_sum<T>(s, red), a.N, a.eps);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f4 x = h[v] * rh;
                if (a.pre) x *= pre[v];
                store4(a.x_out + m * a.N, 4 * (tid + T * v), a.N, x);
            }
        }
    }
}

// Rows of any length, read again for every sum; sums over the row in fp64.
constexpr int kLongThreads = 1024;

__global__ __launch_bounds__(kLongThreads) void long_norm_kernel(NormArgs a)
{
    __shared__ double red[kLongThreads / 64];
    const auto sum = [&](double v) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
        for (int w = 0; w < kLongThreads / 64; ++w) v += red[w];
        return (float)v;
    };
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const float *hp = a.h + m * a.N, *yp = a.y ? a.y + m * a.N : nullptr, *gp = a.gate ? a.gate + m * a.gate_stride : nullptr;
        const f4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
        float ry = 1.0f;
        if (a.post) {
            double s = 0.0;
            for (int64_t i = 4 * threadIdx.x; i < a.N; i += 4 * kLongThreads) s += (double)squares(load4(yp, i, a.N));
            ry = inverse_rms(sum(s), a.N, a.eps);
        }
        // (this thread's own values, so h_out may be h)
        const auto value = [&](int64_t i) {
            const f4 h = load4(hp, i, a.N);
            if (!yp) return h;
            return residual(a, h, load4(yp, i, a.N), a.post ? load4(a.post, i, a.N) : zero, gp ? load4(gp, i, a.N) : zero, ry);
        };
        float rh = 0.0f;
        if (a.x_out) {
            double s = 0.0;
            for (int64_t i = 4 * threadIdx.x; i < a.N; i += 4 * kLongThreads) s += (double)squares(value(i));
            rh = inverse_rms(sum(s), a.N, a.eps);
        }
        for (int64_t i = 4 * threadIdx.x; i < a.N; i += 4 * kLongThreads) {
            const f4 h = value(i);
            if (a.h_out) store4(a.h_out + m * a.N, i, a.N, h);
            if (a.x_out) {
                f4 x = h * rh;
                if (a.pre) x *= load4(a.pre, i, a.N);
                store4(a.x_out + m * a.N, i, a.N, x);
            }
        }
    }
}

template <int T, int V>
void run(const NormArgs &a, hipStream_t stream)
{
    constexpr int kRows = T == 64 ? 4 : 1;
    const int64_t groups = (a.M + kRows - 1) / kRows, most = (int64_t)1 << 20;
    norm_kernel<T, V><<<(unsigned)(groups < most ? groups : most), T == 64 ? 256 : T, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, hipStream_t stream)
{
    const int64_t groups = (a.N + 3) / 4;                // of 4 values
    if (groups <= 64) run<64, 1>(a, stream);
    else if (groups <= 128) run<128, 1>(a, stream);
    else if (groups <= 256) run<256, 1>(a, stream);
    else if (groups <= 512) run<512, 1>(a, stream);
    else if (groups <= 1024) run<1024, 1>(a, stream);
    else if (groups <= 2048) run<1024, 2>(a, stream);
    else if (groups <= 4096) run<1024, 4>(a, stream);
    else if (groups <= 8192) run<1024, 8>(a, stream);
    else long_norm_kernel<<<(unsigned)(a.M < 65536 ? a.M : 65536), kLongThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace wq
