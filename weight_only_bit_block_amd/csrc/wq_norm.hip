// wq_norm.hip -- the norms before and after a block, its gate and residual.
//
//   t = y * rsqrt(mean(y^2) + eps) * post,  h' = h + alpha * gate * t,
//   x = h' * rsqrt(mean(h'^2) + eps) * pre
//
// HBM-bound: 12 to 20 bytes a value, one pass. A row is held in registers from
// its first read to its last write: 2 groups of 4 consecutive values a thread
// where 640 threads are enough (3 such workgroups fit a compute unit), then 4
// (rows of 16384); longer rows are read once per sum (8 groups do not fit 128
// registers a thread: 256 x 32768 72.7 us, read again 45.6). One group a thread
// spends more on the barriers of its sums, four leave fewer wavefronts, in us
// for 1 / 2 / 4 groups, gate and both norms: 1 x 1024 3.9 / 3.9 / 4.4, 4096 x 1024
// 16.5 / 15.0 / 14.7 (5.7 TB/s), 1024 x 4096 18.1 / 15.7 / 14.6, 515 x 5003
// - / 15.4 / 17.1, 512 x 8192 - / 19.3 / 15.0. (Between 2560 and 5120 values two groups are
// the better choice for most numbers of rows: 64 x 4096 4.7 / 5.5, 4096 x 4096 60.0 / 62.3, 1024 x 5100
// 23.7 / 24.6 for 2 / 4, though not for 1024 x 4096.) A row of 1024 in one wavefront: 5.0,
// 4096 of them 17.3. Loads and stores of 4 values ask for 4-byte alignment only,
// so odd widths and offset storage take the same path; the last values of an odd
// row go one by one.
#include "wq_internal.h"
#include "wq_device.h"

namespace wq {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kMaxThreads = 1024, kPairThreads = 640;

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over a row's threads; every thread gets it.
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, float *red)
{
    v = wave_sum(v);
    if constexpr (!ONE) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
        for (int w = 0; w < (int)blockDim.x / 64; ++w) v += red[w];
    }
    return v;
}

// 4 values from i on, zeros past the row's end.
template <typename I>
__device__ __forceinline__ f4 load4(const float *p, I i, I N)
{
    if (i + 4 <= N) return *reinterpret_cast<const f4u *>(p + i);
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (i + j < N) v[j] = p[i + j];
    return v;
}

// (Stored non-temporally: lines still dirty in the L2 when the kernel ends delay
// what follows, 2048 x 1024 10.0 -> 8.5 us, 512 x 8192 15.4 -> 13.7.)
template <typename I>
__device__ __forceinline__ void store4(float *p, I i, I N, f4 v)
{
    if (i + 4 <= N) {
        __builtin_nontemporal_store(v, reinterpret_cast<f4u *>(p + i));
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

// V groups of 4 values a thread; workgroups of one row, or, ONE, of 4 rows of a
// wavefront each.
template <bool ONE, int V>
__global__ __launch_bounds__(ONE ? 256 : kMaxThreads) void norm_kernel(NormArgs a)
{
    constexpr int kRows = ONE ? 4 : 1;
    __shared__ float red[kMaxThreads / 64];
    const uint32_t T = ONE ? 64 : blockDim.x, tid = threadIdx.x % T, N = (uint32_t)a.N;       // (32-bit offsets: N is small)
    for (int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / T; m < a.M; m += (int64_t)gridDim.x * kRows) {
        const float *hp = a.h + m * a.N, *yp = a.y ? a.y + m * a.N : nullptr, *gp = a.gate ? a.gate + m * a.gate_stride : nullptr;
        f4 h[V], y[V], gate[V], post[V], pre[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t i = 4 * (tid + T * v);
            h[v] = load4(hp, i, N);
            if (yp) y[v] = load4(yp, i, N);
            if (gp) gate[v] = load4(gp, i, N);
            if (a.post) post[v] = load4(a.post, i, N);
            if (a.pre && a.x_out) pre[v] = load4(a.pre, i, N);
        }
        if (yp) {
            float ry = 1.0f;
            if (a.post) {
                float s = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) s += squares(y[v]);
                ry = inverse_rms(row_sum<ONE>(s, red), a.N, a.eps);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = residual(a, h[v], y[v], post[v], gate[v], ry);
        }
        if (a.h_out) {
#pragma unroll
            for (int v = 0; v < V; ++v) store4(a.h_out + m * a.N, 4 * (tid + T * v), N, h[v]);
        }
        if (a.x_out) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) s += squares(h[v]);
            const float rh = inverse_rms(row_sum<ONE>(s, red), a.N, a.eps);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f4 x = h[v] * rh;
                if (a.pre) x *= pre[v];
                store4(a.x_out + m * a.N, 4 * (tid + T * v), N, x);
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

template <bool ONE, int V>
void run(const NormArgs &a, int threads, hipStream_t stream)
{
    const int64_t rows = ONE ? 4 : 1, groups = (a.M + rows - 1) / rows, most = (int64_t)1 << 20;
    norm_kernel<ONE, V><<<(unsigned)(groups < most ? groups : most), threads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, hipStream_t stream)
{
    const int64_t groups = (a.N + 3) / 4;                // of 4 values
    const auto threads = [&](int v) { return (int)((groups + 64 * v - 1) / (64 * v) * 64); };
    if (groups > 4 * kMaxThreads) long_norm_kernel<<<(unsigned)(a.M < 65536 ? a.M : 65536), kLongThreads, 0, stream>>>(a);
    else if (groups <= 64) run<true, 1>(a, 256, stream);
    else if (threads(2) <= kPairThreads) run<false, 2>(a, threads(2), stream);
    else run<false, 4>(a, threads(4), stream);
    return hipGetLastError();
}

}  // namespace wq
