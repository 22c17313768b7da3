// wq_rope.hip -- norms of queries and keys for each head, and the rotation by
// position, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * weight          over the head's D values
//   (y_i, y_i') -> factor (y_i cos a - y_i' sin a, y_i' cos a + y_i sin a),
//   a = position * inv_freq[i], for `pairs` pairs; the other values keep y
//
// HBM-bound: 8 D bytes for a token and head (8192 tokens of 24 heads of 128: 201 MB,
// 34 us, 5.9 TB/s with inputs partly in the last-level cache; in a program's turns
// of inputs 39). A row is D / 8 lanes with two groups of 4 values each, chosen so
// that a lane holds both sides of its pairs: no value changes lanes, only the sum of
// squares goes over them. Asking for 2 rows ahead instead of 4 costs as much, 6 more
// (36.4); stores past the L2: 2048 tokens 10.9 -> 10.2 us, 8192 34.1 -> 34.9.
//
// Angles: their products and the reduction to a turn in fp64 (a position and a
// factor of 24 bits: off by 2^-53 of the angle), sine and cosine in fp32 of what is
// left, in two parts.
// They are the same for all heads of a token, so a workgroup makes each of them
// once, one a thread, while its rows are on the way.
#include "wq_internal.h"
#include "wq_device.h"

namespace wq {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kAhead = 4;                    // rows a lane asks for at once

template <int CTRL>
__device__ __forceinline__ float add_dpp(float x)
{
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Sum over a row's D / 8 lanes, the same in each of them.
template <int D>
__device__ __forceinline__ float row_sum(float x)
{
    x = add_dpp<0xB1>(x);                    // quad_perm 1 0 3 2, 2 3 0 1, row_half_mirror, row_mirror
    x = add_dpp<0x4E>(x);
    x = add_dpp<0x141>(x);
    return D == 128 ? add_dpp<0x140>(x) : x;
}

__device__ __forceinline__ float squares(f4 v) { return fmaf(v.x, v.x, v.y * v.y) + fmaf(v.z, v.z, v.w * v.w); }

// The row times its inverse root mean square. Squares outside fp32's range (sums
// that are infinite, or so small that eps does not cover what is lost) are taken of
// values brought near 1 by a power of two.
template <int D>
__device__ __forceinline__ void normalise(f4 &x, f4 &y, float eps)
{
    const float s = row_sum<D>(squares(x) + squares(y));
    float r = 1.0f / sqrtf(s / D + eps);
    const bool big = s > 1.7e38f, small = s < 1e-27f && eps < 1e-30f;
    if (__any(big || small)) {
        const int e = big ? -70 : small ? 100 : 0;
        f4 p, q;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p[j] = ldexpf(x[j], e);
            q[j] = ldexpf(y[j], e);
        }
        const float t = row_sum<D>(squares(p) + squares(q));
        if (e != 0) {
            x = p;
            y = q;
            r = 1.0f / sqrtf(t / D + ldexpf(eps, 2 * e));
        }
    }
    x *= r;
    y *= r;
}

// TOK tokens a workgroup, 4 / TOK wavefronts each.
template <int D, int TOK, bool NORM, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a)
{
    constexpr int L = D / 8, kRows = 64 / L, kStep = kRows * (4 / TOK);          // rows of a wavefront, of all that share the token
    __shared__ float2 turn[TOK][D / 2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % L;
    const int64_t token0 = (int64_t)blockIdx.x * TOK, token = token0 + wave / (4 / TOK);
    const bool live = token < a.T;
    // this lane's values: both sides of its pairs
    const int p = 4 * l;
    const int at1 = INTER || p < a.pairs ? p : p + a.pairs;
    const int at2 = INTER ? p + D / 2 : at1 + (p < a.pairs ? a.pairs : D / 2 - a.pairs);
    const int rows = a.heads + a.kv_heads, first = wave % (4 / TOK) * kRows + lane / L;
    const float *const q = a.q + (live ? token : 0) * a.q_stride, *const k = a.k + (live ? token : 0) * a.k_stride;
    f4 x[kAhead], y[kAhead];
    const auto load = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kStep < rows ? r0 + i * kStep : rows - 1;     // (read again, to no use)
            const float *src = r < a.heads ? q + r * D : k + (r - a.heads) * D;
            x[i] = *reinterpret_cast<const f4 *>(src + at1);
            y[i] = *reinterpret_cast<const f4 *>(src + at2);
        }
    };
    load(first);
    for (int i = threadIdx.x; i < TOK * (D / 2); i += 256) {
        const int64_t t = token0 + i / (D / 2);
        const int pair = i % (D / 2);
        float2 z = {1.0f, 0.0f};
        if (pair < a.pairs && t < a.T) {
            const double turns = (double)a.positions[t] * (double)a.inv_freq[pair] * 0.15915494309189533577;
            // half turns in two parts, the second one by its tangent
            const double half = 2.0 * (turns - rint(turns));
            const float x = (float)half, rest = 3.14159265f * (float)(half - (double)x);
            const float c = cospif(x), s = sinpif(x);
            z = float2{fmaf(-rest, s, c) * a.factor, fmaf(rest, c, s) * a.factor};
        }
        turn[i / (D / 2)][pair] = z;
    }
    const int position = live ? a.positions[token] : -1;         // < 0: nothing is written
    f4 qw1, qw2, kw1, kw2;
    if (NORM) {
        qw1 = qw2 = kw1 = kw2 = f4{1.0f, 1.0f, 1.0f, 1.0f};
        if (a.q_weight) {
            qw1 = *reinterpret_cast<const f4 *>(a.q_weight + at1);
            qw2 = *reinterpret_cast<const f4 *>(a.q_weight + at2);
        }
        if (a.k_weight) {
            kw1 = *reinterpret_cast<const f4 *>(a.k_weight + at1);
            kw2 = *reinterpret_cast<const f4 *>(a.k_weight + at2);
        }
    }
    __syncthreads();
    const float2 *z = turn[wave / (4 / TOK)];
    float2 t[4];                             // of the lane's pairs
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = z[INTER ? 2 * l + (j & 1) + (j >> 1) * (D / 4) : p + j];
    // Values that are not rotated go round the rotation: by an angle of 0 one that is not finite would spoil its
    // partner. (pairs is a multiple of 4, so that a lane's four values on a side are of one kind)
    const bool turns1 = (INTER ? 2 * l : p) < a.pairs, turns2 = INTER ? 2 * l + D / 4 < a.pairs : turns1;
    for (int r0 = first; r0 - first < rows; r0 += kAhead * kStep) {
        if (r0 != first) load(r0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = r0 + i * kStep;
            if (NORM) {
                normalise<D>(x[i], y[i], a.eps);
                x[i] *= r < a.heads ? qw1 : kw1;
                y[i] *= r < a.heads ? qw2 : kw2;
            }
            f4 u, v;
            if (INTER) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    u[2 * j] = fmaf(x[i][2 * j], t[j].x, -(x[i][2 * j + 1] * t[j].y));
                    u[2 * j + 1] = fmaf(x[i][2 * j + 1], t[j].x, x[i][2 * j] * t[j].y);
                    v[2 * j] = fmaf(y[i][2 * j], t[2 + j].x, -(y[i][2 * j + 1] * t[2 + j].y));
                    v[2 * j + 1] = fmaf(y[i][2 * j + 1], t[2 + j].x, y[i][2 * j] * t[2 + j].y);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u[j] = fmaf(x[i][j], t[j].x, -(y[i][j] * t[j].y));
                    v[j] = fmaf(y[i][j], t[j].x, x[i][j] * t[j].y);
                }
            }
            if (!turns1) u = x[i];
            if (!turns2) v = y[i];
            if (r < rows && position >= 0) {
                float *dst = r < a.heads ? a.q_out + token * a.q_out_stride + r * D : a.k_out + token * a.k_out_stride + (r - a.heads) * D;
                *reinterpret_cast<f4 *>(dst + at1) = u;
                *reinterpret_cast<f4 *>(dst + at2) = v;
            }
        }
    }
}

template <int D, int TOK>
hipError_t launch(const RopeArgs &a, bool norm, bool interleaved, hipStream_t stream)
{
    const unsigned grid = (unsigned)((a.T + TOK - 1) / TOK);
    if (norm) {
        if (interleaved) rope_kernel<D, TOK, true, true><<<grid, 256, 0, stream>>>(a);
        else rope_kernel<D, TOK, true, false><<<grid, 256, 0, stream>>>(a);
    } else {
        if (interleaved) rope_kernel<D, TOK, false, true><<<grid, 256, 0, stream>>>(a);
        else rope_kernel<D, TOK, false, false><<<grid, 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs &a, bool norm, bool interleaved, hipStream_t stream)
{
    // Few tokens: a workgroup each, whose wavefronts share its heads; else one wavefront a token, which
    // computes angles for 4 tokens at once. us in a graph, 1 / 4 tokens: 24 heads of 128, 1 token 3.0 / 4.3, 512 4.2 / 6.1,
    // 1024 7.1 / 7.3, 2048 11.4 / 10.9, 8192 35.8 / 34.1; 16 heads of 64, 512 3.5 / 3.4, 1003 4.5 / 3.7, 4096 12.4 / 8.5.
    if (a.T * (128 / a.head_dim) < 1024) return a.head_dim == 128 ? launch<128, 1>(a, norm, interleaved, stream) : launch<64, 1>(a, norm, interleaved, stream);
    return a.head_dim == 128 ? launch<128, 4>(a, norm, interleaved, stream) : launch<64, 4>(a, norm, interleaved, stream);
}

}  // namespace wq
