// wq_prompt.hip -- causal attention over packed prompts (fp32, grouped heads).
#include "wq_internal.h"
#include "wq_device.h"
#include "wq_seq.h"

namespace wq {
namespace {

// A value, or NaN in the place of an infinity.
__device__ __forceinline__ float finite(float x) { return fabsf(x) <= 3.4028235e38f ? x : __builtin_nanf(""); }

// One wavefront per (token, query head): lane l owns values l, l + 64, ... of
// the head, and walks the keys with a running maximum and sum.
template <int D>
__global__ __launch_bounds__(64) void prompt_kernel(PromptArgs a)
{
    constexpr int E = D / 64;
    const int64_t id = blockIdx.x;
    const int t = (int)(id / a.heads), j = (int)(id % a.heads), lane = threadIdx.x;
    const int b = seq_of_token(a.cu, a.B, t);
    const SeqRange r = seq_range(a.cu, (int)a.T, b);
    if (t < r.begin || t >= r.end) return;
    const int kj = j / (a.heads / a.kv_heads);
    const float c = a.scale * 1.44269504088896341f;
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = finite(a.q[(int64_t)t * a.q_stride + j * D + e * 64 + lane]);
        o[e] = 0.0f;
    }
    float m = -3.0e38f, l = 0.0f;
    for (int u = r.begin; u <= t; ++u) {
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], finite(a.k[(int64_t)u * a.k_stride + kj * D + e * 64 + lane]), s);
        for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
        s *= c;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
        for (int e = 0; e < E; ++e) {
            // a non-finite value makes its element NaN whatever its weight
            o[e] = fmaf(p, finite(a.v[(int64_t)u * a.v_stride + kj * D + e * 64 + lane]), o[e] * f);
        }
    }
    for (int e = 0; e < E; ++e) a.out[(int64_t)t * a.out_stride + j * D + e * 64 + lane] = o[e] / l;
}

}  // namespace

uint64_t prompt_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_attn_prefill(const PromptArgs &a, hipStream_t stream)
{
    const unsigned grid = (unsigned)(a.T * a.heads);
    if (a.head_dim == 128) prompt_kernel<128><<<grid, 64, 0, stream>>>(a);
    else prompt_kernel<64><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace wq
