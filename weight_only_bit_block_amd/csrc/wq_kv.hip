// wq_kv.hip -- the int4 key/value cache: append, and attention of single tokens.
#include "wq_internal.h"
#include "wq_device.h"
#include "wq_seq.h"

namespace wq {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- append
// 8 lanes per block of 32 values, 4 consecutive values each: a wavefront reads
// 1 KiB of consecutive floats and writes 128 bytes of codes. The maximum of a
// block and its code dwords go over the 8 lanes by cross-lane moves. Division
// is the correctly rounded fp32 one, as in wq_pack.
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a)
{
    const int D = a.cache.head_dim, H = a.cache.kv_heads;
    const int per_row = D / 4;                           // threads per row of one head
    const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = gid / per_row;                   // (token, head)
    const int c = (int)(gid - row * per_row);            // 4-value group within the row
    const bool values = blockIdx.y != 0;
    const int64_t t = row / H;
    const int h = (int)(row - t * H);
    int64_t dst = -1;                                    // cache row
    f4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (t < a.T) {
        const int b = seq_of_token(a.cu, a.B, (int)t);
        const SeqRange r = seq_range(a.cu, (int)a.T, b);
        if (t >= r.begin && t < r.end) {
            const int64_t pos = (a.start ? (int64_t)a.start[b] : 0) + (t - r.begin);
            if (pos >= 0 && pos < a.max_pages * WQ_KV_PAGE) {
                const int64_t page = a.table[(int64_t)b * a.max_pages + pos / WQ_KV_PAGE];
                if (page >= 0 && page < a.cache.n_pages)
                    dst = (page * H + h) * WQ_KV_PAGE + pos % WQ_KV_PAGE;
            }
        }
        if (dst >= 0) {
            const float *src = values ? a.v + t * a.v_stride : a.k + t * a.k_stride;
            x = *reinterpret_cast<const f4 *>(src + h * D + c * 4);
        }
    }
    float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
    // not finite anywhere: a NaN block (fmaxf drops NaN, so it is asked for apart)
    const float big = 3.4028235e38f;
    bool bad = !(fabsf(x.x) <= big && fabsf(x.y) <= big && fabsf(x.z) <= big && fabsf(x.w) <= big);
    int badi = bad;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        amax = fmaxf(amax, __shfl_xor(amax, o));
        badi |= __shfl_xor(badi, o);
    }
    const _Float16 s16 = (_Float16)(amax / 7.0f);
    const float sf = (float)s16;
    uint16_t sbits = __builtin_bit_cast(uint16_t, s16);
    uint32_t codes = 0;
    if (badi || !(sf <= 65504.0f)) {
        sbits = 0x7E00;
    } else if (sf != 0.0f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float q = fminf(fmaxf(rintf(x[j] / sf), -8.0f), 7.0f);
            codes |= ((uint32_t)(int)q & 0xFu) << (4 * j);
        }
    } else {
        sbits = 0;
    }
    if (dst < 0) return;
    uint16_t *q = reinterpret_cast<uint16_t *>(values ? a.cache.vq : a.cache.kq);
    uint16_t *s = values ? a.cache.vs : a.cache.ks;
    q[dst * per_row + c] = (uint16_t)codes;              // D / 2 bytes a row, 2 bytes a thread
    if ((c & 7) == 0) s[dst * (D / 32) + (c >> 3)] = sbits;
}

// ---------------------------------------------------------------- decode attention
__device__ __forceinline__ float cached(const void *q, const uint16_t *s, int64_t row, int D, int d)
{
    const uint8_t byte = reinterpret_cast<const uint8_t *>(q)[row * (D / 2) + d / 2];
    const int code = (int)((uint32_t)((byte >> (4 * (d & 1))) & 15) << 28) >> 28;
    return (float)code * (float)__builtin_bit_cast(_Float16, s[row * (D / 32) + d / 32]);
}

// One wavefront per (sequence, query head), keys in order.
template <int D>
__global__ __launch_bounds__(64) void decode_kernel(DecodeArgs a)
{
    constexpr int E = D / 64;
    const int b = blockIdx.x / a.heads, j = blockIdx.x % a.heads, lane = threadIdx.x;
    const int H = a.cache.kv_heads, kj = j / (a.heads / H);
    float *out = a.out + (int64_t)b * a.out_stride + j * D;
    const int64_t len = a.lens[b];
    const int32_t *pages = a.table + (int64_t)b * a.max_pages;
    bool bad = len < 0 || len > a.max_pages * WQ_KV_PAGE;
    if (!bad)
        for (int64_t i = 0; i < (len + WQ_KV_PAGE - 1) / WQ_KV_PAGE; ++i) bad |= pages[i] < 0 || pages[i] >= a.cache.n_pages;
    if (bad || len == 0) {
        for (int e = 0; e < E; ++e) out[e * 64 + lane] = bad ? __builtin_nanf("") : 0.0f;
        return;
    }
    float q[E], o[E];
    for (int e = 0; e < E; ++e) {
        q[e] = a.q[(int64_t)b * a.q_stride + j * D + e * 64 + lane];
        if (!(fabsf(q[e]) <= 3.4028235e38f)) q[e] = __builtin_nanf("");
        o[e] = 0.0f;
    }
    const float c = a.scale * 1.44269504088896341f;
    float m = -3.0e38f, l = 0.0f;
    for (int64_t u = 0; u < len; ++u) {
        const int64_t row = ((int64_t)pages[u / WQ_KV_PAGE] * H + kj) * WQ_KV_PAGE + u % WQ_KV_PAGE;
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], cached(a.cache.kq, a.cache.ks, row, D, e * 64 + lane), s);
        for (int x = 32; x; x >>= 1) s += __shfl_xor(s, x);
        s *= c;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, cached(a.cache.vq, a.cache.vs, row, D, e * 64 + lane), o[e] * f);
    }
    for (int e = 0; e < E; ++e) out[e * 64 + lane] = o[e] / l;
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t stream)
{
    const int64_t threads = a.T * a.cache.kv_heads * (a.cache.head_dim / 4);
    const dim3 grid((unsigned)((threads + 255) / 256), 2);
    append_kernel<<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

uint64_t decode_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t stream)
{
    const unsigned grid = (unsigned)((int64_t)a.B * a.heads);
    if (a.cache.head_dim == 128) decode_kernel<128><<<grid, 64, 0, stream>>>(a);
    else decode_kernel<64><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace wq
