// wq_kv.hip -- the int4 key/value cache: append, and attention of single tokens.
#include "wq_internal.h"
#include "wq_device.h"
#include "wq_kv_decode.h"
#include "wq_seq.h"

#include <type_traits>

namespace wq {
namespace {

// ---------------------------------------------------------------- append
// HBM-bound: 8 D bytes read and 1.125 D written for a token and head. A row of
// D values is D / 4 lanes, 4 values each: a wavefront reads 1 KiB of consecutive
// floats, the maximum of a block goes over its 8 lanes by cross-lane moves.
// Every thread takes kAppendRows rows, keys and values, and asks for all of
// them before it looks up where they go (three dependent reads). 4096 tokens, 8
// heads of 128, calls back to back: 10.3 us, 3.7 TB/s (rows read with cached loads: 10.9;
// inputs still in the last-level cache 8.9, six sets in turn 11.1); 16384: 31, 4.9. With slots given:
// 4096 tokens 9.7 (one read in place of three), 48 of one each 3.3 in a graph.
//
// The quotients of wq_pack's rule are correctly rounded; here they cost three
// operations each instead of a division's ten: q0 = x r, q = q0 + r (x - q0 s)
// with r the correctly rounded 1 / s is the correctly rounded x / s unless s has
// a mantissa of all ones (s is a binary16 number, or 7) or the quotient is far below 1,
// where the code is 0 either way (Markstein's theorem).
constexpr int kAppendRows = 2;

__device__ __forceinline__ float quotient(float x, float s, float r)
{
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
}

// Largest of the block's 8 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x)
{
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
    return x > y ? x : y;
}

__device__ __forceinline__ void quantize4(f4 x, uint16_t &codes, uint16_t &scale)
{
    // magnitudes as whole numbers: what is not finite is the largest
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float y = x[j];
        const uint32_t m = __builtin_bit_cast(uint32_t, y) & 0x7FFFFFFFu;
        top = m > top ? m : top;
    }
    top = max_dpp<0xB1>(top);                            // quad_perm 1 0 3 2
    top = max_dpp<0x4E>(top);                            // quad_perm 2 3 0 1
    top = max_dpp<0x141>(top);                           // row_half_mirror: the other quad of 8
    const float amax = __builtin_bit_cast(float, top);
    float s32 = quotient(amax, 7.0f, 1.0f / 7.0f);
    asm("" : "+v"(s32));                                 // rounded to fp32 first, not at once to binary16
    const _Float16 s16 = (_Float16)s32;
    const float sf = (float)s16, r = 1.0f / sf;
    scale = __builtin_bit_cast(uint16_t, s16);
    // rounded by adding 1.5 2^23, which leaves the code in the lowest bits
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float q = __builtin_amdgcn_fmed3f(quotient(x[j], sf, r), -8.0f, 7.0f) + 12582912.0f;
        c[j] = __builtin_bit_cast(uint32_t, q);
    }
    const uint32_t lo = (c[0] & 0xFu) | (c[1] << 4 & ~0xFu), hi = (c[2] & 0xFu) | (c[3] << 4 & ~0xFu);
    const bool bad = !(amax <= 3.4028235e38f) || !(sf <= 65504.0f);
    codes = bad || sf == 0.0f ? 0 : (uint16_t)((lo & 0xFFu) | (hi << 8 & ~0xFFu));
    if (bad) scale = 0x7E00;
}

// by_heads, shift: a row number below 2^27 divided by the heads is the upper half of its
// product with by_heads = ceil(2^(32 + shift) / heads), shifted (heads <= 2^(shift + 1) keeps by_heads
// within 32 bits and what it is too large by below 2^(shift + 5)).
// SLOTS: the rows' places in the cache are given, one number a token.
template <int D, bool SLOTS>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, uint32_t by_heads, int shift)
{
    constexpr int kLanes = D / 4, kRows = 256 / kLanes;  // lanes of a row, rows of a workgroup at a time
    const uint32_t H = a.cache.kv_heads, rows = (uint32_t)(a.T * H);
    const int c = threadIdx.x % kLanes;                  // 4-value group within the row
    f4 k[kAppendRows], v[kAppendRows];
    int64_t dst[kAppendRows];                            // cache row
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
        const uint32_t row = (blockIdx.x * kAppendRows + i) * kRows + threadIdx.x / kLanes, t = by_heads ? __umulhi(row, by_heads) >> shift : row, h = row - t * H;
        k[i] = v[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        if (row < rows) {
            k[i] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(a.k + t * a.k_stride + h * D + c * 4));
            v[i] = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(a.v + t * a.v_stride + h * D + c * 4));
        }
    }
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
        const uint32_t row = (blockIdx.x * kAppendRows + i) * kRows + threadIdx.x / kLanes, t = by_heads ? __umulhi(row, by_heads) >> shift : row, h = row - t * H;
        dst[i] = -1;
        if (SLOTS && row < rows) {
            const int64_t slot = a.slots[t];
            if (slot >= 0 && slot < a.cache.n_pages * WQ_KV_PAGE)
                dst[i] = (slot / WQ_KV_PAGE * H + h) * WQ_KV_PAGE + slot % WQ_KV_PAGE;
        } else if (row < rows) {
            const int b = seq_of_token(a.cu, a.B, (int)t);
            const SeqRange r = seq_range(a.cu, (int)a.T, b);
            if ((int)t >= r.begin && (int)t < r.end) {
                const int64_t pos = (a.start ? (int64_t)a.start[b] : 0) + ((int)t - r.begin);
                if (pos >= 0 && pos < a.max_pages * WQ_KV_PAGE) {
                    const int64_t page = a.table[(int64_t)b * a.max_pages + pos / WQ_KV_PAGE];
                    if (page >= 0 && page < a.cache.n_pages) dst[i] = (page * H + h) * WQ_KV_PAGE + pos % WQ_KV_PAGE;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
        uint16_t kc, ks, vc, vs;
        quantize4(k[i], kc, ks);
        quantize4(v[i], vc, vs);
        if (dst[i] < 0) continue;
        reinterpret_cast<uint16_t *>(a.cache.kq)[dst[i] * kLanes + c] = kc;      // D / 2 bytes a row, 2 bytes a thread
        reinterpret_cast<uint16_t *>(a.cache.vq)[dst[i] * kLanes + c] = vc;
        if ((c & 7) == 0) {
            a.cache.ks[dst[i] * (D / 32) + (c >> 3)] = ks;
            a.cache.vs[dst[i] * (D / 32) + (c >> 3)] = vs;
        }
    }
}

// ---------------------------------------------------------------- decode attention
// (the work of a workgroup: wq_kv_decode.h)
template <int D, int H, int WPS, Form FORM>
__global__ __launch_bounds__(64 * kDecodeWaves, WPS) void decode_kernel(DecodeArgs a, int groups, int cut, float c_man, int c_exp)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[decode_lds_bytes(D, H)];
    decode_job<D, H, FORM>(a, groups, cut, c_man, c_exp, lds, blockIdx.x, threadIdx.x);
}

// Joins the pieces of a head in order; writes the rows of empty sequences and
// of lengths out of range. A thread takes 4 values of every kJoinParts-th piece and
// asks for all it needs of kJoinAhead pieces at once, since the kernel is all latency.
constexpr int kJoinParts = 8, kJoinAhead = 8;

template <int D>
__global__ __launch_bounds__(D / 4 * kJoinParts) void join_kernel(DecodeArgs a, int groups)
{
    constexpr int V = D / 4;                     // threads of a part
    __shared__ f4 red[kJoinParts][V];
    __shared__ float ml[kJoinParts][2];
    const int b = blockIdx.x / a.heads, j = blockIdx.x % a.heads, c = threadIdx.x % V, part = threadIdx.x / V;
    const Pieces at = ((const Pieces *)a.ws)[b];
    const int64_t len = a.lens[b];
    f4 *out = (f4 *)(a.out + (int64_t)b * a.out_stride + j * D) + c;
    if (len <= 0 || len > a.max_pages * kTile) {
        const float y = len == 0 ? 0.0f : __builtin_nanf("");
        if (part == 0) *out = f4{y, y, y, y};
        return;
    }
    if (at.count == 1) return;                   // written already
    const int kv = a.cache.kv_heads, group = a.heads / kv, per_step = kv * groups, per = (group + groups - 1) / groups;
    const int kh = j / group, hg = j % group / per, hh = j % group % per;
    float m = -3.0e38f, l = 0.0f;
    f4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = part; i0 < at.count; i0 += kJoinAhead * kJoinParts) {
        float pm[kJoinAhead], pl[kJoinAhead];
        f4 po[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const int i = i0 + k * kJoinParts;
            pm[k] = -3.0e38f;
            pl[k] = 0.0f;
            po[k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            if (i < at.count) {
                const float *p = partial<D>(a, (int64_t)(at.first + i) * per_step + hg * kv + kh, i == 0 ? at.slot : 0, hh);
                pm[k] = p[D];
                pl[k] = p[D + 1];
                po[k] = ((const f4 *)p)[c];
            }
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) mn = fmaxf(mn, pm[k]);
        const float by = __builtin_amdgcn_exp2f(m - mn);
        l *= by;
        o *= by;
        m = mn;
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const float f = __builtin_amdgcn_exp2f(pm[k] - m);
            l = fmaf(f, pl[k], l);
            o += f * po[k];
        }
    }
    red[part][c] = o;
    if (c == 0) {
        ml[part][0] = m;
        ml[part][1] = l;
    }
    __syncthreads();
    if (part == 0) {
        float mn = ml[0][0];
#pragma unroll
        for (int w = 1; w < kJoinParts; ++w) mn = fmaxf(mn, ml[w][0]);
        float ll = 0.0f;
        f4 oo = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kJoinParts; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml[w][0] - mn);
            ll = fmaf(f, ml[w][1], ll);
            oo += f * red[w][c];
        }
        *out = oo / ll;
    }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t stream)
{
    const int64_t rows = a.T * a.cache.kv_heads, each = kAppendRows * 256 / (a.cache.head_dim / 4);
    const unsigned grid = (unsigned)((rows + each - 1) / each);
    int shift = 0;
    while ((2 << shift) < a.cache.kv_heads) ++shift;
    const uint64_t H = a.cache.kv_heads, by = (((uint64_t)1 << (32 + shift)) + H - 1) / H;
    // one head: 2^32 does not fit, the quotient is the row
    const uint32_t by_heads = H == 1 ? 0 : (uint32_t)by;
    if (a.slots) {
        if (a.cache.head_dim == 128) append_kernel<128, true><<<grid, 256, 0, stream>>>(a, by_heads, shift);
        else append_kernel<64, true><<<grid, 256, 0, stream>>>(a, by_heads, shift);
    } else {
        if (a.cache.head_dim == 128) append_kernel<128, false><<<grid, 256, 0, stream>>>(a, by_heads, shift);
        else append_kernel<64, false><<<grid, 256, 0, stream>>>(a, by_heads, shift);
    }
    return hipGetLastError();
}

uint64_t decode_ws_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    return decode_window_ws_bytes(B, heads, kv_heads, head_dim, max_pages, 0, 0);
}

uint64_t decode_window_ws_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages, int64_t window, int64_t sinks)
{
    const int per_step = (int)kv_heads * head_groups((int)heads, (int)kv_heads);
    return cut_call(B, per_step, max_pages, window, sinks) ? pieces_bytes(per_step, runs_per_head(per_step), head_dim) : 0;
}

hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t stream)
{
    const int kv = a.cache.kv_heads, group = a.heads / kv, groups = head_groups(a.heads, kv), per_step = kv * groups;
    const int cut = cut_call(a.B, per_step, a.max_pages, a.window, a.sinks) ? runs_per_head(per_step) : 0;
    const unsigned grid = (unsigned)((int64_t)per_step * (cut ? cut : a.B));
    int c_exp = 0;
    const double c = frexp((double)a.scale * 1.4426950408889634, &c_exp);      // softmax in powers of two
    const float c_man = (float)(2.0 * c);
    const int per = (group + groups - 1) / groups;
    constexpr int T = 64 * kDecodeWaves;
    const auto start = [&](auto kernel) { kernel<<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1); };
    const auto pick = [&](auto form) {
        constexpr Form F = decltype(form)::value;
        if (a.cache.head_dim == 128) {
            if (per <= 2) start(decode_kernel<128, 2, 2, F>);
            else if (per <= 4) start(decode_kernel<128, 4, 2, F>);
            else start(decode_kernel<128, 8, 2, F>);
        } else {
            if (per <= 4) start(decode_kernel<64, 4, 3, F>);
            else start(decode_kernel<64, 8, 3, F>);
        }
    };
    // (a window as long as the table hides nothing)
    if (a.window > 0 && a.window < a.max_pages * kTile) pick(std::integral_constant<Form, Form::window>{});
    else pick(std::integral_constant<Form, Form::plain>{});
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !cut) return e;
    const unsigned jobs = (unsigned)(a.B * a.heads);
    if (a.cache.head_dim == 128) join_kernel<128><<<jobs, 128 / 4 * kJoinParts, 0, stream>>>(a, groups);
    else join_kernel<64><<<jobs, 64 / 4 * kJoinParts, 0, stream>>>(a, groups);
    return hipGetLastError();
}

}  // namespace wq
