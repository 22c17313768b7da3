// wq_kv.hip -- the int4 key/value cache: append, and attention of single tokens.
#include "wq_internal.h"
#include "wq_device.h"
#include "wq_seq.h"

#include <math.h>

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
//
// One query token per sequence: out = sum_u p_u v_u / sum_u p_u over the cached
// rows, p_u = exp2(x_u - m), x_u = scale log2(e) <q, k_u>. HBM-bound: 9 / 8
// bytes a value pair of k and v, read once for all query heads that share it.
//
// A wavefront walks tiles of 64 tokens (a page of one key/value head), copied
// into its own LDS by direct-to-LDS loads. All arithmetic on codes is on the
// matrix cores, 16 x 16 x 32, whose 32 is one quantization block or 32 tokens,
// with the query heads' side split into two binary16 parts (22 bits):
//   scores   A = q, 16 rows (part, head of H, block of BC), zero outside the
//     row's block, B = k codes (one block x 16 tokens): a chain of BC products
//     gives BC blocks' partial sums side by side. A lane holds one token and the
//     BC blocks of H / 2 heads, scales and adds them, and exchanges the part
//     with the lane 32 away: a score per lane, none computed twice over.
//   output   A = weights p_u s_u, rows as above (each block of the row's BC has
//     its own scale), 32 tokens; B = v codes. Every lane makes its token's 4 rows
//     and they change sides through 2 KiB of LDS (ds_read_b64_tr_b16). Only the
//     columns of a row's own block are used at the end.
// BC H = 8: few heads put blocks side by side, so that a lane has more to do per
// token; more heads take that room.
//
// Codes become exact binary16 values by the mantissa of 1024: (1024 + 8 + c) -
// 1032. (Offset codes as subnormals, (c + 8) 2^-24 with the offset's share
// taken off the sum, need 5 operations for 8 codes instead of 9, but the matrix
// cores' sums of the larger products cost three bits: error 2.4e-6 against
// 4e-7.) v is wanted with tokens along the lane's registers:
// ds_read_b64_tr_b4 transposes 16 x 16 codes on the way.
//
// The weights carry 2^kWeightBits over the largest value scale seen (v_exp), so
// both binary16 parts stay normal; m moves only when a score passes it by
// kSlack.
//
// A tile goes from LDS to registers at once and the copies of the next tile
// into the same LDS go out before anything is computed, so that copies are
// under way all the time and 12 wavefronts of 11 KiB share a compute unit's LDS.
//
// Lengths are device data, so the split is made on the device: every workgroup
// adds up the lengths, cuts the sequences into equal chunks that fill the card
// once and finds its own; a second kernel joins the chunks in order.
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef int i2 __attribute__((ext_vector_type(2)));

constexpr int kDecodeWaves = 4;
constexpr int kTile = WQ_KV_PAGE;
constexpr int kDecodeStep = kDecodeWaves * kTile;      // chunks are multiples of this many tokens
constexpr int kMaxGroup = 8;                           // query heads of a workgroup
constexpr int kWeightBits = 12;
constexpr float kSlack = 3.0f;
constexpr int kMinScaleExp = -24;                      // 2^-24 is binary16's smallest

__device__ __forceinline__ f4 mfma16(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// x plus the value 32 lanes away.
__device__ __forceinline__ float add_halves(float x)
{
    const uint32_t v = __builtin_bit_cast(uint32_t, x);
    const auto both = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const uint32_t lo = both[0], hi = both[1];       // (a bit cast of a vector's element takes element 0)
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// Transposed LDS read of four tokens of 16 rows each, 512 bytes apart, with its
// wait. (As builtins these make the compiler wait for every direct-to-LDS copy
// under way, also those into other buffers.)
__device__ __forceinline__ void read_rows(const uint8_t *p, h4 &a, h4 &b, h4 &c, h4 &d)
{
    const uint32_t at = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)p;
    asm volatile("ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:512\n\t"
                 "ds_read_b64_tr_b16 %2, %4 offset:1024\n\tds_read_b64_tr_b16 %3, %4 offset:1536\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d) : "v"(at) : "memory");
}

// 8 codes of a dword, in the order of nibbles 0 4 1 5 2 6 3 7.
__device__ __forceinline__ int nibble_of(int e) { return (e >> 1) + 4 * (e & 1); }

// The codes of a dword as exact binary16 values.
__device__ __forceinline__ h8 codes8(uint32_t x)
{
    const h2 off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const h2 off16 = {(_Float16)-72.0f, (_Float16)-72.0f}, inv16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t y = x >> 8;
    const h2 a = __builtin_bit_cast(h2, (x & 0x000F000Fu) ^ 0x64086408u) + off;
    const h2 b = __builtin_elementwise_fma(__builtin_bit_cast(h2, (x & 0x00F000F0u) ^ 0x64806480u), inv16, off16);
    const h2 c = __builtin_bit_cast(h2, (y & 0x000F000Fu) ^ 0x64086408u) + off;
    const h2 d = __builtin_elementwise_fma(__builtin_bit_cast(h2, (y & 0x00F000F0u) ^ 0x64806480u), inv16, off16);
    return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// ---- how sequences are cut (host: decode_ws_bytes and the launch sizes agree with it)
// A step is 4 tiles, one per wavefront. Sequences are cut into chunks of equally
// many steps, as few as give about kFill workgroups in all (4 on each of 256
// compute units). Cutting needs every workgroup to look at all lengths, so it
// is left out for many sequences (they fill the card by themselves) and where
// no sequence can be longer than a step.
constexpr int kFill = 1024;
constexpr int kCutMaxSeqs = 512;

__host__ __device__ inline int head_groups(int heads, int kv_heads) { return (heads / kv_heads + kMaxGroup - 1) / kMaxGroup; }
__host__ __device__ inline bool cut_sequences(int64_t B, int64_t max_pages)
{
    return B <= kCutMaxSeqs && max_pages > kDecodeWaves;
}
// Most chunks times workgroups per chunk: sum ceil(n_b / c) <= sum n_b / c + B, c >= sum n_b per / kFill.
__host__ __device__ inline int64_t max_items(int64_t B, int64_t per_chunk) { return kFill + B * per_chunk; }

struct Cut {
    int b;               // the sequence, -1: none
    int first;           // number of its first chunk among all
    int chunks;          // of the sequence
    int64_t steps;       // of a chunk, below 2^31
};

__device__ __forceinline__ int steps_of(const DecodeArgs &a, int b)
{
    const int64_t len = b < a.B ? a.lens[b] : 0;
    return len < 0 || len > a.max_pages * kTile ? 0 : (int)((len + kDecodeStep - 1) / kDecodeStep);
}

// The cut, and the sequence that holds chunk `chunk` (or the one of number seq
// when seq >= 0). A whole wavefront calls it.
__device__ __forceinline__ Cut find_cut(const DecodeArgs &a, int per_chunk, int64_t chunk, int seq)
{
    const int lane = threadIdx.x & 63;
    int64_t total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        int n = steps_of(a, b0 + lane);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
        total += n;
    }
    const int64_t steps = total * per_chunk <= kFill ? 1 : (total * per_chunk + kFill - 1) / kFill;
    int before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int n = steps_of(a, b0 + lane);
        const int mine = (int)((n + steps - 1) / steps);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(upto, o);
            if (lane >= o) upto += x;
        }
        const int first = before + upto - mine;
        const bool hit = seq >= 0 ? b0 + lane == seq : chunk >= first && chunk < first + mine;
        const uint64_t who = __ballot(hit);
        if (who) {
            const int l = __ffsll((unsigned long long)who) - 1;
            return {b0 + l, __shfl(first, l), __shfl(mine, l), steps};
        }
        before += __shfl(upto, 63);
    }
    return {-1, 0, 0, steps};
}

constexpr int kPartialExtra = 2;             // a partial result: D values, then m and l

template <int D, int H, int WPS>
__global__ __launch_bounds__(64 * kDecodeWaves, WPS) void decode_kernel(DecodeArgs a, int groups, bool cut, float c_man, int c_exp)
{
    constexpr int NB = D / 32, BC = 8 / H, R = NB / BC;          // blocks, of them side by side, chains
    constexpr int HL = H / 2;                                    // heads of a lane's scores
    static_assert(BC * H == 8 && BC * R == NB, "rows");
    constexpr int kCodeBytes = kTile * D / 2, kScaleBytes = kTile * NB * 2, kHalf = kCodeBytes + kScaleBytes;
    constexpr int kWeightBytes = kTile * 32;
    static_assert(2 * kHalf >= 16 * D * 4, "the wave's result fits its buffers");
    typedef _Float16 hb __attribute__((ext_vector_type(NB)));    // a token's scales
    __shared__ __attribute__((aligned(16))) uint8_t lds[kDecodeWaves][2 * kHalf + kWeightBytes];
    __shared__ float state[kDecodeWaves][H][2];
    const int kv = a.cache.kv_heads, group = a.heads / kv, per_chunk = kv * groups;
    const int kh = blockIdx.x % kv, hg = blockIdx.x / kv % groups;
    int b = blockIdx.x / per_chunk, chunks = 1;
    int64_t t0 = 0, span = a.max_pages * kTile;
    if (cut) {
        const Cut at = find_cut(a, per_chunk, b, -1);
        const int seq = __builtin_amdgcn_readfirstlane(at.b);
        if (seq < 0) return;
        span = (int64_t)__builtin_amdgcn_readfirstlane((int)at.steps) * kDecodeStep;
        t0 = (b - __builtin_amdgcn_readfirstlane(at.first)) * span;
        b = seq;
        chunks = __builtin_amdgcn_readfirstlane(at.chunks);
    }
    const int per = (group + groups - 1) / groups;               // heads of this workgroup: per or fewer
    const int head0 = kh * group + hg * per, heads = group - hg * per < per ? group - hg * per : per;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t len = a.lens[b];
    if (len <= 0 || len > a.max_pages * kTile) {                 // (not reached where sequences are cut)
        for (int i = tid; i < heads * D; i += 64 * kDecodeWaves)
            a.out[(int64_t)b * a.out_stride + head0 * D + i] = len == 0 ? 0.0f : __builtin_nanf("");
        return;
    }
    const int64_t end = len < t0 + span ? len : t0 + span;
    const int tile0 = (int)(t0 / kTile) + wave, tile_end = (int)((end + kTile - 1) / kTile);
    // (constant address space: scalar loads, which wait for nothing else)
    const __attribute__((address_space(4))) int32_t *pages =
        (const __attribute__((address_space(4))) int32_t *)(uintptr_t)(a.table + (int64_t)b * a.max_pages);
    const int c = lane & 15, g = lane >> 4;

    // copies of a tile: 16-byte pieces (a block of a token each), swizzled by token so that the reads below
    // take 64 banks
    const int64_t rows = (int64_t)kv * kTile;
    bool bad = false;
    auto row_of = [&](int page) -> int64_t {
        if (page < 0 || page >= a.cache.n_pages) {
            bad = true;
            page = 0;
        }
        return (int64_t)page * rows + (int64_t)kh * kTile;
    };
    auto copy = [&](const void *codes, const uint16_t *scales, int64_t row, uint8_t *dst, bool values) {
        const uint8_t *src = (const uint8_t *)codes + row * (D / 2);
#pragma unroll
        for (int i = 0; i < kCodeBytes / 1024; ++i) {
            const int p = i * 64 + lane, t = p / NB, s = p % NB;
            const int blk = s ^ ((t >> (values ? 4 : D == 128 ? 2 : 3)) & (NB - 1));
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(src + t * (D / 2) + blk * 16),
                                             (__attribute__((address_space(3))) void *)(dst + i * 1024), 16, 0, kNonTemporal);
        }
        if (lane < kScaleBytes / 16)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)((const uint8_t *)(scales + row * NB) + lane * 16),
                                             (__attribute__((address_space(3))) void *)(dst + kCodeBytes), 16, 0, kNonTemporal);
    };
    uint8_t *kbuf = lds[wave], *vbuf = kbuf + kHalf, *pbuf = vbuf + kHalf;
    const bool any_page = a.cache.n_pages > 0;
    int page2 = 0;                                               // page of the tile after the next
    if (tile0 < tile_end) {
        const int64_t row = row_of(pages[tile0]);
        if (tile0 + kDecodeWaves < tile_end) page2 = pages[tile0 + kDecodeWaves];
        if (any_page) {
            copy(a.cache.kq, a.cache.ks, row, kbuf, false);
            copy(a.cache.vq, a.cache.vs, row, vbuf, true);
        }
    }

    // the query: row n = c of the operand is part c / 8 of head (c / 4 % 2) HL + c % 4 / BC, and of blocks
    // r BC + c % BC
    h8 q[NB];
    float f[HL];                                                 // scores in powers of two = sums times this
    {
        const int part = c >> 3, bc = c & (BC - 1), h = ((c >> 2) & 1) * HL + (c & 3) / BC;
        const bool live = h < heads;
        const float *src = a.q + (int64_t)b * a.q_stride + (head0 + (live ? h : 0)) * D;
        float x[R][8], top = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[r][e] = live ? src[32 * (r * BC + bc) + 8 * g + nibble_of(e)] : 0.0f;
                const float y = fabsf(x[r][e]);
                if (y <= 3.4028235e38f) top = fmaxf(top, y);
            }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1)
            if (o < BC || o >= 16) top = fmaxf(top, __shfl_xor(top, o));
        const int e2 = top > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
        const float fe = ldexpf(1.0f, c_exp - e2 > 127 ? 127 : c_exp - e2);
#pragma unroll
        for (int i = 0; i < HL; ++i) f[i] = __shfl(fe, 4 * (g & 1) + i * BC);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y = ldexpf(x[r][e], e2) * c_man;
                asm("" : "+v"(y));                               // one rounding of y, whoever uses it
                const _Float16 hi = (_Float16)y;
                v[e] = part ? (_Float16)(y - (float)hi) : hi;
            }
#pragma unroll
            for (int i = 0; i < BC; ++i) q[r * BC + i] = i == bc ? v : h8{};
        }
    }

    // From here on a lane is token 16 u + c of a tile, and the 4 rows 4 g + i: part g / 2, heads (g % 2) HL + i / BC
    f4 acc[D / 16];
#pragma unroll
    for (int n = 0; n < D / 16; ++n) acc[n] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m[HL], l[HL];
#pragma unroll
    for (int i = 0; i < HL; ++i) {
        m[i] = -3.0e38f;
        l[i] = 0.0f;
    }
    int v_exp = kMinScaleExp;
    const float minus = g >> 1 ? -1.0f : 0.0f;                   // this lane keeps the second part of a weight
    // Tokens of the output's operands: element e of product x is token 16 (2 x + e / 4) + 4 g + e % 4. The
    // codes' transposed read puts row c of the lanes into nibble c % 8 of dword c / 8, nibble_of(e) = c % 8.
    const int vn = c & 7, ve = vn < 4 ? 2 * vn : 2 * (vn - 4) + 1;
    const int vt = 16 * (2 * (c >> 3) + (ve >> 2)) + 4 * g + (ve & 3);
    uint8_t *const pw = pbuf + c * 32 + g * 8;                                    // weights are written by token
    uint8_t *const pr = pbuf + (4 * g + (c >> 2)) * 32 + (c & 3) * 8;             // and read by row

    for (int tile = tile0; tile < tile_end; tile += kDecodeWaves) {
        const bool more = tile + kDecodeWaves < tile_end;
        int64_t next = 0;
        if (more) next = row_of(page2);
        if (tile + 2 * kDecodeWaves < tile_end) page2 = pages[tile + 2 * kDecodeWaves];
        __builtin_amdgcn_s_waitcnt(0x0F70);                      // vmcnt(0): the tile has arrived
        asm volatile("" ::: "memory");
        uint32_t kc[4][NB];                                      // codes of the lane's tokens, 8 of each block
        hb ks[4], w[4];                                          // scales of the lane's tokens
        i2 vc[D / 16];                                           // codes of 16 tokens, one value each
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = 16 * u + c;
#pragma unroll
            for (int i = 0; i < NB; ++i)
                kc[u][i] = *(const uint32_t *)(kbuf + t * (D / 2) + (i ^ ((t >> (D == 128 ? 2 : 3)) & (NB - 1))) * 16 + g * 4);
            ks[u] = *(const hb *)(kbuf + kCodeBytes + t * NB * 2);
            w[u] = *(const hb *)(vbuf + kCodeBytes + t * NB * 2);
        }
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
            vc[n] = __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) i2 *)(
                vbuf + vt * (D / 2) + ((n >> 1) ^ ((vt >> 4) & (NB - 1))) * 16 + (n & 1) * 8));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0): read, the buffers may be filled again
        if (more && any_page) {
            copy(a.cache.kq, a.cache.ks, next, kbuf, false);
            copy(a.cache.vq, a.cache.vs, next, vbuf, true);
        }
        const int left = (int)(len - (int64_t)tile * kTile);     // tokens of the tile that count
        float x[HL][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float s[HL];
#pragma unroll
            for (int i = 0; i < HL; ++i) s[i] = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < BC; ++i) z = mfma16(q[r * BC + i], codes8(kc[u][r * BC + i]), z);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i / BC] = fmaf(z[i], (float)ks[u][r * BC + i % BC], s[i / BC]);
            }
#pragma unroll
            for (int i = 0; i < HL; ++i) x[i][u] = add_halves(s[i]);      // the other part is 32 lanes away
        }
        if (left < kTile) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (16 * u + c >= left) {
                    w[u] = hb{};
#pragma unroll
                    for (int i = 0; i < HL; ++i) x[i][u] = -__builtin_inff();
                }
        }
        hb wmax = __builtin_elementwise_max(__builtin_elementwise_max(w[0], w[1]), __builtin_elementwise_max(w[2], w[3]));
        _Float16 vtop = wmax[0];
#pragma unroll
        for (int i = 1; i < NB; ++i) vtop = __builtin_fmaxf16(vtop, wmax[i]);
        float top[HL];
        bool raise = (float)vtop > ldexpf(1.0f, v_exp);
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            top[i] = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])) * f[i];
            raise |= top[i] > m[i] + kSlack;
        }
        if (__any(raise)) {
            float vmax = (float)vtop;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, o));
            const int en = vmax > ldexpf(1.0f, v_exp) ? __builtin_amdgcn_frexp_expf(vmax) : v_exp;
#pragma unroll
            for (int i = 0; i < HL; ++i) {
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) top[i] = fmaxf(top[i], __shfl_xor(top[i], o));
                const float mn = fmaxf(m[i], top[i]);
                const float by = ldexpf(__builtin_amdgcn_exp2f(m[i] - mn), v_exp - en);
                l[i] *= by;
                m[i] = mn;
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
#pragma unroll
                    for (int k = 0; k < BC; ++k) acc[n][i * BC + k] *= by;
            }
            v_exp = en;
        }
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            const float up = (float)(kWeightBits - v_exp) - m[i];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[i][u] = __builtin_amdgcn_exp2f(fmaf(x[i][u], f[i], up));
                l[i] += x[i][u];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                h4 p;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y = x[i / BC][u] * (float)w[u][r * BC + i % BC];
                    asm("" : "+v"(y));
                    p[i] = (_Float16)fmaf(minus, (float)(_Float16)y, y);
                }
                *(h4 *)(pw + u * 512) = p;
            }
            h4 w0, w1, w2, w3;
            read_rows(pr, w0, w1, w2, w3);
            const h8 p0 = __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
            const h8 p1 = __builtin_shufflevector(w2, w3, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int n = 2 * r * BC; n < 2 * (r + 1) * BC; ++n) acc[n] = mfma16(p0, codes8((uint32_t)vc[n].x), acc[n]);
#pragma unroll
            for (int n = 2 * r * BC; n < 2 * (r + 1) * BC; ++n) acc[n] = mfma16(p1, codes8((uint32_t)vc[n].y), acc[n]);
        }
    }

    // join the waves: the 16 rows of a wave's result go through its buffers
    float *res = (float *)lds[wave];
    asm volatile("" ::: "memory");
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) res[(4 * g + i) * D + 16 * n + c] = ldexpf(acc[n][i], v_exp - kWeightBits);
#pragma unroll
    for (int i = 0; i < HL; ++i) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor(l[i], o);
        if (c == 0 && g < 2) {
            state[wave][g * HL + i][0] = m[i];
            state[wave][g * HL + i][1] = bad ? __builtin_nanf("") : ldexpf(l[i], v_exp - kWeightBits);
        }
    }
    __syncthreads();
    for (int i = tid; i < heads * D; i += 64 * kDecodeWaves) {
        const int hh = i / D, d = i % D, rw = hh / HL * 4 + hh % HL * BC + ((d / 32) & (BC - 1));
        float mm = state[0][hh][0];
#pragma unroll
        for (int w = 1; w < kDecodeWaves; ++w) mm = fmaxf(mm, state[w][hh][0]);
        float ll = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) {
            const float by = __builtin_amdgcn_exp2f(state[w][hh][0] - mm);
            const float *rs = (const float *)lds[w];
            ll = fmaf(by, state[w][hh][1], ll);
            o = fmaf(by, rs[rw * D + d] + rs[(8 + rw) * D + d], o);
        }
        if (chunks == 1) {
            a.out[(int64_t)b * a.out_stride + head0 * D + i] = o / ll;
        } else {
            float *p = (float *)a.ws + ((int64_t)blockIdx.x * kMaxGroup + hh) * (D + kPartialExtra);
            p[d] = o;
            if (d == 0) {
                p[D] = mm;
                p[D + 1] = ll;
            }
        }
    }
}

// Joins the chunks of a head in order; writes the rows of empty sequences and
// of lengths out of range. D lanes add up a quarter of the chunks each.
constexpr int kJoinParts = 4;
constexpr int kJoinBlock = 256;              // chunks whose factors are held at once

template <int D>
__global__ __launch_bounds__(D * kJoinParts) void join_kernel(DecodeArgs a, int groups)
{
    __shared__ float factor[kJoinBlock], red[kJoinParts][D + 1], top[D * kJoinParts / 64];
    const int b = blockIdx.x / a.heads, j = blockIdx.x % a.heads, d = threadIdx.x % D, part = threadIdx.x / D;
    const int64_t len = a.lens[b];
    float *out = a.out + (int64_t)b * a.out_stride + j * D + d;
    if (len <= 0 || len > a.max_pages * kTile) {
        if (part == 0) *out = len == 0 ? 0.0f : __builtin_nanf("");
        return;
    }
    const int kv = a.cache.kv_heads, group = a.heads / kv, per_chunk = kv * groups, per = (group + groups - 1) / groups;
    const Cut at = find_cut(a, per_chunk, 0, b);
    if (at.chunks == 1) return;                  // written already
    const int kh = j / group, hg = j % group / per, hh = j % group % per;
    const float *p = (const float *)a.ws +
                     (((int64_t)at.first * per_chunk + hg * kv + kh) * kMaxGroup + hh) * (D + kPartialExtra);
    const int64_t stride = (int64_t)per_chunk * kMaxGroup * (D + kPartialExtra);
    float m = -3.0e38f;
    for (int i = threadIdx.x; i < at.chunks; i += D * kJoinParts) m = fmaxf(m, p[i * stride + D]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < D * kJoinParts / 64; ++w) m = fmaxf(m, top[w]);
    float l = 0.0f, o = 0.0f;
    for (int i0 = 0; i0 < at.chunks; i0 += kJoinBlock) {
        const int n = at.chunks - i0 < kJoinBlock ? at.chunks - i0 : kJoinBlock;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += D * kJoinParts) factor[i] = __builtin_amdgcn_exp2f(p[(i0 + i) * stride + D] - m);
        __syncthreads();
        if (d == 0)
            for (int i = part; i < n; i += kJoinParts) l = fmaf(factor[i], p[(i0 + i) * stride + D + 1], l);
#pragma unroll 8
        for (int i = part; i < n; i += kJoinParts) o = fmaf(factor[i], p[(i0 + i) * stride + d], o);
    }
    red[part][d] = o;
    if (d == 0) red[part][D] = l;
    __syncthreads();
    if (part == 0) {
#pragma unroll
        for (int w = 1; w < kJoinParts; ++w) o += red[w][d];
        *out = o / (red[0][D] + red[1][D] + red[2][D] + red[3][D]);
    }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t stream)
{
    const int64_t threads = a.T * a.cache.kv_heads * (a.cache.head_dim / 4);
    const dim3 grid((unsigned)((threads + 255) / 256), 2);
    append_kernel<<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

uint64_t decode_ws_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    if (!cut_sequences(B, max_pages)) return 0;
    const int64_t per_chunk = kv_heads * head_groups((int)heads, (int)kv_heads);
    return (uint64_t)max_items(B, per_chunk) * kMaxGroup * (uint64_t)(head_dim + kPartialExtra) * 4;
}

hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t stream)
{
    const int kv = a.cache.kv_heads, group = a.heads / kv, groups = head_groups(a.heads, kv);
    const bool cut = cut_sequences(a.B, a.max_pages);
    const unsigned grid = (unsigned)(cut ? max_items(a.B, (int64_t)kv * groups) : (int64_t)a.B * kv * groups);
    int c_exp = 0;
    const double c = frexp((double)a.scale * 1.4426950408889634, &c_exp);      // softmax in powers of two
    const float c_man = (float)(2.0 * c);
    const int per = (group + groups - 1) / groups;
    constexpr int T = 64 * kDecodeWaves;
    if (a.cache.head_dim == 128) {
        if (per <= 2) decode_kernel<128, 2, 3><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
        else if (per <= 4) decode_kernel<128, 4, 3><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
        else decode_kernel<128, 8, 3><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
    } else {
        if (per <= 4) decode_kernel<64, 4, 4><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
        else decode_kernel<64, 8, 4><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !cut) return e;
    const unsigned jobs = (unsigned)(a.B * a.heads);
    if (a.cache.head_dim == 128) join_kernel<128><<<jobs, 128 * kJoinParts, 0, stream>>>(a, groups);
    else join_kernel<64><<<jobs, 64 * kJoinParts, 0, stream>>>(a, groups);
    return hipGetLastError();
}

}  // namespace wq
