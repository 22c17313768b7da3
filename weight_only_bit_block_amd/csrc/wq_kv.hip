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
// one tile ahead into its own LDS by direct-to-LDS loads. All arithmetic on
// codes is on the matrix cores, 16 x 16 x 32, whose 32 is one quantization
// block or 32 tokens:
//   scores   A = k codes (16 tokens x one block), B = q, 16 columns. q is split
//     into two binary16 parts; a column is (part, block of BC, head of H), zero
//     outside its block, so that one chain of BC products gives BC blocks'
//     partial sums side by side. Each lane then scales its 4 tokens by its
//     block's scale and the columns of a head are added by cross-lane moves.
//   output   A = weights p_u s_u (16 rows (part, block of BC, head of H) x 32
//     tokens): every lane forms the weight for its own block's scales and keeps its
//     own part of it, where the scores left the token; B = v codes. Only the
//     rows of a column's own block are used at the end.
// BC * H = 8: few heads put blocks side by side, so that no lane repeats
// another's scaling; more heads take that room.
//
// Codes become binary16 without conversions. k: the offset code (c + 8) as the
// low mantissa bits of a subnormal, (c + 8) 2^-24 or 16 times that (q carries
// 1/16 there), 5 operations for 8 codes; the chain starts at -8 2^-24 sum q, so
// the offset costs nothing (the matrix cores keep subnormals). v: the same
// would cancel a sum that grows with the length, so its codes are made exact
// signed ones, (1024 + 8 + c) - 1032. v is wanted with tokens along
// the lane's registers: ds_read_b64_tr_b4 transposes 16 x 16 codes on the way.
//
// The weights carry 2^kWeightBits over the largest value scale seen (v_exp), so
// both binary16 parts stay normal; m moves only when a score passes it by
// kSlack. The longest sequence decides how many workgroups share one (host),
// every workgroup takes `chunk` tokens, and a second kernel joins them.
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef int i2 __attribute__((ext_vector_type(2)));

constexpr int kDecodeWaves = 4;
constexpr int kTile = WQ_KV_PAGE;
constexpr int kDecodeStep = kDecodeWaves * kTile;      // chunks are multiples of this many tokens
constexpr int kMaxGroup = 8;                           // query heads of a workgroup
constexpr int kWeightBits = 12;
constexpr float kSlack = 3.0f;
constexpr int kMinScaleExp = -24;                      // 2^-24 is binary16's smallest

__device__ __forceinline__ f4 mfma16(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Sum over the 16 lanes' columns of one head: c = part * 8 + bc * H + h.
template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
template <int H>
__device__ __forceinline__ float add_columns(float x)
{
    x += dpp<0x128>(x);                      // row_ror:8, the other part
    if constexpr (H <= 4) x += dpp<0x124>(x);      // row_ror:4
    if constexpr (H <= 2) x += dpp<0x4E>(x);       // quad_perm 2,3,0,1
    return x;
}

// 8 codes of a dword, in the order of nibbles 0 4 1 5 2 6 3 7.
__device__ __forceinline__ int nibble_of(int e) { return (e >> 1) + 4 * (e & 1); }

// Offset codes (c + 8) 2^-24; the pairs of nibbles 1 and 3 come 16 times larger.
__device__ __forceinline__ h8 k_codes(uint32_t x)
{
    u4 r;
    const uint32_t y = x >> 8;
    r.x = (x & 0x000F000Fu) ^ 0x00080008u;
    r.y = (x & 0x00F000F0u) ^ 0x00800080u;
    r.z = (y & 0x000F000Fu) ^ 0x00080008u;
    r.w = (y & 0x00F000F0u) ^ 0x00800080u;
    return __builtin_bit_cast(h8, r);
}

// Signed codes.
__device__ __forceinline__ h8 v_codes(uint32_t x)
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

struct DecodePlan {
    int64_t chunk;           // tokens of a workgroup, multiple of kDecodeStep
    int64_t splits;          // workgroups of the longest possible sequence
};

constexpr int kPartialExtra = 2;             // a partial result: D values, then m and l

template <int D, int H>
__global__ __launch_bounds__(64 * kDecodeWaves, 2) void decode_kernel(DecodeArgs a, int64_t chunk, int splits, int groups,
                                                                      float c_man, int c_exp)
{
    constexpr int NB = D / 32, BC = 8 / H < NB ? 8 / H : NB, R = NB / BC;      // blocks, of them side by side, chains
    static_assert(BC * H <= 8 && BC * R == NB, "columns");
    constexpr int kCodeBytes = kTile * D / 2, kScaleBytes = kTile * NB * 2;
    constexpr int kBuf = 2 * kCodeBytes + 2 * kScaleBytes;
    static_assert(kBuf >= 16 * D * 4, "the wave's result fits its buffer");
    __shared__ __attribute__((aligned(16))) uint8_t lds[kDecodeWaves][2][kBuf];
    __shared__ float state[kDecodeWaves][H][2];
    const int kv = a.cache.kv_heads, group = a.heads / kv;
    int id = blockIdx.x;
    const int kh = id % kv;
    id /= kv;
    const int hg = id % groups;
    id /= groups;
    const int split = id % splits, b = id / splits;
    const int per = (group + groups - 1) / groups;               // heads of this workgroup: per or fewer
    const int head0 = kh * group + hg * per, heads = group - hg * per < per ? group - hg * per : per;
    const int64_t len = a.lens[b], cap = a.max_pages * kTile;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool bad_len = len < 0 || len > cap;
    const int64_t t0 = split * chunk;
    if (splits > 1 && (bad_len || t0 >= len)) return;            // the join knows
    if (bad_len || len == 0) {
        for (int i = tid; i < heads * D; i += 64 * kDecodeWaves)
            a.out[(int64_t)b * a.out_stride + head0 * D + i] = bad_len ? __builtin_nanf("") : 0.0f;
        return;
    }
    const int64_t end = len < t0 + chunk ? len : t0 + chunk;
    const int tile0 = (int)(t0 / kTile) + wave, tile_end = (int)((end + kTile - 1) / kTile);
    const int32_t *pages = a.table + (int64_t)b * a.max_pages;

    const int c = lane & 15, g = lane >> 4, part = c >> 3, h = c & (H - 1), bc = (c / H) & (BC - 1);
    // the query: column c holds part `part` of head h, its blocks r BC + bc
    h8 q[NB];
    float f;                                                     // scores in powers of two = sums times this
    {
        const bool live = h < heads && (c & 7) < BC * H;
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
        for (int o = H; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
        const int e2 = top > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
        const int fe = 24 + c_exp - e2;
        f = ldexpf(1.0f, fe > 127 ? 127 : fe);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y = ldexpf(x[r][e], e2) * c_man;
                asm("" : "+v"(y));                               // one rounding of y, whoever uses it
                const _Float16 hi = (_Float16)y;
                const float z = part ? y - (float)hi : (float)hi;
                v[e] = (_Float16)((nibble_of(e) & 1) ? z * 0.0625f : z);
            }
#pragma unroll
            for (int i = 0; i < BC; ++i) q[r * BC + i] = i == bc ? v : h8{};
        }
    }
    f4 start[R];                                                 // minus the codes' offset
#pragma unroll
    for (int r = 0; r < R; ++r) {
        f4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < BC; ++i) z = mfma16(k_codes(0), q[r * BC + i], z);
        start[r] = -z;
    }

    // copies of a tile: 16-byte pieces (a block of a token each), swizzled by token so that the reads below
    // take 64 banks; both kinds of scales in one instruction
    const int64_t rows = (int64_t)kv * kTile;
    bool bad = false;
    auto copy = [&](int tile, int buf) {
        int page = pages[tile];
        if (page < 0 || page >= a.cache.n_pages) {
            bad = true;
            page = 0;
            if (a.cache.n_pages == 0) return;
        }
        const int64_t row = (int64_t)page * rows + (int64_t)kh * kTile;
        uint8_t *dst = lds[wave][buf];
        const uint8_t *kq = (const uint8_t *)a.cache.kq + row * (D / 2), *vq = (const uint8_t *)a.cache.vq + row * (D / 2);
#pragma unroll
        for (int i = 0; i < kCodeBytes / 1024; ++i) {
            const int p = i * 64 + lane, t = p / NB, s = p % NB;
            const int bk = D == 128 ? s ^ ((t >> 2) & 3) : s ^ ((t >> 3) & 1);
            const int bv = s ^ ((t >> 4) & (NB - 1));
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(kq + t * (D / 2) + bk * 16),
                                             (__attribute__((address_space(3))) void *)(dst + i * 1024), 16, 0, kNonTemporal);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(vq + t * (D / 2) + bv * 16),
                                             (__attribute__((address_space(3))) void *)(dst + kCodeBytes + i * 1024), 16, 0, kNonTemporal);
        }
        constexpr int kPieces = kScaleBytes / 16;                // of each kind
        const uint8_t *sc = lane < kPieces ? (const uint8_t *)(a.cache.ks + row * NB) + lane * 16
                                           : (const uint8_t *)(a.cache.vs + row * NB) + (lane - kPieces) * 16;
        if (lane < 2 * kPieces)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)sc,
                                             (__attribute__((address_space(3))) void *)(dst + 2 * kCodeBytes), 16, 0, kNonTemporal);
    };
    constexpr int kCopies = 2 * (kCodeBytes / 1024) + 1;

    f4 acc[D / 16];
#pragma unroll
    for (int n = 0; n < D / 16; ++n) acc[n] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -3.0e38f, l = 0.0f;
    int v_exp = kMinScaleExp;
    // tokens of the transposed reads: register nibble n of dword x is token 16 (2 x + e / 4) + 4 g + e % 4,
    // nibble_of(e) = n, so that weights stay where the scores came out
    const int vn = c & 7, ve = vn < 4 ? 2 * vn : 2 * (vn - 4) + 1;
    const int vt = 16 * (2 * (c >> 3) + (ve >> 2)) + 4 * g + (ve & 3);

    if (tile0 < tile_end) copy(tile0, 0);
    int buf = 0;
    for (int tile = tile0; tile < tile_end; tile += kDecodeWaves, buf ^= 1) {
        const bool more = tile + kDecodeWaves < tile_end;
        if (more) {
            copy(tile + kDecodeWaves, buf ^ 1);
            __builtin_amdgcn_s_waitcnt(0x0F70 | kCopies);        // vmcnt(kCopies): this tile has arrived
        } else {
            __builtin_amdgcn_s_waitcnt(0x0F70);                  // vmcnt(0)
        }
        asm volatile("" ::: "memory");
        const uint8_t *base = lds[wave][buf];
        const _Float16 *ks = (const _Float16 *)(base + 2 * kCodeBytes), *vs = ks + kTile * NB;
        const int left = (int)(len - (int64_t)tile * kTile);     // tokens of the tile that count
        float x[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const int t = 16 * u + c;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f4 z = start[r];
#pragma unroll
                for (int i = 0; i < BC; ++i) {
                    const int blk = r * BC + i, sw = D == 128 ? blk ^ ((t >> 2) & 3) : blk ^ ((t >> 3) & 1);
                    z = mfma16(k_codes(*(const uint32_t *)(base + t * (D / 2) + sw * 16 + g * 4)), q[blk], z);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = fmaf(z[i], (float)ks[(16 * u + 4 * g + i) * NB + r * BC + bc], s[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * u + i] = add_columns<BC == 1 ? 8 : 8 / BC>(s[i]);
        }
        float w[R][16];                                          // value scales of this lane's blocks
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) w[r][i] = (float)vs[(16 * (i >> 2) + 4 * g + (i & 3)) * NB + r * BC + bc];
        if (left < kTile) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * (i >> 2) + 4 * g + (i & 3) >= left) {
                    x[i] = -__builtin_inff();
#pragma unroll
                    for (int r = 0; r < R; ++r) w[r][i] = 0.0f;
                }
        }
        float top = x[0], vtop = w[0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) vtop = fmaxf(vtop, w[r][i]);
        top *= f;
        if (__any(top > m + kSlack || vtop > ldexpf(1.0f, v_exp))) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) vtop = fmaxf(vtop, __shfl_xor(vtop, o));
            const float mn = fmaxf(m, top);
            const int en = vtop > ldexpf(1.0f, v_exp) ? __builtin_amdgcn_frexp_expf(vtop) : v_exp;
            const float by = ldexpf(__builtin_amdgcn_exp2f(m - mn), v_exp - en);
            l *= by;
            // the factor of row 4 g + i of the output belongs to the lanes of that column
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float rb = __shfl(by, 4 * g + i);
#pragma unroll
                for (int n = 0; n < D / 16; ++n) acc[n][i] *= rb;
            }
            m = mn;
            v_exp = en;
        }
        const float up = (float)(kWeightBits - v_exp) - m;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], f, up));
            l += x[i];
        }
        h8 wp[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float y = x[i] * w[r][i];
                asm("" : "+v"(y));
                const _Float16 hi = (_Float16)y;
                wp[r][i >> 3][i & 7] = part ? (_Float16)(y - (float)hi) : hi;
            }
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            const int blk = n >> 1, sw = blk ^ ((vt >> 4) & (NB - 1));
            const i2 v = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (__attribute__((address_space(3))) i2 *)(base + kCodeBytes + vt * (D / 2) + sw * 16 + (n & 1) * 8));
            acc[n] = mfma16(wp[blk / BC][0], v_codes((uint32_t)v.x), acc[n]);
            acc[n] = mfma16(wp[blk / BC][1], v_codes((uint32_t)v.y), acc[n]);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);                      // the reads are done: the buffer may be filled again
    }

    // join the waves: rows (part, bc, h) of a wave's result go through its buffer
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    l = ldexpf(l, v_exp - kWeightBits);
    if (bad) l = __builtin_nanf("");
    float *res = (float *)lds[wave][0];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) res[(4 * g + i) * D + 16 * n + c] = ldexpf(acc[n][i], v_exp - kWeightBits);
    if (lane < H) {
        state[wave][lane][0] = m;
        state[wave][lane][1] = l;
    }
    __syncthreads();
    for (int i = tid; i < heads * D; i += 64 * kDecodeWaves) {
        const int hh = i / D, d = i % D, row = ((d / 32) & (BC - 1)) * H + hh;
        float mm = state[0][hh][0];
#pragma unroll
        for (int w = 1; w < kDecodeWaves; ++w) mm = fmaxf(mm, state[w][hh][0]);
        float ll = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) {
            const float by = __builtin_amdgcn_exp2f(state[w][hh][0] - mm);
            const float *rw = (const float *)lds[w][0];
            ll = fmaf(by, state[w][hh][1], ll);
            o = fmaf(by, rw[row * D + d] + rw[(8 + row) * D + d], o);
        }
        if (splits == 1) {
            a.out[(int64_t)b * a.out_stride + head0 * D + i] = o / ll;
        } else {
            float *p = (float *)a.ws + (((int64_t)b * a.heads + head0 + hh) * splits + split) * (D + kPartialExtra);
            p[d] = o;
            if (d == 0) {
                p[D] = mm;
                p[D + 1] = ll;
            }
        }
    }
}

// Joins the partial results of a head's splits, in order.
template <int D>
__global__ __launch_bounds__(D) void join_kernel(DecodeArgs a, int64_t chunk, int splits)
{
    const int b = blockIdx.x / a.heads, j = blockIdx.x % a.heads, d = threadIdx.x;
    const int64_t len = a.lens[b];
    float *out = a.out + (int64_t)b * a.out_stride + j * D + d;
    if (len < 0 || len > a.max_pages * kTile || len == 0) {
        *out = len == 0 ? 0.0f : __builtin_nanf("");
        return;
    }
    const int n = (int)((len + chunk - 1) / chunk);
    const float *p = (const float *)a.ws + (int64_t)blockIdx.x * splits * (D + kPartialExtra);
    float m = -3.0e38f;
    for (int i = 0; i < n; ++i) m = fmaxf(m, p[i * (D + kPartialExtra) + D]);
    float l = 0.0f, o = 0.0f;
    for (int i = 0; i < n; ++i) {
        const float *s = p + i * (D + kPartialExtra);
        const float by = __builtin_amdgcn_exp2f(s[D] - m);
        l = fmaf(by, s[D + 1], l);
        o = fmaf(by, s[d], o);
    }
    *out = o / l;
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t stream)
{
    const int64_t threads = a.T * a.cache.kv_heads * (a.cache.head_dim / 4);
    const dim3 grid((unsigned)((threads + 255) / 256), 2);
    append_kernel<<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

namespace {

int head_groups(int64_t heads, int64_t kv_heads) { return (int)((heads / kv_heads + kMaxGroup - 1) / kMaxGroup); }

// Workgroups that the longest possible sequence is split over: enough to fill
// the card with B such sequences (2 workgroups on each of 256 compute units, two
// rounds of them to even out unequal lengths), at least kDecodeStep tokens each.
DecodePlan plan_decode(int64_t B, int64_t heads, int64_t kv_heads, int64_t max_pages)
{
    const int64_t cap = max_pages * kTile, each = B * kv_heads * head_groups(heads, kv_heads);
    int64_t want = 1024 / each;
    if (want < 1) want = 1;
    int64_t steps = (cap + kDecodeStep - 1) / kDecodeStep;
    if (steps < 1) steps = 1;
    if (want > steps) want = steps;
    DecodePlan p;
    p.chunk = (steps + want - 1) / want * kDecodeStep;
    p.splits = (steps * kDecodeStep + p.chunk - 1) / p.chunk;
    return p;
}

template <int D, int H>
void run_decode(const DecodeArgs &a, const DecodePlan &p, hipStream_t stream)
{
    const int groups = head_groups(a.heads, a.cache.kv_heads);
    int c_exp = 0;
    const double c = frexp((double)a.scale * 1.4426950408889634, &c_exp);
    const unsigned grid = (unsigned)((int64_t)a.B * a.cache.kv_heads * groups * p.splits);
    decode_kernel<D, H><<<grid, 64 * kDecodeWaves, 0, stream>>>(a, p.chunk, (int)p.splits, groups, (float)(2.0 * c), c_exp - 1);
}

}  // namespace

uint64_t decode_ws_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    const DecodePlan p = plan_decode(B, heads, kv_heads, max_pages);
    return p.splits == 1 ? 0 : (uint64_t)(B * heads * p.splits) * (uint64_t)(head_dim + kPartialExtra) * 4;
}

hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t stream)
{
    const DecodePlan p = plan_decode(a.B, a.heads, a.cache.kv_heads, a.max_pages);
    const int group = a.heads / a.cache.kv_heads;
    if (a.cache.head_dim == 128) {
        if (group <= 2) run_decode<128, 2>(a, p, stream);
        else if (group <= 4) run_decode<128, 4>(a, p, stream);
        else run_decode<128, 8>(a, p, stream);
    } else {
        if (group <= 4) run_decode<64, 4>(a, p, stream);
        else run_decode<64, 8>(a, p, stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    if (a.cache.head_dim == 128) join_kernel<128><<<(unsigned)(a.B * a.heads), 128, 0, stream>>>(a, p.chunk, (int)p.splits);
    else join_kernel<64><<<(unsigned)(a.B * a.heads), 64, 0, stream>>>(a, p.chunk, (int)p.splits);
    return hipGetLastError();
}

}  // namespace wq
