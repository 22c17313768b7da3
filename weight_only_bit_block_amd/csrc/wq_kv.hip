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
// HBM-bound: 8 D bytes read and 1.125 D written for a token and head. A row of
// D values is D / 4 lanes, 4 values each: a wavefront reads 1 KiB of consecutive
// floats, the maximum of a block goes over its 8 lanes by cross-lane moves.
// Every thread takes kAppendRows rows, keys and values, and asks for all of
// them before it looks up where they go (three dependent reads). 4096 tokens, 8
// heads of 128, calls back to back: 10.3 us, 3.7 TB/s (rows read with cached loads: 10.9;
// inputs still in the last-level cache 8.9, six sets in turn 11.1); 16384: 31, 4.9.
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
template <int D>
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
        if (row < rows) {
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
//     BC blocks of H / 2 heads, one part of each; it scales and adds them, and
//     one exchange with the lane 32 away leaves it with the whole scores of
//     two of its four tokens.
//   output   A = weights p_u s_u, rows as above (each block of the row's BC has
//     its own scale), 32 tokens; B = v codes. Every lane makes both parts of its
//     two tokens' rows, and they change sides through 2 KiB of LDS
//     (ds_read_b64_tr_b16). Only the columns of a row's own block are used at the end.
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
// under way all the time with one buffer of 11 KiB a wavefront (heads of 128;
// 8 wavefronts a compute unit, by their registers and by kFill).
//
// Lengths are device data, so the split is made on the device: the sequences'
// steps of 256 tokens (4 tiles, one per wavefront) are laid end to end and every
// workgroup takes an equal run of them, whatever sequences it meets. Going from
// one sequence to the next costs a workgroup as much as 3 steps (its length, its pages and
// the first tile one after another, the join before: 6 us), so so many stand between
// sequences (64 of 262139 in all, 4 heads each: 85 us without, 74 with). A sequence
// that lies in one run is finished there; the pieces of others go to a workspace
// and a second kernel joins them in order.
//
// 8 heads of 128: one sequence of 131072, 2 query heads each, 30 us (5.0 TB/s), joining
// them 5.9; 64 sequences of 262139 in all, 4 query heads each, 63 us (4.8 TB/s, bound by the
// vector instructions that make weights of scores and numbers of codes), joining 4.8.
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

// Sums over the two lanes 32 apart: of x for the lower one, of y for the upper.
__device__ __forceinline__ float add_halves(float x, float y)
{
    const auto both = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
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

// Binary16 bits in the order of their magnitudes, the sign shifted out; infinities and NaNs wrap round to below zero.
constexpr uint32_t kRankZero = 0x800;
template <typename V>
__device__ __forceinline__ V scale_rank(V bits)
{
    return bits * (uint16_t)2 + (uint16_t)kRankZero;
}

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

// ---- how the work is cut
// kFill workgroups in all, 2 on each of 256 compute units; for every kv head and
// group of query heads equally many. Finding its place makes every workgroup look
// at all lengths, and the pieces cost a second kernel, so thousands of sequences
// are not cut, one workgroup each, and neither are short ones: tables of up to 16 pages, or 32
// where there are kFill / 2 workgroups without (us, uncut / cut, 8 kv heads of 128, 2 query
// heads each: 1 x 500 tokens 8.1 / 10.8, 1 x 1000 10.9 / 10.9, 1 x 2040 17.0 / 11.1, 16 x 1500
// 15.7 / 16.9, 32 x 777 12.7 / 17.6, 32 x 2040 20.4 / 23.7; 520 x 300 and one of 65536
// 365 / 107, 1024 x 2560 497 / 526, 2048 ragged of 500 in the mean 359 / 350, 4096 of 300
// 527 / 555). The limits do not follow all of these: batches of 16 to 31 sequences of 17 to 32
// pages are cut and would be faster without (16 x 1100 13.4 / 15.5, 16 x 1500 15.3 / 17.9, 31 x 2040
// 19.3 / 24.1; 8 x 2040 18.1 / 15.6). It is the table's width that decides, since the lengths are on the
// device: short sequences in a table made for long ones are cut (1 x 300 7.6 us, 10.4 in a
// table of 256 pages; 32 x 777 12.4, 18.3; 64 x 1000 19.2, 20.5).
constexpr int kFill = 512;
constexpr int kCutMaxSeqs = 2048;
constexpr int kShortPages = 16;
constexpr int kChangeSteps = 3;              // 2 and 4 measure the same

__host__ __device__ inline int head_groups(int heads, int kv_heads) { return (heads / kv_heads + kMaxGroup - 1) / kMaxGroup; }
__host__ __device__ inline bool cut_sequences(int64_t B, int per_step, int64_t max_pages)
{
    return B <= kCutMaxSeqs && max_pages > (B * per_step >= kFill / 2 ? 2 * kShortPages : kShortPages);
}
__host__ __device__ inline int runs_per_head(int per_step) { return per_step < kFill ? kFill / per_step : 1; }

// Where a sequence's pieces are: runs first .. first + count - 1; the first one's
// piece is its run's last, slot 1, unless the run begins with it.
struct Pieces {
    int first, count, slot, pad;
};
constexpr int kSlots = 2;                    // pieces of a run that are not whole sequences: its first and its last

__device__ __forceinline__ int steps_of(const DecodeArgs &a, int b)
{
    const int64_t len = a.lens[b];
    return len < 0 || len > a.max_pages * kTile ? 0 : (int)((len + kDecodeStep - 1) / kDecodeStep);
}

// A run: sequence b from its step `skip` on, `left` steps in all, those that stand
// for the changes between sequences among them.
struct Run {
    int b, skip, left;
    int span;                                // of a run
};

// A whole wavefront calls it. left <= 0: nothing.
__device__ __forceinline__ Run find_run(const DecodeArgs &a, int run, int runs)
{
    const int lane = threadIdx.x & 63;
    const auto cost = [&](int b) {
        const int n = b < a.B ? steps_of(a, b) : 0;
        return n > 0 ? n + kChangeSteps : 0;
    };
    const auto scan = [&](int n) {           // sum of the lanes up to this one
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(n, o);
            if (lane >= o) n += x;
        }
        return n;
    };
    const int head = cost(lane), head_upto = scan(head);         // the first 64 sequences, often all
    int64_t total = __shfl(head_upto, 63);
    for (int b0 = 64; b0 < a.B; b0 += 64) {
        int n = cost(b0 + lane);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
        total += n;
    }
    // (no change before the first sequence)
    const int64_t span = (total - kChangeSteps + runs - 1) / runs, from = kChangeSteps + run * span;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B && from < total; b0 += 64) {
        const int n = b0 ? cost(b0 + lane) : head, upto = b0 ? scan(n) : head_upto;
        const int64_t first = before + upto - n;
        const uint64_t who = __ballot(from >= first && from < first + n);
        if (who) {
            const int l = __ffsll((unsigned long long)who) - 1;
            const int at = __builtin_amdgcn_readfirstlane(__shfl((int)(from - first), l)) - kChangeSteps;      // < 0: in the change
            const int left = __builtin_amdgcn_readfirstlane((int)(total - from < span ? total - from : span));
            return {__builtin_amdgcn_readfirstlane(b0 + l), at < 0 ? 0 : at, at < 0 ? left + at : left,
                    __builtin_amdgcn_readfirstlane((int)span)};
        }
        before += __shfl(upto, 63);
    }
    return {0, 0, 0, 0};
}

constexpr int kPartialExtra = 4;             // a partial result: D values, then m and l, 16-byte aligned

// Piece `slot` of a workgroup, head hh.
template <int D>
__device__ __forceinline__ float *partial(const DecodeArgs &a, int64_t group, int slot, int hh)
{
    return (float *)((Pieces *)a.ws + kCutMaxSeqs) + ((group * kSlots + slot) * kMaxGroup + hh) * (D + kPartialExtra);
}

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
    const int kv = a.cache.kv_heads, group = a.heads / kv, per_step = kv * groups;
    const int kh = blockIdx.x % kv, hg = blockIdx.x / kv % groups, run = blockIdx.x / per_step;
    const int per = (group + groups - 1) / groups;               // heads of this workgroup: per or fewer
    const int head0 = kh * group + hg * per, heads = group - hg * per < per ? group - hg * per : per;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t cap = a.max_pages * kTile;
    Run at = {run, 0, 0x7FFFFFFF, 0};                            // not cut: a whole sequence
    if (cut) {
        at = find_run(a, run, runs_per_head(per_step));
        if (at.left <= 0) return;
    } else if (a.lens[run] <= 0 || a.lens[run] > cap) {
        for (int i = tid; i < heads * D; i += 64 * kDecodeWaves)
            a.out[(int64_t)run * a.out_stride + head0 * D + i] = a.lens[run] == 0 ? 0.0f : __builtin_nanf("");
        return;
    }
    // (constant address space: scalar loads, which wait for nothing else)
    typedef __attribute__((address_space(4))) int32_t const_i32;
    const const_i32 *lens = (const const_i32 *)(uintptr_t)a.lens;
    int done = 0;                                                // steps of the run that are finished
next_sequence:
    // (one value for the whole wavefront: said so, for the compiler's loops and descriptors)
    const int b = __builtin_amdgcn_readfirstlane(at.b);
    const int c = lane & 15, g = lane >> 4;
    // the query, asked for before anything that waits: row n = c of the operand is part c / 8 of head
    // (c / 4 % 2) HL + c % 4 / BC, and of blocks r BC + c % BC
    const int part = c >> 3, bc = c & (BC - 1);
    float x[R][8];
    {
        const int h = ((c >> 2) & 1) * HL + (c & 3) / BC;
        const bool live = h < heads;
        const float *src = a.q + (int64_t)b * a.q_stride + (head0 + (live ? h : 0)) * D;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[r][e] = live ? src[32 * (r * BC + bc) + 8 * g + nibble_of(e)] : 0.0f;
    }
    // its length and its first two pages at once (a page number that is not needed may be any of the row's)
    const const_i32 *pages = (const const_i32 *)(uintptr_t)(a.table + (int64_t)b * a.max_pages);
    const int tile0 = __builtin_amdgcn_readfirstlane(at.skip) * kDecodeWaves + wave, tile1 = tile0 + kDecodeWaves;
    const int last_page = (int)a.max_pages - 1;
    const int page1 = pages[tile0 < last_page ? tile0 : last_page];
    int page2 = pages[tile1 < last_page ? tile1 : last_page];    // page of the tile after the next
    const int64_t len = __builtin_amdgcn_readfirstlane(lens[b]);
    const int all = (int)((len + kDecodeStep - 1) / kDecodeStep);      // steps of the sequence
    const int mine = __builtin_amdgcn_readfirstlane(all - at.skip < at.left - done ? all - at.skip : at.left - done);
    const bool whole = mine == all;
    const int64_t t0 = (int64_t)__builtin_amdgcn_readfirstlane(at.skip) * kDecodeStep, end = len < t0 + (int64_t)mine * kDecodeStep ? len : t0 + (int64_t)mine * kDecodeStep;
    const int tile_end = (int)((end + kTile - 1) / kTile);

    // copies of a tile: 16-byte pieces (a block of a token each), swizzled by token so that the reads below
    // take 64 banks
    const int64_t rows = (int64_t)kv * kTile;
    bool bad = false;
    auto row_of = [&](int id) -> int64_t {
        int page = __builtin_amdgcn_readfirstlane(id);
        if (page < 0 || page >= a.cache.n_pages) {
            bad = true;
            page = 0;
        }
        return (int64_t)page * rows + (int64_t)kh * kTile;
    };
    // Instruction i brings tokens (64 / NB) i + lane / NB: its swizzle of k does not depend on i, that of v
    // is block ^ i at 128 values.
    const int kat = lane / NB * (D / 2) + (lane % NB ^ (lane >> 4 & (NB - 1))) * 16;
    const int vat = lane / NB * (D / 2) + (D == 128 ? lane % NB : lane % NB ^ (lane >> 5)) * 16;
    auto copy = [&](const void *codes, const uint16_t *scales, int64_t row, uint8_t *dst, bool values) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc((const uint8_t *)codes + row * (D / 2), kCodeBytes);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(scales + row * NB, kScaleBytes);
#pragma unroll
        for (int i = 0; i < kCodeBytes / 1024; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(dst + i * 1024), 16,
                                                     values ? (D == 128 ? vat ^ i << 4 : vat) : kat, i * 1024, 0, kNonTemporal);
        // (4 bytes a lane: with 16, half of the lanes would be left out and the compiler doubles what follows)
#pragma unroll
        for (int i = 0; i < kScaleBytes / 256; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)(dst + kCodeBytes + i * 256), 4,
                                                     lane * 4, i * 256, 0, kNonTemporal);
    };
    uint8_t *kbuf = lds[wave], *vbuf = kbuf + kHalf, *pbuf = vbuf + kHalf;
    const bool any_page = a.cache.n_pages > 0;
    if (tile0 < tile_end) {
        const int64_t row = row_of(page1);
        if (any_page) {
            copy(a.cache.kq, a.cache.ks, row, kbuf, false);
            copy(a.cache.vq, a.cache.vs, row, vbuf, true);
        }
    }

    h8 q[NB];
    float f[HL];                                                 // scores in powers of two = sums times this
    {
        float top = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = fabsf(x[r][e]);
                if (y <= 3.4028235e38f) top = fmaxf(top, y);
            }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1)
            if (o < BC || o >= 16) top = fmaxf(top, __shfl_xor(top, o));
        const int e2 = top > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
        // (never 0: times a masked token's -inf that is no number. Sums are below 2^42, so such scores are as good as equal)
        const float fe = ldexpf(1.0f, c_exp - e2 > 127 ? 127 : c_exp - e2 < -126 ? -126 : c_exp - e2);
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

    // From here on a lane is tokens 16 u + c of a tile, and the 4 rows 4 g + i: part g / 2, heads (g % 2) HL + i / BC.
    // Of the whole scores it holds those of u = 2 (g / 2) + j, j < 2.
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
    uint32_t v_limit = kRankZero + 2;                            // scale_rank of 2^v_exp (past 16 bits for 2^16: never passed)
    // Tokens of the output's operands: element e of product x is token 16 (2 x + e / 4) + 4 g + e % 4. The
    // codes' transposed read puts row c of the lanes into nibble c % 8 of dword c / 8, nibble_of(e) = c % 8.
    const int vn = c & 7, ve = vn < 4 ? 2 * vn : 2 * (vn - 4) + 1;
    const int vt = 16 * (2 * (c >> 3) + (ve >> 2)) + 4 * g + (ve & 3);
    uint8_t *const pw = pbuf + (g >> 1) * 1024 + c * 32 + (g & 1) * 8;             // weights are written by token
    uint8_t *const pr = pbuf + (4 * g + (c >> 2)) * 32 + (c & 3) * 8;             // and read by row

    for (int tile = tile0; tile < tile_end; tile += kDecodeWaves) {
        const bool more = tile + kDecodeWaves < tile_end;
        int64_t next = 0;
        if (more) next = row_of(page2);
        if (tile + 2 * kDecodeWaves < tile_end) page2 = pages[tile + 2 * kDecodeWaves];
        __builtin_amdgcn_s_waitcnt(0x0F70);                      // vmcnt(0): the tile has arrived
        asm volatile("" ::: "memory");
        uint32_t kc[4][NB];                                      // codes of the lane's tokens, 8 of each block
        hb ks[4], w[2];                                          // scales of the lane's tokens
        i2 vc[D / 16];                                           // codes of 16 tokens, one value each
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = 16 * u + c;
#pragma unroll
            for (int i = 0; i < NB; ++i)
                kc[u][i] = *(const uint32_t *)(kbuf + t * (D / 2) + (i ^ ((t >> (D == 128 ? 2 : 3)) & (NB - 1))) * 16 + g * 4);
            ks[u] = *(const hb *)(kbuf + kCodeBytes + t * NB * 2);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) w[j] = *(const hb *)(vbuf + kCodeBytes + (16 * (2 * (g >> 1) + j) + c) * NB * 2);
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
        float s[4][HL], x[HL][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < HL; ++i) s[u][i] = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f4 z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < BC; ++i) z = mfma16(q[r * BC + i], codes8(kc[u][r * BC + i]), z);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[u][i / BC] = fmaf(z[i], (float)ks[u][r * BC + i % BC], s[u][i / BC]);
            }
        }
#pragma unroll
        for (int i = 0; i < HL; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) x[i][j] = add_halves(s[j][i], s[2 + j][i]);
        if (left < kTile) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (16 * (2 * (g >> 1) + j) + c >= left) {
                    w[j] = hb{};
#pragma unroll
                    for (int i = 0; i < HL; ++i) x[i][j] = -__builtin_inff();
                }
        }
        // largest magnitude of the value scales, in the order of scale_rank (those that are not finite spoil their own
        // blocks only: the others are held against the finite ones)
        typedef uint16_t ub __attribute__((ext_vector_type(NB)));
        const ub wmax = __builtin_elementwise_max(scale_rank(__builtin_bit_cast(ub, w[0])), scale_rank(__builtin_bit_cast(ub, w[1])));
        uint16_t vtop = wmax[0];
#pragma unroll
        for (int i = 1; i < NB; ++i) vtop = vtop > wmax[i] ? vtop : wmax[i];
        float top[HL];
        bool raise = vtop > v_limit;
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            top[i] = fmaxf(x[i][0], x[i][1]) * f[i];
            raise |= top[i] > m[i] + kSlack;
        }
        if (__any(raise)) {
            float vmax = vtop > kRankZero ? (float)__builtin_bit_cast(_Float16, (uint16_t)((vtop - kRankZero) >> 1)) : 0.0f;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, o));
            const int en = vmax > ldexpf(1.0f, v_exp) ? __builtin_amdgcn_frexp_expf(vmax) : v_exp;
#pragma unroll
            for (int i = 0; i < HL; ++i) {
#pragma unroll
                for (int o = 1; o < 64; o <<= 1)
                    if (o != 16) top[i] = fmaxf(top[i], __shfl_xor(top[i], o));
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
            v_limit = kRankZero + 2 * (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)ldexpf(1.0f, en));
        }
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            const float up = (float)(kWeightBits - v_exp) - m[i];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[i][j] = __builtin_amdgcn_exp2f(fmaf(x[i][j], f[i], up));
                l[i] += x[i][j];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                h4 p1, p2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y = x[i / BC][j] * (float)w[j][r * BC + i % BC];
                    asm("" : "+v"(y));                           // one rounding of y, whoever uses it
                    p1[i] = (_Float16)y;
                    p2[i] = (_Float16)(y - (float)p1[i]);
                }
                *(h4 *)(pw + j * 512) = p1;
                *(h4 *)(pw + j * 512 + 16) = p2;
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
        for (int o = 1; o < 64; o <<= 1)
            if (o != 16) l[i] += __shfl_xor(l[i], o);
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
        if (whole) {
            a.out[(int64_t)b * a.out_stride + head0 * D + i] = o / ll;
        } else {
            float *p = partial<D>(a, blockIdx.x, done != 0, hh);
            p[d] = o;
            if (d == 0) {
                p[D] = mm;
                p[D + 1] = ll;
            }
        }
    }
    if (!cut) return;
    if (at.skip == 0 && kh == 0 && hg == 0 && tid == 0) {
        // the rest of the sequence fills runs of `span` from the next run's beginning on
        const int rest = all - mine;
        Pieces *p = (Pieces *)a.ws + b;
        *p = Pieces{run, 1 + (rest + at.span - 1) / at.span, done != 0, 0};
    }
    done += mine + kChangeSteps;
    if (done >= at.left) return;
    do {
        ++at.b;
        if (at.b >= a.B) return;                                 // (not reached: `left` steps are there)
    } while (lens[at.b] <= 0 || lens[at.b] > cap);
    at.skip = 0;
    __syncthreads();                                             // the results have been read
    goto next_sequence;
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
    if (a.cache.head_dim == 128) append_kernel<128><<<grid, 256, 0, stream>>>(a, by_heads, shift);
    else append_kernel<64><<<grid, 256, 0, stream>>>(a, by_heads, shift);
    return hipGetLastError();
}

uint64_t decode_ws_bytes(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    const int per_step = (int)kv_heads * head_groups((int)heads, (int)kv_heads);
    if (!cut_sequences(B, per_step, max_pages)) return 0;
    return kCutMaxSeqs * sizeof(Pieces) +
           (uint64_t)per_step * runs_per_head(per_step) * kSlots * kMaxGroup * (uint64_t)(head_dim + kPartialExtra) * 4;
}

hipError_t launch_attn_decode(const DecodeArgs &a, hipStream_t stream)
{
    const int kv = a.cache.kv_heads, group = a.heads / kv, groups = head_groups(a.heads, kv), per_step = kv * groups;
    const bool cut = cut_sequences(a.B, per_step, a.max_pages);
    const unsigned grid = (unsigned)((int64_t)per_step * (cut ? runs_per_head(per_step) : a.B));
    int c_exp = 0;
    const double c = frexp((double)a.scale * 1.4426950408889634, &c_exp);      // softmax in powers of two
    const float c_man = (float)(2.0 * c);
    const int per = (group + groups - 1) / groups;
    constexpr int T = 64 * kDecodeWaves;
    if (a.cache.head_dim == 128) {
        if (per <= 2) decode_kernel<128, 2, 2><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
        else if (per <= 4) decode_kernel<128, 4, 2><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
        else decode_kernel<128, 8, 2><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
    } else {
        if (per <= 4) decode_kernel<64, 4, 3><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
        else decode_kernel<64, 8, 3><<<grid, T, 0, stream>>>(a, groups, cut, c_man, c_exp - 1);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !cut) return e;
    const unsigned jobs = (unsigned)(a.B * a.heads);
    if (a.cache.head_dim == 128) join_kernel<128><<<jobs, 128 / 4 * kJoinParts, 0, stream>>>(a, groups);
    else join_kernel<64><<<jobs, 64 / 4 * kJoinParts, 0, stream>>>(a, groups);
    return hipGetLastError();
}

}  // namespace wq
