// wq_kv_decode.h -- attention of single tokens over the int4 cache: the work of a
// workgroup, how it is cut, and where the pieces of a sequence are. The kernels
// around it are in wq_kv.hip, and, behind a shared prefix, in wq_shared.hip.
#pragma once

#include "wq_internal.h"
#include "wq_device.h"

#include <hip/hip_runtime.h>
#include <math.h>

namespace wq {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

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
// With a window only its tiles are walked, and those of the first tokens (Tiles); their
// pages follow from the length, so that they are asked for after it.
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

// With a window that takes at most kWindowPages pages, whole sequences that fill the card
// are even enough, and a join less (us, cut / uncut, 16/8 heads of 128, ragged: 64 sequences, window 2048
// 31.3 / 27.5; 32/8 heads 40.1 / 32.3; 4096 44.2 / 44.3; 8192 77 / 82, and 50 sequences, which do not
// fill it, of 3000 31.5 / 33.6).
constexpr int kWindowPages = 64;
inline bool cut_call(int64_t B, int per_step, int64_t max_pages, int64_t window, int64_t sinks)
{
    const int64_t pages = seen_pages(max_pages, window, sinks);
    if (window > 0 && pages < max_pages && pages <= kWindowPages && B * per_step >= kFill) return false;
    return cut_sequences(B, per_step, pages);
}

// Where a sequence's pieces are: runs first .. first + count - 1; the first one's
// piece is its run's last, slot 1, unless the run begins with it.
struct Pieces {
    int first, count, slot, pad;
};
constexpr int kSlots = 2;                    // pieces of a run that are not whole sequences: its first and its last

// The tiles of a sequence that its query sees. With a window: the last `window`
// tokens' and the first `sinks` ones'; what lies between is not walked, its pages
// are not looked at.
template <bool WIN>
struct Tiles {
    int64_t low, sink_end;                   // seen: tokens from low on, and those before sink_end
    int sinks, skip, count;                  // tiles of first tokens, tiles left out behind them, tiles in all
    __device__ __forceinline__ Tiles(const DecodeArgs &a, int64_t len) : low(0), sink_end(0), sinks(0), skip(0), count((int)((len + kTile - 1) / kTile))
    {
        if constexpr (WIN) {
            low = len > a.window ? len - a.window : 0;
            sink_end = a.sinks < low ? a.sinks : low;
            const int from = (int)(low / kTile), first = (int)((sink_end + kTile - 1) / kTile);
            sinks = first < from ? first : from;
            skip = from - sinks;
            count -= skip;
        }
    }
    __device__ __forceinline__ int tile(int v) const { return WIN && v >= sinks ? v + skip : v; }
    __device__ __forceinline__ int steps() const { return (count + kDecodeWaves - 1) / kDecodeWaves; }
};

template <bool WIN>
__device__ __forceinline__ int steps_of(const DecodeArgs &a, int b)
{
    const int64_t len = a.lens[b];
    return len < 0 || len > a.max_pages * kTile ? 0 : Tiles<WIN>(a, len).steps();
}

// A run: sequence b from its step `skip` on, `left` steps in all, those that stand
// for the changes between sequences among them.
struct Run {
    int b, skip, left;
    int span;                                // of a run
};

// A whole wavefront calls it. left <= 0: nothing.
template <bool WIN>
__device__ __forceinline__ Run find_run(const DecodeArgs &a, int run, int runs)
{
    const int lane = threadIdx.x & 63;
    const auto cost = [&](int b) {
        const int n = b < a.B ? steps_of<WIN>(a, b) : 0;
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

// Bytes of the pieces of a launch that is cut into so many runs for every kv head and group of heads.
inline uint64_t pieces_bytes(int per_step, int runs, int64_t head_dim)
{
    return kCutMaxSeqs * sizeof(Pieces) + (uint64_t)per_step * runs * kSlots * kMaxGroup * (uint64_t)(head_dim + kPartialExtra) * 4;
}

// Piece `slot` of a workgroup, head hh.
template <int D>
__device__ __forceinline__ float *partial(const DecodeArgs &a, int64_t group, int slot, int hh)
{
    return (float *)((Pieces *)a.ws + kCutMaxSeqs) + ((group * kSlots + slot) * kMaxGroup + hh) * (D + kPartialExtra);
}

// What a call asks for: all keys, those of a window, all with the maximum and sum
// of each whole sequence's weights beside its output, or parts of one sequence, a
// prefix, for the queries of a batch (its heads are the batch's rows).
enum class Form { plain, window, sums, prefix };

// The runs of pages of a prefix, from its length, which is on the device: whole
// numbers of `unit` pages.
struct PrefixRuns {
    int64_t len;
    int pages, per, count;                   // pages in all, of a run, runs
    bool bad;
};
__device__ __forceinline__ PrefixRuns prefix_runs(const int32_t *len, int64_t most_pages, int runs, int unit)
{
    PrefixRuns r;
    r.len = *len;
    r.bad = r.len < 0 || r.len > most_pages * kTile;
    if (r.bad) r.len = 0;
    r.pages = (int)((r.len + kTile - 1) / kTile);
    const int units = (r.pages + unit - 1) / unit;
    r.per = runs > 0 ? (units + runs - 1) / runs * unit : 0;
    r.count = r.per > 0 ? (r.pages + r.per - 1) / r.per : 0;
    return r;
}

// Where a run's result for a row of a key/value head is: D values, then maximum and sum.
__device__ __forceinline__ float *prefix_part(float *parts, int64_t run, int kv_heads, int kh, int64_t rows, int64_t row, int D)
{
    return parts + ((run * kv_heads + kh) * rows + row) * (D + kPartialExtra);
}

// LDS of a job: every wavefront's buffers, then the state they are joined by.
constexpr int decode_wave_bytes(int D) { return 2 * (kTile * D / 2 + kTile * D / 32 * 2) + kTile * 32; }
constexpr int decode_lds_bytes(int D, int H) { return kDecodeWaves * (decode_wave_bytes(D) + H * 8); }

// The work of kDecodeWaves wavefronts, job `job` of a launch, thread `tid` of it.
// `cut`: into how many runs the work of a kv head and group of heads is cut, 0: not.
// (Where a workgroup does two jobs at once, shared_kernel's, their wavefronts come to unequal numbers of barriers, which
// HIP leaves undefined. It is right by the instruction the barriers are on this machine: s_barrier counts arrivals of a
// workgroup's wavefronts wherever in the program they are, and waits only for those that have not ended. So the n-th
// arrivals of all eight meet, a job's four among them, a barrier more than a job needs only delays it, and a job
// that is done holds up nobody. The condition around a job is the same for whole wavefronts.)
template <int D, int H, Form FORM>
__device__ __forceinline__ void decode_job(const DecodeArgs &a, int groups, int cut, float c_man, int c_exp, uint8_t *lds, unsigned job, int tid)
{
    constexpr bool WIN = FORM == Form::window;
    constexpr int NB = D / 32, BC = 8 / H, R = NB / BC;          // blocks, of them side by side, chains
    constexpr int HL = H / 2;                                    // heads of a lane's scores
    static_assert(BC * H == 8 && BC * R == NB, "rows");
    constexpr int kCodeBytes = kTile * D / 2, kScaleBytes = kTile * NB * 2, kHalf = kCodeBytes + kScaleBytes;
    constexpr int kWaveBytes = decode_wave_bytes(D);
    static_assert(2 * kHalf >= 16 * D * 4 && kWaveBytes == 2 * kHalf + kTile * 32, "the wave's result fits its buffers");
    typedef _Float16 hb __attribute__((ext_vector_type(NB)));    // a token's scales
    float(*const state)[H][2] = reinterpret_cast<float(*)[H][2]>(lds + kDecodeWaves * kWaveBytes);
    const int kv = a.cache.kv_heads, group = a.heads / kv, per_step = kv * groups;
    const int kh = job % kv, hg = job / kv % groups, run = job / per_step;
    const int per = (group + groups - 1) / groups;               // heads of this workgroup: per or fewer
    const int head0 = kh * group + hg * per, heads = group - hg * per < per ? group - hg * per : per;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t cap = a.max_pages * kTile;
    Run at = {run, 0, 0x7FFFFFFF, 0};                            // not cut: a whole sequence
    if constexpr (FORM == Form::prefix) {
        const PrefixRuns runs = prefix_runs(a.lens, a.max_pages, cut, kDecodeWaves);
        if (run >= runs.count) return;
        at = Run{0, run * (runs.per / kDecodeWaves), runs.per / kDecodeWaves, 0};
    } else if (cut) {
        at = find_run<WIN>(a, run, cut);
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
        if constexpr (FORM == Form::prefix) {
            const int row = hg * per + (live ? h : 0), q = row / a.query_heads;
            src = a.q + q * a.q_stride + (kh * a.query_heads + (row - q * a.query_heads)) * D;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[r][e] = live ? src[32 * (r * BC + bc) + 8 * g + nibble_of(e)] : 0.0f;
    }
    // its length and its first two pages at once (a page number that is not needed may be any of the row's)
    const const_i32 *pages = (const const_i32 *)(uintptr_t)(a.table + (int64_t)b * a.max_pages);
    const int tile0 = __builtin_amdgcn_readfirstlane(at.skip) * kDecodeWaves + wave, tile1 = tile0 + kDecodeWaves;
    const int last_page = (int)a.max_pages - 1;
    int page1 = 0, page2 = 0;                                    // page2: of the tile after the next
    if constexpr (!WIN) {
        page1 = pages[tile0 < last_page ? tile0 : last_page];
        page2 = pages[tile1 < last_page ? tile1 : last_page];
    }
    const int64_t len = __builtin_amdgcn_readfirstlane(lens[b]);
    const Tiles<WIN> walk(a, len);
    if constexpr (WIN) {                                         // (which pages these are follows from the length)
        page1 = pages[walk.tile(tile0 < walk.count ? tile0 : 0)];
        page2 = pages[walk.tile(tile1 < walk.count ? tile1 : 0)];
    }
    const int all = walk.steps();                                // steps of the sequence
    const int mine = __builtin_amdgcn_readfirstlane(all - at.skip < at.left - done ? all - at.skip : at.left - done);
    const bool whole = mine == all;
    const int upto = (__builtin_amdgcn_readfirstlane(at.skip) + mine) * kDecodeWaves, tile_end = walk.count < upto ? walk.count : upto;

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
    uint8_t *kbuf = lds + wave * kWaveBytes, *vbuf = kbuf + kHalf, *pbuf = vbuf + kHalf;
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
        if (tile + 2 * kDecodeWaves < tile_end) page2 = pages[walk.tile(tile + 2 * kDecodeWaves)];
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
        const int64_t token0 = (int64_t)walk.tile(tile) * kTile;
        const int left = (int)(len - token0 < kTile ? len - token0 : kTile);      // tokens of the tile that count
        // (with a window: those from `low` on and those before `sink`)
        const int low = WIN && walk.low > token0 ? (int)(walk.low - token0) : 0, sink = WIN && walk.sink_end > token0 ? (int)(walk.sink_end - token0 < kTile ? walk.sink_end - token0 : kTile) : 0;
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
        if (left < kTile || (WIN && low > sink)) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (16 * (2 * (g >> 1) + j) + c >= left || (WIN && 16 * (2 * (g >> 1) + j) + c < low && 16 * (2 * (g >> 1) + j) + c >= sink)) {
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
                for (int i = 0; i < 4; i += 2) {
                    half2_t hi, lo;
                    split2(x[i / BC][j] * (float)w[j][r * BC + i % BC], x[(i + 1) / BC][j] * (float)w[j][r * BC + (i + 1) % BC], hi, lo);
                    p1[i] = hi.x;
                    p1[i + 1] = hi.y;
                    p2[i] = lo.x;
                    p2[i + 1] = lo.y;
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
    float *res = (float *)(lds + wave * kWaveBytes);
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
            const float *rs = (const float *)(lds + w * kWaveBytes);
            ll = fmaf(by, state[w][hh][1], ll);
            o = fmaf(by, rs[rw * D + d] + rs[(8 + rw) * D + d], o);
        }
        if constexpr (FORM == Form::prefix) {
            float *p = prefix_part((float *)a.ws, run, kv, kh, group, hg * per + hh, D);
            p[d] = o;
            if (d == 0) {
                p[D] = mm;
                p[D + 1] = ll;
            }
        } else if (whole) {
            a.out[(int64_t)b * a.out_stride + head0 * D + i] = o / ll;
            if (FORM == Form::sums && d == 0) {
                float *sums = a.sums + ((int64_t)b * a.heads + head0 + hh) * 2;
                sums[0] = mm;
                sums[1] = ll;
            }
        } else {
            float *p = partial<D>(a, job, done != 0, hh);
            p[d] = o;
            if (d == 0) {
                p[D] = mm;
                p[D + 1] = ll;
            }
        }
    }
    if (FORM == Form::prefix || !cut) return;
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

}  // namespace
}  // namespace wq
