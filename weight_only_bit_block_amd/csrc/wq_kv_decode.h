// wq_kv_decode.h -- how the attention of single tokens cuts its work, and where
// the pieces of a sequence are: what its kernels (wq_kv.hip) and the join behind a
// shared prefix (wq_shared.hip) have in common.
#pragma once

#include "wq_internal.h"

#include <hip/hip_runtime.h>

namespace wq {
namespace {

constexpr int kDecodeWaves = 4;
constexpr int kTile = WQ_KV_PAGE;
constexpr int kDecodeStep = kDecodeWaves * kTile;      // chunks are multiples of this many tokens
constexpr int kMaxGroup = 8;                           // query heads of a workgroup

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

constexpr int kPartialExtra = 4;             // a partial result: D values, then m and l, 16-byte aligned

// Piece `slot` of a workgroup, head hh.
template <int D>
__device__ __forceinline__ float *partial(const DecodeArgs &a, int64_t group, int slot, int hh)
{
    return (float *)((Pieces *)a.ws + kCutMaxSeqs) + ((group * kSlots + slot) * kMaxGroup + hh) * (D + kPartialExtra);
}

}  // namespace
}  // namespace wq
