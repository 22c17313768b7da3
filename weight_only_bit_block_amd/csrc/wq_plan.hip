// wq_plan.hip -- the plan of a serving step from request lengths: token offsets,
// lengths, positions, pages for the new tokens, and their places in the cache.
//
// Bound by latency: a few bytes a token (64 requests of one token 4.5 us, 24 of
// 65521 tokens in all 5.1). One launch, whatever the sizes: every workgroup adds up
// all requests' tokens and pages (kChunk requests at a time, in LDS), and takes its
// share of the tokens, of the new pages and of the requests. Nothing that one
// workgroup writes is read by another: a new token's page comes from the list of free
// ones where it is new, from the table where it was there.
#include "wq_internal.h"

namespace wq {
namespace {

constexpr int kThreads = 256, kEach = 4, kChunk = kThreads * kEach;
constexpr int64_t kMost = 0x7FFFFFFF;

struct Request {
    int fresh, start, have, grow;            // new tokens, tokens before, pages before, new pages
    int len;                                 // -1: not a valid request, which gets nothing
};

__device__ __forceinline__ int pages_of(int64_t tokens, int64_t most)
{
    const int64_t n = (tokens + WQ_KV_PAGE - 1) / WQ_KV_PAGE;
    return (int)(n < most ? n : most);
}

__device__ __forceinline__ Request request(const PlanArgs &a, int64_t b)
{
    if (b >= a.B) return {0, 0, 0, 0, 0};
    const int64_t n = a.fresh[b], s = a.start ? a.start[b] : 0;
    if (n < 0 || s < 0 || n + s > kMost) return {0, 0, 0, 0, -1};
    const int have = pages_of(s, a.max_pages);
    return {(int)n, (int)s, have, pages_of(s + n, a.max_pages) - have, (int)(s + n)};
}

// Last entry of up to n ascending ones that is not above x.
__device__ __forceinline__ int find(const int64_t *from, int n, int64_t x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (from[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void plan_kernel(PlanArgs a)
{
    __shared__ int64_t token_at[kChunk], page_at[kChunk];
    __shared__ int start_of[kChunk], have_of[kChunk];
    __shared__ int64_t sums[kThreads / 64][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t all = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + tid;
    const int64_t taken = a.taken ? *a.taken : 0;
    int64_t tokens = 0, pages = 0;           // of the requests before the chunk
    const auto free_page = [&](int64_t nth) -> int64_t {
        const int64_t at = taken + nth;
        return at >= 0 && at < a.n_free ? a.free_pages[at] : -1;
    };
    for (int64_t b0 = 0; b0 < a.B; b0 += kChunk) {
        Request r[kEach];
        int64_t t = 0, p = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            r[i] = request(a, b0 + tid * kEach + i);
            t += r[i].fresh;
            p += r[i].grow;
        }
        int64_t tu = t, pu = p;              // up to this thread
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t x = __shfl_up(tu, o), y = __shfl_up(pu, o);
            if (lane >= o) {
                tu += x;
                pu += y;
            }
        }
        if (lane == 63) {
            sums[wave][0] = tu;
            sums[wave][1] = pu;
        }
        __syncthreads();                     // (the chunk before has been read, too)
        int64_t chunk_tokens = 0, chunk_pages = 0;
        tu -= t;
        pu -= p;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) {
            if (w < wave) {
                tu += sums[w][0];
                pu += sums[w][1];
            }
            chunk_tokens += sums[w][0];
            chunk_pages += sums[w][1];
        }
        const bool mine = b0 / kChunk % gridDim.x == blockIdx.x;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = tid * kEach + i;
            token_at[at] = tu;
            page_at[at] = pu;
            start_of[at] = r[i].start;
            have_of[at] = r[i].have;
            if (mine && b0 + at < a.B) {
                a.cu[b0 + at] = (int32_t)(tokens + tu < kMost ? tokens + tu : kMost);
                a.lens[b0 + at] = r[i].len;
            }
            tu += r[i].fresh;
            pu += r[i].grow;
        }
        __syncthreads();
        const int n = (int)(a.B - b0 < kChunk ? a.B - b0 : kChunk);
        for (int64_t k = me; k < chunk_pages; k += all) {
            const int i = find(page_at, n, k);
            a.table[(b0 + i) * a.max_pages + have_of[i] + (k - page_at[i])] = (int32_t)free_page(pages + k);
        }
        // this chunk's tokens among those this thread would take of all
        const int64_t end = tokens + chunk_tokens < a.T ? tokens + chunk_tokens : a.T;
        for (int64_t row = tokens <= me ? me : me + (tokens - me + all - 1) / all * all; row < end; row += all) {
            const int i = find(token_at, n, row - tokens);
            const int64_t pos = start_of[i] + (row - tokens - token_at[i]), page = pos / WQ_KV_PAGE;
            if (a.positions) a.positions[row] = (int32_t)pos;
            if (a.slots) {
                int64_t id = -1;
                if (page < have_of[i]) id = a.table[(b0 + i) * a.max_pages + page];
                else if (page < a.max_pages) id = free_page(pages + page_at[i] + (page - have_of[i]));
                a.slots[row] = id >= 0 ? id * WQ_KV_PAGE + pos % WQ_KV_PAGE : -1;
            }
        }
        tokens += chunk_tokens;
        pages += chunk_pages;
    }
    for (int64_t row = tokens <= me ? me : me + (tokens - me + all - 1) / all * all; row < a.T; row += all) {
        if (a.positions) a.positions[row] = -1;
        if (a.slots) a.slots[row] = -1;
    }
    if (me == 0) {
        a.cu[a.B] = (int32_t)(tokens < kMost ? tokens : kMost);
        a.taken_out[0] = (int32_t)(taken + pages < kMost ? taken + pages : kMost);
    }
}

}  // namespace

hipError_t launch_kv_plan(const PlanArgs &a, hipStream_t stream)
{
    const int64_t want = (a.T + kThreads - 1) / kThreads;
    plan_kernel<<<(unsigned)(want < 1 ? 1 : want > 1024 ? 1024 : want), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace wq
