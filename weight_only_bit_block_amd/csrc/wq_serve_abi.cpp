// wq_serve_abi.cpp -- the C ABI of the operators a serving step adds to those of
// wq_layer_abi.cpp, by the same rules: every check runs before anything is
// launched, nothing is allocated, synchronized or kept.
#include "wq_layer_checks.h"

namespace {

// A window's sizes: past the longest sequence they mean what that means.
int64_t at_most(int64_t x, int64_t top) { return x < top ? x : top; }

int check_window(int64_t window, int64_t sinks) { return window >= 1 && sinks >= 0 ? WQ_OK : WQ_ERR_SHAPE; }

// Rows of a head operator that reads and writes them, with `heads` of any number.
int check_rows(const float *in, int64_t in_stride, const float *out, int64_t out_stride, int64_t heads, int64_t head_dim)
{
    int st = check_stride(in_stride, heads, head_dim);
    if (st || (st = check_stride(out_stride, heads, head_dim))) return st;
    if (!in || !out) return WQ_ERR_NULL;
    return aligned(in, 16) && aligned(out, 16) ? WQ_OK : WQ_ERR_ALIGN;
}

// Memory of a plan's call.
struct Span {
    const void *at;
    uint64_t bytes;
};
bool meet(const Span &a, const Span &b)
{
    return a.at && b.at && a.bytes && b.bytes && (uintptr_t)a.at < (uintptr_t)b.at + b.bytes && (uintptr_t)b.at < (uintptr_t)a.at + a.bytes;
}

// Rows of a call's memory: n of `bytes` each, `stride` bytes apart.
struct Rows {
    const void *at;
    int64_t bytes, stride, n;
};

// Whether one of `a`'s rows shares memory with one of `b`'s: columns of one buffer do not, though their spans meet.
bool rows_meet(const Rows &a, const Rows &b)
{
    if (!a.at || !b.at || a.bytes <= 0 || b.bytes <= 0 || a.n <= 0 || b.n <= 0) return false;
    const int64_t pa = (int64_t)(uintptr_t)a.at, pb = (int64_t)(uintptr_t)b.at;
    if (pa >= pb + (b.n - 1) * b.stride + b.bytes || pb >= pa + (a.n - 1) * a.stride + a.bytes) return false;
    // Rows first to last of `a` against b's `bytes` from `begin` on: the first that ends behind it decides.
    const auto any = [&](int64_t first, int64_t last, int64_t begin) {
        int64_t i = first;
        if (last > first) {
            const int64_t gap = begin - pa - a.bytes, past = gap / a.stride - (gap % a.stride < 0) + 1;
            i = past > first ? past : first;
        }
        return i <= last && pa + i * a.stride + a.bytes > begin && pa + i * a.stride < begin + b.bytes;
    };
    if (b.n == 1) return any(0, a.n - 1, pb);
    if (a.n == 1) return rows_meet(b, a);
    if (a.stride == b.stride) return any(1 - b.n, a.n - 1, pb);  // only the difference of two rows' numbers counts
    for (int64_t j = 0; j < b.n; ++j)
        if (any(0, a.n - 1, pb + j * b.stride)) return true;
    return false;
}

int check_shared(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages, int64_t prefix_pages)
{
    int st = check_decode(B, heads, kv_heads, head_dim, max_pages);
    if (st) return st;
    return prefix_pages < 0 || prefix_pages >= (int64_t)1 << 25 ? WQ_ERR_SHAPE : WQ_OK;
}

}  // namespace

extern "C" {

int wq_qk_norm_rope(const float *q, int64_t q_stride, int64_t heads, const float *k, int64_t k_stride,
                    int64_t kv_heads, int64_t head_dim, int64_t T, const int32_t *positions, const float *inv_freq,
                    int64_t pairs, int interleaved, float factor, int norm, const float *q_weight,
                    const float *k_weight, float eps, float *q_out, int64_t q_out_stride, float *k_out,
                    int64_t k_out_stride, hipStream_t stream)
{
    if (head_dim != 64 && head_dim != 128) return WQ_ERR_SHAPE;
    // workgroups of 256 threads for 1 token or more, below 2^32 threads in all
    if (T < 0 || T >= (int64_t)1 << 24 || heads < 0 || kv_heads < 0 || heads >= kLim / head_dim || kv_heads >= kLim / head_dim)
        return WQ_ERR_SHAPE;
    if (pairs < 0 || pairs > head_dim / 2 || pairs % 4 != 0) return WQ_ERR_SHAPE;
    if (T == 0 || heads + kv_heads == 0) return WQ_OK;
    int st;
    if (heads > 0 && (st = check_rows(q, q_stride, q_out, q_out_stride, heads, head_dim))) return st;
    if (kv_heads > 0 && (st = check_rows(k, k_stride, k_out, k_out_stride, kv_heads, head_dim))) return st;
    if (!positions || (pairs > 0 && !inv_freq)) return WQ_ERR_NULL;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return WQ_ERR_ALIGN;
    // in place row by row only: with other strides a row would be written over one that is still to be read
    if (T > 1 && ((heads > 0 && q == q_out && q_stride != q_out_stride) || (kv_heads > 0 && k == k_out && k_stride != k_out_stride)))
        return WQ_ERR_SHAPE;
    const wq::RopeArgs a = {q, k, q_stride, k_stride, (int)heads, (int)kv_heads, (int)head_dim, T, positions, inv_freq,
                            (int)pairs, factor, norm ? q_weight : nullptr, norm ? k_weight : nullptr, eps, q_out, k_out,
                            q_out_stride, k_out_stride};
    return hip_status(wq::launch_qk_norm_rope(a, norm != 0, interleaved != 0, stream));
}

int wq_kv_plan(const int32_t *fresh, const int32_t *start, int64_t B, int32_t *table, int64_t max_pages,
               const int32_t *free_pages, int64_t n_free, const int32_t *taken, int64_t T, int32_t *cu, int32_t *lens,
               int32_t *positions, int64_t *slots, int32_t *taken_out, hipStream_t stream)
{
    if (B < 0 || B >= kMaxSeqs || max_pages < 0 || max_pages >= (int64_t)1 << 25 || n_free < 0 || n_free >= (int64_t)1 << 31 ||
        T < 0 || T >= kLim)
        return WQ_ERR_SHAPE;
    if (taken_out && taken_out == taken) return WQ_ERR_SHAPE;     // read by all workgroups, written by one
    if (!cu || !taken_out || (B > 0 && (!fresh || !lens)) || (B > 0 && max_pages > 0 && !table) || (n_free > 0 && !free_pages))
        return WQ_ERR_NULL;
    if (!aligned(fresh, 4) || !aligned(start, 4) || !aligned(table, 4) || !aligned(free_pages, 4) || !aligned(taken, 4) ||
        !aligned(cu, 4) || !aligned(lens, 4) || !aligned(positions, 4) || !aligned(slots, 8) || !aligned(taken_out, 4))
        return WQ_ERR_ALIGN;
    // Every workgroup reads all inputs and writes its share of the outputs, in no order: start of the next step in
    // the lengths of this one would be read before or after they are written.
    const uint64_t n = (uint64_t)B * 4;
    const Span in[] = {{fresh, n}, {start, n}, {free_pages, (uint64_t)n_free * 4}, {taken, 4}};
    const Span outs[] = {{table, n * (uint64_t)max_pages}, {cu, n + 4}, {lens, n}, {positions, (uint64_t)T * 4}, {slots, (uint64_t)T * 8}, {taken_out, 4}};
    for (const Span &o : outs) {
        for (const Span &i : in)
            if (meet(o, i)) return WQ_ERR_SHAPE;
        for (const Span *p = outs; p != &o; ++p)
            if (meet(o, *p)) return WQ_ERR_SHAPE;
    }
    const wq::PlanArgs a = {fresh, start, B, table, max_pages, free_pages, n_free, taken, T, cu, lens, positions, slots, taken_out};
    return hip_status(wq::launch_kv_plan(a, stream));
}

int wq_kv_append_slots(const wq_kv_cache *cache, const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                       int64_t T, const int64_t *slots, hipStream_t stream)
{
    int st = check_cache(cache, 1, 0);
    if (st) return st;
    if (T < 0 || T >= kLim || T * cache->kv_heads >= (int64_t)1 << 27) return WQ_ERR_SHAPE;
    if (T == 0) return WQ_OK;
    if ((st = check_stride(k_stride, cache->kv_heads, cache->head_dim)) ||
        (st = check_stride(v_stride, cache->kv_heads, cache->head_dim)))
        return st;
    if (!k || !v || !slots) return WQ_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return WQ_ERR_ALIGN;
    if ((st = check_cache_pointers(cache, nullptr, 0))) return st;
    if (cache->n_pages == 0) return WQ_OK;                        // every row is dropped
    wq::AppendArgs a = {*cache, k, v, k_stride, v_stride, T, nullptr, nullptr, 0, nullptr, 0, slots};
    return hip_status(wq::launch_kv_append(a, stream));
}

int wq_attn_prefill_window(const float *q, int64_t q_stride, const float *k, int64_t k_stride, const float *v,
                           int64_t v_stride, int64_t T, const int32_t *cu, int64_t B, int64_t heads, int64_t kv_heads,
                           int64_t head_dim, float scale, int64_t window, int64_t sinks, float *out,
                           int64_t out_stride, void *workspace, uint64_t workspace_bytes, hipStream_t stream)
{
    int st = check_prompt(T, B, heads, kv_heads, head_dim);
    if (st || (st = check_window(window, sinks))) return st;
    if (T == 0 || B == 0) return WQ_OK;
    if ((st = check_stride(q_stride, heads, head_dim)) || (st = check_stride(k_stride, kv_heads, head_dim)) ||
        (st = check_stride(v_stride, kv_heads, head_dim)) || (st = check_stride(out_stride, heads, head_dim)))
        return st;
    if (!cu && B != 1) return WQ_ERR_NULL;
    if (!q || !k || !v || !out) return WQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu, 4)) return WQ_ERR_ALIGN;
    st = check_ws(workspace, workspace_bytes, wq::prompt_ws_bytes(T, B, heads, kv_heads, head_dim));
    if (st) return st;
    const wq::PromptArgs a = {q, k, v, q_stride, k_stride, v_stride, T, cu, (int)B, (int)heads, (int)kv_heads, (int)head_dim,
                              scale, out, out_stride, workspace, (int)at_most(window, T), (int)at_most(sinks, T)};
    return hip_status(wq::launch_attn_prefill(a, stream));
}

uint64_t wq_attn_decode_window_ws(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages,
                                  int64_t window, int64_t sinks)
{
    if (check_decode(B, heads, kv_heads, head_dim, max_pages) || check_window(window, sinks) || B == 0) return 0;
    const int64_t most = max_pages * WQ_KV_PAGE;
    return wq::decode_window_ws_bytes(B, heads, kv_heads, head_dim, max_pages, at_most(window, most), at_most(sinks, most));
}

int wq_attn_decode_window(const wq_kv_cache *cache, const float *q, int64_t q_stride, int64_t heads,
                          const int32_t *lens, int64_t B, const int32_t *table, int64_t max_pages, float scale,
                          int64_t window, int64_t sinks, float *out, int64_t out_stride, void *workspace,
                          uint64_t workspace_bytes, hipStream_t stream)
{
    int st = check_cache(cache, B, max_pages);
    if (st) return st;
    st = check_decode(B, heads, cache->kv_heads, cache->head_dim, max_pages);
    if (st || (st = check_window(window, sinks))) return st;
    if (B == 0) return WQ_OK;
    if ((st = check_stride(q_stride, heads, cache->head_dim)) || (st = check_stride(out_stride, heads, cache->head_dim)))
        return st;
    if (!q || !lens || !out) return WQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4)) return WQ_ERR_ALIGN;
    if ((st = check_cache_pointers(cache, table, max_pages))) return st;
    st = check_ws(workspace, workspace_bytes,
                  wq_attn_decode_window_ws(B, heads, cache->kv_heads, cache->head_dim, max_pages, window, sinks));
    if (st) return st;
    const int64_t most = max_pages * WQ_KV_PAGE;
    // (no pages: every length but 0 is out of range, whatever the window)
    const wq::DecodeArgs a = {*cache, q, q_stride, (int)heads, lens, (int)B, table, max_pages, scale, out, out_stride, workspace,
                              at_most(window, most), at_most(sinks, most), 0, nullptr};
    return hip_status(wq::launch_attn_decode(a, stream));
}

uint64_t wq_attn_decode_shared_ws(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages,
                                  int64_t prefix_pages)
{
    if (check_shared(B, heads, kv_heads, head_dim, max_pages, prefix_pages) || B == 0) return 0;
    return wq::shared_ws_bytes(B, heads, kv_heads, head_dim, max_pages, prefix_pages);
}

int wq_attn_decode_shared(const wq_kv_cache *cache, const float *q, int64_t q_stride, int64_t heads,
                          const int32_t *prefix, int64_t prefix_pages, const int32_t *prefix_len, const int32_t *lens,
                          int64_t B, const int32_t *table, int64_t max_pages, float scale, float *out,
                          int64_t out_stride, void *workspace, uint64_t workspace_bytes, hipStream_t stream)
{
    int st = check_cache(cache, B, max_pages);
    if (st) return st;
    st = check_shared(B, heads, cache->kv_heads, cache->head_dim, max_pages, prefix_pages);
    if (st) return st;
    if (B == 0) return WQ_OK;
    if ((st = check_stride(q_stride, heads, cache->head_dim)) || (st = check_stride(out_stride, heads, cache->head_dim)))
        return st;
    if (!q || !lens || !out || !prefix_len || (prefix_pages > 0 && !prefix)) return WQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) || !aligned(prefix, 4) || !aligned(prefix_len, 4)) return WQ_ERR_ALIGN;
    if ((st = check_cache_pointers(cache, table, max_pages))) return st;
    st = check_ws(workspace, workspace_bytes,
                  wq::shared_ws_bytes(B, heads, cache->kv_heads, cache->head_dim, max_pages, prefix_pages));
    if (st) return st;
    // Finished rows of own tokens go to out while other workgroups may still have to read any of the inputs.
    const int64_t row = heads * cache->head_dim * 4, codes = cache->n_pages * cache->kv_heads * WQ_KV_PAGE * (cache->head_dim / 2);
    const Rows y = {out, row, out_stride * 4, B};
    const Rows in[] = {{q, row, q_stride * 4, B},           {lens, B * 4, 0, 1},
                       {table, B * max_pages * 4, 0, 1},    {prefix, prefix_pages * 4, 0, 1},
                       {prefix_len, 4, 0, 1},               {cache->kq, codes, 0, 1},
                       {cache->vq, codes, 0, 1},            {cache->ks, codes / 8, 0, 1},
                       {cache->vs, codes / 8, 0, 1}};
    for (const Rows &i : in)
        if (rows_meet(y, i)) return WQ_ERR_SHAPE;
    const wq::SharedArgs a = {{*cache, q, q_stride, (int)heads, lens, (int)B, table, max_pages, scale, out, out_stride, workspace, 0, 0, 0, nullptr},
                              prefix, prefix_len, prefix_pages};
    return hip_status(wq::launch_attn_decode_shared(a, stream));
}

}  // extern "C"
