// wq_layer_checks.h -- host-side checks shared by the entry points between the
// projections (wq_layer_abi.cpp, wq_serve_abi.cpp).
#pragma once

#include <stdint.h>

#include "wq_internal.h"

namespace {

constexpr int64_t kLim = (int64_t)1 << 30;        // tokens, rows, strides
constexpr int64_t kMaxSeqs = (int64_t)1 << 24;
constexpr int64_t kMaxGroups = (int64_t)1 << 24;  // workgroups of a launch

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? WQ_OK : WQ_ERR_HIP; }

[[maybe_unused]] int check_heads(int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    if (head_dim != 64 && head_dim != 128) return WQ_ERR_SHAPE;
    if (kv_heads < 1 || kv_heads > 1024 || heads < 1 || heads % kv_heads != 0) return WQ_ERR_SHAPE;
    if (heads >= kLim / head_dim) return WQ_ERR_SHAPE;
    return WQ_OK;
}

// Rows of `heads` heads, `stride` floats apart.
[[maybe_unused]] int check_stride(int64_t stride, int64_t heads, int64_t head_dim)
{
    return stride >= heads * head_dim && stride % 4 == 0 && stride < kLim ? WQ_OK : WQ_ERR_SHAPE;
}

[[maybe_unused]] int check_prompt(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    int st = check_heads(heads, kv_heads, head_dim);
    if (st) return st;
    if (T < 0 || T >= kLim || B < 0 || B >= kMaxSeqs) return WQ_ERR_SHAPE;
    // workgroups of at most 256 threads, below 2^32 threads in all
    if ((T / 32 + B) * heads >= kMaxGroups) return WQ_ERR_SHAPE;
    return WQ_OK;
}

[[maybe_unused]] int check_cache(const wq_kv_cache *c, int64_t B, int64_t max_pages)
{
    if (!c) return WQ_ERR_NULL;
    int st = check_heads(c->kv_heads, c->kv_heads, c->head_dim);
    if (st) return st;
    if (c->n_pages < 0 || c->n_pages >= (int64_t)1 << 31) return WQ_ERR_SHAPE;
    if (B < 0 || B >= kMaxSeqs || max_pages < 0 || max_pages >= (int64_t)1 << 25) return WQ_ERR_SHAPE;
    return WQ_OK;
}

// Pointers of a cache and of the table into it, for a call that reads or writes them.
[[maybe_unused]] int check_cache_pointers(const wq_kv_cache *c, const int32_t *table, int64_t max_pages)
{
    if (c->n_pages > 0) {
        if (!c->kq || !c->ks || !c->vq || !c->vs) return WQ_ERR_NULL;
        if (!aligned(c->kq, 16) || !aligned(c->ks, 16) || !aligned(c->vq, 16) || !aligned(c->vs, 16)) return WQ_ERR_ALIGN;
    }
    if (max_pages > 0 && !table) return WQ_ERR_NULL;
    return aligned(table, 4) ? WQ_OK : WQ_ERR_ALIGN;
}

[[maybe_unused]] int check_decode(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    int st = check_heads(heads, kv_heads, head_dim);
    if (st) return st;
    if (B < 0 || B >= kMaxSeqs || max_pages < 0 || max_pages >= (int64_t)1 << 25) return WQ_ERR_SHAPE;
    // the join's workgroups of up to 512 threads, below 2^32 threads in all; steps are counted in 31 bits
    if (B * heads >= kMaxGroups / 2 || B * max_pages >= (int64_t)1 << 32) return WQ_ERR_SHAPE;
    return WQ_OK;
}

[[maybe_unused]] int check_ws(const void *ws, uint64_t have, uint64_t need)
{
    if (need == 0) return WQ_OK;
    if (!ws) return WQ_ERR_NULL;
    if (!aligned(ws, 256)) return WQ_ERR_ALIGN;
    return have >= need ? WQ_OK : WQ_ERR_SHAPE;
}

}  // namespace
