// wq_layer_abi.cpp -- the C ABI of the operators between the projections:
// host-side validation and workspace sizes. As in wq_abi.cpp, every check runs
// before anything is launched, a failing check touches no HIP state, and
// nothing is allocated, synchronized or kept.
#include <stdint.h>

#include "wq_internal.h"

namespace {

constexpr int64_t kLim = (int64_t)1 << 30;        // tokens, rows, strides
constexpr int64_t kMaxSeqs = (int64_t)1 << 24;
constexpr int64_t kMaxGroups = (int64_t)1 << 24;  // workgroups of a launch

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? WQ_OK : WQ_ERR_HIP; }

int check_heads(int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    if (head_dim != 64 && head_dim != 128) return WQ_ERR_SHAPE;
    if (kv_heads < 1 || kv_heads > 1024 || heads < 1 || heads % kv_heads != 0) return WQ_ERR_SHAPE;
    if (heads >= kLim / head_dim) return WQ_ERR_SHAPE;
    return WQ_OK;
}

// Rows of `heads` heads, `stride` floats apart.
int check_stride(int64_t stride, int64_t heads, int64_t head_dim)
{
    return stride >= heads * head_dim && stride % 4 == 0 && stride < kLim ? WQ_OK : WQ_ERR_SHAPE;
}

int check_prompt(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    int st = check_heads(heads, kv_heads, head_dim);
    if (st) return st;
    if (T < 0 || T >= kLim || B < 0 || B >= kMaxSeqs) return WQ_ERR_SHAPE;
    // workgroups of at most 256 threads, below 2^32 threads in all
    if ((T / 32 + B) * heads >= kMaxGroups) return WQ_ERR_SHAPE;
    return WQ_OK;
}

int check_cache(const wq_kv_cache *c, int64_t B, int64_t max_pages)
{
    if (!c) return WQ_ERR_NULL;
    int st = check_heads(c->kv_heads, c->kv_heads, c->head_dim);
    if (st) return st;
    if (c->n_pages < 0 || c->n_pages >= (int64_t)1 << 31) return WQ_ERR_SHAPE;
    if (B < 0 || B >= kMaxSeqs || max_pages < 0 || max_pages >= (int64_t)1 << 25) return WQ_ERR_SHAPE;
    return WQ_OK;
}

// Pointers of a cache and of the table into it, for a call that reads or writes them.
int check_cache_pointers(const wq_kv_cache *c, const int32_t *table, int64_t max_pages)
{
    if (c->n_pages > 0) {
        if (!c->kq || !c->ks || !c->vq || !c->vs) return WQ_ERR_NULL;
        if (!aligned(c->kq, 16) || !aligned(c->ks, 16) || !aligned(c->vq, 16) || !aligned(c->vs, 16)) return WQ_ERR_ALIGN;
    }
    if (max_pages > 0 && !table) return WQ_ERR_NULL;
    return aligned(table, 4) ? WQ_OK : WQ_ERR_ALIGN;
}

int check_decode(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    int st = check_heads(heads, kv_heads, head_dim);
    if (st) return st;
    if (B < 0 || B >= kMaxSeqs || max_pages < 0 || max_pages >= (int64_t)1 << 25) return WQ_ERR_SHAPE;
    // the join's workgroups of up to 512 threads, below 2^32 threads in all; steps are counted in 31 bits
    if (B * heads >= kMaxGroups / 2 || B * max_pages >= (int64_t)1 << 32) return WQ_ERR_SHAPE;
    return WQ_OK;
}

int check_ws(const void *ws, uint64_t have, uint64_t need)
{
    if (need == 0) return WQ_OK;
    if (!ws) return WQ_ERR_NULL;
    if (!aligned(ws, 256)) return WQ_ERR_ALIGN;
    return have >= need ? WQ_OK : WQ_ERR_SHAPE;
}

}  // namespace

extern "C" {

uint64_t wq_attn_prefill_ws(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim)
{
    if (check_prompt(T, B, heads, kv_heads, head_dim) || T == 0 || B == 0) return 0;
    return wq::prompt_ws_bytes(T, B, heads, kv_heads, head_dim);
}

int wq_attn_prefill(const float *q, int64_t q_stride, const float *k, int64_t k_stride, const float *v,
                    int64_t v_stride, int64_t T, const int32_t *cu, int64_t B, int64_t heads, int64_t kv_heads,
                    int64_t head_dim, float scale, float *out, int64_t out_stride, void *workspace,
                    uint64_t workspace_bytes, hipStream_t stream)
{
    int st = check_prompt(T, B, heads, kv_heads, head_dim);
    if (st) return st;
    if (T == 0 || B == 0) return WQ_OK;
    if ((st = check_stride(q_stride, heads, head_dim)) || (st = check_stride(k_stride, kv_heads, head_dim)) ||
        (st = check_stride(v_stride, kv_heads, head_dim)) || (st = check_stride(out_stride, heads, head_dim)))
        return st;
    if (!cu && B != 1) return WQ_ERR_NULL;
    if (!q || !k || !v || !out) return WQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu, 4)) return WQ_ERR_ALIGN;
    st = check_ws(workspace, workspace_bytes, wq::prompt_ws_bytes(T, B, heads, kv_heads, head_dim));
    if (st) return st;
    const wq::PromptArgs a = {q, k, v, q_stride, k_stride, v_stride, T, cu, (int)B, (int)heads, (int)kv_heads,
                              (int)head_dim, scale, out, out_stride, workspace};
    return hip_status(wq::launch_attn_prefill(a, stream));
}

int wq_kv_append(const wq_kv_cache *cache, const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                 int64_t T, const int32_t *cu, const int32_t *start, int64_t B, const int32_t *table,
                 int64_t max_pages, hipStream_t stream)
{
    int st = check_cache(cache, B, max_pages);
    if (st) return st;
    if (T < 0 || T >= kLim || T * cache->kv_heads >= (int64_t)1 << 27) return WQ_ERR_SHAPE;
    if (T == 0 || B == 0) return WQ_OK;
    if ((st = check_stride(k_stride, cache->kv_heads, cache->head_dim)) ||
        (st = check_stride(v_stride, cache->kv_heads, cache->head_dim)))
        return st;
    if (!cu && B != 1) return WQ_ERR_NULL;
    if (!k || !v) return WQ_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cu, 4) || !aligned(start, 4)) return WQ_ERR_ALIGN;
    if ((st = check_cache_pointers(cache, table, max_pages))) return st;
    if (max_pages == 0 || cache->n_pages == 0) return WQ_OK;      // every row is dropped
    const wq::AppendArgs a = {*cache, k, v, k_stride, v_stride, T, cu, start, (int)B, table, max_pages};
    return hip_status(wq::launch_kv_append(a, stream));
}

uint64_t wq_attn_decode_ws(int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t max_pages)
{
    if (check_decode(B, heads, kv_heads, head_dim, max_pages) || B == 0) return 0;
    return wq::decode_ws_bytes(B, heads, kv_heads, head_dim, max_pages);
}

int wq_attn_decode(const wq_kv_cache *cache, const float *q, int64_t q_stride, int64_t heads, const int32_t *lens,
                   int64_t B, const int32_t *table, int64_t max_pages, float scale, float *out, int64_t out_stride,
                   void *workspace, uint64_t workspace_bytes, hipStream_t stream)
{
    int st = check_cache(cache, B, max_pages);
    if (st) return st;
    st = check_decode(B, heads, cache->kv_heads, cache->head_dim, max_pages);
    if (st) return st;
    if (B == 0) return WQ_OK;
    if ((st = check_stride(q_stride, heads, cache->head_dim)) || (st = check_stride(out_stride, heads, cache->head_dim)))
        return st;
    if (!q || !lens || !out) return WQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4)) return WQ_ERR_ALIGN;
    if ((st = check_cache_pointers(cache, table, max_pages))) return st;
    st = check_ws(workspace, workspace_bytes,
                  wq::decode_ws_bytes(B, heads, cache->kv_heads, cache->head_dim, max_pages));
    if (st) return st;
    const wq::DecodeArgs a = {*cache, q, q_stride, (int)heads, lens, (int)B, table, max_pages, scale, out, out_stride, workspace};
    return hip_status(wq::launch_attn_decode(a, stream));
}

int wq_residual_norm(const float *h, const float *y, const float *post_weight, const float *gate, int64_t gate_stride,
                     float alpha, const float *pre_weight, float eps, int64_t M, int64_t N, float *h_out, float *x_out,
                     hipStream_t stream)
{
    if (M < 0 || M >= kLim || N < 0 || N >= kLim) return WQ_ERR_SHAPE;
    if (gate && gate_stride != 0 && gate_stride != N) return WQ_ERR_SHAPE;
    if (M == 0 || N == 0) return WQ_OK;
    if (!h || (!h_out && !x_out)) return WQ_ERR_NULL;
    if (!y && (post_weight || gate)) return WQ_ERR_NULL;
    if (!aligned(h, 4) || !aligned(y, 4) || !aligned(post_weight, 4) || !aligned(gate, 4) || !aligned(pre_weight, 4) ||
        !aligned(h_out, 4) || !aligned(x_out, 4))
        return WQ_ERR_ALIGN;
    const wq::NormArgs a = {h, y, post_weight, gate, gate_stride, alpha, pre_weight, eps, M, N, h_out, x_out};
    return hip_status(wq::launch_residual_norm(a, stream));
}

}  // extern "C"
