"""Weight-only block-32 int4/int8 matmul for MI355X (gfx950).

Public API (all computation runs in libwq.so's HIP kernels; PyTorch supplies
device memory and the current stream):

    pack(w, bits) -> (q, scales)        quantize + pack fp32 weights [N, K]
    unpack(q, K, bits) -> codes         int8 codes [N, K]
    gemv(x, q, scales, bits)            decode path, 1 <= M <= 16
    gemm(x, q, scales, bits)            prefill path (fp16 matrix cores)
    gemm_noalloc(x, q, scales, bits)    the same on the library's fixed per-device scratch
    linear(x, q, scales, bits)          dispatch by M
    embed(ids, q, scales, K, bits)      tied-embedding rows of a packed table, fp32
    Package / GroupedCall               64-byte-aligned package + one-launch decode step

Between the projections of a layer:

    attn_prefill(q, k, v, cu)           causal attention over packed prompts
    KVCache                             paged key/value cache in int4 block-32
    kv_append(cache, k, v, table, cu)   quantize new rows into the cache
    attn_decode(q, cache, table, lens)  attention of one token per sequence over the cache
    residual_norm(h, y, ...)            norms around a block, its gate and its residual

A serving step:

    kv_plan(fresh, table, free, ...)    block tables, positions and slots from request lengths
    qk_norm_rope(q, k, positions, ...)  norms of queries and keys, rotated by position
    attn_prefill / attn_decode(..., window, sinks)   attention through a sliding window
    attn_decode_shared(q, cache, ...)   attention of one token per sequence behind a shared prefix

The library is loaded on first use and must have been built
(``python -m weight_only_bit_block_amd.build``); there is no fallback.
"""
from .wq import (BLOCK, GEMV_MAX_M, GroupedCall, Package, WqError, embed, gemm, gemm_noalloc, gemv,
                 header_symbols, linear, load, pack, table_layout, table_plan, table_plan_gemm, unpack)

_LAYER = ("KV_PAGE", "KVCache", "KVPlan", "attn_decode", "attn_decode_shared", "attn_prefill", "kv_append", "kv_plan",
          "qk_norm_rope", "residual_norm")


def __getattr__(name):
    # imported on first use, since it imports torch
    if name in _LAYER:
        from . import layer
        globals().update({n: getattr(layer, n) for n in _LAYER})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


__all__ = ["BLOCK", "GEMV_MAX_M", "GroupedCall", "Package", "WqError", "embed", "gemm", "gemm_noalloc", "gemv",
           "header_symbols", "linear", "load", "pack", "table_layout", "table_plan", "table_plan_gemm", "unpack",
           "KV_PAGE", "KVCache", "KVPlan", "attn_decode", "attn_decode_shared", "attn_prefill", "kv_append", "kv_plan",
           "qk_norm_rope", "residual_norm"]
