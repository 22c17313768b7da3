"""Operators between the packed projections of a decoder layer: attention over
packed prompts, the int4 key/value cache with the attention that reads it, and
the residual norms.

As in wq.py the binding marshals arguments only. Every tensor of a call lives
on one device, which need not be the current one; work goes to `stream`, else
to that device's current stream, and outputs and workspaces allocated here
belong to that stream (tensors of another stream have to be ready for it and stay
until it is done with them, as everywhere in torch). Bad arguments raise ValueError (or WqError where the
library refuses them) before anything is launched.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .wq import BLOCK, WqError, WqKVCache, _need, _stream, load

KV_PAGE = 64
_WS_ALIGN = 256
_F32, _I32, _I16, _U8 = torch.float32, torch.int32, torch.int16, torch.uint8
_Tensor = torch.Tensor
_CONTIGUOUS = torch.contiguous_format
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class KVCache(NamedTuple):
    """A paged key/value cache in int4 block-32: codes uint8
    [n_pages, kv_heads, 64, head_dim / 2] and scales int16 (binary16 bits)
    [n_pages, kv_heads, 64, head_dim / 32], for keys and for values."""
    kq: torch.Tensor
    ks: torch.Tensor
    vq: torch.Tensor
    vs: torch.Tensor

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache of zero rows."""
        _need(head_dim in (64, 128), "head_dim must be 64 or 128")

        def codes():
            return torch.zeros((n_pages, kv_heads, KV_PAGE, head_dim // 2), dtype=_U8, device=device)

        def scales():
            return torch.zeros((n_pages, kv_heads, KV_PAGE, head_dim // BLOCK), dtype=_I16, device=device)
        return cls(codes(), scales(), codes(), scales())

    @property
    def n_pages(self) -> int:
        return self.kq.shape[0]

    @property
    def kv_heads(self) -> int:
        return self.kq.shape[1]

    @property
    def head_dim(self) -> int:
        return self.kq.shape[3] * 2

    def _struct(self, at: int) -> WqKVCache:
        """The library's view of the cache, whose arrays must lie on device `at`."""
        kq, ks, vq, vs = self
        if not (isinstance(kq, _Tensor) and kq.dim() == 4):
            raise ValueError("cache.kq must be a 4-D device tensor")
        shape = kq.shape
        n, h, page, half = shape
        if page != KV_PAGE:
            raise ValueError("cache pages hold 64 tokens")
        scales = (n, h, page, half // 16)
        if not (kq.dtype is _U8 and vq.dtype is _U8 and ks.dtype is _I16 and vs.dtype is _I16 and vq.shape == shape
                and ks.shape == scales and vs.shape == scales):
            raise ValueError(f"the cache must be uint8 codes {list(shape)} and int16 scales {list(scales)}")
        if not (kq.get_device() == at and ks.get_device() == at and vq.get_device() == at and vs.get_device() == at
                and kq.is_contiguous() and ks.is_contiguous() and vq.is_contiguous() and vs.is_contiguous()):
            raise ValueError(f"the cache's arrays must be contiguous and on device {at}")
        return WqKVCache(kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), n, h, 2 * half)


def _heads(t, name, at=None):
    """[tokens, heads, head_dim] fp32 with heads and values contiguous, on
    device `at` where given; returns (tokens, heads, head_dim, floats between
    tokens)."""
    if not (isinstance(t, _Tensor) and t.dtype is _F32 and t.dim() == 3 and t.is_cuda):
        raise ValueError(f"{name} must be a float32 device tensor [tokens, heads, head_dim]")
    if at is not None and t.get_device() != at:
        raise ValueError(f"{name} must be on device {at}")
    n, h, d = t.shape
    if t.is_contiguous() and d % 4 == 0:
        return n, h, d, h * d
    row, head, value = t.stride()
    if (value != 1 and d > 1) or (head != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    # (the distance to a next token that is not there is never used)
    return n, h, d, row if n > 1 else -(-h * d // 4) * 4


def _index(t, shape, name, at):
    if not (isinstance(t, _Tensor) and t.dtype is _I32 and t.shape == shape and t.get_device() == at and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on device {at}")
    return t.data_ptr()


def _cu(cu, at):
    """Address and number of sequences of cu."""
    if cu is None:
        return None, 1
    if not (isinstance(cu, _Tensor) and cu.dim() == 1 and cu.shape[0] >= 1):
        raise ValueError("cu must be [sequences + 1]")
    shape = cu.shape
    return _index(cu, shape, "cu", at), shape[0] - 1


def _table(table, B, at):
    if not (isinstance(table, _Tensor) and table.dim() == 2):
        raise ValueError("table must be [sequences, max_pages]")
    W = table.shape[1]
    return _index(table, (B, W), "table", at), W


class _On:
    """A device made current, and allocations taken from `stream`."""

    def __init__(self, at, stream):
        _need(stream is None or stream.device.index == at, "stream belongs to another device")
        self.guards = [torch.cuda.device(at)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _run(launch, at, stream):
    """launch(raw stream) with device `at` current and allocations from the stream."""
    if stream is None and at == _current_device():
        return launch(_stream(None, at))
    with _On(at, stream):
        return launch(_stream(stream, at))


def _workspace(nbytes, like):
    """A workspace of nbytes, 256-byte aligned: (tensor to keep, address)."""
    if nbytes == 0:
        return None, None
    t = torch.empty(nbytes + _WS_ALIGN, dtype=_U8, device=like.device)
    p = t.data_ptr()
    return t, p + (-p) % _WS_ALIGN


def _out_heads(out, q, shape, at):
    """`out` of q's shape, made here if None, and the floats between its tokens."""
    if out is None:
        return torch.empty_like(q, memory_format=_CONTIGUOUS), shape[1] * shape[2]
    n, h, d, stride = _heads(out, "out", at)
    if (n, h, d) != shape:
        raise ValueError("out must have q's shape")
    return out, stride


def attn_prefill(q, k, v, cu: Optional[torch.Tensor] = None, scale: Optional[float] = None, out=None, stream=None):
    """Causal attention over packed prompts: q [T, heads, head_dim], k and v
    [T, kv_heads, head_dim] in fp32, rows of any 16-byte stride (slices of a
    fused projection's output); cu int32 [sequences + 1] token offsets on the
    device (None: one prompt). scale defaults to head_dim ** -0.5. Returns out
    [T, heads, head_dim], which must not alias an input; rows of no sequence are
    not written."""
    T, H, D, qs = _heads(q, "q")
    at = q.get_device()
    Tk, Hk, Dk, ks = _heads(k, "k", at)
    Tv, Hv, Dv, vs = _heads(v, "v", at)
    if not (Tk == T and Tv == T and Dk == D and Dv == D and Hv == Hk):
        raise ValueError("k and v must be [T, kv_heads, head_dim] for q's T and head_dim")
    pcu, B = _cu(cu, at)
    lib = load()

    def launch(s):
        y, ys = _out_heads(out, q, (T, H, D), at)
        nb = lib.wq_attn_prefill_ws(T, B, H, Hk, D)
        keep, ws = _workspace(nb, q)
        st = lib.wq_attn_prefill(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, B, H, Hk, D,
                                 D ** -0.5 if scale is None else scale, y.data_ptr(), ys, ws, nb, s)
        if st:
            raise WqError(st, "wq_attn_prefill")
        return y
    return _run(launch, at, stream)


def kv_append(cache: KVCache, k, v, table, cu: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """Quantize k and v [T, kv_heads, head_dim] into the cache: token t of
    sequence b goes to position start[b] + t - cu[b] (start None: 0), page
    table[b, position // 64]. table int32 [sequences, max_pages], cu int32
    [sequences + 1] (None: one sequence), start int32 [sequences]. Rows without
    a page in the cache are dropped."""
    T, H, D, ks = _heads(k, "k")
    at = k.get_device()
    Tv, Hv, Dv, vs = _heads(v, "v", at)
    c = cache._struct(at)
    if not (Tv == T and Hv == H and Dv == D and H == c.kv_heads and D == c.head_dim):
        raise ValueError("k and v must be [T, kv_heads, head_dim] of the cache")
    pcu, B = _cu(cu, at)
    pt, W = _table(table, B, at)
    pst = None if start is None else _index(start, (B,), "start", at)

    def launch(s):
        st = load().wq_kv_append(c, k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, pst, B, pt, W, s)
        if st:
            raise WqError(st, "wq_kv_append")
    _run(launch, at, stream)


def attn_decode(q, cache: KVCache, table, lens, scale: Optional[float] = None, out=None, stream=None):
    """Attention of one query token per sequence over the cache: q
    [sequences, heads, head_dim] fp32, table int32 [sequences, max_pages], lens
    int32 [sequences] cached tokens (the new one included). scale defaults to
    head_dim ** -0.5. Returns out like q (not aliasing an input): zeros where
    lens is 0, NaN where a length or page lies outside the table or the cache."""
    B, H, D, qs = _heads(q, "q")
    at = q.get_device()
    c = cache._struct(at)
    _need(D == c.head_dim, "q must have the cache's head_dim")
    pt, W = _table(table, B, at)
    pl = _index(lens, (B,), "lens", at)
    lib = load()

    def launch(s):
        y, ys = _out_heads(out, q, (B, H, D), at)
        nb = lib.wq_attn_decode_ws(B, H, c.kv_heads, D, W)
        keep, ws = _workspace(nb, q)
        st = lib.wq_attn_decode(c, q.data_ptr(), qs, H, pl, B, pt, W, D ** -0.5 if scale is None else scale,
                                y.data_ptr(), ys, ws, nb, s)
        if st:
            raise WqError(st, "wq_attn_decode")
        return y
    return _run(launch, at, stream)


def _rows(t, shape, name, at):
    """Address of a contiguous fp32 tensor, None for none."""
    if t is None:
        return None
    if not (isinstance(t, _Tensor) and t.dtype is _F32 and t.shape == shape and t.get_device() == at and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 tensor {list(shape)} on device {at}")
    return t.data_ptr()


def residual_norm(h, y=None, post_weight=None, gate=None, alpha: float = 1.0, pre_weight=None, eps: float = 1e-6,
                  norm: Optional[bool] = None, h_out=None, x_out=None, stream=None):
    """The norms around a block, its gate and its residual:
        t = rmsnorm(y) * post_weight (y where post_weight is None),
        h_out = h + alpha * gate * t,   x_out = rmsnorm(h_out) * pre_weight.
    h and y [M, N] fp32; gate [M, N] or [N] (one row for all); weights [N].
    y None: h_out is h (the norm before the first block, not stored unless
    h_out is given). x_out is computed where pre_weight or x_out is given, or
    where norm is True (weight 1). Returns (h_out, x_out), None for what was
    not computed. h_out may be h; no other output may alias an input or the
    other output."""
    if not (isinstance(h, _Tensor) and h.dtype is _F32 and h.dim() == 2 and h.is_cuda and h.is_contiguous()):
        raise ValueError("h must be a contiguous float32 device tensor [M, N]")
    at, shape = h.get_device(), h.shape
    M, N = shape
    py = _rows(y, shape, "y", at)
    pp = _rows(post_weight, (N,), "post_weight", at)
    pw = _rows(pre_weight, (N,), "pre_weight", at)
    pg, gs = None, 0
    if gate is not None:
        one = isinstance(gate, _Tensor) and gate.dim() == 1
        pg, gs = _rows(gate, (N,) if one else shape, "gate", at), 0 if one else N
    want_x = (pre_weight is not None or x_out is not None) if norm is None else norm
    _need(want_x or (pre_weight is None and x_out is None), "norm=False with a pre_weight or x_out")
    _need(y is not None or (post_weight is None and gate is None), "post_weight and gate need y")
    _need(want_x or y is not None, "nothing to compute: neither a block output nor a norm")
    ph, px = _rows(h_out, shape, "h_out", at), _rows(x_out, shape, "x_out", at)

    def launch(s):
        ho = torch.empty_like(h) if h_out is None and y is not None else h_out
        xo = torch.empty_like(h) if x_out is None and want_x else x_out
        st = load().wq_residual_norm(h.data_ptr(), py, pp, pg, gs, alpha, pw, eps, M, N,
                                     ho.data_ptr() if ph is None and ho is not None else ph,
                                     xo.data_ptr() if px is None and xo is not None else px, s)
        if st:
            raise WqError(st, "wq_residual_norm")
        return ho, xo
    return _run(launch, at, stream)
