"""Operators between the packed projections of a decoder layer: attention over
packed prompts, the int4 key/value cache with the attention that reads it, and
the residual norms.

As in wq.py the binding marshals arguments only. Every tensor of a call lives
on one device, which need not be the current one; work goes to `stream`, else
to that device's current stream, and outputs and workspaces allocated here
belong to that stream. Bad arguments raise ValueError (or WqError where the
library refuses them) before anything is launched.
"""
from __future__ import annotations

import ctypes
from typing import TYPE_CHECKING, NamedTuple, Optional

from .wq import BLOCK, WqError, WqKVCache, _need, _stream, _torch, load

if TYPE_CHECKING:
    import torch

KV_PAGE = 64
_WS_ALIGN = 256


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
        torch = _torch()
        _need(head_dim in (64, 128), "head_dim must be 64 or 128")

        def codes():
            return torch.zeros((n_pages, kv_heads, KV_PAGE, head_dim // 2), dtype=torch.uint8, device=device)

        def scales():
            return torch.zeros((n_pages, kv_heads, KV_PAGE, head_dim // BLOCK), dtype=torch.int16, device=device)
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

    def _struct(self, device) -> WqKVCache:
        torch = _torch()
        n, h, page, half = _shape4(self.kq, "cache.kq")
        _need(page == KV_PAGE, "cache pages hold 64 tokens")
        for t, dt, shape, name in ((self.kq, torch.uint8, (n, h, page, half), "cache.kq"),
                                   (self.vq, torch.uint8, (n, h, page, half), "cache.vq"),
                                   (self.ks, torch.int16, (n, h, page, half // 16), "cache.ks"),
                                   (self.vs, torch.int16, (n, h, page, half // 16), "cache.vs")):
            if not (t.dtype == dt and t.shape == shape and t.is_contiguous() and t.device == device):
                raise ValueError(f"{name} must be a contiguous {dt} tensor {list(shape)} on {device}")
        return WqKVCache(self.kq.data_ptr(), self.ks.data_ptr(), self.vq.data_ptr(), self.vs.data_ptr(), n, h, 2 * half)


def _shape4(t, name):
    torch = _torch()
    _need(isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 4, f"{name} must be a 4-D device tensor")
    return t.shape


def _heads(t, name, device=None):
    """[tokens, heads, head_dim] fp32 with heads and values contiguous; returns
    (tokens, heads, head_dim, floats between tokens)."""
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.float32 and t.dim() == 3):
        raise ValueError(f"{name} must be a float32 device tensor [tokens, heads, head_dim]")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    n, h, d = t.shape
    st = t.stride()
    if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if n <= 1:
        return n, h, d, -(-h * d // 4) * 4        # the distance to a next token is never used
    return n, h, d, st[0]


def _index(t, shape, name, device):
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.device == device and t.is_contiguous()
            and t.shape == shape):
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on {device}")
    return t.data_ptr()


def _cu(cu, B, name, device):
    torch = _torch()
    if cu is None:
        return None, 1
    _need(isinstance(cu, torch.Tensor) and cu.dim() == 1 and cu.shape[0] >= 1, f"{name} must be [sequences + 1]")
    B = cu.shape[0] - 1 if B is None else B
    return _index(cu, (B + 1,), name, device), B


class _On:
    """The tensors' device made current, and allocations taken from `stream`."""

    def __init__(self, device, stream):
        torch = _torch()
        _need(stream is None or stream.device == device, "stream belongs to another device")
        self.guard = torch.cuda.device(device) if device.index != torch.cuda.current_device() else None
        self.on = torch.cuda.stream(stream) if stream is not None else None
        self.device, self.stream = device, stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.on is not None:
            self.on.__enter__()
        return _stream(self.stream, self.device.index)

    def __exit__(self, *exc):
        if self.on is not None:
            self.on.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _workspace(nbytes, device):
    """A workspace of nbytes, 256-byte aligned: (tensor to keep, address)."""
    torch = _torch()
    if nbytes == 0:
        return None, None
    t = torch.empty(nbytes + _WS_ALIGN, dtype=torch.uint8, device=device)
    p = t.data_ptr()
    return t, p + (-p) % _WS_ALIGN


def attn_prefill(q, k, v, cu: Optional[torch.Tensor] = None, scale: Optional[float] = None, out=None, stream=None):
    """Causal attention over packed prompts: q [T, heads, head_dim], k and v
    [T, kv_heads, head_dim] in fp32, rows of any 16-byte stride (slices of a
    fused projection's output); cu int32 [sequences + 1] token offsets on the
    device (None: one prompt). scale defaults to head_dim ** -0.5. Returns out
    [T, heads, head_dim]; rows of no sequence are not written."""
    torch = _torch()
    T, H, D, qs = _heads(q, "q")
    dev = q.device
    Tk, Hk, Dk, ks = _heads(k, "k", dev)
    Tv, Hv, Dv, vs = _heads(v, "v", dev)
    if not (Tk == T and Tv == T and Dk == D and Dv == D and Hv == Hk):
        raise ValueError("k and v must be [T, kv_heads, head_dim] for q's T and head_dim")
    pcu, B = _cu(cu, None, "cu", dev)
    lib = load()
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((T, H, D), dtype=torch.float32, device=dev)
        To, Ho, Do, os_ = _heads(out, "out", dev)
        if (To, Ho, Do) != (T, H, D):
            raise ValueError("out must have q's shape")
        nb = lib.wq_attn_prefill_ws(T, B, H, Hk, D)
        keep, ws = _workspace(nb, dev)
        st = lib.wq_attn_prefill(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, B, H, Hk, D,
                                 D ** -0.5 if scale is None else scale, out.data_ptr(), os_, ws, nb, s)
    if st:
        raise WqError(st, "wq_attn_prefill")
    return out


def kv_append(cache: KVCache, k, v, table, cu: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """Quantize k and v [T, kv_heads, head_dim] into the cache: token t of
    sequence b goes to position start[b] + t - cu[b] (start None: 0), page
    table[b, position // 64]. table int32 [sequences, max_pages], cu int32
    [sequences + 1] (None: one sequence), start int32 [sequences]. Rows without
    a page in the cache are dropped."""
    torch = _torch()
    T, H, D, ks = _heads(k, "k")
    dev = k.device
    Tv, Hv, Dv, vs = _heads(v, "v", dev)
    c = cache._struct(dev)
    if not (Tv == T and Hv == H and Dv == D and H == c.kv_heads and D == c.head_dim):
        raise ValueError("k and v must be [T, kv_heads, head_dim] of the cache")
    pcu, B = _cu(cu, None, "cu", dev)
    _need(isinstance(table, torch.Tensor) and table.dim() == 2, "table must be [sequences, max_pages]")
    W = table.shape[1]
    pt = _index(table, (B, W), "table", dev)
    pst = None if start is None else _index(start, (B,), "start", dev)
    with _On(dev, stream) as s:
        st = load().wq_kv_append(ctypes.byref(c), k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, pst, B, pt, W, s)
    if st:
        raise WqError(st, "wq_kv_append")


def attn_decode(q, cache: KVCache, table, lens, scale: Optional[float] = None, out=None, stream=None):
    """Attention of one query token per sequence over the cache: q
    [sequences, heads, head_dim] fp32, table int32 [sequences, max_pages], lens
    int32 [sequences] cached tokens (the new one included). scale defaults to
    head_dim ** -0.5. Returns out like q: zeros where lens is 0, NaN where a
    length or page lies outside the table or the cache."""
    torch = _torch()
    B, H, D, qs = _heads(q, "q")
    dev = q.device
    c = cache._struct(dev)
    _need(D == c.head_dim, "q must have the cache's head_dim")
    _need(isinstance(table, torch.Tensor) and table.dim() == 2, "table must be [sequences, max_pages]")
    W = table.shape[1]
    pt = _index(table, (B, W), "table", dev)
    pl = _index(lens, (B,), "lens", dev)
    lib = load()
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((B, H, D), dtype=torch.float32, device=dev)
        Bo, Ho, Do, os_ = _heads(out, "out", dev)
        if (Bo, Ho, Do) != (B, H, D):
            raise ValueError("out must have q's shape")
        nb = lib.wq_attn_decode_ws(B, H, c.kv_heads, D, W)
        keep, ws = _workspace(nb, dev)
        st = lib.wq_attn_decode(ctypes.byref(c), q.data_ptr(), qs, H, pl, B, pt, W,
                                D ** -0.5 if scale is None else scale, out.data_ptr(), os_, ws, nb, s)
    if st:
        raise WqError(st, "wq_attn_decode")
    return out


def _rows(t, shape, name, device):
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.device == device and t.is_contiguous()
            and t.shape == shape):
        raise ValueError(f"{name} must be a contiguous float32 tensor {list(shape)} on {device}")
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
    not computed. h_out may be h."""
    torch = _torch()
    if not (isinstance(h, torch.Tensor) and h.is_cuda and h.dtype == torch.float32 and h.dim() == 2 and h.is_contiguous()):
        raise ValueError("h must be a contiguous float32 device tensor [M, N]")
    dev, shape = h.device, h.shape
    M, N = shape
    py = None if y is None else _rows(y, shape, "y", dev)
    pp = None if post_weight is None else _rows(post_weight, (N,), "post_weight", dev)
    pw = None if pre_weight is None else _rows(pre_weight, (N,), "pre_weight", dev)
    pg, gs = None, 0
    if gate is not None:
        one = isinstance(gate, torch.Tensor) and gate.dim() == 1
        pg, gs = _rows(gate, (N,) if one else shape, "gate", dev), 0 if one else N
    want_x = (pre_weight is not None or x_out is not None) if norm is None else norm
    _need(want_x or (pre_weight is None and x_out is None), "norm=False with a pre_weight or x_out")
    _need(y is not None or (post_weight is None and gate is None), "post_weight and gate need y")
    _need(want_x or y is not None, "nothing to compute: neither a block output nor a norm")
    with _On(dev, stream) as s:
        if h_out is None and y is not None:
            h_out = torch.empty(shape, dtype=torch.float32, device=dev)
        if x_out is None and want_x:
            x_out = torch.empty(shape, dtype=torch.float32, device=dev)
        ph = None if h_out is None else _rows(h_out, shape, "h_out", dev)
        px = None if x_out is None else _rows(x_out, shape, "x_out", dev)
        st = load().wq_residual_norm(h.data_ptr(), py, pp, pg, gs, alpha, pw, eps, M, N, ph, px, s)
    if st:
        raise WqError(st, "wq_residual_norm")
    return h_out, x_out
