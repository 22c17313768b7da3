"""Operators between the packed projections of a decoder layer: attention over
packed prompts, the int4 key/value cache with the attention that reads it, the
residual norms, and what a serving step adds: its plan, the norms and rotation
of queries and keys, attention through a window or behind a shared prefix.

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
_F32, _I64, _I32, _I16, _U8 = torch.float32, torch.int64, torch.int32, torch.int16, torch.uint8
_MOST = 1 << 40             # a window as long as any sequence
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


def _out_heads(out, q, shape, at, name="out"):
    """`out` of q's shape, made here if None, and the floats between its tokens."""
    if out is None:
        return torch.empty_like(q, memory_format=_CONTIGUOUS), shape[1] * shape[2]
    n, h, d, stride = _heads(out, name, at)
    if (n, h, d) != shape:
        raise ValueError(f"{name} must have {'k' if name == 'k_out' else 'q'}'s shape")
    return out, stride


def _count(x, name, least):
    """A whole number (of any integer type), at least `least`."""
    if type(x) is not int:
        if isinstance(x, bool) or not hasattr(x, "__index__") or isinstance(x, _Tensor):
            raise ValueError(f"{name} must be a whole number")
        x = x.__index__()
    if x < least:
        raise ValueError(f"{name} must be {least} at least")
    return x if x < _MOST else _MOST


def attn_prefill(q, k, v, cu: Optional[torch.Tensor] = None, scale: Optional[float] = None, out=None, stream=None,
                 window: Optional[int] = None, sinks: int = 0):
    """Causal attention over packed prompts: q [T, heads, head_dim], k and v
    [T, kv_heads, head_dim] in fp32, rows of any 16-byte stride (slices of a
    fused projection's output); cu int32 [sequences + 1] token offsets on the
    device (None: one prompt). scale defaults to head_dim ** -0.5. Returns out
    [T, heads, head_dim], which must not alias an input; rows of no sequence are
    not written. window: a token sees itself and the window - 1 tokens before it,
    and its sequence's first `sinks` tokens (None: all before it)."""
    T, H, D, qs = _heads(q, "q")
    at = q.get_device()
    Tk, Hk, Dk, ks = _heads(k, "k", at)
    Tv, Hv, Dv, vs = _heads(v, "v", at)
    if not (Tk == T and Tv == T and Dk == D and Dv == D and Hv == Hk):
        raise ValueError("k and v must be [T, kv_heads, head_dim] for q's T and head_dim")
    pcu, B = _cu(cu, at)
    _need(window is not None or sinks == 0, "sinks need a window")
    if window is not None:
        window, sinks = _count(window, "window", 1), _count(sinks, "sinks", 0)
    lib = load()

    def launch(s):
        y, ys = _out_heads(out, q, (T, H, D), at)
        nb = lib.wq_attn_prefill_ws(T, B, H, Hk, D)
        keep, ws = _workspace(nb, q)
        if window is not None:
            st = lib.wq_attn_prefill_window(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, B, H, Hk, D,
                                            D ** -0.5 if scale is None else scale, window, sinks, y.data_ptr(), ys, ws, nb, s)
            if st:
                raise WqError(st, "wq_attn_prefill_window")
            return y
        st = lib.wq_attn_prefill(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, B, H, Hk, D,
                                 D ** -0.5 if scale is None else scale, y.data_ptr(), ys, ws, nb, s)
        if st:
            raise WqError(st, "wq_attn_prefill")
        return y
    return _run(launch, at, stream)


def kv_append(cache: KVCache, k, v, table=None, cu: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
              stream=None, slots: Optional[torch.Tensor] = None) -> None:
    """Quantize k and v [T, kv_heads, head_dim] into the cache: token t of
    sequence b goes to position start[b] + t - cu[b] (start None: 0), page
    table[b, position // 64]. table int32 [sequences, max_pages], cu int32
    [sequences + 1] (None: one sequence), start int32 [sequences]. Rows without
    a page in the cache are dropped. slots int64 [T] in place of all these: token t
    goes to row slots[t] % 64 of page slots[t] // 64 (kv_plan makes them; those of
    different tokens must differ, and negative ones are dropped)."""
    T, H, D, ks = _heads(k, "k")
    at = k.get_device()
    Tv, Hv, Dv, vs = _heads(v, "v", at)
    c = cache._struct(at)
    if not (Tv == T and Hv == H and Dv == D and H == c.kv_heads and D == c.head_dim):
        raise ValueError("k and v must be [T, kv_heads, head_dim] of the cache")
    if slots is not None:
        _need(table is None and cu is None and start is None, "slots take the place of table, cu and start")
        if not (isinstance(slots, _Tensor) and slots.dtype is _I64 and slots.shape == (T,) and slots.get_device() == at
                and slots.is_contiguous()):
            raise ValueError(f"slots must be a contiguous int64 tensor [{T}] on device {at}")

        def launch(s):
            st = load().wq_kv_append_slots(c, k.data_ptr(), ks, v.data_ptr(), vs, T, slots.data_ptr(), s)
            if st:
                raise WqError(st, "wq_kv_append_slots")
        return _run(launch, at, stream)
    pcu, B = _cu(cu, at)
    pt, W = _table(table, B, at)
    pst = None if start is None else _index(start, (B,), "start", at)

    def launch(s):
        st = load().wq_kv_append(c, k.data_ptr(), ks, v.data_ptr(), vs, T, pcu, pst, B, pt, W, s)
        if st:
            raise WqError(st, "wq_kv_append")
    _run(launch, at, stream)


def attn_decode(q, cache: KVCache, table, lens, scale: Optional[float] = None, out=None, stream=None,
                window: Optional[int] = None, sinks: int = 0):
    """Attention of one query token per sequence over the cache: q
    [sequences, heads, head_dim] fp32, table int32 [sequences, max_pages], lens
    int32 [sequences] cached tokens (the new one included). scale defaults to
    head_dim ** -0.5. Returns out like q (not aliasing an input): zeros where
    lens is 0, NaN where a length or page lies outside the table or the cache.
    window: only the last `window` cached tokens and the first `sinks` ones are
    seen; pages without any of them are not looked at."""
    B, H, D, qs = _heads(q, "q")
    at = q.get_device()
    c = cache._struct(at)
    _need(D == c.head_dim, "q must have the cache's head_dim")
    pt, W = _table(table, B, at)
    pl = _index(lens, (B,), "lens", at)
    _need(window is not None or sinks == 0, "sinks need a window")
    if window is not None:
        window, sinks = _count(window, "window", 1), _count(sinks, "sinks", 0)
    lib = load()

    def launch(s):
        y, ys = _out_heads(out, q, (B, H, D), at)
        if window is not None:
            nb = lib.wq_attn_decode_window_ws(B, H, c.kv_heads, D, W, window, sinks)
            keep, ws = _workspace(nb, q)
            st = lib.wq_attn_decode_window(c, q.data_ptr(), qs, H, pl, B, pt, W, D ** -0.5 if scale is None else scale,
                                           window, sinks, y.data_ptr(), ys, ws, nb, s)
            if st:
                raise WqError(st, "wq_attn_decode_window")
            return y
        nb = lib.wq_attn_decode_ws(B, H, c.kv_heads, D, W)
        keep, ws = _workspace(nb, q)
        st = lib.wq_attn_decode(c, q.data_ptr(), qs, H, pl, B, pt, W, D ** -0.5 if scale is None else scale,
                                y.data_ptr(), ys, ws, nb, s)
        if st:
            raise WqError(st, "wq_attn_decode")
        return y
    return _run(launch, at, stream)


def attn_decode_shared(q, cache: KVCache, prefix, prefix_len, table, lens, scale: Optional[float] = None, out=None,
                       stream=None):
    """Attention of one query token per sequence where all sequences begin with
    the same cached tokens: q [sequences, heads, head_dim] fp32; prefix int32
    [prefix_pages] and prefix_len int32 [1], the shared tokens' pages and number,
    read once for all queries; table int32 [sequences, max_pages] and lens int32
    [sequences] as in attn_decode, of each sequence's own tokens behind them (rotated,
    where they are, as tokens prefix_len + 0, 1, ...).
    Returns out like q (sharing no memory with an input): zeros where there is no
    token, NaN where a length or page lies outside its table or the cache (of the
    prefix: in all rows)."""
    B, H, D, qs = _heads(q, "q")
    at = q.get_device()
    c = cache._struct(at)
    _need(D == c.head_dim, "q must have the cache's head_dim")
    if not (isinstance(prefix, _Tensor) and prefix.dim() == 1):
        raise ValueError("prefix must be [prefix_pages]")
    P = prefix.shape[0]
    pp, pn = _index(prefix, (P,), "prefix", at), _index(prefix_len, (1,), "prefix_len", at)
    pt, W = _table(table, B, at)
    pl = _index(lens, (B,), "lens", at)
    lib = load()

    def launch(s):
        y, ys = _out_heads(out, q, (B, H, D), at)
        nb = lib.wq_attn_decode_shared_ws(B, H, c.kv_heads, D, W, P)
        keep, ws = _workspace(nb, q)
        st = lib.wq_attn_decode_shared(c, q.data_ptr(), qs, H, pp, P, pn, pl, B, pt, W, D ** -0.5 if scale is None else scale,
                                       y.data_ptr(), ys, ws, nb, s)
        if st:
            raise WqError(st, "wq_attn_decode_shared")
        return y
    return _run(launch, at, stream)


class KVPlan(NamedTuple):
    """What kv_plan makes, besides the pages in the table: cu int32
    [requests + 1], lens int32 [requests], positions int32 [tokens], slots int64
    [tokens], taken int32 [1]."""
    cu: torch.Tensor
    lens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    taken: torch.Tensor


def kv_plan(fresh, table, free, taken: Optional[torch.Tensor] = None, tokens: int = 0,
            start: Optional[torch.Tensor] = None, out: Optional[KVPlan] = None, stream=None) -> KVPlan:
    """The plan of a step, made on the device: `fresh` int32 [requests] new
    tokens each, behind the start int32 [requests] (None: 0) cached ones. New
    pages come from free int32 [pages], from entry taken int32 [1] (None: 0) on,
    into table int32 [requests, max_pages], which is written (-1 where the list
    is used up); returns the token offsets cu, the lengths after the step, each
    token's position and its slot in the cache for up to `tokens` tokens (-1
    past the last one, slots also where there is no page), and the new `taken`
    (past len(free): the list was too short). `out`: a plan to write into, which
    shares no memory with the inputs (start and taken are copies of the last step's
    lens and taken, or those of another plan). A request with a bad length gets
    lens -1 and no tokens. Of requests behind a shared prefix these are their own
    tokens: for qk_norm_rope add the prefix's length to the positions that are not -1."""
    if not (isinstance(fresh, _Tensor) and fresh.dim() == 1 and fresh.is_cuda):
        raise ValueError("fresh must be an int32 device tensor [requests]")
    B, at = fresh.shape[0], fresh.get_device()
    pf = _index(fresh, (B,), "fresh", at)
    pt, W = _table(table, B, at)
    if not (isinstance(free, _Tensor) and free.dim() == 1):
        raise ValueError("free must be [pages]")
    n_free = free.shape[0]
    pfree = _index(free, (n_free,), "free", at)
    ptaken = None if taken is None else _index(taken, (1,), "taken", at)
    pst = None if start is None else _index(start, (B,), "start", at)
    tokens = _count(tokens, "tokens", 0)
    if out is not None:
        for t, n, name in ((out.cu, B + 1, "cu"), (out.lens, B, "lens"), (out.positions, tokens, "positions"), (out.taken, 1, "taken")):
            _index(t, (n,), "out." + name, at)
        s = out.slots
        if not (isinstance(s, _Tensor) and s.dtype is _I64 and s.shape == (tokens,) and s.get_device() == at and s.is_contiguous()):
            raise ValueError(f"out.slots must be a contiguous int64 tensor [{tokens}] on device {at}")
        _need(out.taken.data_ptr() != ptaken, "out.taken must not be taken")

    def launch(s):
        p = out
        if p is None:                            # (two allocations instead of five: 2 us a call)
            cu, lens, positions, took = fresh.new_empty(2 * B + tokens + 2).split_with_sizes((B + 1, B, tokens, 1))
            p = KVPlan(cu, lens, positions, fresh.new_empty(tokens, dtype=_I64), took)
        st = load().wq_kv_plan(pf, pst, B, pt, W, pfree, n_free, ptaken, tokens, p.cu.data_ptr(), p.lens.data_ptr(),
                               p.positions.data_ptr(), p.slots.data_ptr(), p.taken.data_ptr(), s)
        if st:
            raise WqError(st, "wq_kv_plan")
        return p
    return _run(launch, at, stream)


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 interleaved: bool = False, factor: float = 1.0, q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head and their rotation by position:
        y = rmsnorm(x) * weight                                (norm False: x)
        (y_i, y_j) -> factor * (y_i cos a - y_j sin a, y_j cos a + y_i sin a),
    a = positions[t] * inv_freq[i]; j = i + pairs, or, interleaved, values 2 i
    and 2 i + 1. q [T, heads, head_dim] and k [T, kv_heads, head_dim] fp32 with rows
    of any 16-byte stride (k None: no keys); positions int32 [T] (rows with a
    negative one are not written); inv_freq fp32 [pairs], pairs a multiple of 4 and
    at most head_dim / 2 (fewer: the values from 2 pairs on are normed only);
    weights fp32 [head_dim] (None: 1). Returns (q_out, k_out); they may be q and
    k themselves, and must not alias other inputs."""
    T, H, D, qs = _heads(q, "q")
    at = q.get_device()
    Hk, ks, pk = 0, 0, None
    if k is not None:
        Tk, Hk, Dk, ks = _heads(k, "k", at)
        _need(Tk == T and Dk == D, "k must be [T, kv_heads, head_dim] for q's T and head_dim")
        pk = k.data_ptr()
    _need(k is not None or (k_weight is None and k_out is None), "k_weight and k_out need k")
    _need(norm or (q_weight is None and k_weight is None), "weights need the norm")
    ppos = _index(positions, (T,), "positions", at)
    if not (isinstance(inv_freq, _Tensor) and inv_freq.dim() == 1):
        raise ValueError("inv_freq must be [pairs]")
    pairs = inv_freq.shape[0]
    pfreq = _rows(inv_freq, (pairs,), "inv_freq", at)
    pqw, pkw = _rows(q_weight, (D,), "q_weight", at), _rows(k_weight, (D,), "k_weight", at)

    def launch(s):
        yq, yqs = _out_heads(q_out, q, (T, H, D), at, "q_out")
        yk, yks = (None, 0) if k is None else _out_heads(k_out, k, (T, Hk, D), at, "k_out")
        st = load().wq_qk_norm_rope(q.data_ptr(), qs, H, pk, ks, Hk, D, T, ppos, pfreq, pairs, interleaved, factor, norm,
                                    pqw, pkw, eps, yq.data_ptr(), yqs, None if yk is None else yk.data_ptr(), yks, s)
        if st:
            raise WqError(st, "wq_qk_norm_rope")
        return yq, yk
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
