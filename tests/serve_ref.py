"""Plain 64-bit forms of the operators of a serving step (numpy), and the error
bounds the GPU tests hold the kernels to (attention's: tests/layer_ref.py)."""
import numpy as np

from tests.layer_ref import PAGE, U32, _attend

TILE = 32                   # keys of a prompt that are normalised together


# ------------------------------------------------------------------ norms and rotation
def rope(x, positions, inv_freq, weight, eps, norm, interleaved, factor):
    """Heads x [T, heads, D] normed and rotated, and each value's error bound.

    Norm: the sum of D squares takes 8 roundings of half a step on the way to a
    value (4 in the lane, 4 over lanes), half of that after the root; eps, root,
    reciprocal and the products with it and the weight 4.5 more: below 10 halves.
    A rotated value takes those of both sides (at most sqrt 2 of the larger: 14),
    for each side the sine's or cosine's (half a step of the turn, pi / 2 of
    2^-24, and 2 steps of the function, 4 of 2^-24: 12 for both), and two products
    and a factor: below 28 in all. The angle itself is off by 2^-53, taken 4 times.
    """
    y = x.astype(np.float64)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps)))
        if weight is not None:
            y = y * weight.astype(np.float64)
    n = len(inv_freq)
    a = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    c, s = np.cos(a)[:, None] * float(np.float32(factor)), np.sin(a)[:, None] * float(np.float32(factor))
    lim = 28 * U32 * np.abs(y)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    p, r = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = p * c - r * s, r * c + p * s
    big = np.maximum(np.abs(p), np.abs(r)) * abs(float(np.float32(factor)))
    lim[..., i] = lim[..., j] = big * (28 * U32 + 4 * 2.0 ** -53 * np.abs(a)[:, None])
    return y, lim + 1e-44


# ------------------------------------------------------------------ plans
def plan(fresh, start, table, free, taken, tokens):
    """(table, cu, lens, positions, slots, taken) by the definition, one token at a time."""
    table, width, most = table.copy(), table.shape[1], 2 ** 31 - 1
    positions, slots = np.full(tokens, -1, np.int64), np.full(tokens, -1, np.int64)
    cu, lens, t, at = [0], [], 0, taken
    for b, (n, s) in enumerate(zip(fresh, start)):
        if n < 0 or s < 0 or n + s > most:
            lens.append(-1)
            cu.append(min(t, most))
            continue
        for page in range(-(-s // PAGE), min(-(-(s + n) // PAGE), width)):
            table[b, page] = free[at] if 0 <= at < len(free) else -1
            at += 1
        for i in range(min(n, max(0, tokens - t))):
            positions[t + i] = s + i
            page = int(table[b, (s + i) // PAGE]) if (s + i) // PAGE < width else -1
            slots[t + i] = page * PAGE + (s + i) % PAGE if page >= 0 else -1
        t += n
        lens.append(s + n)
        cu.append(min(t, most))
    return table, np.array(cu), np.array(lens), positions, slots, np.array([min(at, most)])


# ------------------------------------------------------------------ attention
def window_prompt(q, k, v, lens, scale, window, sinks):
    """As layer_ref.prompt with a window. The largest value of a row is taken over
    whole tiles of every key it sees: hidden rows of those share their units."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    out, sums = np.full(q.shape, np.nan), np.full((3,) + q.shape, np.nan)
    group, at = q.shape[1] // k.shape[1], 0
    for n in lens:
        t = np.arange(n)
        see = (t[:, None] >= t) & ((t > t[:, None] - window) | (t < sinks))
        tiles = np.add.reduceat(see, np.arange(0, n, TILE), axis=1) > 0 if n else see
        for j in range(q.shape[1]):
            here = slice(at, at + n)
            if n:
                kk, vv = k[here, j // group], v[here, j // group]
                o, pv, first = _attend(q[here, j], kk, vv, scale, see)
                out[here, j] = o
                top = np.array([np.abs(vv[i:i + TILE]).max() for i in range(0, n, TILE)])
                sums[0, here, j], sums[1, here, j] = pv, first
                sums[2, here, j] = np.where(tiles, top, 0).max(1)[:, None]
        at += n
    return out, sums


def seen(n, window, sinks):
    t = np.arange(n)
    return (t >= n - window) | (t < sinks)


def rows_of(vals, scales, ids, j, n):
    d = vals.shape[-1]
    ids = np.asarray(ids, np.int64)[: -(-n // PAGE)]
    return vals[ids, j].reshape(-1, d)[:n], scales[ids, j].astype(np.float64).reshape(-1, d // 32)[:n]


def decode(q, kval, vval, vscale, scale, rows):
    """Single-token attention; rows(b) gives the (table row, length, mask or None)
    parts whose tokens sequence b sees. The largest value of a head is taken as
    16 of its largest scale (layer_ref.decode)."""
    q = q.astype(np.float64)
    out, sums = np.zeros(q.shape), np.zeros((3,) + q.shape)
    kv, d = kval.shape[1], q.shape[2]
    group = q.shape[1] // kv
    for b in range(len(q)):
        parts = [x for x in rows(b) if x[1] > 0]
        if not parts:
            continue
        for j in range(kv):
            kk, vv, sc = [], [], []
            for ids, n, mask in parts:
                mask = np.ones(n, bool) if mask is None else mask
                kk.append(rows_of(kval, vscale, ids, j, n)[0][mask])
                x, s = rows_of(vval, vscale, ids, j, n)
                vv.append(x[mask])
                sc.append(s[mask])
            kk, vv, sc = (np.concatenate(x) for x in (kk, vv, sc))
            mine = slice(j * group, (j + 1) * group)
            o, pv, first = _attend(q[b, mine], kk, vv, scale, np.ones((group, len(kk)), bool))
            out[b, mine] = o
            sums[0, b, mine], sums[1, b, mine], sums[2, b, mine] = pv, first, 16 * float(np.abs(sc).max())
    return out, sums
