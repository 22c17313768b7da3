"""Plain 64-bit forms of the operators between the projections (numpy), and the
error bounds the GPU tests hold the kernels to."""
import numpy as np

PAGE = 64
U32 = 2.0 ** -24            # half a step of fp32, relative


def _attend(q, k, v, scale, visible):
    """One head: q [n, d], k and v [m, d], visible [n, m]. Returns the output,
    sum p |v|, and the largest |logit| operand product |scale| |q| |k|."""
    s = (q @ k.T) * scale
    s = np.where(visible, s, -np.inf)
    top = s.max(1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    p = e / np.where(total == 0, 1.0, total)
    qk = abs(scale) * np.linalg.norm(q, axis=1)[:, None] * np.linalg.norm(k, axis=1)[None, :]
    # what a key's logit error does to the output goes with its weight
    spread = np.where(visible, p, 0.0) * qk
    o = p @ v
    av = np.abs(v)
    first = spread @ av + spread.sum(1, keepdims=True) * (p @ av)
    return o, p @ av, first


def prompt(q, k, v, lens, scale):
    """Causal attention over packed prompts. Returns out, and per output the
    sums its error bound is made of (see prompt_bound)."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    out = np.full(q.shape, np.nan)
    sums = np.full((3,) + q.shape, np.nan)
    group = q.shape[1] // k.shape[1]
    at = 0
    for n in lens:
        see = np.tril(np.ones((n, n), bool))
        for j in range(q.shape[1]):
            here = slice(at, at + n)
            if n:
                kk, vv = k[here, j // group], v[here, j // group]
                o, pv, first = _attend(q[here, j], kk, vv, scale, see)
                out[here, j] = o
                sums[0, here, j] = pv
                sums[1, here, j] = first
                sums[2, here, j] = np.maximum.accumulate(np.abs(vv).max(1))[:, None]
        at += n
    return out, sums


def bound(sums, n, d):
    """Error bound of an attention output over n visible keys of d values.

    Logits: q and k are held in two binary16 parts (2^-22 relative each, and
    2^-22 for the product of the low parts that is left out), 3 d / 16 partial
    sums rounded to fp32 at half a step each, the scale folded into q and the
    subtraction of the running maximum at half a step each, and the exponential
    at 2^-22: (3 2^-22 + (3 d / 16 + 4) 2^-24) |scale| |q| |k|, taken twice for
    the cross terms Cauchy-Schwarz leaves out. Each weight's error moves the
    output by its share of sum p |v| both directly and through the sum: `first`.
    Weights and values: two parts each (3 2^-22), one fp32 rounding per
    partial sum (n 3 / 16 of the product, n / 2 of the weight sum), 8 for the
    normalisation, rescaling and final division; values
    far below the largest one of the head keep an absolute error of 2^-36 of it,
    and every weight one of 2^-37 of the largest: a weight of 1 is held as 2^12
    or more, in parts that go down to 2^-24, off by half of that, so n keys
    may add n 2^-37 of the largest value.
    """
    logit = 2.0 * (3 * 2.0 ** -22 + (3 * d / 16 + 4) * U32)
    value = 3 * 2.0 ** -22 + 2.0 ** -21 + (3 * n / 16 + n / 2 + 8) * U32
    return logit * sums[1] + value * sums[0] + (2.0 ** -36 + n * 2.0 ** -37) * sums[2] + 1e-44


def quantize(x):
    """Block-32 int4 rows of x [..., d]: (codes int8, scales float16), a NaN
    scale where a block is not finite or its scale passes binary16."""
    b = x.astype(np.float32).reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(over="ignore", invalid="ignore"):
        s = (np.abs(b).max(-1) / np.float32(7)).astype(np.float16)
        bad = ~np.isfinite(b).all(-1) | ~np.isfinite(s)
        sf = np.where(bad | (s == 0), np.float16(1), s).astype(np.float32)[..., None]
        c = np.clip(np.rint(b / sf), -8, 7)
    c = np.where((bad | (s == 0))[..., None], 0, c).astype(np.int8)
    return c.reshape(x.shape), np.where(bad, np.float16(np.nan), s)


def nibbles(codes):
    u = codes.astype(np.uint8) & 15
    return u[..., 0::2] | (u[..., 1::2] << 4)


def values(codes, scales):
    """float64 values of codes [..., d] with scales [..., d / 32]."""
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32, -1)


def decode(q, kval, vval, vscale, table, lens, scale):
    """q [b, heads, d], kval and vval [pages, kv, PAGE, d] in float64, vscale the
    scales of vval [pages, kv, PAGE, d / 32]. The largest value of a head is
    taken as 16 of its largest scale: weights times scales are held against the
    power of two above the largest scale (at most twice it), and codes reach 8."""
    q = q.astype(np.float64)
    out = np.zeros(q.shape)
    sums = np.zeros((3,) + q.shape)
    kv = kval.shape[1]
    group = q.shape[1] // kv
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = np.asarray(table[b][: -(-n // PAGE)])
        for j in range(kv):
            kk = kval[ids, j].reshape(-1, q.shape[2])[:n]
            vv = vval[ids, j].reshape(-1, q.shape[2])[:n]
            sc = vscale[ids, j].astype(np.float64).reshape(-1, q.shape[2] // 32)[:n]
            mine = slice(j * group, (j + 1) * group)
            o, pv, first = _attend(q[b, mine], kk, vv, scale, np.ones((group, n), bool))
            out[b, mine] = o
            sums[0, b, mine], sums[1, b, mine], sums[2, b, mine] = pv, first, 16 * float(sc.max())
    return out, sums


def residual_norm(h, y, post, gate, alpha, pre, eps):
    h = h.astype(np.float64)
    if y is not None:
        t = y.astype(np.float64)
        if post is not None:
            t = t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * post
        if gate is not None:
            t = t * gate
        size = np.abs(h) + np.abs(alpha * t)
        h = h + alpha * t
    else:
        size = np.abs(h)
    x = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, size, x if pre is None else x * pre
