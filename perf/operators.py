"""Cases of the operators around the packed projections of a decoder: attention
over a whole prompt, the int4 key/value cache (append and single-token
attention), and the residual norms.

`run` computes a case in elementary torch operations where `own` is false and
through the library's entry points where it is true; `exact` states the same
operators in 64 bits.
"""
import random

import numpy as np
import torch

own = False

PAGE = 64           # tokens per cache page
BLOCK = 32          # values per quantization block

# (query heads, key/value heads, head size): the decoder's own layout first,
# then plain multi-head, wider groups, one shared head and the smaller head.
LAYOUTS = [(16, 8, 128), (8, 8, 128), (32, 8, 128), (16, 2, 128), (12, 1, 128), (16, 8, 64), (14, 2, 64)]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the prompt signature of 128 tokens, one layer: a call whose latency counts
        dict(name="prompt_128", op="prompt", count=1, total=128, heads=16, kv=8, dim=128, mix=0),
        # the prompt signature of 1024 tokens, one layer
        dict(name="prompt_1024", op="prompt", count=1, total=1024, heads=16, kv=8, dim=128, mix=0),
        # eleven minutes of audio in one prompt
        dict(name="prompt_8192", op="prompt", count=1, total=8192, heads=16, kv=8, dim=128, mix=0),
        # a serving batch of prompts of different lengths, packed; small heads in wide groups
        dict(name="prompt_packed", op="prompt", count=13, total=5003, heads=14, kv=2, dim=64, mix=5),
        # a prompt's keys and values go into the cache
        dict(name="append_prompt", op="append", count=1, total=4096, heads=16, kv=8, dim=128, mix=0),
        # one decode step of a batch: one row per sequence, each at its own length
        dict(name="append_step", op="append", count=48, total=48, heads=16, kv=8, dim=128, mix=3),
        # one transcript being decoded: one short row
        dict(name="decode_one", op="decode", count=1, total=777, heads=16, kv=8, dim=128, mix=0),
        # one very long context, where the split over its length has to fill the card
        dict(name="decode_long", op="decode", count=1, total=131072, heads=16, kv=8, dim=128, mix=0),
        # a full serving batch, lengths of all sizes, wide groups
        dict(name="decode_batch", op="decode", count=64, total=262139, heads=32, kv=8, dim=128, mix=7),
        # between two blocks of one decode step
        dict(name="norm_step", op="norm", rows=1, cols=1024, gate="row", post=True, pre=True),
        # between two blocks of a long prefill
        dict(name="norm_prefill", op="norm", rows=4096, cols=1024, gate="all", post=True, pre=True),
        # an odd width that fills no vector, without gate
        dict(name="norm_odd", op="norm", rows=515, cols=5003, gate="none", post=False, pre=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "decode", "decode", "norm"])
    if op == "norm":
        cols = _spread(rng, 64, 16384)
        rows = _spread(rng, 1, max(1, min(8192, (4096 * 1024) // cols)))
        return dict(op=op, rows=rows, cols=cols, gate=rng.choice(["none", "row", "all"]), post=rng.random() < 0.6,
                    pre=rng.random() < 0.8)
    heads, kv, dim = rng.choice(LAYOUTS)
    mix = rng.randrange(1, 1 << 20)
    if op == "prompt":
        total = _spread(rng, 16, 4096)
        count = min(_spread(rng, 1, 24), total)
        return dict(op=op, count=count, total=total, heads=heads, kv=kv, dim=dim, mix=mix)
    if op == "append":
        total = _spread(rng, 1, 4096)
        count = total if rng.random() < 0.4 and total <= 256 else min(_spread(rng, 1, 16), total)
        return dict(op=op, count=count, total=total, heads=heads, kv=kv, dim=dim, mix=mix)
    count = _spread(rng, 1, 96)
    total = max(count, _spread(rng, 48, 262139))
    return dict(op=op, count=count, total=total, heads=heads, kv=kv, dim=dim, mix=mix)


def _lens(case):
    """`count` lengths that add up to `total`: even parts where mix is 0, else
    spread, with an empty sequence among them where there are ten or more."""
    n, total = case["count"], case["total"]
    if n == 1:
        return [total]
    if n == total:
        return [1] * n
    r = random.Random(case["mix"])
    w = [np.exp(1.2 * r.gauss(0.0, 1.0)) for _ in range(n)]
    lens = [1 + int((total - n) * x / sum(w)) for x in w]
    if n >= 10:
        lens[r.randrange(n)] = 0
    lens[int(np.argmax(lens))] += total - sum(lens)
    return lens


def _starts(case):
    """Tokens already in the cache before an append."""
    r = random.Random(case["mix"] + 1)
    return [r.randrange(0, 300) if case["mix"] else 0 for _ in range(case["count"])]


def work(case):
    if case["op"] == "norm":
        m, n = case["rows"], case["cols"]
        elems = 2 * m * n + (m * n if case["pre"] else 0) + m * n
        elems += {"none": 0, "row": n, "all": m * n}[case["gate"]] + (n if case["post"] else 0) + (n if case["pre"] else 0)
        return {"bytes": 4 * elems, "flops": 10 * m * n}
    h, kv, d, t = case["heads"], case["kv"], case["dim"], case["total"]
    packed = kv * (d // 2 + d // 16)             # codes and scales of one token, keys or values
    if case["op"] == "prompt":
        return {"bytes": 4 * t * d * (2 * h + 2 * kv), "flops": sum(2 * d * h * n * (n + 1) for n in _lens(case))}
    if case["op"] == "append":                   # rows in, packed rows out; their values come back
        return {"bytes": 2 * t * (4 * kv * d + packed) + 2 * t * (4 * kv * d + packed), "flops": 6 * t * kv * d}
    return {"bytes": 2 * t * packed + 8 * case["count"] * h * d, "flops": 4 * t * h * d}


# ------------------------------------------------------------------ inputs
def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pages(lens, g):
    """Block table of sequences of these lengths over shuffled pages, and the
    number of pages (a few are nobody's)."""
    need = [-(-n // PAGE) for n in lens]
    width, total = max(1, max(need)), sum(need) + 3
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu().tolist()
    rows, at = [], 0
    for k in need:
        rows.append(ids[at:at + k] + [0] * (width - k))
        at += k
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), total


def _quantize(x):
    """Block-32 int4 of x [..., D]: codes as whole numbers, scales in binary16."""
    b = x.unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1).double() / 7).float().half()
    d = s.double()[..., None]
    c = torch.where(d == 0, 0.0, (b.double() / torch.where(d == 0, 1.0, d)).float().round()).clamp(-8, 7)
    return c.to(torch.int32).flatten(-2), s


def _nibbles(c):
    c = c & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _values(q, s):
    """Values of packed rows q [..., D/2] with scales s [..., D/32] (binary16 bits)."""
    u = q.to(torch.int32)
    c = torch.stack((u & 15, u >> 4), -1).flatten(-2)
    c = ((c ^ 8) - 8).float()
    return (c.unflatten(-1, (-1, BLOCK)) * s.view(torch.float16).float()[..., None]).flatten(-2)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "norm":
        m, n = case["rows"], case["cols"]
        st["h"] = _rand(g, m, n) * 3.0
        st["y"] = _rand(g, m, n) * torch.exp(0.5 * _rand(g, m, 1))
        st["post"] = 1.0 + 0.2 * _rand(g, n) if case["post"] else None
        st["pre"] = 1.0 + 0.2 * _rand(g, n) if case["pre"] else None
        st["gate"] = {"none": None, "row": 0.5 * _rand(g, n), "all": 0.5 * _rand(g, m, n) if case["gate"] == "all" else None}[case["gate"]]
        st["alpha"], st["eps"] = 0.75, 1e-6
        return st
    h, kv, d, t, n = case["heads"], case["kv"], case["dim"], case["total"], case["count"]
    st["scale"] = d ** -0.5
    lens = _lens(case)
    shape = torch.exp(0.3 * _rand(g, kv, d))      # keys have channels of different size
    if case["op"] == "decode":
        table, pages = _pages(lens, g)
        ck, sk = _quantize(_rand(g, pages, kv, PAGE, d) * shape[:, None])
        st["kq"], st["ks"] = _nibbles(ck), sk.view(torch.int16)
        del ck
        cv, sv = _quantize(_rand(g, pages, kv, PAGE, d) * 0.5)
        st["vq"], st["vs"] = _nibbles(cv), sv.view(torch.int16)
        del cv
        st["q"] = _rand(g, n, h, d) * 1.5
        st["table"], st["lens"] = table, _ints(lens)
        return st
    # q, k and v are slices of one fused projection's output
    y = _rand(g, t, (h + 2 * kv) * d)
    y[:, :h * d] *= 1.5
    y[:, h * d:(h + kv) * d] *= shape.reshape(-1)
    y[:, (h + kv) * d:] *= 0.5
    st["q"] = y[:, :h * d].view(t, h, d)
    st["k"] = y[:, h * d:(h + kv) * d].view(t, kv, d)
    st["v"] = y[:, (h + kv) * d:].view(t, kv, d)
    st["cu"] = _ints([0] + np.cumsum(lens).tolist())
    if case["op"] == "append":
        starts = _starts(case)
        st["table"], pages = _pages([a + b for a, b in zip(starts, lens)], g)
        st["start"] = _ints(starts)
        for x in ("k", "v"):
            st[x + "q"] = torch.zeros(pages, kv, PAGE, d // 2, dtype=torch.uint8, device="cuda")
            st[x + "s"] = torch.zeros(pages, kv, PAGE, d // BLOCK, dtype=torch.int16, device="cuda")
        # the cache rows of the appended tokens, [token][head]
        rows = []
        table = st["table"].cpu().numpy()
        for b, (a, c) in enumerate(zip(starts, lens)):
            p = np.arange(a, a + c)
            rows.append((table[b, p // PAGE][:, None] * kv + np.arange(kv)) * PAGE + (p % PAGE)[:, None])
        st["rows"] = torch.from_numpy(np.concatenate(rows).reshape(-1).astype(np.int32)).cuda()
    return st


# ------------------------------------------------------------------ plain forms
def _plain_prompt(q, k, v, cu, scale):
    t, h, d = q.shape
    kv = k.shape[1]
    at = torch.arange(t, device=q.device, dtype=torch.int32)
    seq = torch.bucketize(at, cu, right=True)
    mask = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
    qh = q.transpose(0, 1).reshape(kv, (h // kv) * t, d)
    s = torch.matmul(qh, k.permute(1, 2, 0).contiguous()).view(h, t, t) * scale
    s = s.masked_fill_(~mask, float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(kv, (h // kv) * t, t), v.transpose(0, 1).contiguous())
    return o.view(h, t, d).transpose(0, 1).contiguous()


def _plain_append(st):
    out = []
    rows = st["rows"].long()
    for x in ("k", "v"):
        c, s = _quantize(st[x].flatten(0, 1))
        q, z = st[x + "q"].flatten(0, 2), st[x + "s"].flatten(0, 2)
        q[rows] = _nibbles(c)
        z[rows] = s.view(torch.int16)
        out.append(_values(q[rows], z[rows]))
    return out


def _plain_decode(q, kq, ks, vq, vs, table, lens, scale):
    n, h, d = q.shape
    kv = kq.shape[1]
    at = table.long()

    def rows(codes, scales):                     # [n * kv, tokens, d]
        x = _values(codes[at], scales[at])       # [n, pages, kv, PAGE, d]
        return x.transpose(1, 2).reshape(n * kv, -1, d)

    qt = q.view(n * kv, h // kv, d).transpose(1, 2).contiguous()
    s = torch.matmul(rows(kq, ks), qt).transpose(1, 2) * scale       # [n * kv, group, tokens]
    s = s.contiguous().view(n, h, -1)
    dead = torch.arange(s.shape[-1], device=q.device)[None, None, :] >= lens[:, None, None]
    s = s.masked_fill(dead, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, 1.0, l)
    return torch.matmul(p.view(n * kv, h // kv, -1), rows(vq, vs)).view(n, h, d)


def _plain_norm(st):
    t = st["y"]
    if st["post"] is not None:
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + st["eps"]) * st["post"]
    if st["gate"] is not None:
        t = t * st["gate"]
    h = st["h"] + st["alpha"] * t
    if st["pre"] is None:
        return [h]
    return [h, h * torch.rsqrt(h.square().mean(-1, keepdim=True) + st["eps"]) * st["pre"]]


# ------------------------------------------------------------------ one pass
def run(state):
    st = state
    op = st["case"]["op"]
    if own:
        import weight_only_bit_block_amd as wqa
        if op == "prompt":
            return wqa.attn_prefill(st["q"], st["k"], st["v"], cu=st["cu"], scale=st["scale"])
        if op == "norm":
            h, x = wqa.residual_norm(st["h"], st["y"], post_weight=st["post"], gate=st["gate"], alpha=st["alpha"],
                                     pre_weight=st["pre"], eps=st["eps"])
            return [h] if x is None else [h, x]
        cache = wqa.KVCache(st["kq"], st["ks"], st["vq"], st["vs"])
        if op == "decode":
            return wqa.attn_decode(st["q"], cache, st["table"], st["lens"], scale=st["scale"])
        wqa.kv_append(cache, st["k"], st["v"], st["table"], cu=st["cu"], start=st["start"])
        d = st["case"]["dim"]
        return [wqa.embed(st["rows"], st[x + "q"].view(-1, d // 2), st[x + "s"].view(-1, d // BLOCK), d, 4)
                for x in ("k", "v")]
    if op == "prompt":
        return _plain_prompt(st["q"], st["k"], st["v"], st["cu"], st["scale"])
    if op == "append":
        return _plain_append(st)
    if op == "decode":
        return _plain_decode(st["q"], st["kq"], st["ks"], st["vq"], st["vs"], st["table"], st["lens"], st["scale"])
    return _plain_norm(st)


# ------------------------------------------------------------------ in 64 bits
def _softmax_rows(s):
    e = torch.exp(s - s.max(dim=-1, keepdim=True).values)
    return e / e.sum(dim=-1, keepdim=True)


def _signed(byte_rows):
    """Two's complement codes of packed rows, as float64."""
    low = byte_rows.to(torch.int64) % 16
    high = torch.div(byte_rows.to(torch.int64), 16, rounding_mode="floor")
    both = torch.empty(byte_rows.shape[:-1] + (2 * byte_rows.shape[-1],), dtype=torch.float64, device=byte_rows.device)
    both[..., 0::2] = low.double()
    both[..., 1::2] = high.double()
    return torch.where(both >= 8, both - 16, both)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        y, h = st["y"].double(), st["h"].double()
        if st["post"] is not None:
            y = st["post"].double() * y / torch.sqrt((y * y).sum(1, keepdim=True) / case["cols"] + st["eps"])
        gate = 1.0 if st["gate"] is None else st["gate"].double()
        h = h + st["alpha"] * gate * y
        if st["pre"] is None:
            return [h]
        return [h, st["pre"].double() * h / torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + st["eps"])]
    lens, group, d = _lens(case), case["heads"] // case["kv"], case["dim"]
    if op == "append":
        out = []
        for x in ("k", "v"):
            w = st[x].cpu().numpy().reshape(-1, d // BLOCK, BLOCK)
            s = (np.abs(w).max(-1) / np.float32(7)).astype(np.float16)
            sf = s.astype(np.float32)[..., None]
            c = np.where(sf == 0, np.float32(0), np.rint(w / np.where(sf == 0, np.float32(1), sf)))
            out.append((np.clip(c, -8, 7).astype(np.float64) * s.astype(np.float64)[..., None]).reshape(-1, d))
        return out
    if op == "prompt":
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for n in lens:
            here = slice(at, at + n)
            at += n
            if n == 0:
                continue
            later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            for j in range(case["heads"]):
                s = st["q"][here, j].double() @ st["k"][here, j // group].double().t().contiguous() * st["scale"]
                s[later] = float("-inf")
                out[here, j] = _softmax_rows(s) @ st["v"][here, j // group].double()
        return out
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = st["table"][b, :-(-n // PAGE)].long()
        for j in range(case["kv"]):
            rows = []
            for x in ("k", "v"):
                sc = st[x + "s"][ids, j].view(torch.float16).double().repeat_interleave(BLOCK, -1)
                rows.append((_signed(st[x + "q"][ids, j]) * sc).reshape(-1, d)[:n])
            mine = slice(j * group, (j + 1) * group)
            s = st["q"][b, mine].double() @ rows[0].t().contiguous() * st["scale"]
            out[b, mine] = _softmax_rows(s) @ rows[1]
    return out
