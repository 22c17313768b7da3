"""Cases of the operators that a serving step needs around the int4 key/value
cache: norms and rotation of queries and keys, the plan of a step (block tables,
positions, slots), attention through a sliding window with first tokens that
stay visible, and single-token attention of a batch that shares a prefix.

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
        # one token of a transcript, far into it: a call whose latency counts
        dict(name="rotate_step", op="rotate", tokens=1, heads=16, kv=8, dim=128, pairs=64, inter=False, far=40000, mix=0),
        # a long prompt's queries and keys
        dict(name="rotate_prompt", op="rotate", tokens=8192, heads=16, kv=8, dim=128, pairs=64, inter=False, far=0, mix=0),
        # packed prompts, small heads, a quarter of each rotated, neighbours paired
        dict(name="rotate_part", op="rotate", tokens=1003, heads=14, kv=2, dim=64, pairs=8, inter=True, far=131072, mix=5),
        # one decode step of a full batch: a token each, a page now and then
        dict(name="plan_step", op="plan", count=64, total=64, before=262139, short=False, mix=3),
        # prompts of different lengths arrive together
        dict(name="plan_prompts", op="plan", count=24, total=65521, before=0, short=False, mix=7),
        # eleven minutes of audio; each token sees about eighty seconds
        dict(name="window_prompt", op="wprompt", count=1, total=8192, heads=16, kv=8, dim=128, window=1024, sinks=4, mix=0),
        # a batch of packed prompts, some shorter than the window; small heads in wide groups
        dict(name="window_packed", op="wprompt", count=13, total=5003, heads=14, kv=2, dim=64, window=300, sinks=1, mix=5),
        # one transcript that has grown very long
        dict(name="window_one", op="wdecode", count=1, total=131072, heads=16, kv=8, dim=128, window=4096, sinks=4, mix=0),
        # a full serving batch, lengths of all sizes, wide groups
        dict(name="window_batch", op="wdecode", count=64, total=262139, heads=32, kv=8, dim=128, window=2048, sinks=64, mix=7),
        # a few requests behind one short instruction
        dict(name="shared_few", op="shared", count=5, total=1001, prefix=777, heads=16, kv=8, dim=128, mix=2),
        # many questions about one long transcript
        dict(name="shared_batch", op="shared", count=64, total=16384, prefix=32768, heads=16, kv=8, dim=128, mix=4),
        # small heads in wide groups, an odd prefix, more rows than fit one workgroup
        dict(name="shared_wide", op="shared", count=75, total=40009, prefix=8191, heads=14, kv=2, dim=64, mix=6),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rotate", "plan", "wprompt", "wprompt", "wdecode", "wdecode", "shared", "shared"])
    mix = rng.randrange(1, 1 << 20)
    if op == "plan":
        count = _spread(rng, 1, 512)
        step = rng.random() < 0.5
        total = count if step else max(count, _spread(rng, 16, 65521))
        before = _spread(rng, 64, 262139) if step or rng.random() < 0.5 else 0
        return dict(op=op, count=count, total=total, before=before, short=rng.random() < 0.2, mix=mix)
    heads, kv, dim = rng.choice(LAYOUTS)
    if op == "rotate":
        pairs = rng.choice([dim // 2, dim // 2, dim // 4, dim // 8])
        most = 8192 * 24 * 128 // ((heads + kv) * dim)
        return dict(op=op, tokens=_spread(rng, 1, min(8192, most)), heads=heads, kv=kv, dim=dim, pairs=pairs,
                    inter=rng.random() < 0.4, far=rng.choice([0, 500, 131072, 1000003]), mix=mix)
    window = _spread(rng, 1, 4096)
    sinks = rng.choice([0, 1, 4, 5, 64, 130])
    if op == "wprompt":
        total = _spread(rng, 16, 4096)
        count = min(_spread(rng, 1, 24), total)
        return dict(op=op, count=count, total=total, heads=heads, kv=kv, dim=dim, window=window, sinks=sinks, mix=mix)
    if op == "wdecode":
        count = _spread(rng, 1, 96)
        total = max(count, _spread(rng, 48, 262139))
        return dict(op=op, count=count, total=total, heads=heads, kv=kv, dim=dim, window=window, sinks=sinks, mix=mix)
    count = _spread(rng, 1, 96)
    total = max(count, _spread(rng, 48, 40009))
    prefix = _spread(rng, 16, max(16, min(32768, (32768 * 64 * 16) // (count * heads))))
    return dict(op=op, count=count, total=total, prefix=prefix, heads=heads, kv=kv, dim=dim, mix=mix)


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


def _before(case):
    """Tokens in the cache before a step."""
    n, total = case["count"], case["before"]
    if total < n:
        return [0] * n
    return _lens(dict(count=n, total=total, mix=case["mix"] + 1))


def _need(lens):
    return [-(-n // PAGE) for n in lens]


def _pairs_seen(n, window, sinks):
    """Key/query pairs of a prompt of n tokens."""
    t = np.arange(n, dtype=np.int64)
    near = np.minimum(t + 1, window)
    return int((near + np.minimum(sinks, t + 1 - near)).sum())


def work(case):
    op = case["op"]
    if op == "rotate":
        rows = case["tokens"] * (case["heads"] + case["kv"])
        return {"bytes": 8 * rows * case["dim"] + 4 * case["tokens"], "flops": 10 * rows * case["dim"]}
    if op == "plan":
        lens, before = _lens(case), _before(case)
        pages = sum(_need([a + b for a, b in zip(lens, before)])) - sum(_need(before))
        return {"bytes": 12 * case["total"] + 16 * case["count"] + 8 * pages, "flops": 4 * case["total"]}
    h, kv, d, t = case["heads"], case["kv"], case["dim"], case["total"]
    packed = kv * (d // 2 + d // 16)             # codes and scales of one token, keys or values
    if op == "wprompt":
        return {"bytes": 4 * t * d * (2 * h + 2 * kv),
                "flops": sum(4 * d * h * _pairs_seen(n, case["window"], case["sinks"]) for n in _lens(case))}
    if op == "wdecode":
        seen = sum(min(n, case["window"]) + min(case["sinks"], max(0, n - case["window"])) for n in _lens(case))
        return {"bytes": 2 * seen * packed + 8 * case["count"] * h * d, "flops": 4 * seen * h * d}
    rows = case["prefix"] + t
    return {"bytes": 2 * rows * packed + 8 * case["count"] * h * d,
            "flops": 4 * d * h * (case["count"] * case["prefix"] + t)}


# ------------------------------------------------------------------ inputs
def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(lens, g, more=3):
    """Block table of sequences of these lengths over shuffled pages, and the
    pages that are nobody's."""
    need = _need(lens)
    width, total = max(1, max(need)), sum(need) + more
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32).cpu().tolist()
    rows, at = [], 0
    for k in need:
        rows.append(ids[at:at + k] + [0] * (width - k))
        at += k
    return _ints(rows), ids[at:]


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, st = case["op"], {"case": case}
    if op == "plan":
        lens, before = _lens(case), _before(case)
        have, need = _need(before), _need([a + b for a, b in zip(lens, before)])
        grow = sum(need) - sum(have)
        left = max(0, grow - 1 - grow // 3) if case["short"] else grow + 5
        old, free = _pages(before, g, left)
        taken = 7                                # pages that earlier steps took
        st["table"] = torch.full((case["count"], max(1, max(need)) + 1), -1, dtype=torch.int32, device="cuda")
        st["table"][:, :old.shape[1]] = old
        st["free"] = _ints([0] * taken + free)
        st["taken"] = _ints([taken])
        st["new"], st["start"] = _ints(lens), _ints(before)
        return st
    h, kv, d = case["heads"], case["kv"], case["dim"]
    if op == "rotate":
        t, n = case["tokens"], case["pairs"]
        y = _rand(g, t, (h + 2 * kv) * d) * 2.0  # q, k and v are slices of one fused projection's output
        st["q"] = y[:, :h * d].view(t, h, d)
        st["k"] = y[:, h * d:(h + kv) * d].view(t, kv, d)
        if case["mix"]:                          # tokens of several requests, each at its own place
            cuts = torch.randint(0, t, (t // 100 + 1,), generator=g, device="cuda")
            seq = torch.bucketize(torch.arange(t, device="cuda"), cuts.sort().values, right=True)
            base = torch.randint(0, case["far"] + 1, (t // 100 + 2,), generator=g, device="cuda")
            st["positions"] = (base[seq] + torch.arange(t, device="cuda")).to(torch.int32)
        else:
            st["positions"] = torch.arange(case["far"], case["far"] + t, dtype=torch.int32, device="cuda")
        st["inv_freq"] = (1e6 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)).float()
        st["wq"], st["wk"] = 1.0 + 0.2 * _rand(g, d), 1.0 + 0.2 * _rand(g, d)
        st["eps"], st["factor"] = 1e-6, 1.0 if n == d // 2 else 1.125
        return st
    st["scale"] = d ** -0.5
    lens, n, t = _lens(case), case["count"], case["total"]
    shape = torch.exp(0.3 * _rand(g, kv, d))     # keys have channels of different size
    if op == "wprompt":
        y = _rand(g, t, (h + 2 * kv) * d)
        y[:, :h * d] *= 1.5
        y[:, h * d:(h + kv) * d] *= shape.reshape(-1)
        y[:, (h + kv) * d:] *= 0.5
        st["q"] = y[:, :h * d].view(t, h, d)
        st["k"] = y[:, h * d:(h + kv) * d].view(t, kv, d)
        st["v"] = y[:, (h + kv) * d:].view(t, kv, d)
        st["cu"] = _ints([0] + np.cumsum(lens).tolist())
        return st
    more = _need([case["prefix"]])[0] + 3 if op == "shared" else 3
    table, free = _pages(lens, g, more)
    pages = sum(_need(lens)) + more
    ck, sk = _quantize(_rand(g, pages, kv, PAGE, d) * shape[:, None])
    st["kq"], st["ks"] = _nibbles(ck), sk.view(torch.int16)
    del ck
    cv, sv = _quantize(_rand(g, pages, kv, PAGE, d) * 0.5)
    st["vq"], st["vs"] = _nibbles(cv), sv.view(torch.int16)
    del cv
    st["q"] = _rand(g, n, h, d) * 1.5
    st["table"], st["lens"] = table, _ints(lens)
    if op == "shared":
        st["prefix"], st["prefix_len"] = _ints(free[:more - 3]), _ints([case["prefix"]])
    return st


# ------------------------------------------------------------------ plain forms
def _plain_rotate(st):
    d, n = st["case"]["dim"], st["case"]["pairs"]
    a = st["positions"].double()[:, None] * st["inv_freq"].double()
    c, s = ((f(a) * st["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w
        if st["case"]["inter"]:
            p, r = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
            turned = torch.stack((p * c - r * s, r * c + p * s), -1).flatten(-2)
        else:
            p, r = y[..., :n], y[..., n:2 * n]
            turned = torch.cat((p * c - r * s, r * c + p * s), -1)
        out.append(torch.cat((turned, y[..., 2 * n:]), -1) if 2 * n < d else turned)
    return out


def _plain_plan(st):
    new, start, table, free = st["new"], st["start"], st["table"], st["free"]
    t, width = st["case"]["total"], table.shape[1]
    cu = torch.cat((torch.zeros(1, dtype=torch.int64, device=new.device), new.cumsum(0)))
    lens = start + new
    have = ((start + PAGE - 1) // PAGE).clamp(max=width)
    grow = ((lens + PAGE - 1) // PAGE).clamp(max=width) - have
    base = grow.cumsum(0) - grow
    col = torch.arange(width, device=new.device)
    nth = col - have[:, None]
    at = st["taken"] + base[:, None] + nth
    got = torch.where(at < free.shape[0], free[at.clamp(0, max(free.shape[0] - 1, 0))], -1)
    table.copy_(torch.where((nth >= 0) & (nth < grow[:, None]), got, table))
    row = torch.arange(t, device=new.device)
    b = torch.bucketize(row, cu[1:], right=True)
    live = b < new.shape[0]
    b = b.clamp(max=new.shape[0] - 1)
    pos = start[b] + row - cu[b]
    page = table[b, (pos // PAGE).clamp(max=width - 1)].long()
    there = live & (pos < width * PAGE) & (page >= 0)
    slots = torch.where(there, page * PAGE + pos % PAGE, -1)
    pos = torch.where(live, pos, -1)
    return [table, cu.to(torch.int32), lens, pos.to(torch.int32), slots, st["taken"] + grow.sum().to(torch.int32)]


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l == 0, 1.0, l)


def _plain_wprompt(st):
    q, k, v, cu = st["q"], st["k"], st["v"], st["cu"]
    t, h, d = q.shape
    kv = k.shape[1]
    at = torch.arange(t, device=q.device, dtype=torch.int32)
    seq = torch.bucketize(at, cu, right=True)
    pos = at - cu[(seq - 1).clamp(min=0)]
    mask = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
    mask &= (at[:, None] - at[None, :] < st["case"]["window"]) | (pos[None, :] < st["case"]["sinks"])
    qh = q.transpose(0, 1).reshape(kv, (h // kv) * t, d)
    s = torch.matmul(qh, k.permute(1, 2, 0).contiguous()).view(h, t, t) * st["scale"]
    p = _softmax(s.masked_fill_(~mask, float("-inf")))
    o = torch.matmul(p.view(kv, (h // kv) * t, t), v.transpose(0, 1).contiguous())
    return o.view(h, t, d).transpose(0, 1).contiguous()


def _cached(st, x, page, row):
    """Values of cache rows: [n, kv, m, d] for pages and rows [n, m]."""
    return _values(st[x + "q"][page, :, row], st[x + "s"][page, :, row]).transpose(1, 2)


def _plain_wdecode(st):
    q, lens = st["q"], st["lens"].long()
    n, h, d = q.shape
    kv, width = st["kq"].shape[1], st["table"].shape[1] * PAGE
    window, sinks = min(st["case"]["window"], width), min(st["case"]["sinks"], width)
    low = (lens - window).clamp(min=0)[:, None]
    first = torch.arange(sinks, device=q.device).expand(n, -1)
    last = low + torch.arange(window, device=q.device)
    at = torch.cat((first, last), 1)
    live = torch.cat((first < low, last < lens[:, None]), 1)
    at = at.clamp(max=width - 1)
    page = st["table"].long().gather(1, at // PAGE)
    keys, vals = (_cached(st, x, page, at % PAGE) for x in ("k", "v"))
    qh = q.view(n, kv, h // kv, d)
    s = torch.matmul(qh, keys.transpose(2, 3).contiguous()) * st["scale"]
    p = _softmax(s.masked_fill(~live[:, None, None], float("-inf")))
    return torch.matmul(p, vals.contiguous()).view(n, h, d)


def _plain_shared(st):
    q, lens, size = st["q"], st["lens"], st["case"]["prefix"]
    n, h, d = q.shape
    kv = st["kq"].shape[1]
    # the prefix once, for all queries of a head at once
    at = torch.arange(st["prefix"].shape[0] * PAGE, device=q.device)[None]
    pk, pv = (_cached(st, x, st["prefix"].long()[at // PAGE], at % PAGE)[0].contiguous() for x in ("k", "v"))
    qt = q.view(n, kv, h // kv, d).transpose(0, 1).reshape(kv, -1, d)
    sp = torch.matmul(qt, pk.transpose(1, 2).contiguous()) * st["scale"]
    sp = sp.masked_fill(at[0] >= st["prefix_len"], float("-inf")).view(kv, n, h // kv, -1)
    # then each one's own rows
    own_at = torch.arange(st["table"].shape[1] * PAGE, device=q.device).expand(n, -1)
    page = st["table"].long().gather(1, own_at // PAGE)
    ok, ov = (_cached(st, x, page, own_at % PAGE).contiguous() for x in ("k", "v"))
    so = torch.matmul(q.view(n, kv, h // kv, d), ok.transpose(2, 3).contiguous()) * st["scale"]
    so = so.masked_fill((own_at >= lens[:, None])[:, None, None], float("-inf"))
    p = _softmax(torch.cat((sp.transpose(0, 1), so), -1))
    pp = p[..., :at.shape[1]].transpose(0, 1).reshape(kv, n * (h // kv), -1)
    o = torch.matmul(pp, pv).view(kv, n, h // kv, d).transpose(0, 1)
    return (o + torch.matmul(p[..., at.shape[1]:].contiguous(), ov)).reshape(n, h, d)


# ------------------------------------------------------------------ one pass
def run(state):
    st = state
    case = st["case"]
    op = case["op"]
    if own:
        import weight_only_bit_block_amd as wqa
        if op == "rotate":
            return list(wqa.qk_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], q_weight=st["wq"], k_weight=st["wk"],
                                         eps=st["eps"], interleaved=case["inter"], factor=st["factor"]))
        if op == "plan":
            p = wqa.kv_plan(st["new"], st["table"], st["free"], st["taken"], tokens=case["total"], start=st["start"])
            return [st["table"], p.cu, p.lens, p.positions, p.slots, p.taken]
        if op == "wprompt":
            return wqa.attn_prefill(st["q"], st["k"], st["v"], cu=st["cu"], scale=st["scale"], window=case["window"],
                                    sinks=case["sinks"])
        cache = wqa.KVCache(st["kq"], st["ks"], st["vq"], st["vs"])
        if op == "wdecode":
            return wqa.attn_decode(st["q"], cache, st["table"], st["lens"], scale=st["scale"], window=case["window"],
                                   sinks=case["sinks"])
        return wqa.attn_decode_shared(st["q"], cache, st["prefix"], st["prefix_len"], st["table"], st["lens"],
                                      scale=st["scale"])
    return {"rotate": _plain_rotate, "plan": _plain_plan, "wprompt": _plain_wprompt, "wdecode": _plain_wdecode,
            "shared": _plain_shared}[op](st)


# ------------------------------------------------------------------ in 64 bits
def _attend(q, k, v, scale, seen=None):
    """Softmax attention of rows q over keys k, in float64."""
    s = q.double() @ k.t().contiguous() * scale
    if seen is not None:
        s[~seen] = float("-inf")
    e = torch.exp(s - s.max(dim=-1, keepdim=True).values)
    return e @ v / e.sum(dim=-1, keepdim=True)


def _rows64(st, x, ids, j):
    """All rows of head j in these pages, as float64."""
    b = st[x + "q"][ids, j].to(torch.int64)
    c = torch.empty(b.shape[:-1] + (2 * b.shape[-1],), dtype=torch.float64, device=b.device)
    c[..., 0::2] = (b % 16).double()
    c[..., 1::2] = torch.div(b, 16, rounding_mode="floor").double()
    c = torch.where(c >= 8, c - 16, c)
    s = st[x + "s"][ids, j].view(torch.float16).double().repeat_interleave(BLOCK, -1)
    return (c * s).reshape(-1, c.shape[-1])


def _exact_plan(st, case):
    new, start, free = (st[x].cpu().tolist() for x in ("new", "start", "free"))
    table, at = st["table"].cpu().numpy().copy(), int(st["taken"][0])
    positions, slots, cu = np.full(case["total"], -1, np.int32), np.full(case["total"], -1, np.int64), [0]
    for b, (n, s) in enumerate(zip(new, start)):
        for page in range(-(-s // PAGE), -(-(s + n) // PAGE)):
            if page < table.shape[1]:
                table[b, page] = free[at] if at < len(free) else -1
                at += 1
        p = np.arange(s, s + n)
        here = np.array([table[b, x // PAGE] for x in p.tolist()], np.int64)
        positions[cu[-1]:cu[-1] + n] = p
        slots[cu[-1]:cu[-1] + n] = np.where(here >= 0, here * PAGE + p % PAGE, -1)
        cu.append(cu[-1] + n)
    lens = np.array([a + b for a, b in zip(new, start)], np.int32)
    return [table, np.array(cu, np.int32), lens, positions, slots, np.array([at], np.int32)]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(st, case)
    if op == "rotate":
        n, out = case["pairs"], []
        turn = torch.polar(torch.full((), st["factor"], dtype=torch.float64, device="cuda"),
                           torch.outer(st["positions"].double(), st["inv_freq"].double()))[:, None]
        for x, w in (("q", "wq"), ("k", "wk")):
            y = st[x].double()
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + st["eps"]) * st[w].double()
            re, im = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["inter"] else (slice(0, n), slice(n, 2 * n))
            z = torch.complex(y[..., re].contiguous(), y[..., im].contiguous()) * turn
            y[..., re], y[..., im] = z.real, z.imag
            out.append(y)
        return out
    lens, group = _lens(case), case["heads"] // case["kv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if op == "wprompt":
        first = 0
        for n in lens:
            here = slice(first, first + n)
            first += n
            if n == 0:
                continue
            t = torch.arange(n, device="cuda")
            seen = (t[:, None] >= t) & ((t > t[:, None] - case["window"]) | (t < case["sinks"]))
            for j in range(case["heads"]):
                out[here, j] = _attend(st["q"][here, j], st["k"][here, j // group].double(), st["v"][here, j // group].double(),
                                       st["scale"], seen)
        return out
    for j in range(case["kv"]):
        mine = slice(j * group, (j + 1) * group)
        shared = [_rows64(st, x, st["prefix"].long(), j)[:case["prefix"]] for x in "kv"] if op == "shared" else None
        for b, n in enumerate(lens):
            k, v = (_rows64(st, x, st["table"][b, :-(-n // PAGE)].long(), j)[:n] for x in "kv")
            if op == "shared":
                k, v = torch.cat((shared[0], k)), torch.cat((shared[1], v))
            elif n > case["window"]:
                t = torch.arange(n, device="cuda")
                keep = (t >= n - case["window"]) | (t < case["sinks"])
                k, v = k[keep], v[keep]
            if len(k):
                out[b, mine] = _attend(st["q"][b, mine], k, v, st["scale"])
    return out
