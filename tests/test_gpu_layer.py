"""GPU parity of the operators between the projections against their plain
64-bit forms (tests/layer_ref.py, where the error bounds are derived)."""
import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import layer_ref as ref
from tests.gpu_util import note, torch_cuda

pytestmark = pytest.mark.gpu

LAYOUTS = [(16, 8, 128), (4, 4, 64), (14, 2, 64), (12, 1, 128)]
WIDE = [(160, 2, 128), (420, 2, 64)]       # so many heads that short prompts fill the card: the other prompt kernel
NAN = float("nan")


def rng_for(*seed):
    return np.random.Generator(np.random.PCG64(np.random.SeedSequence(list(seed))))


def dev(a):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def qkv(rng, T, heads, kv, d):
    """q, k, v as host arrays and as device slices of one fused row."""
    y = rng.standard_normal((T, (heads + 2 * kv) * d)).astype(np.float32)
    return split(y, heads, kv, d)


def split(y, heads, kv, d):
    T = y.shape[0]
    cut = [heads * d, (heads + kv) * d]
    host = [x.reshape(T, -1, d) for x in np.split(y, cut, axis=1)]
    on = dev(y)
    parts = [on[:, :cut[0]].view(T, heads, d), on[:, cut[0]:cut[1]].view(T, kv, d), on[:, cut[1]:].view(T, kv, d)]
    return host, parts


def cu_of(lens, first=0):
    return dev(np.cumsum([first] + list(lens)).astype(np.int32))


def check_prompt(out, host, lens, scale, first=0, what=""):
    """Rows of the sequences within the bound, all others still NaN."""
    q, k, v = (x[first:] for x in host)
    want, sums = ref.prompt(q, k, v, lens, scale)
    got = out.cpu().numpy().astype(np.float64)
    assert np.isnan(got[:first]).all(), what
    got = got[first:]
    live = ~np.isnan(want)
    assert np.isnan(got[~live]).all(), f"{what}: a row of no sequence was written"
    lim = ref.bound(sums, max(lens, default=0), q.shape[2])
    err = np.abs(got - want)
    assert (err[live] <= lim[live]).all(), f"{what}: worst error / bound {np.nanmax(err / lim):.3f}"


# ------------------------------------------------------------------ prompts
@pytest.mark.parametrize("heads,kv,d", LAYOUTS + WIDE)
@pytest.mark.parametrize("lens", [[1], [2, 31, 32, 33], [0, 64, 0, 0, 65, 1, 0], [127, 128, 129], [300], [1] * 70],
                         ids=lambda x: "-".join(map(str, x[:7])))
def test_prompt_parity(heads, kv, d, lens):
    note(f"prompt {heads} {kv} {d} {lens}")
    torch = torch_cuda()
    T = sum(lens) + 3                                  # three tokens of nobody behind the last sequence
    host, (q, k, v) = qkv(rng_for(1, heads, d, T), T, heads, kv, d)
    out = torch.full((T, heads, d), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, cu=cu_of(lens), out=out)
    check_prompt(out, host, lens, d ** -0.5, what=str(lens))


@pytest.mark.parametrize("T,heads", [(1, 16), (5, 16), (100, 16), (1023, 4), (2049, 4), (700, 60), (700, 100)])
def test_prompt_single(T, heads):
    note(f"prompt single {T} {heads}")
    torch = torch_cuda()
    kv, d = heads // 2, 128
    host, (q, k, v) = qkv(rng_for(2, T), T, heads, kv, d)
    out = torch.full((T, heads, d), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, scale=-0.2, out=out)
    check_prompt(out, host, [T], -0.2)


def test_prompt_tokens_before_the_first_sequence():
    note("prompt first 7")
    torch = torch_cuda()
    host, (q, k, v) = qkv(rng_for(3), 90, 4, 2, 64)
    out = torch.full((90, 4, 64), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, cu=cu_of([40, 33], first=7), out=out)
    check_prompt(out, host, [40, 33], 64 ** -0.5, first=7)


def test_prompt_strides():
    """Output rows inside wider rows, inputs contiguous and not; what lies between is left alone."""
    note("prompt strides")
    torch = torch_cuda()
    host, (q, k, v) = qkv(rng_for(4), 150, 6, 3, 64)
    wide = torch.full((150, 6 * 64 + 36), NAN, device="cuda")
    out = wide[:, 16:16 + 6 * 64].unflatten(1, (6, 64))
    wqa.attn_prefill(q.contiguous(), k, v.contiguous(), cu=cu_of([150]), out=out)
    check_prompt(out, host, [150], 0.125)
    assert torch.isnan(wide[:, :16]).all() and torch.isnan(wide[:, 16 + 6 * 64:]).all()


@pytest.mark.parametrize("heads", [4, 160, 2])
@pytest.mark.parametrize("what", ["outlier_keys", "peaked", "tiny", "huge", "value_spread", "key_spread", "equal", "one_channel"])
def test_prompt_range(what, heads):
    """Magnitudes the normalisation has to carry: single rows far above the
    others, logits that leave one key, data near the ends of fp32, values that
    span 2^60 between rows."""
    note(f"prompt range {what} {heads}")
    torch = torch_cuda()
    kv, d, lens = 2, 128, [70, 45] if heads == 2 else [200, 77]          # 2: short enough for one kernel
    T = sum(lens)
    rng = rng_for(5, len(what))
    y = rng.standard_normal((T, (heads + 2 * kv) * d)).astype(np.float32)
    qc, kc, vc = slice(0, heads * d), slice(heads * d, (heads + kv) * d), slice((heads + kv) * d, None)
    scale = d ** -0.5
    if what == "outlier_keys":
        y[::37, kc] *= 300.0
        y[5, vc] *= 3000.0
    elif what == "peaked":
        y[:, qc] *= 40.0
    elif what == "tiny":
        y[:, qc] *= 1e-18
        y[:, kc] *= 1e-17
        y[:, vc] *= 1e-34
        scale = 1e34
    elif what == "huge":
        y[:, qc] *= 1e18
        y[:, kc] *= 1e15
        y[:, vc] *= 1e36
        scale = 1e-34
    elif what == "value_spread":
        y[:, vc] *= np.exp2(rng.integers(-30, 31, T)).astype(np.float32)[:, None]
    elif what == "key_spread":
        y[:, kc] *= np.exp2(rng.integers(-30, 3, T)).astype(np.float32)[:, None]
    elif what == "equal":
        y[:, kc] = y[:1, kc]
    else:
        y[:, kc][:, ::64] *= 500.0
        y[:, qc][:, ::64] *= 1e-3
    host, (q, k, v) = split(y, heads, kv, d)
    out = torch.full((T, heads, d), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, cu=cu_of(lens), scale=scale, out=out)
    check_prompt(out, host, lens, scale, what=what)


@pytest.mark.parametrize("heads", [4, 160, 420])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("at", [0, 31, 70, 150])
def test_prompt_non_finite_stays_with_the_rows_that_see_it(bad, at, heads):
    note(f"prompt non-finite {bad} at {at} {heads}")
    torch = torch_cuda()
    kv, d, lens = 2, 64, [33, 140, 20]
    group = heads // kv
    T = sum(lens)
    first = np.cumsum([0] + lens)
    rng = rng_for(6, at)
    clean, _ = qkv(rng, T, heads, kv, d)
    b = int(np.searchsorted(first, at, side="right")) - 1
    end = first[b + 1]
    for which in range(3):
        arr = [x.copy() for x in clean]
        arr[which][at, 1, 5] = bad
        parts = [dev(x) for x in arr]
        out = torch.full((T, heads, d), NAN, device="cuda")
        wqa.attn_prefill(*parts, cu=cu_of(lens), out=out)
        got = out.cpu().numpy()
        want, sums = ref.prompt(*clean, lens, d ** -0.5)
        hit = np.zeros((T, heads, d), bool)
        if which == 0:
            hit[at, 1] = True
        elif which == 1:
            hit[at:end, group:] = True
        else:
            hit[at:end, group:, 5] = True
        assert np.isnan(got[hit]).all(), (which, at)
        lim = ref.bound(sums, max(lens), d)
        assert (np.abs(got - want)[~hit] <= lim[~hit]).all(), (which, at)


def test_prompt_device_lengths_out_of_range_stay_in_bounds():
    """Offsets past T, below 0 and decreasing: rows of valid ranges come out right, nothing faults."""
    note("prompt bad cu")
    torch = torch_cuda()
    host, (q, k, v) = qkv(rng_for(7), 64, 4, 2, 64)
    for cu in ([-5, 20, 1000], [0, 64, 64, 10], [70, 80], [-9, -3], [30, 20, 64]):
        out = torch.full((64, 4, 64), NAN, device="cuda")
        wqa.attn_prefill(q, k, v, cu=dev(np.array(cu, np.int32)), out=out)
        torch.cuda.synchronize()
    out = torch.full((64, 4, 64), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, cu=dev(np.array([-5, 20, 1000], np.int32)), out=out)
    check_prompt(out, host, [20, 44], 0.125)


# ------------------------------------------------------------------ cache
def table_for(rng, lens, spare=2):
    need = [-(-n // ref.PAGE) for n in lens]
    pages = sum(need) + spare
    ids = rng.permutation(pages)
    width = max(1, max(need)) + 1
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages


def cache_arrays(rng, pages, kv, d, fill=True):
    """Host codes and scales of a cache, and the device cache."""
    host = []
    for _ in range(2):
        c = rng.integers(-8, 8, (pages, kv, ref.PAGE, d)).astype(np.int8)
        s = np.exp2(rng.uniform(-5, -2, (pages, kv, ref.PAGE, d // 32))).astype(np.float16)
        host += [c, s]
    return host, cache_on(host)


def cache_on(host):
    return wqa.KVCache(dev(ref.nibbles(host[0])), dev(host[1].view(np.int16)),
                       dev(ref.nibbles(host[2])), dev(host[3].view(np.int16)))


@pytest.mark.parametrize("kv,d", [(8, 128), (2, 64), (3, 128), (1, 64)])
@pytest.mark.parametrize("lens,starts", [([1], [0]), ([1] * 9, [0, 1, 63, 64, 65, 127, 200, 31, 5]), ([130, 0, 7, 64], [0, 4, 60, 64]),
                                         ([33], None)])
def test_append_is_bit_exact(kv, d, lens, starts):
    note(f"append {kv} {d} {lens} {starts}")
    rng = rng_for(10, kv, d, len(lens))
    T = sum(lens) + 2
    host, (_, k, v) = qkv(rng, T, kv, kv, d)
    ends = [n + s for n, s in zip(lens, starts or [0] * len(lens))]
    table, pages = table_for(rng, ends)
    want, cache = cache_arrays(rng, pages, kv, d)
    wqa.kv_append(cache, k, v, dev(table), cu=cu_of(lens), start=None if starts is None else dev(np.array(starts, np.int32)))
    at = 0
    for b, n in enumerate(lens):
        for i in range(n):
            pos = ends[b] - n + i
            page, row = table[b, pos // ref.PAGE], pos % ref.PAGE
            for j, x in ((0, host[1]), (2, host[2])):
                want[j][page, :, row], want[j + 1][page, :, row] = ref.quantize(x[at])
            at += 1
    for j, t in enumerate(cache):
        exp = ref.nibbles(want[j]) if j % 2 == 0 else want[j].view(np.int16)
        assert np.array_equal(t.cpu().numpy(), exp), j


def test_append_ties():
    """Blocks whose scale lies exactly midway between two binary16 numbers, and
    values midway between two codes, or a step of fp32 off: the fp32 quotients
    decide."""
    note("append ties")
    torch_cuda()
    rng = rng_for(30)
    half = np.arange(0x0400, 0x7000, 5, dtype=np.uint16)
    low, high = half.view(np.float16).astype(np.float32), (half + 1).astype(np.uint16).view(np.float16).astype(np.float32)
    amax = np.float32(7) * ((low + high) / np.float32(2))                         # exact: 15 bits
    assert ((amax / np.float32(7)).astype(np.float64) * 7 == amax).all()
    s = (amax / np.float32(7)).astype(np.float16).astype(np.float32)[:, None]
    x = (rng.integers(-6, 6, (len(amax), 32)) + 0.5).astype(np.float32) * s      # exact: the middle of two codes
    x = np.nextafter(x, x * rng.integers(0, 3, x.shape).astype(np.float32))       # a step down, none, a step up
    x = np.clip(x, -amax[:, None], amax[:, None])
    x[:, 0] = amax
    T = len(amax) // 4
    x = x[:T * 4].reshape(T, 1, 128)
    pages = -(-T // ref.PAGE)
    cache = wqa.KVCache.empty(pages, 1, 128)
    wqa.kv_append(cache, dev(x), dev(-x), dev(np.arange(pages, dtype=np.int32)[None]))
    for y, codes, scales in ((x, cache.kq, cache.ks), (-x, cache.vq, cache.vs)):
        c, sc = ref.quantize(y[:, 0])
        assert np.array_equal(scales.cpu().numpy().reshape(-1, 4)[:T], sc.view(np.int16))
        assert np.array_equal(codes.cpu().numpy().reshape(-1, 64)[:T], ref.nibbles(c))


def test_append_values_and_bad_blocks():
    """Ties, zeros, tiny and huge blocks as the packing rule has them; blocks
    that are not finite read back as NaN and change no other block."""
    note("append values")
    rng = rng_for(11)
    x = rng.standard_normal((64, 1, 128)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e-7
    x[2] *= 1e-12
    x[3] = np.float32(7) * np.sign(x[3])
    x[4] = np.tile(np.arange(-16, 16, dtype=np.float32) / 2, 4)
    x[5] *= 1e5
    x[6, 0, 0] = 458751.0          # / 7 rounds below binary16's overflow or above it: the rule decides
    x[7, 0, 33] = np.inf
    x[8, 0, 64] = np.nan
    x[9, 0, 127] = -np.inf
    x[10] = 1e30
    k = dev(x)
    cache = wqa.KVCache.empty(1, 1, 128)
    wqa.kv_append(cache, k, k, dev(np.array([[0]], np.int32)))
    codes, scales = ref.quantize(x[:, 0])
    for q, s in ((cache.kq, cache.ks), (cache.vq, cache.vs)):
        got = s.cpu().numpy()[0, 0].view(np.float16)
        assert np.array_equal(np.isnan(got), np.isnan(scales))
        assert np.array_equal(got[~np.isnan(got)], scales[~np.isnan(scales)])
        assert np.array_equal(q.cpu().numpy()[0, 0], ref.nibbles(codes))
    # the cache reads back through the packed-table lookup
    torch = torch_cuda()
    ids = torch.arange(64, dtype=torch.int32, device="cuda")
    back = wqa.embed(ids, cache.kq.view(64, 64), cache.ks.view(64, 4), 128, 4).cpu().numpy()
    want = ref.values(codes, scales)
    assert np.array_equal(np.isnan(back), np.isnan(want)) and np.array_equal(back[~np.isnan(want)], want[~np.isnan(want)])


def test_append_drops_rows_without_a_page():
    note("append bad pages")
    torch = torch_cuda()
    rng = rng_for(12)
    _, (_, k, v) = qkv(rng, 10, 2, 2, 64)
    for table, starts in ([[-1], [5], [1 << 30], [2]], [0, 0, 0, 0]), ([[0], [0], [1], [1]], [-3, 64, -2147483648, 2147483647]):
        cache = wqa.KVCache.empty(2, 2, 64)
        wqa.kv_append(cache, k, v, dev(np.array(table, np.int32)), cu=dev(np.array([0, 2, 4, 6, 8], np.int32)),
                      start=dev(np.array(starts, np.int32)))
        assert all(int(t.to(torch.int64).abs().sum()) == 0 for t in cache)
    # the rows of a sequence that begins before its table are dropped one by one
    cache = wqa.KVCache.empty(2, 2, 64)
    wqa.kv_append(cache, k, v, dev(np.array([[1]], np.int32)), start=dev(np.array([-4], np.int32)))
    assert int(cache.kq[0].to(torch.int64).sum()) == 0
    full = wqa.KVCache.empty(2, 2, 64)
    wqa.kv_append(full, k[4:], v[4:], dev(np.array([[1]], np.int32)))
    assert all(torch.equal(a, b) for a, b in zip(cache, full))


# ------------------------------------------------------------------ decode attention
def check_decode(out, q, host, table, lens, scale, what=""):
    kval, vval = ref.values(*host[:2]), ref.values(*host[2:])
    want, sums = ref.decode(q, kval, vval, host[3], table, lens, scale)
    got = out.cpu().numpy().astype(np.float64)
    lim = ref.bound(sums, max(lens), q.shape[2])
    err = np.abs(got - want)
    assert (err <= lim).all(), f"{what}: worst error / bound {np.nanmax(err / lim):.3f}, {np.isnan(got).sum()} NaN"


@pytest.mark.parametrize("heads,kv,d", LAYOUTS + [(8, 1, 128), (32, 2, 64), (3, 3, 128), (12, 4, 128), (20, 1, 64)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 63, 64, 65, 0, 200, 15], [700], [33] * 20, [1100, 0, 300, 2]], ids=lambda x: "-".join(map(str, x[:8])))
def test_decode_parity(heads, kv, d, lens):
    note(f"decode {heads} {kv} {d} {lens}")
    torch = torch_cuda()
    rng = rng_for(20, heads, kv, d, len(lens))
    table, pages = table_for(rng, lens)
    host, cache = cache_arrays(rng, pages, kv, d)
    q = rng.standard_normal((len(lens), heads, d)).astype(np.float32) * 2
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), out=out)
    check_decode(out, q, host, table, lens, d ** -0.5, str(lens))


@pytest.mark.parametrize("lens", [[20000], [5000, 9, 12345, 0, 4097]])
def test_decode_long(lens):
    """Lengths that are split over workgroups."""
    note(f"decode long {lens}")
    torch = torch_cuda()
    rng = rng_for(21, len(lens))
    table, pages = table_for(rng, lens)
    host, cache = cache_arrays(rng, pages, 2, 64)
    q = rng.standard_normal((len(lens), 4, 64)).astype(np.float32)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), scale=0.3, out=out)
    check_decode(out, q, host, table, lens, 0.3)


@pytest.mark.parametrize("count,longest", [(600, 1300), (600, 2500), (2100, 2500)])
def test_decode_many_sequences(count, longest):
    """More sequences than a workgroup looks at together, some empty, some past a
    step: not cut for short tables, cut, and too many to be cut."""
    note(f"decode many {count} {longest}")
    torch = torch_cuda()
    rng = rng_for(27)
    lens = [int(n) for n in rng.integers(0, 80, count)]
    lens[7], lens[-1] = longest, 600
    table, pages = table_for(rng, lens)
    host, cache = cache_arrays(rng, pages, 1, 64)
    q = rng.standard_normal((count, 2, 64)).astype(np.float32)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), out=out)
    check_decode(out, q, host, table, lens, 0.125)


def test_cache_past_four_gib():
    """Pages whose byte offsets pass 32 bits: append and read them back."""
    note("cache past 4 GiB")
    torch = torch_cuda()
    n, kv, d = 140000, 8, 128                  # 4.27 GiB of codes each for keys and values
    cache = wqa.KVCache(*(torch.empty((n, kv, 64, w), dtype=t, device="cuda")
                          for w, t in ((64, torch.uint8), (4, torch.int16), (64, torch.uint8), (4, torch.int16))))
    rng = rng_for(28)
    T = 1200
    _, (q, k, v) = qkv(rng, T, 16, kv, d)
    ids = [n - 1, 0, 131072, 131071] + list(range(n - 20, n - 5))
    table = np.array([ids], np.int32)
    wqa.kv_append(cache, k, v, dev(table))
    small = wqa.KVCache.empty(len(ids), kv, d)
    stab = np.arange(len(ids), dtype=np.int32)[None]
    wqa.kv_append(small, k, v, dev(stab))
    for a, b in zip(cache, small):
        assert torch.equal(a[torch.tensor(ids, device="cuda")][:18], b[:18])
    ln = dev(np.array([T], np.int32))
    big, want = (wqa.attn_decode(q[:1], c, dev(t), ln) for c, t in ((cache, table), (small, stab)))
    assert torch.equal(big, want) and torch.isfinite(big).all()


def test_calls_on_two_streams_at_once():
    """The same and different calls under way on two streams: the bits of a call alone."""
    note("two streams")
    torch = torch_cuda()
    rng = rng_for(29)
    lens = [3000, 1700]
    table, pages = table_for(rng, lens)
    _, cache = cache_arrays(rng, pages, 2, 128)
    _, (q, k, v) = qkv(rng, 900, 8, 2, 128)
    tab, ln = dev(table), dev(np.array(lens, np.int32))
    qd = q[:2].contiguous()
    want = (wqa.attn_decode(qd, cache, tab, ln), wqa.attn_prefill(q, k, v, cu=cu_of([500, 400])))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        s = streams[i % 2]
        got.append((wqa.attn_decode(qd, cache, tab, ln, stream=s), wqa.attn_prefill(q, k, v, cu=cu_of([500, 400]), stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


@pytest.mark.parametrize("what", ["scales", "zero_values", "peaked", "tiny_q", "huge_q", "negative_scale", "equal"])
def test_decode_range(what):
    """Scales over binary16's whole range, values of zero, logits that leave one key, queries near the ends of fp32."""
    note(f"decode range {what}")
    torch = torch_cuda()
    heads, kv, d, lens = 8, 2, 128, [130, 64, 513]
    rng = rng_for(22, len(what))
    table, pages = table_for(rng, lens)
    host, _ = cache_arrays(rng, pages, kv, d)
    q = rng.standard_normal((len(lens), heads, d)).astype(np.float32)
    scale = d ** -0.5
    if what == "scales":
        for j in (1, 3):
            bits = rng.integers(0, 0x7C00, host[j].shape).astype(np.uint16)
            host[j] = bits.view(np.float16)
        scale = 1e-5
    elif what == "zero_values":
        host[3][:, :, ::2] = 0
        host[2][:, :, 1::4] = 0
        host[1][:, :, 5] = 0
    elif what == "peaked":
        q *= 60
    elif what == "tiny_q":
        q *= 1e-30
        scale = 1e30
    elif what == "huge_q":
        q *= 1e36
        scale = 1e-37
    elif what == "negative_scale":
        scale = -0.3
    else:
        host[0][:] = host[0][:1, :, :1]
        host[1][:] = host[1][:1, :, :1]
    cache = cache_on(host)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), scale=scale, out=out)
    check_decode(out, q, host, table, lens, scale, what)


def test_decode_rows_past_the_length_may_hold_anything():
    note("decode past length")
    torch = torch_cuda()
    heads, kv, d, lens = 4, 2, 128, [70, 1, 64, 100]
    rng = rng_for(23)
    table, pages = table_for(rng, lens, spare=0)
    host, _ = cache_arrays(rng, pages, kv, d)
    for b, n in enumerate(lens):
        page, row = table[b, n // ref.PAGE], n % ref.PAGE
        if row:
            host[1][page, :, row:] = np.nan
            host[3][page, :, row:] = np.inf
    out = torch.full((4, heads, d), NAN, device="cuda")
    q = rng.standard_normal((4, heads, d)).astype(np.float32)
    wqa.attn_decode(dev(q), cache_on(host), dev(table), dev(np.array(lens, np.int32)), out=out)
    clean = [np.where(np.isfinite(x), x, 0).astype(x.dtype) for x in host]
    check_decode(out, q, clean, table, lens, d ** -0.5)


def test_decode_bad_pages_and_lengths():
    note("decode bad pages")
    torch = torch_cuda()
    rng = rng_for(24)
    table, pages = table_for(rng, [64, 100, 128, 64, 30, 64], spare=0)
    host, cache = cache_arrays(rng, pages, 2, 64)
    W = table.shape[1]
    table[0, 0] = pages
    table[1, 1] = -1
    table[2, 1] = 1 << 30
    lens = [64, 100, 128, 64 * W + 1, 30, -1]
    q = rng.standard_normal((6, 4, 64)).astype(np.float32)
    out = torch.zeros((6, 4, 64), device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), out=out)
    got = out.cpu().numpy()
    assert np.isnan(got[[0, 1, 2, 3, 5]]).all()
    check_decode(out[4:5], q[4:5], host, table[4:5], [30], 0.125)
    # a bad page behind the length is not looked at
    lens = [0, 64, 64, 1, 30, 2]
    out = torch.full((6, 4, 64), NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), out=out)
    check_decode(out, q, host, table, lens, 0.125)
    # no pages at all
    empty = wqa.KVCache.empty(0, 2, 64)
    out = wqa.attn_decode(dev(q[:2]), empty, torch.zeros((2, 0), dtype=torch.int32, device="cuda"),
                          dev(np.array([0, 3], np.int32)))
    assert (out[0] == 0).all() and torch.isnan(out[1]).all()


def test_decode_non_finite_data():
    """A NaN scale of a key makes the heads that read it NaN, one of a value the
    block's elements; a query's NaN or infinity its own head."""
    note("decode non-finite")
    torch = torch_cuda()
    heads, kv, d, lens = 4, 2, 128, [90]
    rng = rng_for(25)
    table, pages = table_for(rng, lens)
    q = rng.standard_normal((1, heads, d)).astype(np.float32)
    for which in range(4):
        host, _ = cache_arrays(rng_for(26), pages, kv, d)
        clean = [x.copy() for x in host]
        hit = np.zeros((heads, d), bool)
        qq = q.copy()
        if which == 0:
            host[1][table[0, 1], 1, 7, 2] = np.nan
            hit[2:] = True
        elif which == 1:
            host[3][table[0, 0], 0, 60, 1] = np.nan
            hit[:2, 32:64] = True
        else:
            qq[0, 3, 100] = np.inf if which == 2 else np.nan
            hit[3] = True
        out = torch.full(q.shape, 0.0, device="cuda")
        wqa.attn_decode(dev(qq), cache_on(host), dev(table), dev(np.array(lens, np.int32)), out=out)
        got = out.cpu().numpy()[0]
        want, sums = ref.decode(q, ref.values(*clean[:2]), ref.values(*clean[2:]), clean[3], table, lens, d ** -0.5)
        lim = ref.bound(sums, 90, d)[0]
        assert np.isnan(got[hit]).all(), which
        assert (np.abs(got - want[0])[~hit] <= lim[~hit]).all(), which


def test_decode_value_scales_of_either_sign():
    """A cache filled by other means: value scales below zero, far larger than the
    others, and an infinite one, whose block alone is not finite."""
    note("decode value scale signs")
    torch = torch_cuda()
    heads, kv, d, lens = 4, 2, 128, [700]
    rng = rng_for(27)
    table, pages = table_for(rng, lens)
    q = rng.standard_normal((1, heads, d)).astype(np.float32)
    host, _ = cache_arrays(rng, pages, kv, d)
    host[3][:, :, ::3] *= -1
    host[3][table[0, 2], :, 5, 1] = -20000.0
    host[3][table[0, 9], :, 40, :] = -300.0
    want, sums = ref.decode(q, ref.values(*host[:2]), ref.values(*host[2:]), np.abs(host[3]), table, lens, d ** -0.5)
    lim = ref.bound(sums, 700, d)[0]
    for inf in (False, True):
        hit = np.zeros((heads, d), bool)
        if inf:
            host[3][table[0, 1], 1, 7, 2] = -np.inf
            hit[2:, 64:96] = True
        got = wqa.attn_decode(dev(q), cache_on(host), dev(table), dev(np.array(lens, np.int32))).cpu().numpy()[0]
        assert not np.isfinite(got[hit]).any(), inf
        assert (np.abs(got - want[0])[~hit] <= lim[~hit]).all(), inf


# ------------------------------------------------------------------ norms
def norm_bound(h, y, post, gate, alpha, pre, eps, want_h, size, want_x):
    """h_out: t carries the norm (mean of squares: one rounding a square, half
    a step per level of the sum, at most 64 levels; half of it through the
    square root; root, division and three products half a step each), then one
    fused multiply-add. x_out: the relative error of the same kind plus h_out's
    own, over the row's mean square."""
    rel = (64 / 2 + 8) * ref.U32
    eh = 2 * rel * size + 1e-44
    n = h.shape[1]
    rms = np.sqrt((want_h * want_h).mean(1, keepdims=True) + eps)
    w = 1.0 if pre is None else np.abs(pre)
    # d x / d h_out: w / rms on the element, and through the root at most |x| sum |h_out| eh / (n rms^2)
    through = (np.abs(want_h) * eh).sum(1, keepdims=True) / (n * rms * rms)
    return eh, (eh / rms + np.abs(want_h) / rms * through) * w + 2 * rel * np.abs(want_x) + 1e-44


@pytest.mark.parametrize("M,N", [(1, 1), (3, 2), (1, 1024), (5, 63), (4, 257), (7, 1024), (300, 1000), (2, 4099),
                                 (9, 8192), (2, 20001), (1, 40000), (3, 100003)])
@pytest.mark.parametrize("post,gate,pre", [(True, "all", True), (False, "row", True), (True, "none", False), (False, "none", True)])
def test_norm_parity(M, N, post, gate, pre):
    note(f"norm {M} {N} {post} {gate} {pre}")
    torch = torch_cuda()
    rng = rng_for(30, M, N)
    h, y = (rng.standard_normal((M, N)).astype(np.float32) * s for s in (3, 0.7))
    g = {"none": None, "row": rng.standard_normal(N), "all": rng.standard_normal((M, N))}[gate]
    g = None if g is None else g.astype(np.float32)
    pw = (1 + 0.1 * rng.standard_normal(N)).astype(np.float32) if post else None
    w = (1 + 0.1 * rng.standard_normal(N)).astype(np.float32) if pre else None
    want_h, size, want_x = ref.residual_norm(h, y, pw, g, 0.6, w, 1e-6)
    want_h32, size, want_x = ref.residual_norm(h, y, pw, g, float(np.float32(0.6)), w, float(np.float32(1e-6)))
    eh, ex = norm_bound(h, y, pw, g, 0.6, w, 1e-6, want_h32, size, want_x)
    on = [None if x is None else dev(x) for x in (h, y, pw, g, w)]
    ho = torch.full((M, N), NAN, device="cuda")
    xo = torch.full((M, N), NAN, device="cuda")
    wqa.residual_norm(on[0], on[1], post_weight=on[2], gate=on[3], alpha=0.6, pre_weight=on[4], eps=1e-6, h_out=ho,
                      x_out=xo)
    assert (np.abs(ho.cpu().numpy() - want_h32) <= eh).all()
    assert (np.abs(xo.cpu().numpy() - want_x) <= ex).all()
    # without x_out, without h_out, and with h updated in place: the same bits
    h2, none = wqa.residual_norm(on[0], on[1], post_weight=on[2], gate=on[3], alpha=0.6, eps=1e-6)
    assert none is None and torch.equal(h2, ho)
    a, b = wqa.residual_norm(on[0], on[1], post_weight=on[2], gate=on[3], alpha=0.6, pre_weight=on[4], eps=1e-6,
                             norm=True, h_out=on[0])
    assert a is on[0] and torch.equal(a, ho) and torch.equal(b, xo)


def test_norm_alone_and_unaligned():
    note("norm alone")
    torch = torch_cuda()
    rng = rng_for(31)
    for M, N in ((2, 1024), (3, 37), (2, 9001)):
        h = rng.standard_normal((M, N)).astype(np.float32)
        w = rng.standard_normal(N).astype(np.float32)
        want, size, wx = ref.residual_norm(h, None, None, None, 1.0, w, 1e-5)
        ex = norm_bound(h, None, None, None, 1.0, w, 1e-5, want, size, wx)[1]
        ho, xo = wqa.residual_norm(dev(h), pre_weight=dev(w), eps=1e-5)
        assert ho is None and (np.abs(xo.cpu().numpy() - wx) <= ex).all()
        # storage that starts 4 bytes off every wider alignment
        buf = torch.zeros(M * N + 1, device="cuda")
        hs = buf[1:].view(M, N)
        hs.copy_(dev(h))
        _, x2 = wqa.residual_norm(hs, pre_weight=dev(w), eps=1e-5)
        assert torch.equal(x2, xo)


def test_norm_extremes():
    """Rows of zeros, rows whose squares leave fp32's range on neither side, and non-finite rows that stay rows."""
    note("norm extremes")
    rng = rng_for(32)
    h = rng.standard_normal((5, 300)).astype(np.float32)
    h[0] = 0
    h[1] *= 1e15
    h[2] *= 1e-15
    h[3, 7] = np.inf
    _, x = wqa.residual_norm(dev(h), norm=True, eps=1e-6)
    x = x.cpu().numpy()
    assert (x[0] == 0).all() and np.isfinite(x[[1, 2, 4]]).all() and np.isnan(x[3, 7])
    want = ref.residual_norm(h[[1, 2, 4]], None, None, None, 1, None, float(np.float32(1e-6)))[2]
    assert np.allclose(x[[1, 2, 4]], want, rtol=80 * ref.U32, atol=1e-44)


# ------------------------------------------------------------------ streams, graphs, threads of calls
def layer_state(rng, lens, heads, kv, d):
    T = sum(lens)
    hidden = heads * d
    st = {"h": dev(rng.standard_normal((T, hidden)).astype(np.float32)),
          "w1": dev((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32)),
          "w2": dev((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32))}
    for name, n in (("qkv", (heads + 2 * kv) * d), ("o", hidden)):
        st[name] = wqa.pack(dev((rng.standard_normal((n, hidden)) * hidden ** -0.5).astype(np.float32)), 4)
    return st


def split_heads(y, heads, kv, d):
    T = y.shape[0]
    return (y[:, :heads * d].view(T, heads, d), y[:, heads * d:(heads + kv) * d].view(T, kv, d),
            y[:, (heads + kv) * d:].view(T, kv, d))


def test_layer_prefill_then_decode():
    """The operators in the order of use: a packed prompt through norm, fused
    projection, attention, output projection and residual, its keys and values
    into the cache, then one token per sequence over the cache."""
    note("layer run")
    torch = torch_cuda()
    heads, kv, d, lens = 4, 2, 64, [70, 1, 129]
    rng = rng_for(40)
    st = layer_state(rng, lens, heads, kv, d)
    T = sum(lens)
    cu = cu_of(lens)
    table, pages = table_for(rng, [n + 1 for n in lens])
    cache = wqa.KVCache.empty(pages, kv, d)
    tab = dev(table)
    # prompt
    _, x = wqa.residual_norm(st["h"], pre_weight=st["w1"])
    y = wqa.linear(x, *st["qkv"], 4)
    q, k, v = split_heads(y, heads, kv, d)
    o = wqa.attn_prefill(q, k, v, cu=cu)
    wqa.kv_append(cache, k, v, tab, cu=cu)
    z = wqa.linear(o.view(T, -1), *st["o"], 4)
    h1, x1 = wqa.residual_norm(st["h"], z, post_weight=st["w2"], alpha=0.5, pre_weight=st["w1"])
    # the attention of the prompt over its own projections
    yh = y.cpu().numpy()
    host = [a.reshape(T, -1, d) for a in np.split(yh, [heads * d, (heads + kv) * d], axis=1)]
    check_prompt(o, host, lens, d ** -0.5)
    want = ref.residual_norm(st["h"].cpu().numpy(), z.cpu().numpy(), st["w2"].cpu().numpy(), None, 0.5,
                             st["w1"].cpu().numpy(), float(np.float32(1e-6)))
    assert np.allclose(h1.cpu().numpy(), want[0], rtol=0, atol=80 * ref.U32 * want[1].max())
    assert np.allclose(x1.cpu().numpy(), want[2], rtol=0, atol=400 * ref.U32 * np.abs(want[2]).max())
    # one token more for every sequence
    hb = h1[:len(lens)].contiguous()
    _, xb = wqa.residual_norm(hb, pre_weight=st["w1"])
    yb = wqa.linear(xb, *st["qkv"], 4)
    qb, kb, vb = split_heads(yb, heads, kv, d)
    ln = np.array(lens, np.int32)
    wqa.kv_append(cache, kb, vb, tab, cu=cu_of([1] * len(lens)), start=dev(ln))
    ob = wqa.attn_decode(qb, cache, tab, dev(ln + 1))
    # a cache built on the host from the same rows
    hostc = [np.zeros((pages, kv, ref.PAGE, d), np.int8), np.zeros((pages, kv, ref.PAGE, d // 32), np.float16),
             np.zeros((pages, kv, ref.PAGE, d), np.int8), np.zeros((pages, kv, ref.PAGE, d // 32), np.float16)]
    at = 0
    ybh = yb.cpu().numpy()
    new = [a.reshape(len(lens), -1, d) for a in np.split(ybh, [heads * d, (heads + kv) * d], axis=1)]
    for b, n in enumerate(lens):
        for i in range(n + 1):
            page, row = table[b, i // ref.PAGE], i % ref.PAGE
            for j in (0, 1):
                src = host[1 + j][at + i] if i < n else new[1 + j][b]
                hostc[2 * j][page, :, row], hostc[2 * j + 1][page, :, row] = ref.quantize(src)
        at += n
    for j, t in enumerate(cache):
        assert np.array_equal(t.cpu().numpy(), ref.nibbles(hostc[j]) if j % 2 == 0 else hostc[j].view(np.int16))
    check_decode(ob, new[0], hostc, table, [n + 1 for n in lens], d ** -0.5)


def test_layer_on_another_stream_and_in_a_graph():
    """A decode step on a side stream and captured: every replay gives the eager
    bits, for lengths changed on the device between replays."""
    note("layer graph")
    torch = torch_cuda()
    heads, kv, d = 8, 2, 128
    rng = rng_for(41)
    cap = [300, 2100, 64]
    table, pages = table_for(rng, cap)
    _, cache = cache_arrays(rng, pages, kv, d)
    q = dev(rng.standard_normal((3, heads, d)).astype(np.float32))
    k, v = (dev(rng.standard_normal((3, kv, d)).astype(np.float32)) for _ in range(2))
    tab, cu = dev(table), cu_of([1, 1, 1])
    start = dev(np.array([10, 2000, 0], np.int32))
    h = dev(rng.standard_normal((3, heads * d)).astype(np.float32))
    pq, pk, pv = (dev(rng.standard_normal((200, n, d)).astype(np.float32)) for n in (heads, kv, kv))
    pcu = cu_of([150, 50])

    def step():
        wqa.kv_append(cache, k, v, tab, cu=cu, start=start)
        o = wqa.attn_decode(q, cache, tab, start + 1)
        p = wqa.attn_prefill(pq, pk, pv, cu=pcu)
        return wqa.residual_norm(h, o.view(3, -1), norm=True) + (o, p)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = step()
    side.synchronize()
    # the stream argument, from the default stream
    o2 = wqa.attn_decode(q, cache, tab, start + 1, stream=side)
    p2 = wqa.attn_prefill(pq, pk, pv, cu=pcu, stream=side)
    side.synchronize()
    assert torch.equal(o2, warm[2]) and torch.equal(p2, warm[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i, lens in enumerate(([10, 2000, 0], [299, 2099, 63], [0, 0, 0], [128, 1024, 7])):
        start.copy_(dev(np.array(lens, np.int32)))
        q.mul_(1.0 + 0.1 * i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in caught]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), lens


def test_layer_runs_are_bitwise_equal():
    note("layer determinism")
    torch = torch_cuda()
    heads, kv, d, lens = 8, 4, 128, [260, 131]
    rng = rng_for(42)
    _, (q, k, v) = qkv(rng, sum(lens), heads, kv, d)
    table, pages = table_for(rng, [3000, 700])
    _, cache = cache_arrays(rng, pages, kv, d)
    ln = dev(np.array([2999, 700], np.int32))
    qd = q[:2].contiguous()
    first = None
    for _ in range(6):
        now = (wqa.attn_prefill(q, k, v, cu=cu_of(lens)), wqa.attn_decode(qd, cache, dev(table), ln))
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_layer_refusals():
    torch = torch_cuda()
    q, k = torch.zeros((4, 4, 64), device="cuda"), torch.zeros((4, 2, 64), device="cuda")
    cache = wqa.KVCache.empty(2, 2, 64)
    tab, ln = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    bad = [lambda: wqa.attn_prefill(q.half(), k, k), lambda: wqa.attn_prefill(q, k[:3], k), lambda: wqa.attn_prefill(q, k, k, cu=ln.long()),
           lambda: wqa.attn_prefill(q.transpose(0, 1), k, k), lambda: wqa.attn_prefill(q, k, k, out=q[:2]),
           lambda: wqa.attn_prefill(q[..., :32], k[..., :32], k[..., :32]),
           lambda: wqa.kv_append(cache, q, q, tab[:1]), lambda: wqa.kv_append(cache, k, k, tab, cu=ln),
           lambda: wqa.kv_append(cache._replace(ks=cache.ks[:1]), k, k, tab[:1]),
           lambda: wqa.attn_decode(q, cache, tab[:2], ln), lambda: wqa.attn_decode(q, cache, tab, ln[:2]),
           lambda: wqa.attn_decode(q, cache, tab, ln.float()), lambda: wqa.attn_decode(q[..., :32].contiguous(), cache, tab, ln),
           lambda: wqa.attn_decode(q[:, :3].contiguous(), cache, tab, ln),
           lambda: wqa.residual_norm(q[0]), lambda: wqa.residual_norm(q[0], gate=q[0]), lambda: wqa.residual_norm(q[0], q[1, :2]),
           lambda: wqa.residual_norm(q[0], norm=False, x_out=q[1]), lambda: wqa.residual_norm(q[0, :, ::2])]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, wqa.WqError)):
            f()
            pytest.fail(f"call {i} was accepted")
    # nothing to do
    assert wqa.attn_prefill(q[:0], k[:0], k[:0]).shape == (0, 4, 64)
    assert wqa.attn_decode(q[:0], cache, tab[:0], ln[:0]).shape == (0, 4, 64)
    wqa.kv_append(cache, k[:0], k[:0], tab[:1])
