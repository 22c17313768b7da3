"""GPU parity of the operators of a serving step against their plain 64-bit forms
(tests/serve_ref.py, tests/layer_ref.py, where the error bounds are derived)."""
import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import layer_ref as ref
from tests import serve_ref as sref
from tests.gpu_util import note, torch_cuda
from tests.test_gpu_layer import LAYOUTS, NAN, WIDE, cache_arrays, cache_on, cu_of, dev, qkv, rng_for, table_for

pytestmark = pytest.mark.gpu


def ints(a):
    return dev(np.asarray(a, np.int32))


# ------------------------------------------------------------------ plans
def plan_inputs(rng, count, width, most, before, short=0):
    fresh = rng.integers(0, most + 1, count)
    start = rng.integers(0, before + 1, count)
    table = np.full((count, width), -1, np.int32)
    have = np.minimum(-(-start // 64), width)
    ids = rng.permutation(int(have.sum()) + 5000).astype(np.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = ids[at:at + n]
        at += n
    need = int((np.minimum(-(-(start + fresh) // 64), width) - have).sum())
    return fresh, start, table, ids[at:at + max(0, need + 3 - short)]


def check_plan(got, table, want, tokens):
    assert np.array_equal(table.cpu().numpy(), want[0])
    for x, y, name in zip((got.cu, got.lens, got.positions, got.slots, got.taken), want[1:], ("cu", "lens", "positions", "slots", "taken")):
        assert np.array_equal(x.cpu().numpy(), y), name


@pytest.mark.parametrize("count,width,most,before", [(1, 4, 100, 0), (1, 40, 1, 2000), (5, 3, 130, 100), (64, 12, 1, 700), (300, 9, 200, 300),
                                                     (1024, 3, 2, 130), (1025, 3, 70, 64), (2600, 2, 1, 127), (7, 0, 9, 9)])
@pytest.mark.parametrize("short", [0, 3, 1000])
def test_plan(count, width, most, before, short):
    note(f"plan {count} {width} {most} {before} {short}")
    torch_cuda()
    rng = rng_for(60, count, width, most)
    fresh, start, table, free = plan_inputs(rng, count, width, most, before, short)
    total = int(fresh.sum())
    for tokens in sorted({0, 1, total // 2, total, total + 77}):
        dt = dev(table)
        got = wqa.kv_plan(ints(fresh), dt, dev(free), tokens=tokens, start=ints(start))
        check_plan(got, dt, sref.plan(fresh.tolist(), start.tolist(), table, free, 0, tokens), tokens)


def test_plan_without_start_and_with_taken():
    note("plan taken")
    torch = torch_cuda()
    fresh, table, free = [3, 0, 64, 129], np.full((4, 3), -7, np.int32), np.arange(100, 108, dtype=np.int32)
    for taken in (0, 2, 5, 8, 2 ** 31 - 2, -3):
        dt = dev(table)
        got = wqa.kv_plan(ints(fresh), dt, dev(free), ints([taken]), tokens=200)
        check_plan(got, dt, sref.plan(fresh, [0] * 4, table, free, taken, 200), 200)
    dt = dev(table)
    got = wqa.kv_plan(ints([]), dt[:0], dev(free), ints([4]), tokens=5)
    assert got.cu.tolist() == [0] and got.taken.tolist() == [4] and got.slots.tolist() == [-1] * 5 and got.lens.shape == (0,)
    out = wqa.KVPlan(ints([9] * 5), ints([9] * 4), ints([9] * 6), torch.full((6,), 9, device="cuda"), ints([9]))
    back = wqa.kv_plan(ints(fresh), dt, dev(free), tokens=6, out=out)
    assert back is out
    check_plan(out, dt, sref.plan(fresh, [0] * 4, table, free, 0, 6), 6)


def test_plan_bad_requests_and_long_ones():
    """Negative lengths, sums past 31 bits, tokens past the table's row."""
    note("plan bad")
    torch_cuda()
    big = 2 ** 31 - 1
    for fresh, start in (([5, -1, 7], [0, 3, 1]), ([5, 2, 7], [0, -3, 60]), ([big, 4, big], [0, 1, 1]), ([5, 4, 3], [big - 5, big - 2, big]),
                         ([200, 1, 70], [64, 640, 100]), ([big, big, big], [0, 0, 0])):
        table, free = np.full((3, 4), 77, np.int32), np.arange(9, dtype=np.int32)
        dt = dev(table)
        got = wqa.kv_plan(ints(fresh), dt, dev(free), tokens=300, start=ints(start))
        check_plan(got, dt, sref.plan(fresh, start, table, free, 0, 300), 300)
    # bad entries of the row, and of the list
    table, free = np.array([[5, -4, 3]], np.int32), np.array([-9, 8], np.int32)
    dt = dev(table)
    got = wqa.kv_plan(ints([100]), dt, dev(free), tokens=100, start=ints([70]))
    check_plan(got, dt, sref.plan([100], [70], table, free, 0, 100), 100)


@pytest.mark.parametrize("kv,d", [(8, 128), (2, 64), (1, 64), (3, 128)])
def test_append_by_slots_is_append_by_table(kv, d):
    note(f"append slots {kv} {d}")
    torch = torch_cuda()
    rng = rng_for(61, kv, d)
    fresh, start, table, free = plan_inputs(rng, 9, 8, 200, 130)
    T = int(fresh.sum()) + 4
    _, (_, k, v) = qkv(rng, T, kv, kv, d)
    pages = int(max(table.max(), free.max(initial=0))) + 1
    _, one = cache_arrays(rng, pages, kv, d)
    two = wqa.KVCache(*(t.clone() for t in one))
    dt = dev(table)
    p = wqa.kv_plan(ints(fresh), dt, dev(free), tokens=T, start=ints(start))
    wqa.kv_append(one, k, v, dt, cu=p.cu, start=ints(start))
    wqa.kv_append(two, k, v, slots=p.slots)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    # slots outside the cache are dropped
    bad = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    bad[::2] = pages * 64 + torch.arange(0, T, 2, device="cuda")
    bad[1] = -2 ** 62
    bad[3] = 2 ** 62
    wqa.kv_append(two, k, v, slots=bad)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


# ------------------------------------------------------------------ norms and rotation
def check_rope(got, x, *args):
    want, lim = sref.rope(x, *args)
    err = np.abs(got.cpu().numpy().astype(np.float64) - want)
    assert (err <= lim).all(), f"worst error / bound {np.nanmax(err / lim):.3f}"


def freqs(n, base=1e6):
    return (base ** (-np.arange(n) / n)).astype(np.float32)


@pytest.mark.parametrize("heads,kv,d", LAYOUTS + [(1, 0, 64), (70, 3, 128), (33, 33, 64)])
@pytest.mark.parametrize("T", [1, 3, 70, 1030])
@pytest.mark.parametrize("inter", [False, True])
def test_rope(heads, kv, d, T, inter):
    note(f"rope {heads} {kv} {d} {T} {inter}")
    torch = torch_cuda()
    rng = rng_for(62, heads, kv, d, T)
    host, (q, k, _) = qkv(rng, T, heads, kv, d)
    wq, wk = (rng.standard_normal(d).astype(np.float32) for _ in range(2))
    for pairs, norm, weights, factor in ((d // 2, True, True, 1.0), (8, True, False, 1.25), (d // 4, False, False, -0.5), (12, True, True, 1.0), (0, True, True, 1.0)):
        pos = rng.integers(0, 10 ** rng.integers(1, 7), T).astype(np.int32)
        inv = freqs(pairs) if pairs else np.zeros(0, np.float32)
        oq, ok = (torch.full(x.shape, NAN, device="cuda") for x in (q, k))
        w = dict(q_weight=dev(wq), k_weight=dev(wk) if kv else None) if weights else {}
        back = wqa.qk_norm_rope(q, k if kv else None, dev(pos), dev(inv), norm=norm, interleaved=inter, factor=factor,
                                q_out=oq, k_out=ok if kv else None, **w)
        assert back[0] is oq and back[1] is (ok if kv else None)
        check_rope(oq, host[0], pos, inv, wq if weights else None, 1e-6, norm, inter, factor)
        if kv:
            check_rope(ok, host[1], pos, inv, wk if weights else None, 1e-6, norm, inter, factor)


@pytest.mark.parametrize("T", [9, 1500])
def test_rope_in_place_in_a_fused_row(T):
    """q and k rotated where the projection left them; v and skipped rows keep what they held."""
    note(f"rope in place {T}")
    torch_cuda()
    rng = rng_for(63, T)
    heads, kv, d = 16, 8, 128
    y = rng.standard_normal((T, (heads + 2 * kv) * d)).astype(np.float32)
    on = dev(y)
    q, k, v = on[:, :heads * d].view(T, heads, d), on[:, heads * d:-kv * d].view(T, kv, d), on[:, -kv * d:].view(T, kv, d)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    pos[[2, T - 1]] = [-1, -2 ** 31]
    inv = freqs(64)
    wqa.qk_norm_rope(q, k, dev(pos), dev(inv), q_out=q, k_out=k)
    hq, hk = y[:, :heads * d].reshape(T, heads, d), y[:, heads * d:-kv * d].reshape(T, kv, d)
    live = pos >= 0
    for got, x in ((q, hq), (k, hk)):
        got = got.cpu()
        assert np.array_equal(got.numpy()[~live], x[~live])
        check_rope(got[live], x[live], pos[live], inv, None, 1e-6, True, False, 1.0)
    assert np.array_equal(v.cpu().numpy(), y[:, -kv * d:].reshape(T, kv, d))


def test_rope_far_positions_and_odd_frequencies():
    note("rope far")
    torch_cuda()
    rng = rng_for(64)
    pos = np.array([0, 1, 131071, 1 << 24, (1 << 24) + 1, 1000003, (1 << 30) + 12345, 2 ** 31 - 1], np.int32)
    host, (q, k, _) = qkv(rng, len(pos), 4, 2, 64)
    inv = np.concatenate([freqs(28), np.array([0.0, -0.37, 1e-30, 3.0], np.float32)])
    oq, ok = wqa.qk_norm_rope(q, k, dev(pos), dev(inv))
    check_rope(oq, host[0], pos, inv, None, 1e-6, True, False, 1.0)
    check_rope(ok, host[1], pos, inv, None, 1e-6, True, False, 1.0)


@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-20, 1e-31, 1e-38])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_magnitudes(d, eps):
    """Rows whose squares leave fp32 at either end, beside ordinary ones and zeros."""
    note(f"rope magnitudes {d} {eps}")
    torch_cuda()
    rng = rng_for(65, d)
    x = rng.standard_normal((24, 4, d)).astype(np.float32)
    scale = np.exp2(np.linspace(-140, 125, 96)).reshape(24, 4, 1)
    x = (x * scale).astype(np.float32)
    if eps:
        x[5] = 0.0
    x[6, 1, 3:] = 0.0
    x[7, 2] = 0.0
    x[7, 2, 9] = 3.4028235e38
    if eps == 0.0:
        x[np.abs(x).max(-1) == 0] = 1.0
    pos = np.arange(24, dtype=np.int32)
    inv = freqs(d // 2)
    oq, ok = wqa.qk_norm_rope(dev(x), dev(x[:, :2].copy()), dev(pos), dev(inv), eps=eps)
    # (inputs that are themselves subnormal are exact; results below 2^-126 may lose steps of 2^-149)
    check_rope(oq, x, pos, inv, None, eps, True, False, 1.0)
    check_rope(ok, x[:, :2], pos, inv, None, eps, True, False, 1.0)


@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_rope_non_finite_stays_in_its_head(bad):
    note(f"rope non-finite {bad}")
    torch_cuda()
    rng = rng_for(66)
    host, _ = qkv(rng, 6, 5, 3, 64)
    x = host[0].copy()
    x[3, 2, 7] = bad
    pos, inv = np.arange(6, dtype=np.int32), freqs(32)
    oq, _ = wqa.qk_norm_rope(dev(x), None, dev(pos), dev(inv))
    got = oq.cpu().numpy()
    assert not np.isfinite(got[3, 2, [7, 39]]).any()
    want, lim = sref.rope(host[0], pos, inv, None, 1e-6, True, False, 1.0)
    ok = np.ones((6, 5), bool)
    ok[3, 2] = False
    assert (np.abs(got - want)[ok] <= lim[ok]).all()


# ------------------------------------------------------------------ prompts through a window
def check_window_prompt(out, host, lens, scale, window, sinks, what=""):
    want, sums = sref.window_prompt(*host, lens, scale, window, sinks)
    got = out.cpu().numpy().astype(np.float64)
    live = ~np.isnan(want)
    assert np.isnan(got[~live]).all(), f"{what}: a row of no sequence was written"
    lim = ref.bound(sums, min(max(lens, default=0), window + sinks), want.shape[2])
    err = np.abs(got - want)
    assert (err[live] <= lim[live]).all(), f"{what}: worst error / bound {np.nanmax(err / lim):.3f}"


@pytest.mark.parametrize("heads,kv,d", LAYOUTS + WIDE)
@pytest.mark.parametrize("lens", [[1], [2, 31, 32, 33], [0, 64, 0, 65, 1, 0], [97], [300], [127, 260, 128, 129]],
                         ids=lambda x: "-".join(map(str, x[:7])))
def test_window_prompt(heads, kv, d, lens):
    note(f"window prompt {heads} {kv} {d} {lens}")
    torch = torch_cuda()
    T = sum(lens) + 3
    host, (q, k, v) = qkv(rng_for(70, heads, d, T), T, heads, kv, d)
    for window, sinks in ((1, 0), (2, 1), (31, 5), (32, 0), (33, 32), (64, 33), (100, 4), (5, 1000), (1000, 3)):
        out = torch.full((T, heads, d), NAN, device="cuda")
        wqa.attn_prefill(q, k, v, cu=cu_of(lens), out=out, window=window, sinks=sinks)
        check_window_prompt(out, host, lens, d ** -0.5, window, sinks, f"{lens} {window} {sinks}")


@pytest.mark.parametrize("T,heads,d", [(1023, 4, 128), (2049, 4, 64), (700, 60, 128), (1400, 100, 64), (4200, 16, 128)])
@pytest.mark.parametrize("window,sinks", [(200, 4), (513, 0), (7, 70)])
def test_window_prompt_long(T, heads, d, window, sinks):
    note(f"window prompt long {T} {heads} {d} {window} {sinks}")
    torch = torch_cuda()
    host, (q, k, v) = qkv(rng_for(71, T), T, heads, 2, d)
    out = torch.full((T, heads, d), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, scale=-0.2, out=out, window=window, sinks=sinks)
    # (a few heads: the plain form is slow)
    some = [0, heads // 2 - 1, heads // 2, heads - 1] if heads > 4 else list(range(heads))
    part = [host[0][:, some], host[1][:, [j // (heads // 2) for j in some]], host[2][:, [j // (heads // 2) for j in some]]]
    check_window_prompt(out[:, some], part, [T], -0.2, window, sinks)


@pytest.mark.parametrize("heads,d,lens", [(4, 128, [90]), (14, 64, [300, 77]), (160, 128, [300])])
def test_a_window_as_long_as_the_prompts_is_no_window(heads, d, lens):
    note(f"window all {heads} {d} {lens}")
    torch = torch_cuda()
    _, (q, k, v) = qkv(rng_for(72, heads), sum(lens), heads, 2, d)
    want = wqa.attn_prefill(q, k, v, cu=cu_of(lens))
    for window, sinks in ((sum(lens), 0), (sum(lens) + 5, 9), (1 << 62, 1 << 62)):
        assert torch.equal(wqa.attn_prefill(q, k, v, cu=cu_of(lens), window=window, sinks=sinks), want)
    # a window that hides nothing of the longest prompt, by the other path
    window = max(lens)
    if window < sum(lens):
        got = wqa.attn_prefill(q, k, v, cu=cu_of(lens), window=window)
        assert torch.equal(got, want)


@pytest.mark.parametrize("heads,d", [(4, 64), (160, 128), (420, 64)])
@pytest.mark.parametrize("T", [100, 330])
@pytest.mark.parametrize("window,sinks", [(40, 0), (64, 3), (1, 40)])
def test_window_prompt_hides_what_it_hides(heads, d, T, window, sinks):
    """Keys and values that are not finite, or far larger, change only the rows that see them."""
    note(f"window prompt hidden {heads} {d} {T} {window} {sinks}")
    torch = torch_cuda()
    kv, group = 2, heads // 2
    host, _ = qkv(rng_for(73, T), T, heads, kv, d)
    some = [0, group - 1, group, heads - 1]
    want, sums = sref.window_prompt(host[0][:, some], host[1][:, [j // group for j in some]], host[2][:, [j // group for j in some]],
                                    [T], d ** -0.5, window, sinks)
    lim = ref.bound(sums, min(T, window + sinks), d)
    t = np.arange(T)
    for at in (0, 2, 33, T // 2):
        sees = (t >= at) & ((at > t - window) | (at < sinks))
        for which in (1, 2):
            for bad in (NAN, float("inf"), 1e20):
                arr = [x.copy() for x in host]
                arr[which][at, 1, 5] = bad
                out = torch.full((T, heads, d), NAN, device="cuda")
                wqa.attn_prefill(*(dev(x) for x in arr), out=out, window=window, sinks=sinks)
                got = out.cpu().numpy()[:, some]
                hit = np.zeros(got.shape, bool)
                hit[sees, 2:] = True
                if bad != 1e20:
                    hard = hit.copy()
                    if which == 2:
                        hard[..., :5] = hard[..., 6:] = False
                        hit = hard
                    assert np.isnan(got[hard]).all() if which == 1 or bad != float("inf") else not np.isfinite(got[hard]).any()
                # (1e20 is more than 2^14 above its tile, so hidden rows keep units of their own)
                assert (np.abs(got - want)[~hit] <= lim[~hit]).all(), (at, which, bad)


# ------------------------------------------------------------------ decode through a window
def check_rows(out, want, sums, n, d, what=""):
    got = out.cpu().numpy().astype(np.float64)
    lim = ref.bound(sums, n, d)
    err = np.abs(got - want)
    assert (err <= lim).all(), f"{what}: worst error / bound {np.nanmax(err / lim):.3f}"


@pytest.mark.parametrize("heads,kv,d", LAYOUTS + [(8, 1, 128), (32, 2, 64), (3, 3, 128), (20, 1, 64)])
@pytest.mark.parametrize("lens", [[1], [0, 1, 63, 64, 65, 0, 200, 15], [700], [1100, 0, 300, 2], [5000, 9, 2300, 0, 4097]], ids=lambda x: "-".join(map(str, x[:8])))
def test_window_decode(heads, kv, d, lens):
    """Pages of hidden tokens are given away: their table entries point nowhere, their scales are NaN."""
    note(f"window decode {heads} {kv} {d} {lens}")
    torch = torch_cuda()
    rng = rng_for(75, heads, kv, d, len(lens))
    table, pages = table_for(rng, lens)
    host, _ = cache_arrays(rng, pages, kv, d)
    kval, vval = ref.values(host[0], host[1]), ref.values(host[2], host[3])
    q = rng.standard_normal((len(lens), heads, d)).astype(np.float32) * 2
    for window, sinks in ((1, 0), (2, 1), (64, 0), (65, 64), (100, 4), (129, 130), (3000, 5), (10000, 0)):
        want, sums = sref.decode(q, kval, vval, host[3], d ** -0.5, lambda b: [(table[b], lens[b], sref.seen(lens[b], window, sinks))])
        tab = table.copy()
        spoilt = [x.copy() for x in host]
        for b, n in enumerate(lens):
            see = sref.seen(n, window, sinks)
            for p in range(-(-n // 64)):
                if not see[p * 64:(p + 1) * 64].any():
                    tab[b, p] = rng.choice([-1, pages + 5, 2 ** 31 - 1])
                else:
                    gone = np.flatnonzero(~np.pad(see[p * 64:(p + 1) * 64], (0, 64))[:64])
                    for j in (1, 3):
                        spoilt[j][table[b, p], :, gone] = np.nan
        out = torch.full(q.shape, NAN, device="cuda")
        wqa.attn_decode(dev(q), cache_on(spoilt), dev(tab), ints(lens), out=out, window=window, sinks=sinks)
        check_rows(out, want, sums, min(max(lens), window + sinks), d, f"{lens} {window} {sinks}")


def test_window_decode_of_a_short_sequence_is_decode():
    note("window decode short")
    torch = torch_cuda()
    rng = rng_for(76)
    lens = [40, 64, 1, 0, 63]
    table, pages = table_for(rng, [900] * 5)
    _, cache = cache_arrays(rng, pages, 2, 64)
    q = dev(rng.standard_normal((5, 4, 64)).astype(np.float32))
    want = wqa.attn_decode(q, cache, dev(table[:, :3].copy()), ints(lens))
    assert torch.equal(wqa.attn_decode(q, cache, dev(table), ints(lens), window=64), want)
    assert torch.equal(wqa.attn_decode(q, cache, dev(table[:, :3].copy()), ints(lens), window=1 << 60, sinks=1 << 60), want)


def test_window_decode_bad_pages_and_lengths():
    note("window decode bad")
    torch_cuda()
    rng = rng_for(77)
    lens = [300, 300, 300, 300, -1, 2 ** 31 - 1]
    table, pages = table_for(rng, [300] * 6)
    host, cache = cache_arrays(rng, pages, 2, 64)
    table[1, 4] = pages                            # seen: the last page
    table[2, 0] = -1                               # seen: the first tokens' page
    table[3, 1:3] = -5                             # hidden
    q = rng.standard_normal((6, 4, 64)).astype(np.float32)
    got = wqa.attn_decode(dev(q), cache, dev(table), ints(lens), window=70, sinks=2).cpu().numpy()
    assert np.isnan(got[[1, 2, 4, 5]]).all()
    kval, vval = ref.values(host[0], host[1]), ref.values(host[2], host[3])
    want, sums = sref.decode(q[[0, 3]], kval, vval, host[3], 0.125, lambda b: [(table[[0, 3]][b], 300, sref.seen(300, 70, 2))])
    assert (np.abs(got[[0, 3]] - want) <= ref.bound(sums, 72, 64)).all()


# ------------------------------------------------------------------ a shared prefix
def shared_case(rng, heads, kv, d, prefix, lens, spare=2):
    table, pages = table_for(rng, [prefix] + list(lens), spare)
    host, cache = cache_arrays(rng, pages, kv, d)
    q = rng.standard_normal((len(lens), heads, d)).astype(np.float32) * 2
    return table[0, :-(-prefix // 64) + 1].copy(), table[1:].copy(), host, cache, q


def check_shared(out, q, host, pre, prefix, table, lens, scale, what=""):
    kval, vval = ref.values(host[0], host[1]), ref.values(host[2], host[3])
    want, sums = sref.decode(q, kval, vval, host[3], scale, lambda b: [(pre, prefix, None), (table[b], lens[b], None)])
    check_rows(out, want, sums, prefix + max(lens), q.shape[2], what)


@pytest.mark.parametrize("heads,kv,d", LAYOUTS + [(8, 1, 128), (40, 2, 64), (3, 3, 128), (20, 1, 64)])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 200, 777])
@pytest.mark.parametrize("lens", [[5], [0, 1, 64, 200, 0, 15, 33]], ids=lambda x: "-".join(map(str, x[:8])))
def test_shared(heads, kv, d, prefix, lens):
    note(f"shared {heads} {kv} {d} {prefix} {lens}")
    torch = torch_cuda()
    rng = rng_for(80, heads, kv, d, prefix)
    pre, table, host, cache, q = shared_case(rng, heads, kv, d, prefix, lens)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([prefix]), dev(table), ints(lens), out=out)
    check_shared(out, q, host, pre, prefix, table, lens, d ** -0.5, f"{prefix} {lens}")


@pytest.mark.parametrize("count,heads,kv,d,prefix,longest", [(16, 16, 8, 128, 1300, 2000), (33, 4, 2, 64, 4000, 100), (70, 14, 2, 64, 2111, 300),
                                                              (300, 8, 2, 64, 500, 40), (9, 32, 2, 128, 6000, 1500), (150, 2, 1, 128, 1000, 30),
                                                              (1, 16, 2, 128, 40000, 700), (3, 16, 8, 128, 6000, 300), (8, 4, 2, 64, 9000, 700), (5, 6, 2, 64, 2500, 1200), (17, 2, 2, 128, 3000, 64)])
def test_shared_large(count, heads, kv, d, prefix, longest):
    """More rows than a workgroup holds, prefixes in many runs, own tokens that are cut."""
    note(f"shared large {count} {heads} {kv} {d} {prefix} {longest}")
    torch = torch_cuda()
    rng = rng_for(81, count, prefix)
    lens = [int(x) for x in rng.integers(0, longest, count)]
    lens[-1], lens[count // 2] = longest, 0
    pre, table, host, cache, q = shared_case(rng, heads, kv, d, prefix, lens)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([prefix]), dev(table), ints(lens), scale=-0.07, out=out)
    check_shared(out, q, host, pre, prefix, table, lens, -0.07)


@pytest.mark.parametrize("count,heads,kv,d,prefix,longest", [(40, 4, 2, 128, 9000, 60), (70, 2, 2, 128, 9001, 700), (33, 4, 2, 64, 17000, 50),
                                                              (200, 14, 2, 64, 16700, 20), (65, 8, 1, 128, 8300, 9)])
@pytest.mark.parametrize("shown", [1.0, 0.03, 0.0])
def test_shared_long_tables(count, heads, kv, d, prefix, longest, shown):
    """Workgroups of 128 rows, with all of a long prefix and with little of it in a table made for all."""
    note(f"shared long {count} {heads} {kv} {d} {prefix} {longest} {shown}")
    torch = torch_cuda()
    rng = rng_for(87, count, prefix)
    lens = [int(x) for x in rng.integers(0, longest, count)]
    lens[-1], lens[count // 2] = longest, 0
    pre, table, host, cache, q = shared_case(rng, heads, kv, d, prefix, lens)
    seen = int(prefix * shown)
    pre[-(-seen // 64):] = -3                      # past it: anything
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([seen]), dev(table), ints(lens), out=out)
    check_shared(out, q, host, pre, seen, table, lens, d ** -0.5)


def test_shared_strides_and_wide_rows():
    note("shared strides")
    torch = torch_cuda()
    rng = rng_for(82)
    pre, table, host, cache, q = shared_case(rng, 6, 3, 64, 150, [70, 0, 9])
    wide_q = torch.zeros(3, 6 * 64 + 20, device="cuda")
    wide_q[:, 8:8 + 384] = dev(q).view(3, -1)
    wide = torch.full((3, 6 * 64 + 36), NAN, device="cuda")
    out = wide[:, 16:16 + 384].unflatten(1, (6, 64))
    wqa.attn_decode_shared(wide_q[:, 8:8 + 384].unflatten(1, (6, 64)), cache, dev(pre), ints([150]), dev(table), ints([70, 0, 9]), out=out)
    check_shared(out, q, host, pre, 150, table, [70, 0, 9], 0.125)
    assert torch.isnan(wide[:, :16]).all() and torch.isnan(wide[:, 16 + 384:]).all()


@pytest.mark.parametrize("what", ["peaked", "key_scales", "value_scales", "tiny", "huge", "equal", "zero_values", "negative_scales", "below_range"])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_range(what, d):
    note(f"shared range {what} {d}")
    torch = torch_cuda()
    rng = rng_for(83, d, len(what))
    prefix, lens, heads, kv, scale = 333, [100, 3, 0], 6, 2, d ** -0.5
    pre, table, host, _, q = shared_case(rng, heads, kv, d, prefix, lens)
    if what == "peaked":
        q *= 60.0
    elif what == "key_scales":
        host[1][:] = np.exp2(rng.uniform(-24, 0, host[1].shape))
    elif what == "value_scales":
        host[3][:] = np.exp2(rng.uniform(-24, 15, host[3].shape))
    elif what == "tiny":
        q *= 1e-30
        scale = 1e30
        host[3][:] = np.exp2(-24.0)
    elif what == "huge":
        q *= 1e30
        scale = 1e-31
        host[3][:] = 60000.0
    elif what == "equal":
        host[0][:] = host[0][:1, :, :1]
        host[1][:] = host[1][:1, :, :1]
    elif what == "zero_values":
        host[3][pre[0]] = 0.0
        host[2][pre[1]] = 0
    elif what == "negative_scales":
        host[1][:] *= rng.choice([-1, 1], host[1].shape)
        host[3][:] *= rng.choice([-1, 1], host[3].shape)
    else:
        q *= 1e-38
        scale = 1e-30
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode_shared(dev(q), cache_on(host), dev(pre), ints([prefix]), dev(table), ints(lens), scale=scale, out=out)
    check_shared(out, q, host, pre, prefix, table, lens, scale, what)


def test_shared_rows_past_the_lengths_may_hold_anything():
    note("shared past")
    torch = torch_cuda()
    rng = rng_for(84)
    prefix, lens = 70, [1, 0, 65]
    pre, table, host, _, q = shared_case(rng, 4, 2, 64, prefix, lens)
    dirty = [x.copy() for x in host]
    for ids, n in [(pre, prefix)] + list(zip(table, lens)):
        if n % 64:
            for j, bad in ((0, -8), (1, np.nan), (2, 7), (3, np.inf)):
                dirty[j][ids[n // 64], :, n % 64:] = bad
    want, got = (wqa.attn_decode_shared(dev(q), cache_on(h), dev(pre), ints([prefix]), dev(table), ints(lens)) for h in (host, dirty))
    assert torch.equal(want, got)
    check_shared(got, q, host, pre, prefix, table, lens, 0.125)


def test_shared_bad_pages_and_lengths():
    note("shared bad")
    torch = torch_cuda()
    rng = rng_for(85)
    prefix, lens = 200, [100, 0, 30, 64]
    pre, table, host, cache, q = shared_case(rng, 4, 2, 64, prefix, lens)
    pages = cache.n_pages

    def call(pre=pre, prefix=prefix, table=table, lens=lens, cache=cache):
        out = torch.full(q.shape, -3.0, device="cuda")
        wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([prefix]), dev(table), ints(lens), out=out)
        return out.cpu().numpy()
    good = call()
    for n in (-1, 64 * len(pre) + 1, 2 ** 31 - 1, -2 ** 31):
        assert np.isnan(call(prefix=n)).all(), n
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        p = pre.copy()
        p[2] = bad
        assert np.isnan(call(pre=p)).all()
        p = pre.copy()
        p[4] = bad                                 # past the prefix
        assert np.array_equal(call(pre=p), good)
        t = table.copy()
        t[0, 1] = bad
        got = call(table=t)
        assert np.isnan(got[0]).all() and np.array_equal(got[1:], good[1:])
    got = call(lens=[100, -1, 2 ** 30, 64])
    assert np.isnan(got[[1, 2]]).all() and np.array_equal(got[[0, 3]], good[[0, 3]])
    zeros = call(prefix=0, lens=[0, 0, 30, 0])
    assert (zeros[[0, 1, 3]] == 0).all()
    # an empty cache, and tables without columns
    none = wqa.KVCache.empty(0, 2, 64)
    assert np.isnan(call(cache=none)).all()
    assert (call(cache=none, prefix=0, lens=[0] * 4) == 0).all()
    assert (call(pre=pre[:0], prefix=0, table=table[:, :0], lens=[0] * 4) == 0).all()
    assert np.isnan(call(pre=pre[:0], prefix=1, table=table[:, :0], lens=[0] * 4)).all()
    own = call(pre=pre[:0], prefix=0)
    want = wqa.attn_decode(dev(q), cache, dev(table), ints(lens)).cpu().numpy()
    assert np.allclose(own, want, rtol=4 * ref.U32, atol=0)      # divided, multiplied and divided again
    assert np.array_equal(call(table=table[:, :0], lens=[0] * 4)[1], good[1])


@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_shared_non_finite(bad):
    note(f"shared non-finite {bad}")
    torch_cuda()
    rng = rng_for(86)
    prefix, lens, d = 100, [20, 5, 0], 64
    pre, table, host, _, q = shared_case(rng, 4, 2, d, prefix, lens)
    kval, vval = ref.values(host[0], host[1]), ref.values(host[2], host[3])
    want, sums = sref.decode(q, kval, vval, host[3], 0.125, lambda b: [(pre, prefix, None), (table[b], lens[b], None)])
    lim = ref.bound(sums, prefix + 20, d)

    def call(q, h):
        return wqa.attn_decode_shared(dev(q), cache_on(h), dev(pre), ints([prefix]), dev(table), ints(lens)).cpu().numpy()
    x = q.copy()
    x[1, 2, 3] = bad
    got = call(x, host)
    hit = np.zeros(q.shape, bool)
    hit[1, 2] = True
    assert np.isnan(got[hit]).all() and (np.abs(got - want)[~hit] <= lim[~hit]).all()
    h = [a.copy() for a in host]
    h[3][pre[0], 1, 40, 1] = bad                   # a value scale of head 1, block 1
    got = call(q, h)
    hit[:] = False
    hit[:, 2:, 32:] = True
    assert not np.isfinite(got[hit]).any() and (np.abs(got - want)[~hit] <= lim[~hit]).all()
    if np.isnan(bad):
        h = [a.copy() for a in host]
        h[1][pre[0], 0, 63, 0] = bad
        got = call(q, h)
        hit[:] = False
        hit[:, :2] = True
        assert np.isnan(got[hit]).all() and (np.abs(got - want)[~hit] <= lim[~hit]).all()


# ------------------------------------------------------------------ together
def test_serving_steps():
    """Prompts arrive, are planned, rotated and cached; then single tokens, through a
    window and all; then a batch behind the first prompt. Every attention is checked
    against the cache's own bytes, and those against the host's."""
    note("serving steps")
    torch = torch_cuda()
    rng = rng_for(90)
    heads, kv, d, width = 8, 2, 128, 9
    pages = 40
    free, taken = dev(rng.permutation(pages).astype(np.int32)), None
    cache = wqa.KVCache.empty(pages, kv, d)
    lens = np.array([130, 0, 300, 64])
    table = dev(np.full((4, width), -1, np.int32))
    hostc = [np.zeros((pages, kv, 64, d), np.int8), np.zeros((pages, kv, 64, d // 32), np.float16)] * 2
    hostc = [x.copy() for x in hostc]
    inv, w = freqs(64), rng.standard_normal(d).astype(np.float32)
    before = np.zeros(4, int)
    used = 0
    for fresh in (lens, np.array([1, 70, 1, 0]), np.array([1, 1, 1, 1])):
        T = int(fresh.sum())
        host, (q, k, v) = qkv(rng, T, heads, kv, d)
        want = sref.plan(fresh.tolist(), before.tolist(), table.cpu().numpy(), free.cpu().numpy(), used, T + 2)
        p = wqa.kv_plan(ints(fresh), table, free, taken, tokens=T + 2, start=ints(before))
        check_plan(p, table, want, T + 2)
        taken, used = p.taken, int(want[5][0])
        qr, kr = wqa.qk_norm_rope(q, k, p.positions[:T], dev(inv), q_weight=dev(w))
        check_rope(qr, host[0], want[3][:T], inv, w, 1e-6, True, False, 1.0)
        wqa.kv_append(cache, kr, v, slots=p.slots[:T])
        krh = kr.cpu().numpy()
        for t in range(T):
            page, row = divmod(int(want[4][t]), 64)
            for j, x in ((0, krh), (2, host[2])):
                hostc[j][page, :, row], hostc[j + 1][page, :, row] = ref.quantize(x[t])
        for j, t in enumerate(cache):
            assert np.array_equal(t.cpu().numpy(), ref.nibbles(hostc[j]) if j % 2 == 0 else hostc[j].view(np.int16)), j
        o = wqa.attn_prefill(qr, kr, v, cu=p.cu, window=100, sinks=4)
        check_window_prompt(o, [qr.cpu().numpy(), krh, host[2]], fresh.tolist(), d ** -0.5, 100, 4)
        before = before + fresh
    kval, vval = ref.values(hostc[0], hostc[1]), ref.values(hostc[2], hostc[3])
    tab = want[0]
    qh = qr.cpu().numpy()
    assert np.array_equal(p.lens.cpu().numpy(), before)
    for window, sinks in ((None, 0), (100, 4)):
        o = wqa.attn_decode(qr, cache, table, p.lens, window=window, sinks=sinks)
        r, sums = sref.decode(qh, kval, vval, hostc[3], d ** -0.5,
                              lambda b: [(tab[b], before[b], None if window is None else sref.seen(before[b], window, sinks))])
        check_rows(o, r, sums, int(before.max()), d)
    # the others as questions about request 2's tokens
    o = wqa.attn_decode_shared(qr, cache, table[2], p.lens[2:3], table, p.lens)
    r, sums = sref.decode(qh, kval, vval, hostc[3], d ** -0.5, lambda b: [(tab[2], before[2], None), (tab[b], before[b], None)])
    check_rows(o, r, sums, 2 * int(before.max()), d)


def test_serving_step_on_another_stream_and_in_a_graph():
    """A whole step on a side stream and captured: every replay gives the eager
    bits, with lengths, positions and pages that change on the device."""
    note("serving graph")
    torch = torch_cuda()
    rng = rng_for(91)
    heads, kv, d, B, width = 8, 2, 128, 3, 40
    pages = 200
    cache = wqa.KVCache.empty(pages, kv, d)
    for t in cache:
        t.copy_(dev(rng.integers(0, 100, tuple(t.shape)).astype(np.uint8)).to(t.dtype) if t.dtype == torch.uint8 else
                torch.full_like(t, 0x3000))
    table = dev(rng.integers(0, pages, (B, width)).astype(np.int32))
    y = dev(rng.standard_normal((B, (heads + 2 * kv) * d)).astype(np.float32))
    q, k, v = y[:, :heads * d].view(B, heads, d), y[:, heads * d:-kv * d].view(B, kv, d), y[:, -kv * d:].view(B, kv, d)
    start, fresh, taken = ints([100, 2000, 63]), ints([1, 1, 1]), ints([0])
    free, inv = ints(rng.permutation(pages)), dev(freqs(64))
    pq, pk, pv = (dev(rng.standard_normal((400, n, d)).astype(np.float32)) for n in (heads, kv, kv))
    prefix, plen = ints(rng.permutation(pages)[:30]), ints([1900])
    pcu = cu_of([350, 50])

    def step(stream=None):
        p = wqa.kv_plan(fresh, table, free, taken, tokens=B, start=start, stream=stream)
        a, b = wqa.qk_norm_rope(q, k, p.positions, inv, stream=stream)
        wqa.kv_append(cache, b, v, slots=p.slots, stream=stream)
        return tuple(p) + (a, b, wqa.attn_decode(a, cache, table, p.lens, window=1500, sinks=4, stream=stream),
                           wqa.attn_decode_shared(a, cache, prefix, plen, table, p.lens, stream=stream),
                           wqa.attn_prefill(pq, pk, pv, cu=pcu, window=90, sinks=1, stream=stream))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = step()
    side.synchronize()
    again = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, warm))
    now = step()
    assert all(torch.equal(a, b) for a, b in zip(now, warm))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = step()
    for i, at in enumerate(([100, 2000, 63], [2540, 64, 128], [0, 0, 0], [10, 1000, 700])):
        start.copy_(ints(at))
        plen.copy_(ints([[1900, 5, 0, 1856][i]]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in caught]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), at


def test_serving_calls_on_two_streams_at_once():
    note("serving two streams")
    torch = torch_cuda()
    rng = rng_for(92)
    lens = [700, 1500, 64]
    pre, table, _, cache, q = shared_case(rng, 8, 2, 128, 3000, lens)
    _, (pq, pk, pv) = qkv(rng, 900, 8, 2, 128)
    args = (dev(q), cache, dev(pre), ints([3000]), dev(table), ints(lens))

    def calls():
        return (wqa.attn_decode_shared(*args), wqa.attn_decode(args[0], cache, args[4], args[5], window=600, sinks=3),
                wqa.attn_prefill(pq, pk, pv, window=77, sinks=5))
    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(calls())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_serving_past_four_gib():
    """Pages whose byte offsets pass 32 bits: slots, windows and a shared prefix."""
    note("serving past 4 GiB")
    torch = torch_cuda()
    n, kv, d, heads = 140000, 8, 128, 16           # 4.27 GiB of codes each for keys and values
    big = wqa.KVCache(*(torch.empty((n, kv, 64, w), dtype=t, device="cuda")
                        for w, t in ((64, torch.uint8), (4, torch.int16), (64, torch.uint8), (4, torch.int16))))
    rng = rng_for(93)
    T = 1200
    _, (q, k, v) = qkv(rng, T, heads, kv, d)
    ids = np.array([n - 1, 0, 131072, 131071] + list(range(n - 20, n - 5)), np.int64)
    small = wqa.KVCache.empty(len(ids), kv, d)
    t = np.arange(T)
    wqa.kv_append(big, k, v, slots=dev(ids[t // 64] * 64 + t % 64))
    wqa.kv_append(small, k, v, slots=dev(t.astype(np.int64)))
    at = torch.from_numpy(ids).cuda()
    assert all(torch.equal(a[at][:18], b[:18]) for a, b in zip(big, small))
    for rows in (2, 40):
        ln = ints([T - 3 * i for i in range(rows)])
        qr = q[:rows].contiguous()
        for c, tab in ((big, ids), (small, np.arange(len(ids)))):
            table = ints(np.tile(tab, (rows, 1)))
            got = (wqa.attn_decode(qr, c, table, ln, window=700, sinks=3),
                   wqa.attn_decode_shared(qr, c, table[0], ln[:1], table[:, :3].contiguous(), ln.clamp(max=150)))
            if c is big:
                want = got
        assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(got, want))


@pytest.mark.parametrize("seed", range(12))
def test_serving_random_shapes(seed):
    """Sizes no list has: windows of prompts and of single tokens, shared prefixes."""
    torch = torch_cuda()
    rng = rng_for(94, seed)
    heads, kv, d = [(16, 8, 128), (4, 4, 64), (14, 2, 64), (12, 1, 128), (6, 3, 128), (9, 1, 64), (34, 2, 64)][rng.integers(7)]
    window, sinks = int(np.exp(rng.uniform(0, 7))), int(rng.choice([0, 1, 5, 31, 64, 100]))
    lens = [int(x) for x in rng.integers(0, int(rng.choice([5, 70, 400])), rng.integers(1, 9))]
    note(f"random {seed} {heads} {kv} {d} {window} {sinks} {lens}")
    host, (q, k, v) = qkv(rng, sum(lens) + 1, heads, kv, d)
    out = torch.full((sum(lens) + 1, heads, d), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, cu=cu_of(lens), out=out, window=window, sinks=sinks)
    check_window_prompt(out, host, lens, d ** -0.5, window, sinks)
    count, prefix = int(rng.integers(1, 60)), int(rng.integers(0, 3000))
    lens = [int(x) for x in rng.integers(0, int(rng.choice([3, 200, 2500])), count)]
    pre, table, host, cache, q = shared_case(rng, heads, kv, d, prefix, lens)
    kval, vval = ref.values(host[0], host[1]), ref.values(host[2], host[3])
    out = wqa.attn_decode(dev(q), cache, dev(table), ints(lens), window=window, sinks=sinks)
    want, sums = sref.decode(q, kval, vval, host[3], d ** -0.5, lambda b: [(table[b], lens[b], sref.seen(lens[b], window, sinks))])
    check_rows(out, want, sums, min(max(lens), window + sinks), d)
    out = wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([prefix]), dev(table), ints(lens))
    check_shared(out, q, host, pre, prefix, table, lens, d ** -0.5)


def test_serving_refusals():
    torch = torch_cuda()
    q, k = torch.zeros((4, 4, 64), device="cuda"), torch.zeros((4, 2, 64), device="cuda")
    cache = wqa.KVCache.empty(2, 2, 64)
    tab, ln = torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    inv, slots = torch.ones(32, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    one = ln[:1].clone()
    plan = wqa.kv_plan(ln, tab, ln, tokens=4)
    bad = [lambda: wqa.attn_prefill(q, k, k, window=0), lambda: wqa.attn_prefill(q, k, k, window=-1), lambda: wqa.attn_prefill(q, k, k, sinks=2),
           lambda: wqa.attn_prefill(q, k, k, window=3, sinks=-1), lambda: wqa.attn_prefill(q, k, k, window=2.0), lambda: wqa.attn_prefill(q, k, k, window=True),
           lambda: wqa.attn_decode(q, cache, tab, ln, window=0), lambda: wqa.attn_decode(q, cache, tab, ln, sinks=1),
           lambda: wqa.attn_decode(q, cache, tab, ln, window=4, sinks=1.5),
           lambda: wqa.kv_append(cache, k, k), lambda: wqa.kv_append(cache, k, k, tab[:1], slots=slots), lambda: wqa.kv_append(cache, k, k, slots=ln),
           lambda: wqa.kv_append(cache, k, k, slots=slots[:3]), lambda: wqa.kv_append(cache, k, k, slots=slots.cpu()),
           lambda: wqa.attn_decode_shared(q, cache, tab, one, tab, ln), lambda: wqa.attn_decode_shared(q, cache, ln, ln, tab, ln),
           lambda: wqa.attn_decode_shared(q, cache, ln.long(), one, tab, ln), lambda: wqa.attn_decode_shared(q, cache, ln, 3, tab, ln),
           lambda: wqa.attn_decode_shared(q, cache, ln, one, tab[:2], ln), lambda: wqa.attn_decode_shared(q[:, :3].contiguous(), cache, ln, one, tab, ln),
           lambda: wqa.qk_norm_rope(q, k[:3], ln, inv), lambda: wqa.qk_norm_rope(q, k, ln[:3], inv), lambda: wqa.qk_norm_rope(q, k, ln.long(), inv),
           lambda: wqa.qk_norm_rope(q, k, ln, inv[:30]), lambda: wqa.qk_norm_rope(q, k, ln, torch.ones(36, device="cuda")),
           lambda: wqa.qk_norm_rope(q, k, ln, inv.double()), lambda: wqa.qk_norm_rope(q, k, ln, inv, q_weight=inv),
           lambda: wqa.qk_norm_rope(q, k, ln, inv, q_weight=torch.ones(64, device="cuda"), norm=False), lambda: wqa.qk_norm_rope(q, None, ln, inv, k_out=k),
           lambda: wqa.qk_norm_rope(q, k, ln, inv, q_out=k), lambda: wqa.qk_norm_rope(q, k, ln, inv, q_weight=torch.ones(65, device="cuda")[1:]),
           lambda: wqa.qk_norm_rope(q[..., :32].contiguous(), None, ln, inv[:16]),
           lambda: wqa.kv_plan(ln, tab[:2], ln), lambda: wqa.kv_plan(ln.long(), tab, ln), lambda: wqa.kv_plan(ln, tab, tab), lambda: wqa.kv_plan(ln, tab, ln, ln),
           lambda: wqa.kv_plan(ln, tab, ln, tokens=-1), lambda: wqa.kv_plan(ln, tab, ln, tokens=2.0), lambda: wqa.kv_plan(ln, tab, ln, start=one),
           lambda: wqa.kv_plan(ln, tab, ln, tokens=5, out=plan), lambda: wqa.kv_plan(ln, tab, ln, plan.taken, tokens=4, out=plan)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, wqa.WqError)):
            f()
            pytest.fail(f"call {i} was accepted")
    # nothing to do
    assert wqa.attn_prefill(q[:0], k[:0], k[:0], window=4).shape == (0, 4, 64)
    assert wqa.attn_decode(q[:0], cache, tab[:0], ln[:0], window=4).shape == (0, 4, 64)
    assert wqa.attn_decode_shared(q[:0], cache, ln, one, tab[:0], ln[:0]).shape == (0, 4, 64)
    assert wqa.qk_norm_rope(q[:0], k[:0], ln[:0], inv)[1].shape == (0, 2, 64)
    wqa.kv_append(cache, k[:0], k[:0], slots=slots[:0])


@pytest.mark.parametrize("count,heads,kv,d", [(4, 8, 2, 128), (40, 4, 2, 64), (70, 2, 1, 128)])
def test_pages_that_are_named_more_than_once(count, heads, kv, d):
    """Rows that share pages with one another, with the prefix and with themselves."""
    note(f"pages twice {count} {heads} {kv} {d}")
    torch = torch_cuda()
    rng = rng_for(95, count)
    host, cache = cache_arrays(rng, 4, kv, d)
    table, pre = rng.integers(0, 4, (count, 9)).astype(np.int32), np.array([2, 2, 0, 1, 2, 3, 3], np.int32)
    table[1] = table[0]
    lens = rng.integers(0, 9 * 64 + 1, count)
    lens[:2] = 9 * 64
    q = (rng.standard_normal((count, heads, d)) * 2).astype(np.float32)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([7 * 64 - 1]), dev(table), ints(lens), out=out)
    check_shared(out, q, host, pre, 7 * 64 - 1, table, lens, d ** -0.5)
    kval, vval = ref.values(host[0], host[1]), ref.values(host[2], host[3])
    out = wqa.attn_decode(dev(q), cache, dev(table), ints(lens), window=150, sinks=70)
    want, sums = sref.decode(q, kval, vval, host[3], d ** -0.5, lambda b: [(table[b], lens[b], sref.seen(lens[b], 150, 70))])
    check_rows(out, want, sums, 220, d)


def test_one_slot_for_two_tokens_spoils_only_itself():
    note("slot twice")
    torch = torch_cuda()
    kv, d, T = 2, 128, 300
    _, (_, k, v) = qkv(rng_for(96), T, kv, kv, d)
    slots = np.arange(T) + 20
    slots[[5, 250]] = 150                          # the place of token 130
    caches = [wqa.KVCache.empty(6, kv, d) for _ in range(2)]
    for c in caches:
        for t in c:
            t.zero_()
    wqa.kv_append(caches[0], k, v, slots=dev(slots))
    slots[[5, 250, 130]] = -1
    wqa.kv_append(caches[1], k, v, slots=dev(slots))
    for a, b in zip(*caches):
        a[150 // 64, :, 150 % 64] = 0
        assert torch.equal(a, b)


def test_plan_of_no_requests_and_into_its_own_inputs():
    note("plan edges")
    torch = torch_cuda()
    none = ints([])
    p = wqa.kv_plan(none, none.view(0, 4), ints([1, 2]), ints([1]), tokens=5)
    assert p.cu.tolist() == [0] and p.lens.numel() == 0 and p.positions.tolist() == [-1] * 5 == p.slots.tolist() and p.taken.tolist() == [1]
    fresh, table, free = ints([1, 1]), ints([[-1] * 3] * 2), ints([4, 5, 6])
    p = wqa.kv_plan(fresh, table, free, tokens=2)
    before = [t.clone() for t in p] + [table.clone()]
    for kw in (dict(start=p.lens), dict(taken=p.taken), dict(start=p.positions)):
        with pytest.raises((ValueError, wqa.WqError)):
            wqa.kv_plan(fresh, table, free, tokens=2, out=p, **kw)
    with pytest.raises(wqa.WqError):
        wqa.kv_plan(p.lens, table, free, tokens=2, out=p)
    with pytest.raises(wqa.WqError):
        wqa.kv_plan(fresh, table, table.view(-1), tokens=2)
    with pytest.raises(wqa.WqError):
        wqa.kv_plan(fresh, table, free, tokens=2, out=p._replace(positions=p.lens))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, tuple(p) + (table,)))


def test_a_captured_step_that_goes_on_by_itself():
    """Lengths and the place in the list of free pages advance on the device: replays are steps."""
    note("captured loop")
    torch = torch_cuda()
    B, width, pages = 5, 6, 40
    rng = rng_for(97)
    first = rng.integers(0, 130, B)
    free, fresh = ints(rng.permutation(pages)), ints([1, 1, 0, 2, 1])

    def state():
        table = ints(np.full((B, width), -1))
        p = wqa.kv_plan(ints(first), table, free)
        return table, p.lens.clone(), p.taken.clone()

    def step(table, start, taken):
        p = wqa.kv_plan(fresh, table, free, taken, tokens=8, start=start)
        start.add_(fresh)
        torch.add(p.taken, 0, out=taken)
        return p

    eager, caught = state(), state()
    step(*state())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = step(*caught)
    for i in range(70):
        graph.replay()
        p = step(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(tuple(p) + eager, tuple(q) + caught)), i
    want = sref.plan((70 * fresh.cpu().numpy() + first).tolist(), [0] * B, np.full((B, width), -1, np.int32), free.cpu().numpy(), 0, 0)
    assert np.array_equal(np.sort(caught[0].cpu().numpy(), None), np.sort(want[0], None)) and np.array_equal(p.taken.cpu().numpy(), want[5])


def test_two_graphs_of_one_pool():
    """Replayed in turns: neither keeps anything of its workspace from one replay to the next."""
    note("two graphs")
    torch = torch_cuda()
    rng = rng_for(98)
    cases, graphs, caught, want = [], [], [], []
    for heads, kv, d, prefix, lens in ((8, 2, 128, 3000, [700, 1500, 64]), (14, 2, 64, 2000, [300] * 40)):
        pre, table, _, cache, q = shared_case(rng, heads, kv, d, prefix, lens)
        cases.append((dev(q), cache, dev(pre), ints([prefix]), dev(table), ints(lens), *qkv(rng, 500, heads, kv, d)[1]))

    def calls(q, cache, pre, n, table, lens, pq, pk, pv):
        return (wqa.attn_decode_shared(q, cache, pre, n, table, lens), wqa.attn_decode(q, cache, table, lens, window=600, sinks=3),
                wqa.attn_prefill(pq, pk, pv, window=77, sinks=5))
    for c in cases:
        want.append(calls(*c))
    torch.cuda.synchronize()
    pool = torch.cuda.graph_pool_handle()
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            caught.append(calls(*c))
    for i in (0, 1, 1, 0, 1, 0, 0, 1):
        for t in caught[i]:
            t.fill_(NAN)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(caught[i], want[i])), i


def test_rows_gigabytes_apart():
    """Tokens 2 GiB from one another: offsets pass 32 bits in every operator that takes rows with a stride."""
    note("rows far apart")
    torch = torch_cuda()
    rng = rng_for(99)
    heads, kv, d, T, far = 8, 2, 128, 6, 1 << 29
    host, (q, k, v) = qkv(rng, T, heads, kv, d)
    big = torch.empty((T - 1) * far + 8 * heads * d, device="cuda")
    spots = iter(range(0, 8 * heads * d, heads * d))

    def away(t=None, n=heads):
        y = big.as_strided((T, n, d), (far, d, 1), next(spots))
        return y if t is None else y.copy_(t)
    fq, fk, fv = away(q), away(k, kv), away(v, kv)
    pos, inv, w = ints(np.arange(T) * 1000), dev(freqs(64)), dev(rng.standard_normal(d).astype(np.float32))
    want = wqa.qk_norm_rope(q, k, pos, inv, q_weight=w)
    got = wqa.qk_norm_rope(fq, fk, pos, inv, q_weight=w, q_out=away(), k_out=away(n=kv))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = away()
    assert torch.equal(wqa.attn_prefill(fq, fk, fv, out=out, window=3, sinks=1), wqa.attn_prefill(q, k, v, window=3, sinks=1))
    slots = dev(np.arange(T, dtype=np.int64) * 70)
    caches = [wqa.KVCache(*(t.zero_() for t in wqa.KVCache.empty(8, kv, d))) for _ in range(2)]
    wqa.kv_append(caches[0], k, v, slots=slots)
    wqa.kv_append(caches[1], fk, fv, slots=slots)
    assert all(torch.equal(a, b) for a, b in zip(*caches))
    table, lens = ints(rng.integers(0, 8, (T, 5))), ints([300, 0, 64, 65, 1, 320])
    pre, n = ints([3, 1, 2]), ints([150])
    out.fill_(NAN)
    assert torch.equal(wqa.attn_decode(fq, caches[0], table, lens, out=out, window=100, sinks=3), wqa.attn_decode(q, caches[0], table, lens, window=100, sinks=3))
    out.fill_(NAN)
    assert torch.equal(wqa.attn_decode_shared(fq, caches[0], pre, n, table, lens, out=out), wqa.attn_decode_shared(q, caches[0], pre, n, table, lens))
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,heads", [(64, 4), (300, 4), (330, 300)])
def test_window_prompt_offsets_out_of_range_stay_in_bounds(T, heads):
    """Offsets past T, below 0 and decreasing: rows of valid ranges come out right, others stay in bounds; tokens before the
    first sequence and behind the last are left alone."""
    note(f"window bad cu {T} {heads}")
    torch = torch_cuda()
    host, (q, k, v) = qkv(rng_for(100, T), T, heads, 2, 64)
    for cu in ([-5, 20, 1000], [0, 64, 64, 10], [T + 6, T + 9], [-9, -3], [30, 20, 64]):
        out = torch.full((T, heads, 64), NAN, device="cuda")
        wqa.attn_prefill(q, k, v, cu=ints(cu), out=out, window=33, sinks=2)
        torch.cuda.synchronize()
        if cu[-1] < 0 or cu[0] > T:
            assert torch.isnan(out).all()
    some = [0, heads // 2 - 1, heads // 2, heads - 1]
    part = [host[0][:, some], host[1][:, [j // (heads // 2) for j in some]], host[2][:, [j // (heads // 2) for j in some]]]
    out = torch.full((T, heads, 64), NAN, device="cuda")
    wqa.attn_prefill(q, k, v, cu=ints([-5, 20, 1000]), out=out, window=33, sinks=2)
    check_window_prompt(out[:, some], part, [20, T - 20], 0.125, 33, 2)
    out.fill_(NAN)
    wqa.attn_prefill(q, k, v, cu=ints([7, 50, T - 3]), out=out, window=33, sinks=2)
    assert torch.isnan(out[:7]).all() and torch.isnan(out[T - 3:]).all()
    check_window_prompt(out[7:T - 3, some], [x[7:T - 3] for x in part], [43, T - 53], 0.125, 33, 2)
