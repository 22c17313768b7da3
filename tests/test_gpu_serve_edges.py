"""The operators of a serving step on calls that strain what their kernels keep
beside the values (plain forms and bounds: tests/serve_ref.py, tests/layer_ref.py)."""
import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import layer_ref as ref
from tests import serve_ref as sref
from tests.gpu_util import note, torch_cuda
from tests.test_gpu_layer import NAN, cu_of, dev, qkv, rng_for
from tests.test_gpu_serve import check_rows, check_shared, check_window_prompt, freqs, ints, shared_case

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norms and rotation
@pytest.mark.parametrize("d,pairs", [(64, 0), (64, 8), (64, 28), (128, 0), (128, 4), (128, 32), (128, 60)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T", [5, 1100])
def test_rope_values_that_are_not_rotated_are_kept(d, pairs, inter, T):
    """Without the norm they are copies, bit by bit, whatever stands beside them; with it each is its own product."""
    note(f"rope tail {d} {pairs} {inter} {T}")
    torch_cuda()
    rng = rng_for(110, d, pairs, T)
    host, _ = qkv(rng, T, 6, 3, d)
    x, y = host[0], host[1]
    tail = slice(2 * pairs, d)
    pos, inv = rng.integers(1, 100000, T).astype(np.int32), freqs(pairs) if pairs else np.zeros(0, np.float32)
    for a in (x, y):
        spots = rng.random(a[..., tail].shape) < 0.1
        a[..., tail][spots] = rng.choice(np.array([np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-44], np.float32), int(spots.sum()))
    oq, ok = wqa.qk_norm_rope(dev(x), dev(y), dev(pos), dev(inv), norm=False, interleaved=inter, factor=1.5)
    for got, a in ((oq.cpu().numpy(), x), (ok.cpu().numpy(), y)):
        assert np.array_equal(got[..., tail].view(np.uint32), a[..., tail].view(np.uint32))
        want, lim = sref.rope(a, pos, inv, None, 0.0, False, inter, 1.5)
        assert (np.abs(got - want)[..., :2 * pairs] <= lim[..., :2 * pairs]).all()
    # with the norm: a weight that is not finite belongs to its own value
    host, (q, _, _) = qkv(rng, T, 6, 3, d)
    for bad in (NAN, np.inf):
        w = rng.standard_normal(d).astype(np.float32)
        w[[2 * pairs, d - 1]] = bad
        got = wqa.qk_norm_rope(q, None, dev(pos), dev(inv), q_weight=dev(w), interleaved=inter)[0].cpu().numpy()
        own = np.zeros(d, bool)
        own[[2 * pairs, d - 1]] = True
        assert not np.isfinite(got[..., own]).any()
        want, lim = sref.rope(host[0], pos, inv, np.where(own, 1, w).astype(np.float32), 1e-6, True, inter, 1.0)
        assert (np.abs(got - want)[..., ~own] <= lim[..., ~own]).all()


# ------------------------------------------------------------------ prompts through a window
def few(heads, T, host, out):
    """Some heads of a wide layout with 2 key/value heads: the plain form is slow."""
    some = [0, heads // 2 - 1, heads // 2, heads - 1]
    return out[:, some], [host[0][:, some], *(x[:, [j // (heads // 2) for j in some]] for x in host[1:])]


@pytest.mark.parametrize("heads,d", [(800, 64), (500, 128)])
@pytest.mark.parametrize("window,sinks", [(40, 0), (64, 3), (1, 40), (100, 33)])
def test_window_of_many_heads_hides_what_it_hides(heads, d, window, sinks):
    """Wavefronts that share tiles of 128 rows: those that they leave out may hold anything, wild rows and rows that
    are not finite among them, at both ends of what is left out."""
    note(f"window many {heads} {d} {window} {sinks}")
    torch = torch_cuda()
    T, kv = 330, 2
    host, _ = qkv(rng_for(111, heads), T, heads, kv, d)
    t = np.arange(T)
    want, lim = None, None
    for at in (0, 2, 33, 70, 127, 128, 190, 256):
        sees = (t >= at) & ((at > t - window) | (at < sinks))
        for which in (1, 2):
            for bad in (NAN, np.inf, 1e20):
                arr = [host[0], host[1].copy(), host[2].copy()]
                arr[which][at, 1, 5] = bad
                out = torch.full((T, heads, d), NAN, device="cuda")
                wqa.attn_prefill(*(dev(x) for x in arr), out=out, window=window, sinks=sinks)
                got, part = few(heads, T, host, out)
                got = got.cpu().numpy()
                if want is None:
                    want, sums = sref.window_prompt(*part, [T], d ** -0.5, window, sinks)
                    lim = ref.bound(sums, min(T, window + sinks), d)
                hit = np.zeros(got.shape, bool)
                hit[sees, 2:] = True
                if which == 2 and bad != 1e20:
                    hit[..., :5] = hit[..., 6:] = False
                if bad != 1e20:
                    assert (np.isnan(got[hit]) if which == 1 else ~np.isfinite(got[hit])).all(), (at, which, bad)
                # (hidden rows of 1e20's tile keep units of their own: it is more than 2^14 above them)
                assert (np.abs(got - want)[~hit] <= lim[~hit]).all(), (at, which, bad)


@pytest.mark.parametrize("heads,d", [(800, 64), (500, 128)])
def test_window_of_many_heads_with_offsets_out_of_range(heads, d):
    """Offsets past T, below 0 and decreasing; tokens of no sequence are left alone."""
    note(f"window many cu {heads} {d}")
    torch = torch_cuda()
    T = 330
    host, (q, k, v) = qkv(rng_for(112, heads), T, heads, 2, d)
    for cu, lens, at in (([-5, 20, 1000], [20, T - 20], 0), ([7, 50, T - 3], [43, T - 53], 7), ([0, 200, 200, 90], [200], 0),
                         ([T + 6, T + 9], [], 0), ([-9, -3], [], 0)):
        out = torch.full((T, heads, d), NAN, device="cuda")
        wqa.attn_prefill(q, k, v, cu=ints(cu), out=out, window=33, sinks=2)
        end = at + sum(lens)
        got, part = few(heads, T, host, out)
        assert torch.isnan(out[:at]).all() and torch.isnan(out[end:]).all()
        if lens:
            check_window_prompt(got[at:end], [x[at:end] for x in part], lens, d ** -0.5, 33, 2, str(cu))


@pytest.mark.parametrize("lens,heads,d", [([330], 450, 64), ([330], 170, 128), ([90, 100, 80, 60], 260, 64), ([330], 500, 64), ([330], 160, 128), ([200, 130], 310, 64)])
def test_window_of_any_width_on_either_side_of_the_limits(lens, heads, d):
    """Numbers of groups of rows between the limits of narrow and wide windows: the same values whatever the width."""
    note(f"window widths {lens} {heads} {d}")
    torch = torch_cuda()
    T = sum(lens)
    host, (q, k, v) = qkv(rng_for(113, heads), T, heads, 2, d)
    for window, sinks in ((1, 3), (100, 0), (263, 0), (264, 70), (265, 0), (T - 1, 0)):
        out = torch.full((T, heads, d), NAN, device="cuda")
        wqa.attn_prefill(q, k, v, cu=cu_of(lens), out=out, window=window, sinks=sinks)
        got, part = few(heads, T, host, out)
        check_window_prompt(got, part, lens, d ** -0.5, window, sinks, f"{window} {sinks}")


# ------------------------------------------------------------------ a shared prefix
def test_shared_out_beside_its_query_but_not_in_it():
    """Columns of one buffer are apart; anything that shares memory is refused."""
    note("shared out")
    torch = torch_cuda()
    rng = rng_for(114)
    heads, kv, d, B = 6, 2, 64, 70
    pre, table, host, cache, q = shared_case(rng, heads, kv, d, 1000, [50] * B)
    args = (cache, dev(pre), ints([1000]), dev(table), ints([50] * B))
    want = wqa.attn_decode_shared(dev(q), *args)
    w = heads * d
    both = torch.full((B, 3 * w), NAN, device="cuda")
    qs = both[:, w:2 * w].unflatten(1, (heads, d))
    for at in (0, 2 * w):
        qs.copy_(dev(q))
        out = both[:, at:at + w].unflatten(1, (heads, d))
        assert torch.equal(wqa.attn_decode_shared(qs, *args, out=out), want) and torch.equal(qs, dev(q))
    before = both.clone()
    for at in (w, w - 64, 64, 2 * w - 64):
        with pytest.raises(wqa.WqError):
            wqa.attn_decode_shared(qs, *args, out=both[:, at:at + w].unflatten(1, (heads, d)))
    flat = dev(q).view(-1)
    with pytest.raises(wqa.WqError):
        wqa.attn_decode_shared(flat[:-w].view(B - 1, heads, d), cache, args[1], args[2], args[3][1:], args[4][1:], out=flat[w:].view(B - 1, heads, d))
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(both), torch.nan_to_num(before))


@pytest.mark.parametrize("count,heads,kv,d,prefix,longest", [(1, 16, 8, 128, 70, 100000), (40, 4, 2, 128, 100, 12500), (4, 16, 8, 128, 50, 27000),
                                                              (60, 14, 2, 64, 30, 7000), (1, 8, 1, 64, 300, 800000), (90, 20, 4, 64, 0, 2500)])
def test_shared_long_sequences_behind_a_short_prefix(count, heads, kv, d, prefix, longest):
    """Own tokens that take nearly the whole card."""
    note(f"shared short prefix {count} {heads} {kv} {d} {prefix} {longest}")
    torch = torch_cuda()
    rng = rng_for(115, count, longest)
    lens = [int(x) for x in rng.integers(0, longest // 4, count)]
    lens[-1] = longest
    if count > 1:
        lens[count // 2] = 0
    pre, table, host, cache, q = shared_case(rng, heads, kv, d, prefix, lens)
    out = torch.full(q.shape, NAN, device="cuda")
    for n in (prefix, prefix // 2):
        wqa.attn_decode_shared(dev(q), cache, dev(pre), ints([n]), dev(table), ints(lens), out=out)
        check_shared(out, q, host, pre, n, table, lens, d ** -0.5, str(n))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("prefix", [128, 100])
def test_own_tokens_are_rotated_behind_the_prefix(prefix):
    """Requests planned and cached whole, and the same as own tokens behind one copy of their common beginning: the same
    cache rows and the same attention."""
    note(f"rotated behind {prefix}")
    torch = torch_cuda()
    rng = rng_for(116, prefix)
    heads, kv, d, pages, width = 8, 2, 128, 40, 6
    own = [70, 1, 64]
    inv, free, n = dev(freqs(64)), ints(rng.permutation(pages)), ints([prefix])
    _, first = qkv(rng, prefix, heads, kv, d)
    rest = [qkv(rng, m, heads, kv, d)[1] for m in own]

    def fill(parts, fresh, shift):
        """Plans, rotates and caches requests of these tokens; one more token in hand than there is."""
        q, k, v = (torch.cat([p[i] for p in parts] + [parts[0][i][:1]]) for i in range(3))
        cache, table = wqa.KVCache.empty(pages, kv, d), ints(np.full((len(fresh), width), -1))
        p = wqa.kv_plan(ints(fresh), table, free, tokens=len(q))
        at = torch.where(p.positions < 0, p.positions, p.positions + shift)
        q, k = wqa.qk_norm_rope(q, k, at, inv)
        wqa.kv_append(cache, k, v, slots=p.slots)
        return q[p.cu[1:].long() - 1], cache, table, p

    def rows(cache, table, b, lo, hi):
        t = np.arange(lo, hi)
        page = table.cpu().numpy()[b, t // 64]
        return [x.cpu().numpy()[page, :, t % 64] for x in cache]
    q, whole, tables, p = fill([x for r in rest for x in (first, r)], [prefix + m for m in own], 0)
    _, pre, pre_table, _ = fill([first], [prefix], 0)
    # the prefix's pages are the first of the list, own tokens' those behind them
    free = free[-(-prefix // 64):].contiguous()
    q2, cache, table, p2 = fill(rest, own, n)
    for b, m in enumerate(own):
        for x, y in zip(rows(whole, tables, b, prefix, prefix + m), rows(cache, table, b, 0, m)):
            assert np.array_equal(x, y), b
        for x, y in zip(rows(whole, tables, b, 0, prefix), rows(pre, pre_table, 0, 0, prefix)):
            assert np.array_equal(x, y), b
    assert torch.equal(q, q2)
    for x, y in zip(cache, pre):
        at = pre_table[0][pre_table[0] >= 0].long()
        x[at] = y[at]
    out = wqa.attn_decode_shared(q2, cache, pre_table[0], n, table, p2.lens)
    codes = [t.cpu().numpy() for t in (cache.kq, cache.vq)]
    codes = [np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], d).astype(np.int8) for c in codes]
    kval, vval = (ref.values(np.where(c > 7, c - 16, c), t.view(torch.float16).cpu().numpy()) for c, t in zip(codes, (cache.ks, cache.vs)))
    tab, first = table.cpu().numpy(), pre_table[0].cpu().numpy()
    want, sums = sref.decode(q.cpu().numpy(), kval, vval, cache.vs.view(torch.float16).cpu().numpy(), d ** -0.5,
                             lambda b: [(first, prefix, None), (tab[b], own[b], None)])
    check_rows(out, want, sums, prefix + max(own), d)
    check_rows(wqa.attn_decode(q, whole, tables, p.lens), want, sums, prefix + max(own), d)
