"""Operators between the projections on data that strains what the kernels keep
beside the values: the units of a tile, the power of two of the scores, the
largest value scale. Against the plain 64-bit forms of tests/layer_ref.py, within
the bounds derived there."""
import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import layer_ref as ref
from tests.gpu_util import note, torch_cuda
from tests.test_gpu_layer import NAN, cache_arrays, cache_on, check_decode, cu_of, dev, qkv, rng_for, table_for

pytestmark = pytest.mark.gpu

# heads, kv heads, head size, tokens of one prompt, for each prompt kernel: it splits k and v itself (one and two
# tiles a wavefront), wavefronts share 32 rows, wavefronts of 32 rows each
KERNELS = [(16, 8, 128, 128), (14, 2, 64, 256), (4, 2, 128, 530), (4, 2, 64, 530), (288, 2, 128, 200), (602, 2, 64, 200)]


def prompt_of(host, cu=None, scale=None):
    torch = torch_cuda()
    out = torch.full(host[0].shape, NAN, device="cuda")
    wqa.attn_prefill(*(dev(x) for x in host), cu=cu, scale=scale, out=out)
    return out.cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ tiles of zeros
@pytest.mark.parametrize("heads,kv,d,T", KERNELS)
@pytest.mark.parametrize("where", ["first", "middle", "last", "first_two", "all", "not_finite"])
def test_prompt_tile_of_zero_values(heads, kv, d, T, where):
    """32 keys whose values are all zero (padding, silence) have no largest value
    and must not set the units of the others; neither must 32 keys none of whose
    values is finite. Values of any size around them: the output is
    proportional, exactly so for powers of two."""
    note(f"prompt zero tile {heads} {kv} {d} {T} {where}")
    host, _ = qkv(rng_for(50, heads, d), T, heads, kv, d)
    last = (T - 1) // 32
    tiles = {"first": [0], "middle": [3], "last": [last], "first_two": [0, 1], "all": range(last + 1), "not_finite": [2]}[where]
    for t in tiles:
        host[2][32 * t:32 * t + 32] = 0
    want, sums = ref.prompt(*host, [T], d ** -0.5)
    lim = ref.bound(sums, T, d)
    for size in (2.0 ** 60, 1.0, 2.0 ** -10, 2.0 ** -20, 2.0 ** -30, 2.0 ** -100):
        v = host[2] * np.float32(size)
        seen = np.ones(want.shape, bool)
        if where == "not_finite":
            v[64:96] = np.inf
            seen[64:] = False
        got = prompt_of([host[0], host[1], v])
        err, most = np.abs(got - want * size), (lim - 1e-44) * size + 1e-44
        assert (err[seen] <= most[seen]).all(), f"values {size}: worst error / bound {np.nanmax((err / most)[seen]):.3g}"
        assert np.isnan(got[~seen]).all()


# ------------------------------------------------------------------ scores below fp32
@pytest.mark.parametrize("heads,kv,d,T", KERNELS)
@pytest.mark.parametrize("qs,ks,scale", [(1e-20, 1e-17, None), (1e-37, 1.0, None), (1.0, 1e-41, 1e-3), (1e-25, 1e-25, -0.1),
                                         (1.0, 1.0, 1e-44), (1.0, 1.0, 0.0)])
def test_prompt_scores_below_the_range(heads, kv, d, T, qs, ks, scale):
    """Products whose powers of two are below fp32's: the weights are equal, and
    keys that a query does not see still have none."""
    note(f"prompt tiny scores {heads} {kv} {d} {T} {qs} {ks} {scale}")
    T = T - 9
    host, _ = qkv(rng_for(51, heads, d), T, heads, kv, d)
    host[0], host[1] = (host[0] * qs).astype(np.float32), (host[1] * ks).astype(np.float32)
    used = d ** -0.5 if scale is None else float(np.float32(scale))
    want, sums = ref.prompt(*host, [T], used)
    got = prompt_of(host, scale=scale)
    assert np.isfinite(got).all(), f"{np.isnan(got).sum()} NaN"
    assert (np.abs(got - want) <= ref.bound(sums, T, d)).all()


@pytest.mark.parametrize("heads,kv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 128), (4, 2, 64), (16, 2, 64)])
@pytest.mark.parametrize("lens", [[70, 1, 333], [1100, 0, 2000, 3]])
@pytest.mark.parametrize("qs,scale", [(1e-41, None), (1e-36, 1e-8), (1.0, 1e-44), (1e-38, -1e-3), (1.0, 0.0)])
def test_decode_scores_below_the_range(heads, kv, d, lens, qs, scale):
    """The same over the cache, whose last pages end inside a tile."""
    note(f"decode tiny scores {heads} {kv} {d} {lens} {qs} {scale}")
    torch = torch_cuda()
    rng = rng_for(52, heads, d, len(lens))
    table, pages = table_for(rng, lens)
    host, cache = cache_arrays(rng, pages, kv, d)
    q = (rng.standard_normal((len(lens), heads, d)) * qs).astype(np.float32)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), scale=scale, out=out)
    check_decode(out, q, host, table, lens, d ** -0.5 if scale is None else float(np.float32(scale)))


# ------------------------------------------------------------------ scales that are not finite
@pytest.mark.parametrize("heads,kv,d", [(4, 2, 128), (8, 2, 128), (16, 2, 128), (4, 2, 64), (16, 2, 64)])
@pytest.mark.parametrize("lens", [[900], [2000, 1100]])
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_decode_value_scale_that_is_not_finite(heads, kv, d, lens, bad):
    """One value block that is not finite makes its own elements so; all others keep
    the precision that the finite scales give them."""
    note(f"decode bad value scale {heads} {kv} {d} {lens} {bad}")
    torch = torch_cuda()
    rng = rng_for(53, heads, d, len(lens))
    table, pages = table_for(rng, lens)
    host, _ = cache_arrays(rng, pages, kv, d)
    host[3] = (host[3].astype(np.float32) * 2.0 ** -7).astype(np.float16)        # about 1e-3
    q = rng.standard_normal((len(lens), heads, d)).astype(np.float32)
    want, sums = ref.decode(q, ref.values(*host[:2]), ref.values(*host[2:]), host[3], table, lens, d ** -0.5)
    lim = ref.bound(sums, max(lens), d)
    host[3][table[0, 0], 1, 9, 1] = bad
    host[2][table[0, 0], 1, 9, 32:64] = 3
    hit = np.zeros(q.shape, bool)
    hit[0, heads // 2:, 32:64] = True
    out = torch.zeros(q.shape, device="cuda")
    wqa.attn_decode(dev(q), cache_on(host), dev(table), dev(np.array(lens, np.int32)), out=out)
    got = out.cpu().numpy().astype(np.float64)
    assert not np.isfinite(got[hit]).any()
    err = np.abs(got - want)
    assert (err[~hit] <= lim[~hit]).all(), f"worst error / bound {np.nanmax((err / lim)[~hit]):.3g}"


def test_decode_after_a_token_that_is_not_finite():
    """The same through the append: a token with a NaN among its values costs the
    others nothing."""
    note("decode after a NaN token")
    torch_cuda()
    heads, kv, d, n = 8, 2, 128, 960
    rng = rng_for(54)
    table, pages = table_for(rng, [n])
    k = rng.standard_normal((n, kv, d)).astype(np.float32)
    v = (rng.standard_normal((n, kv, d)) * 2.0 ** -12).astype(np.float32)
    clean = [np.zeros((pages, kv, ref.PAGE, w), t) for w, t in ((d, np.int8), (d // 32, np.float16)) * 2]
    for j, x in ((0, k), (2, v)):
        codes, scales = ref.quantize(x)
        at = table[0, np.arange(n) // ref.PAGE], np.arange(n) % ref.PAGE
        clean[j][at[0], :, at[1]], clean[j + 1][at[0], :, at[1]] = codes, scales
    clean[2][table[0, 0], 0, 5, 96:], clean[3][table[0, 0], 0, 5, 3] = 0, 0
    v[5, 0, 100] = np.nan
    cache = wqa.KVCache.empty(pages, kv, d)
    wqa.kv_append(cache, dev(k), dev(v), dev(table))
    q = rng.standard_normal((1, heads, d)).astype(np.float32)
    got = wqa.attn_decode(dev(q), cache, dev(table), dev(np.array([n], np.int32))).cpu().numpy()
    want, sums = ref.decode(q, ref.values(*clean[:2]), ref.values(*clean[2:]), clean[3], table, [n], d ** -0.5)
    lim = ref.bound(sums, n, d)
    hit = np.zeros(q.shape, bool)
    hit[0, :4, 96:] = True
    assert np.isnan(got[hit]).all()
    assert (np.abs(got - want)[~hit] <= lim[~hit]).all()


# ------------------------------------------------------------------ larger values that a query does not see
@pytest.mark.parametrize("heads,kv,d,T", KERNELS)
@pytest.mark.parametrize("bits", [3, 8, 13, 14])
def test_prompt_larger_values_behind_a_query(heads, kv, d, T, bits):
    """The last keys of every 32 have values 2^bits above the others, and set the
    units of the tile also for queries that do not see them. A tile's operands
    are off by 2^-25 at most where its largest value has become 2^14 or more,
    that is by 2^-39 of it: within the bound's 2^-36 up to 8 times larger ones.
    Rows keep a common factor up to 2^15 between them, so it is never more
    than 2^-24 of the row's own largest value."""
    note(f"prompt larger values behind {heads} {kv} {d} {T} {bits}")
    host, _ = qkv(rng_for(55, heads, d), T, heads, kv, d)
    v = host[2]
    v[:, :, 1::2] *= np.float32(2.0 ** -11)              # elements far below their row's largest
    late = np.arange(T) % 32 >= 30
    v[late] *= np.float32(2.0 ** bits)
    want, sums = ref.prompt(*host, [T], d ** -0.5)
    lim = ref.bound(sums, T, d)
    rows = np.abs(v).max(2)                              # [T, kv]
    if bits > 3:
        extra = ref.prompt(host[0], host[1], np.repeat(rows[:, :, None], d, 2), [T], d ** -0.5)[0]
        lim = lim + 2.0 ** -24 * extra
    got = prompt_of(host)
    err = np.abs(got - want)
    assert (err <= lim).all(), f"worst error / bound {np.nanmax(err / lim):.3g}"


# ------------------------------------------------------------------ walks that nothing else takes
@pytest.mark.parametrize("heads,kv,d,lens", [(24, 8, 128, [2900]), (8, 2, 128, [6000, 3000, 31]), (40, 8, 64, [4000]), (16, 2, 64, [33, 7000, 3300, 0, 64])])
def test_prompt_long_walk(heads, kv, d, lens):
    """Hundreds of tiles through the double buffer of the kernel for long prompts,
    some rows checked against the 64-bit form of their own."""
    note(f"prompt long walk {heads} {kv} {d} {lens}")
    T = sum(lens)
    rng = rng_for(56, heads, d)
    host, _ = qkv(rng, T, heads, kv, d)
    got = prompt_of(host, cu=cu_of(lens))
    q, k, v = (x.astype(np.float64) for x in host)
    at = 0
    for n in lens:
        rows = sorted({0, n // 2, n - 1, *rng.integers(0, n, 20).tolist()}) if n else []
        for j in range(heads):
            kk, vv = k[at:at + n, j // (heads // kv)], v[at:at + n, j // (heads // kv)]
            if not rows:
                continue
            see = np.arange(n)[None, :] <= np.array(rows)[:, None]
            o, pv, first = ref._attend(q[at:at + n][rows, j], kk, vv, d ** -0.5, see)
            top = np.maximum.accumulate(np.abs(vv).max(1))[rows][:, None] * np.ones((1, d))
            lim = ref.bound(np.stack([pv, first, top]), n, d)
            assert (np.abs(got[at:at + n][rows, j] - o) <= lim).all(), (n, j)
        at += n
    assert np.isfinite(got).all()


@pytest.mark.parametrize("heads,kv,d,lens,width", [(300, 300, 64, [2300, 0, 5, 400], 0), (600, 600, 128, [2200], 0),
                                                   (600, 300, 64, [70, 2100, 256], 0), (16, 8, 128, [1, 64, 65, 0, 300], 256),
                                                   (16, 8, 128, [0, 0, 0], 64), (8, 8, 64, [16], 4096), (14, 2, 64, [40] * 9, 300)])
def test_decode_cut_of_few_steps_and_many_heads(heads, kv, d, lens, width):
    """So many heads that a run of steps is the whole batch, and tables of a fixed
    width far beyond the lengths, where most workgroups find nothing to do."""
    note(f"decode cut {heads} {kv} {d} {lens} {width}")
    torch = torch_cuda()
    rng = rng_for(57, heads, d, len(lens))
    table, pages = table_for(rng, lens)
    if width:
        table = np.pad(table, ((0, 0), (0, width - table.shape[1])), constant_values=-1)
    host, cache = cache_arrays(rng, pages, kv, d)
    q = rng.standard_normal((len(lens), heads, d)).astype(np.float32)
    out = torch.full(q.shape, NAN, device="cuda")
    wqa.attn_decode(dev(q), cache, dev(table), dev(np.array(lens, np.int32)), out=out)
    check_decode(out, q, host, table, lens, d ** -0.5)


@pytest.mark.parametrize("lens", [[300, 5], [3000, 5, 0, 1500]])
def test_decode_rows_of_wider_rows(lens):
    """Queries and outputs inside wider rows, in groups of five and six heads; what lies between is left alone."""
    note(f"decode strides {lens}")
    torch = torch_cuda()
    for heads, kv, d in ((11, 1, 128), (10, 2, 64)):
        rng = rng_for(58, heads, d, len(lens))
        table, pages = table_for(rng, lens)
        host, cache = cache_arrays(rng, pages, kv, d)
        q = rng.standard_normal((len(lens), heads, d)).astype(np.float32)
        qw = torch.full((len(lens), heads * d + 20), NAN, device="cuda")
        qs = qw[:, 8:8 + heads * d].unflatten(1, (heads, d))
        qs.copy_(dev(q))
        wide = torch.full((len(lens), heads * d + 52), NAN, device="cuda")
        out = wide[:, 4:4 + heads * d].unflatten(1, (heads, d))
        wqa.attn_decode(qs, cache, dev(table), dev(np.array(lens, np.int32)), out=out)
        check_decode(out, q, host, table, lens, d ** -0.5)
        assert torch.isnan(wide[:, :4]).all() and torch.isnan(wide[:, 4 + heads * d:]).all()


# ------------------------------------------------------------------ norms
@pytest.mark.parametrize("N", [5, 300, 3000, 9000, 20001])
def test_norm_of_squares_past_the_range(N):
    """A row whose sum of squares passes fp32's range is normed to zeros, the block's output too; the other rows are not touched by it."""
    note(f"norm past the range {N}")
    rng = rng_for(59, N)
    h, y = rng.standard_normal((2, 4, N)).astype(np.float32)
    h[1] *= np.float32(1e25)
    y[2] *= np.float32(1e30)
    h_out, x = (t.cpu().numpy() for t in wqa.residual_norm(dev(h), dev(y), post_weight=dev(np.ones(N, np.float32)), norm=True))
    assert np.array_equal(h_out[2], h[2]) and (x[1] == 0).all()
    want = ref.residual_norm(h[[0, 3]], y[[0, 3]], np.ones(N), None, 1.0, None, float(np.float32(1e-6)))
    # a norm is off by 40 half steps (64 levels of its sum halved by the root, root, division, products); twice, and h_out in between
    assert np.allclose(h_out[[0, 3]], want[0], rtol=0, atol=80 * ref.U32 * want[1].max())
    assert np.allclose(x[[0, 3]], want[2], rtol=0, atol=400 * ref.U32 * np.abs(want[2]).max())
