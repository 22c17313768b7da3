"""Host-side checks of the operators between the projections (no GPU): every
refusal of the C ABI happens before a launch, and the binding refuses tensors
the library could not take."""
import ctypes

import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import layer_ref as ref
from weight_only_bit_block_amd.wq import WqKVCache

OK, NULL, SHAPE, BITS, ALIGN, MRANGE, HIP, TABLE, SCRATCH = range(9)
FAKE = 0x10000          # 256-byte aligned, never dereferenced (validation fails first)
MIS = 0x10004


@pytest.fixture(scope="module")
def lib():
    return wqa.load()


def _prefill(lib, **kw):
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, v=FAKE, vs=1024, T=8, cu=FAKE, B=2, H=16, Hk=8, D=128, scale=0.1,
             out=FAKE, os=2048, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.wq_attn_prefill(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["cu"], a["B"], a["H"],
                               a["Hk"], a["D"], a["scale"], a["out"], a["os"], a["ws"], a["wsb"], None)


def test_prefill_refusals(lib):
    assert _prefill(lib, T=0) == OK and _prefill(lib, B=0) == OK
    assert _prefill(lib, T=0, q=None, k=None, v=None, out=None, cu=None, ws=None) == OK
    for bad in (dict(D=96), dict(D=0), dict(H=15), dict(H=0), dict(Hk=0), dict(H=2048, Hk=1025), dict(T=-1), dict(B=-1),
                dict(T=1 << 30), dict(B=1 << 24), dict(T=1 << 25, H=16), dict(T=8, B=1 << 20), dict(qs=2047), dict(qs=2050), dict(ks=1020),
                dict(vs=1 << 30), dict(os=1024)):
        assert _prefill(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None)):
        assert _prefill(lib, **bad) == NULL, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(out=MIS), dict(cu=FAKE + 2)):
        assert _prefill(lib, **bad) == ALIGN, bad


def test_prefill_workspace(lib):
    need = lib.wq_attn_prefill_ws(800, 2, 16, 8, 128)
    assert need > 0 and need % 256 == 0
    assert lib.wq_attn_prefill_ws(800, 2, 15, 8, 128) == 0 and lib.wq_attn_prefill_ws(0, 2, 16, 8, 128) == 0
    assert _prefill(lib, T=800, ws=None) == NULL and _prefill(lib, T=800, ws=MIS) == ALIGN
    assert _prefill(lib, T=800, wsb=need - 1) == SHAPE
    # the shortest prompts take none
    assert lib.wq_attn_prefill_ws(8, 2, 16, 8, 128) == 0 and lib.wq_attn_prefill_ws(8, 2000, 16, 8, 128) > 0
    # a tile of 32 keys is 4 binary16 operands; sequences may begin anywhere, so each adds one tile
    tile = 4 * 128 * 32 * 2
    for T, B in ((129, 1), (191, 1), (192, 1), (193, 3), (4096, 9)):
        slots = T // 32 + B
        got = lib.wq_attn_prefill_ws(T, B, 16, 8, 128)
        assert slots * 8 * tile <= got <= slots * 8 * (tile + 512) + 256


def _cache(**kw):
    c = WqKVCache(FAKE, FAKE, FAKE, FAKE, 10, 8, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(lib, cache=None, **kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, T=8, cu=FAKE, start=FAKE, B=2, table=FAKE, W=4)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.wq_kv_append(ctypes.byref(c), a["k"], a["ks"], a["v"], a["vs"], a["T"], a["cu"], a["start"], a["B"],
                            a["table"], a["W"], None)


def test_append_refusals(lib):
    assert _append(lib, T=0) == OK and _append(lib, B=0) == OK
    assert _append(lib, _cache(n_pages=0, kq=None)) == OK and _append(lib, W=0, table=None) == OK   # every row is dropped
    assert lib.wq_kv_append(None, FAKE, 1024, FAKE, 1024, 8, FAKE, FAKE, 2, FAKE, 4, None) == NULL
    for bad in (dict(head_dim=32), dict(kv_heads=0), dict(n_pages=-1), dict(n_pages=1 << 31)):
        assert _append(lib, _cache(**bad)) == SHAPE, bad
    for bad in (dict(T=-1), dict(T=1 << 30), dict(T=1 << 24), dict(B=-1), dict(W=-1), dict(W=1 << 25), dict(ks=1000),
                dict(vs=1026)):
        assert _append(lib, **bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(cu=None), dict(table=None)):
        assert _append(lib, **bad) == NULL, bad
    for name in ("kq", "ks", "vq", "vs"):
        assert _append(lib, _cache(**{name: None})) == NULL
        assert _append(lib, _cache(**{name: MIS})) == ALIGN
    for bad in (dict(k=MIS), dict(v=MIS), dict(cu=FAKE + 1), dict(start=FAKE + 2), dict(table=FAKE + 3)):
        assert _append(lib, **bad) == ALIGN, bad


def _decode(lib, cache=None, **kw):
    a = dict(q=FAKE, qs=2048, H=16, lens=FAKE, B=2, table=FAKE, W=4, scale=0.1, out=FAKE, os=2048, ws=FAKE, wsb=1 << 50)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.wq_attn_decode(ctypes.byref(c), a["q"], a["qs"], a["H"], a["lens"], a["B"], a["table"], a["W"], a["scale"],
                              a["out"], a["os"], a["ws"], a["wsb"], None)


def test_decode_refusals(lib):
    assert _decode(lib, B=0) == OK
    for bad in (dict(head_dim=256), dict(kv_heads=3), dict(n_pages=-1)):
        assert _decode(lib, _cache(**bad)) == SHAPE, bad
    for bad in (dict(H=12), dict(H=0), dict(B=-1), dict(W=-1), dict(W=1 << 25), dict(qs=1024), dict(os=2046),
                dict(B=1 << 16, H=256, qs=1 << 15, os=1 << 15), dict(B=1 << 20, H=16)):
        assert _decode(lib, **bad) == SHAPE, bad
    for bad in (dict(B=1 << 13, H=1 << 10, qs=1 << 17, os=1 << 17), dict(B=1 << 8, W=1 << 24)):
        assert _decode(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(lens=None), dict(out=None), dict(table=None)):
        assert _decode(lib, **bad) == NULL, bad
    for bad in (dict(q=MIS), dict(lens=FAKE + 2), dict(out=MIS), dict(table=FAKE + 1)):
        assert _decode(lib, **bad) == ALIGN, bad
    for name in ("kq", "ks", "vq", "vs"):
        assert _decode(lib, _cache(**{name: None})) == NULL
        assert _decode(lib, _cache(**{name: MIS})) == ALIGN
    need = lib.wq_attn_decode_ws(1, 16, 8, 128, 1 << 11)
    assert need > 0 and lib.wq_attn_decode_ws(1, 12, 8, 128, 4) == 0 and lib.wq_attn_decode_ws(0, 16, 8, 128, 4) == 0
    assert lib.wq_attn_decode_ws(1, 16, 8, 128, 4) == 0 and lib.wq_attn_decode_ws(5000, 16, 8, 128, 1 << 11) == 0    # not cut
    assert _decode(lib, B=1, W=1 << 11, ws=None) == NULL and _decode(lib, B=1, W=1 << 11, wsb=need - 1) == SHAPE
    assert _decode(lib, B=1, W=1 << 11, ws=FAKE + 64) == ALIGN


def test_norm_refusals(lib):
    def f(h=FAKE, y=FAKE, post=FAKE, gate=FAKE, gs=0, pre=FAKE, M=3, N=5, ho=FAKE, xo=FAKE):
        return lib.wq_residual_norm(h, y, post, gate, gs, 1.0, pre, 1e-6, M, N, ho, xo, None)
    assert f(M=0) == OK and f(N=0) == OK
    assert f(M=-1) == SHAPE and f(N=-1) == SHAPE and f(M=1 << 30) == SHAPE and f(gs=4) == SHAPE
    assert f(h=None) == NULL and f(ho=None, xo=None) == NULL and f(y=None) == NULL and f(y=None, gate=None) == NULL
    for name in ("h", "y", "post", "gate", "pre", "ho", "xo"):
        assert f(**{name: FAKE + 2}) == ALIGN, name


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 2, 64)
    cache = wqa.KVCache.empty(2, 2, 64, device="cpu")
    table = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: wqa.attn_prefill(q, q, q), lambda: wqa.kv_append(cache, q, q, table[:1]),
                 lambda: wqa.attn_decode(q, cache, table, table[:, 0]), lambda: wqa.residual_norm(torch.zeros(2, 8))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        wqa.KVCache.empty(2, 2, 96, device="cpu")
    assert (cache.n_pages, cache.kv_heads, cache.head_dim) == (2, 2, 64)


def test_reference_quantizer_is_the_packing_rule(oracle_mod):
    """The cache's rows are packed rows: the plain quantizer of the layer tests agrees with the oracle's."""
    x = np.random.default_rng(5).standard_normal((37, 128)).astype(np.float32)
    x[3] = 0
    x[4, :32] = 1e-9
    codes, scales = ref.quantize(x)
    q, s = oracle_mod.quantize(x, 4)
    assert np.array_equal(ref.nibbles(codes), q.reshape(37, 64)) and np.array_equal(scales.view(np.uint16), s.reshape(37, 4))


def test_reference_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(6)
    q, k, v = (rng.standard_normal((5, 2, 64)) for _ in range(3))
    out, _ = ref.prompt(q, k, v, [1, 0, 4], 0.3)
    assert np.array_equal(out[0], v[0]) and np.array_equal(out[1], v[1])
    w = np.exp(0.3 * (q[2, 1] @ k[1:3, 1].T))
    assert np.allclose(out[2, 1], (w @ v[1:3, 1]) / w.sum())
