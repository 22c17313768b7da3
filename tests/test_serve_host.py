"""Host-side checks of the operators of a serving step (no GPU): every refusal of
the C ABI happens before a launch, and the plain forms the GPU tests use agree
with hand-made cases."""
import ctypes
import os

import numpy as np
import pytest

import weight_only_bit_block_amd as wqa
from tests import layer_ref as ref
from tests import serve_ref as sref
from tests.test_layer_host import ALIGN, FAKE, MIS, NULL, OK, SHAPE, _cache, lib  # noqa: F401  (lib is a fixture)
from tests.test_sanitize_host import CSRC, ROOT, SAN, _env, _run, tmp  # noqa: F401  (tmp is a fixture)


def _rope(lib, **kw):  # noqa: F811
    a = dict(q=FAKE, qs=2048, H=16, k=FAKE, ks=1024, Hk=8, D=128, T=3, pos=FAKE, inv=FAKE, pairs=64, inter=0, norm=1, wq=FAKE,
             wk=FAKE, qo=FAKE, qos=2048, ko=FAKE, kos=1024)
    a.update(kw)
    return lib.wq_qk_norm_rope(a["q"], a["qs"], a["H"], a["k"], a["ks"], a["Hk"], a["D"], a["T"], a["pos"], a["inv"], a["pairs"],
                               a["inter"], 1.0, a["norm"], a["wq"], a["wk"], 1e-6, a["qo"], a["qos"], a["ko"], a["kos"], None)


def test_rope_refusals(lib):  # noqa: F811
    assert _rope(lib, T=0) == OK and _rope(lib, H=0, Hk=0, q=None, k=None) == OK
    for bad in (dict(D=96), dict(D=256), dict(T=-1), dict(T=1 << 24), dict(H=-1), dict(Hk=-1), dict(H=1 << 23), dict(Hk=1 << 40), dict(pairs=65),
                dict(pairs=-4), dict(pairs=6), dict(D=64, pairs=36), dict(qs=2044), dict(qs=2050), dict(ks=1 << 30), dict(qos=1024), dict(kos=1026)):
        assert _rope(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(inv=None)):
        assert _rope(lib, **bad) == NULL, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(qo=MIS), dict(ko=MIS), dict(pos=FAKE + 2), dict(inv=FAKE + 1), dict(wq=MIS), dict(wk=MIS)):
        assert _rope(lib, **bad) == ALIGN, bad


def _plan(lib, **kw):  # noqa: F811
    a = dict(fresh=FAKE, start=FAKE, B=3, table=FAKE, W=4, free=FAKE, F=9, taken=FAKE, T=5, cu=FAKE, lens=FAKE, pos=FAKE, slots=FAKE, out=2 * FAKE)
    a.update(kw)
    return lib.wq_kv_plan(a["fresh"], a["start"], a["B"], a["table"], a["W"], a["free"], a["F"], a["taken"], a["T"], a["cu"], a["lens"],
                          a["pos"], a["slots"], a["out"], None)


def test_plan_refusals(lib):  # noqa: F811
    for bad in (dict(B=-1), dict(B=1 << 24), dict(W=-1), dict(W=1 << 25), dict(F=-1), dict(F=1 << 31), dict(T=-1), dict(T=1 << 30), dict(out=FAKE)):
        assert _plan(lib, **bad) == SHAPE, bad
    for bad in (dict(fresh=None), dict(table=None), dict(free=None), dict(cu=None), dict(lens=None), dict(out=None)):
        assert _plan(lib, **bad) == NULL, bad
    for name in ("fresh", "start", "table", "free", "taken", "cu", "lens", "pos", "out"):
        assert _plan(lib, **{name: 3 * FAKE + 2}) == ALIGN, name
    assert _plan(lib, slots=FAKE + 4) == ALIGN


def _spread(**kw):
    """Arguments of a plan that share no memory: 3 requests, rows of 4 pages, 9 free ones, 5 tokens."""
    a = {name: FAKE + 256 * i for i, name in enumerate(("fresh", "start", "free", "taken", "table", "cu", "lens", "pos", "slots", "out"))}
    a.update(kw)
    return a


def test_plan_refuses_outputs_in_other_memory_of_the_call(lib):  # noqa: F811
    """The next step's start in this one's lens would be read before or after it is written."""
    at = _spread()
    size = dict(fresh=12, start=12, free=36, taken=4, table=48, cu=16, lens=12, pos=20, slots=40, out=4)
    outputs = ("table", "cu", "lens", "pos", "slots", "out")
    for name in outputs:
        for other in at:
            if other != name:
                step = 8 if name == "slots" else 4
                last = (size[other] - 1) // step * step
                for where in (at[other], at[other] + last, at[other] - size[name] + step):
                    assert _plan(lib, **_spread(**{name: where})) == SHAPE, (name, other, where)


def test_rope_in_place_needs_the_same_stride(lib):  # noqa: F811
    assert _rope(lib, q=FAKE, qo=FAKE, qs=4096, qos=4100) == SHAPE and _rope(lib, k=FAKE, ko=FAKE, ks=4096, kos=4100) == SHAPE


def _slots(lib, cache=None, **kw):  # noqa: F811
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, T=8, slots=FAKE)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.wq_kv_append_slots(ctypes.byref(c), a["k"], a["ks"], a["v"], a["vs"], a["T"], a["slots"], None)


def test_append_slots_refusals(lib):  # noqa: F811
    assert _slots(lib, T=0) == OK and _slots(lib, _cache(n_pages=0, kq=None)) == OK
    assert lib.wq_kv_append_slots(None, FAKE, 1024, FAKE, 1024, 8, FAKE, None) == NULL
    for bad in (dict(head_dim=32), dict(kv_heads=0), dict(n_pages=-1)):
        assert _slots(lib, _cache(**bad)) == SHAPE, bad
    for bad in (dict(T=-1), dict(T=1 << 30), dict(T=1 << 24), dict(ks=1000), dict(vs=1026)):
        assert _slots(lib, **bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(slots=None)):
        assert _slots(lib, **bad) == NULL, bad
    for bad in (dict(k=MIS), dict(v=MIS), dict(slots=FAKE + 4)):
        assert _slots(lib, **bad) == ALIGN, bad
    for name in ("kq", "ks", "vq", "vs"):
        assert _slots(lib, _cache(**{name: None})) == NULL and _slots(lib, _cache(**{name: MIS})) == ALIGN


def _wprefill(lib, **kw):  # noqa: F811
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, v=FAKE, vs=1024, T=800, cu=FAKE, B=2, H=16, Hk=8, D=128, window=100, sinks=4,
             out=FAKE, os=2048, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.wq_attn_prefill_window(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["cu"], a["B"], a["H"], a["Hk"], a["D"], 0.1,
                                      a["window"], a["sinks"], a["out"], a["os"], a["ws"], a["wsb"], None)


def test_prefill_window_refusals(lib):  # noqa: F811
    assert _wprefill(lib, T=0) == OK and _wprefill(lib, B=0) == OK
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(D=96), dict(H=15), dict(T=-1), dict(T=1 << 30), dict(qs=2047), dict(ks=1020),
                dict(vs=1 << 30), dict(os=1024), dict(T=0, window=0)):
        assert _wprefill(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None), dict(ws=None)):
        assert _wprefill(lib, **bad) == NULL, bad
    for bad in (dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(out=MIS), dict(cu=FAKE + 2), dict(ws=MIS)):
        assert _wprefill(lib, **bad) == ALIGN, bad
    assert _wprefill(lib, wsb=lib.wq_attn_prefill_ws(800, 2, 16, 8, 128) - 1) == SHAPE


def _wdecode(lib, cache=None, **kw):  # noqa: F811
    a = dict(q=FAKE, qs=2048, H=16, lens=FAKE, B=2, table=FAKE, W=4, window=100, sinks=4, out=FAKE, os=2048, ws=FAKE, wsb=1 << 50)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.wq_attn_decode_window(ctypes.byref(c), a["q"], a["qs"], a["H"], a["lens"], a["B"], a["table"], a["W"], 0.1, a["window"],
                                     a["sinks"], a["out"], a["os"], a["ws"], a["wsb"], None)


def test_decode_window_refusals(lib):  # noqa: F811
    assert _wdecode(lib, B=0) == OK
    for bad in (dict(window=0), dict(sinks=-1), dict(H=12), dict(B=-1), dict(W=-1), dict(W=1 << 25), dict(qs=1024), dict(os=2046), dict(B=0, window=0)):
        assert _wdecode(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(lens=None), dict(out=None), dict(table=None)):
        assert _wdecode(lib, **bad) == NULL, bad
    for bad in (dict(q=MIS), dict(lens=FAKE + 2), dict(out=MIS), dict(table=FAKE + 1)):
        assert _wdecode(lib, **bad) == ALIGN, bad
    ws = lib.wq_attn_decode_window_ws
    assert ws(1, 16, 8, 128, 1 << 11, 100, 4) == 0                   # few pages are seen: not cut
    assert ws(1, 16, 8, 128, 1 << 11, 1 << 15, 4) > 0 and ws(1, 16, 8, 128, 1 << 11, 64, 1 << 15) > 0
    assert ws(1, 16, 8, 128, 1 << 11, 1 << 60, 1 << 60) == lib.wq_attn_decode_ws(1, 16, 8, 128, 1 << 11)
    assert ws(1, 16, 8, 128, 4, 0, 4) == 0 and ws(1, 16, 8, 128, 0, 5, 4) == 0
    need = ws(1, 16, 8, 128, 1 << 11, 1 << 15, 4)
    big = dict(B=1, W=1 << 11, window=1 << 15)
    assert _wdecode(lib, ws=None, **big) == NULL and _wdecode(lib, wsb=need - 1, **big) == SHAPE and _wdecode(lib, ws=FAKE + 64, **big) == ALIGN


def _shared(lib, cache=None, **kw):  # noqa: F811
    a = dict(q=FAKE, qs=2048, H=16, pre=FAKE, P=5, plen=FAKE, lens=FAKE, B=2, table=FAKE, W=4, out=FAKE, os=2048, ws=FAKE, wsb=1 << 50)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.wq_attn_decode_shared(ctypes.byref(c), a["q"], a["qs"], a["H"], a["pre"], a["P"], a["plen"], a["lens"], a["B"], a["table"], a["W"],
                                     0.1, a["out"], a["os"], a["ws"], a["wsb"], None)


def test_decode_shared_refusals(lib):  # noqa: F811
    assert _shared(lib, B=0) == OK
    for bad in (dict(P=-1), dict(P=1 << 25), dict(H=12), dict(B=-1), dict(W=-1), dict(W=1 << 25), dict(qs=1024), dict(os=2046),
                dict(B=1 << 20, H=16), dict(B=1 << 8, W=1 << 24)):
        assert _shared(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(lens=None), dict(out=None), dict(table=None), dict(pre=None), dict(plen=None), dict(ws=None)):
        assert _shared(lib, **bad) == NULL, bad
    for bad in (dict(q=MIS), dict(lens=FAKE + 2), dict(out=MIS), dict(table=FAKE + 1), dict(pre=FAKE + 2), dict(plen=FAKE + 1), dict(ws=FAKE + 128)):
        assert _shared(lib, **bad) == ALIGN, bad
    need = lib.wq_attn_decode_shared_ws(2, 16, 8, 128, 4, 5)
    assert need > 0 and _shared(lib, wsb=need - 1) == SHAPE
    assert lib.wq_attn_decode_shared_ws(0, 16, 8, 128, 4, 5) == 0 and lib.wq_attn_decode_shared_ws(2, 16, 8, 128, 4, -1) == 0
    # more pages never ask for less, and a prefix of thousands of pages is not cut into thousands of runs
    sizes = [lib.wq_attn_decode_shared_ws(2, 16, 8, 128, 4, n) for n in (0, 1, 5, 100, 1 << 12, 1 << 24)]
    assert sizes == sorted(sizes) and sizes[-1] < 64 << 20


def test_serve_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 2, 64)
    cache = wqa.KVCache.empty(2, 2, 64, device="cpu")
    table, n = torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: wqa.attn_prefill(q, q, q, window=3), lambda: wqa.kv_append(cache, q, q, slots=n.long()),
                 lambda: wqa.attn_decode(q, cache, table, n, window=3), lambda: wqa.attn_decode_shared(q, cache, n, n[:1], table, n),
                 lambda: wqa.qk_norm_rope(q, q, n, torch.ones(32)), lambda: wqa.kv_plan(n, table, n)):
        with pytest.raises(ValueError):
            call()


def test_serve_abi_under_sanitizers(tmp):  # noqa: F811
    exe = os.path.join(tmp, "serve_abi_sanitize")
    rc, out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(CSRC, "wq_serve_abi.cpp"),
                    os.path.join(ROOT, "tests", "c", "serve_abi_sanitize.cpp"),
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], None, 300)
    assert rc == 0, out
    rc, out = _run([exe], _env(tmp), 300)
    assert rc == 0 and "all checks passed" in out and "runtime error" not in out, out


# ------------------------------------------------------------------ the plain forms
def test_reference_plan():
    table = np.array([[7, -1, -1], [8, 9, -1], [-1, -1, -1]], np.int32)
    got = sref.plan([70, 1, 0], [60, 128, 0], table, np.array([30, 31], np.int32), 0, 73)
    assert got[0].tolist() == [[7, 30, 31], [8, 9, -1], [-1, -1, -1]]        # the third page of request 1 finds the list used up
    assert got[1].tolist() == [0, 70, 71, 71] and got[2].tolist() == [130, 129, 0] and got[5].tolist() == [3]
    assert got[3].tolist() == list(range(60, 130)) + [128, -1, -1]
    assert got[4].tolist() == [7 * 64 + i for i in range(60, 64)] + [30 * 64 + i for i in range(64)] + [31 * 64, 31 * 64 + 1, -1, -1, -1]


def test_reference_rotation():
    x = np.random.default_rng(1).standard_normal((3, 2, 64))
    pos, inv = np.array([0, 1, 5]), np.array([0.25, 1.0, 0.5, 0.0])
    y, _ = sref.rope(x, pos, inv, None, 0.0, False, False, 1.0)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:]) and np.array_equal(y[..., 3], x[..., 3])
    z = (x[..., :4] + 1j * x[..., 4:8]) * np.exp(1j * pos[:, None, None] * inv)
    assert np.allclose(y[..., :4], z.real) and np.allclose(y[..., 4:8], z.imag)
    w, _ = sref.rope(x, pos, inv, None, 0.0, False, True, 2.0)
    z = 2 * (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * np.exp(1j * pos[:, None, None] * inv)
    assert np.allclose(w[..., 0:8:2], z.real) and np.allclose(w[..., 1:8:2], z.imag)


def test_reference_window():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((40, 1, 64)) for _ in range(3))
    out, _ = sref.window_prompt(q, k, v, [40], 0.1, 1, 0)
    assert np.array_equal(out, v)                              # only itself
    full, _ = ref.prompt(q, k, v, [40], 0.1)
    same, _ = sref.window_prompt(q, k, v, [40], 0.1, 40, 0)
    assert np.array_equal(full, same)
    out, _ = sref.window_prompt(q, k, v, [40], 0.1, 2, 1)
    w = np.exp(0.1 * k[[0, 9, 10], 0] @ q[10, 0])
    assert np.allclose(out[10, 0], w @ v[[0, 9, 10], 0] / w.sum())
    assert sref.seen(7, 2, 3).tolist() == [True] * 3 + [False] * 2 + [True] * 2


def test_decode_shared_refuses_an_out_in_other_memory_of_the_call(lib):  # noqa: F811
    """Finished rows would be written where other workgroups have inputs still to read."""
    row, far = 2048 * 4, 1 << 32
    at = dict(q=far, pre=2 * far, plen=3 * far, lens=4 * far, table=5 * far, ws=6 * far)
    cache = _cache(kq=7 * far, ks=8 * far, vq=9 * far, vs=10 * far)
    codes = cache.n_pages * cache.kv_heads * 64 * cache.head_dim // 2
    size = dict(pre=20, plen=4, lens=8, table=32, kq=codes, ks=codes // 8, vq=codes, vs=codes // 8)
    for qs, os in ((2048, 2048), (2048, 4096), (4096, 2048), (8192, 8192), (4096, 6144), (6144, 4096)):
        spans = dict(size, q=(qs + 2048) * 4)
        for name, base in list(at.items())[:-1] + [(n, getattr(cache, n)) for n in ("kq", "ks", "vq", "vs")]:
            begin, end = base, base + spans[name]
            # its first row's beginning or end, or its second row's
            for where in (begin // 16 * 16, (end - 1) // 16 * 16, begin - row + 16, (begin - os * 4) // 16 * 16, (end - 16 - os * 4) // 16 * 16):
                assert _shared(lib, cache, qs=qs, os=os, out=where, **at) == SHAPE, (name, qs, os, where - base)
    # rows that pass between one another do not meet at first, but further on
    assert _shared(lib, cache, qs=4096, os=4160, out=far + row, **dict(at, B=40, table=11 * far)) == SHAPE
    assert _shared(lib, cache, qs=4160, os=4096, out=far + row, **dict(at, B=40, table=11 * far)) == SHAPE


@pytest.mark.parametrize("B,heads,kv,d,pages", [(1, 16, 8, 128, 2048), (64, 32, 8, 128, 128), (1024, 16, 8, 128, 20), (4, 16, 8, 128, 500), (64, 14, 2, 64, 128),
                                                (2, 100, 100, 64, 300), (3, 1024, 512, 128, 90), (1, 8, 1, 64, 16000)])
def test_own_tokens_behind_a_short_prefix_have_room_for_as_many_runs_as_alone(lib, B, heads, kv, d, pages):  # noqa: F811
    alone = lib.wq_attn_decode_ws(B, heads, kv, d, pages)
    sizes = [lib.wq_attn_decode_shared_ws(B, heads, kv, d, pages, n) for n in (0, 1, 2, 4, 16, 64, 128, 129, 1000, 100000, (1 << 25) - 1)]
    assert sizes == sorted(sizes) and sizes[0] >= alone
    # the parts of the prefix and a maximum and a sum for each head come on top
    assert sizes[2] <= alone + 512 + B * heads * (8 + 2 * (d + 4) * 4)
