"""Refusals of the rotary, 8-bit cache and page calls without a GPU: argument
checks come before any CUDA call, so these run anywhere.  Also the host-only
parts: rotary frequencies against the published formulas, plans and workspaces."""
import ctypes
import math

import pytest

from decode_attention_product_gb300 import _lib, build as B

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: checks fail first
ODD = ctypes.c_void_p(0x10008)       # 8-byte but not 16-byte aligned
INV, UNS, WS = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def cfg(D=128, P=16):
    return ctypes.byref(_lib.PQConfig(D, 4, 256, P))


# ---------------------------------------------------------------- rotary ----
def _rope(lib, c=None, T=4, Hq=2, Hkv=2, pos=FAKE, freq=FAKE, rot=128, m=1.0, flags=0, q=FAKE, qo=FAKE, kv=FAKE, kvo=FAKE):
    return lib.aq_rope(cfg() if c is None else c, T, Hq, Hkv, pos, freq, rot, m, flags, q, qo, kv, kvo, None)


def test_rope_refusals(lib):
    assert lib.aq_rope(None, 4, 2, 2, FAKE, FAKE, 128, 1.0, 0, FAKE, FAKE, FAKE, FAKE, None) == INV
    assert _rope(lib, c=cfg(D=64)) == UNS
    for bad in (0, 4, 12, 130, 136, -8):
        assert _rope(lib, rot=bad) == INV
    assert _rope(lib, T=-1) == INV
    assert _rope(lib, Hq=0) == INV and _rope(lib, Hkv=0) == INV
    assert _rope(lib, m=float("nan")) == INV and _rope(lib, m=float("inf")) == INV
    assert _rope(lib, flags=8) == INV
    assert _rope(lib, pos=None) == INV and _rope(lib, freq=None) == INV
    assert _rope(lib, qo=None) == INV and _rope(lib, kvo=None) == INV
    assert _rope(lib, q=None) == INV and _rope(lib, kv=None) == INV          # an output without its input
    assert _rope(lib, q=None, qo=None, kv=None, kvo=None) == INV
    assert _rope(lib, q=ODD) == INV and _rope(lib, kvo=ODD) == INV and _rope(lib, freq=ODD) == INV
    assert _rope(lib, T=0, pos=None, freq=None) == 0


def _freq(lib, rot=128, base=1e4, scaling=0, factor=1.0, orig=0, fast=32.0, slow=1.0):
    w, m = (ctypes.c_double * 64)(), ctypes.c_float()
    st = lib.aq_rope_frequencies(rot, base, scaling, factor, orig, fast, slow, w, ctypes.byref(m))
    return st, list(w)[:max(rot, 0) // 2], m.value


def test_rope_frequency_formulas(lib):
    for rot in (8, 64, 128):
        st, w, m = _freq(lib, rot)
        assert st == 0 and m == 1.0
        assert w == pytest.approx([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], rel=1e-14)
        st, w2, m = _freq(lib, rot, scaling=1, factor=4.0)
        assert st == 0 and m == 1.0 and w2 == pytest.approx([x / 4 for x in w], rel=1e-14)
        st, w3, m = _freq(lib, rot, scaling=2, factor=4.0)
        assert st == 0 and m == 1.0
        b = 10000.0 * 4.0 ** (rot / (rot - 2))
        assert w3 == pytest.approx([b ** (-2 * i / rot) for i in range(rot // 2)], rel=1e-14)
        # the stretched base leaves the fastest pair alone and slows the slowest by the factor
        assert w3[0] == 1.0 and w3[-1] == pytest.approx(w[-1] / 4, rel=1e-12)
    # by parts: fast pairs kept, slow ones divided, in between monotone between the two
    st, w, m = _freq(lib, 128, 1e4, 3, 8.0, 4096)
    plain = _freq(lib, 128, 1e4)[1]
    assert st == 0 and m == pytest.approx(0.1 * math.log(8.0) + 1.0, rel=1e-6)
    lo = math.floor(128 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(1e4)))
    hi = math.ceil(128 * math.log(4096 / (1 * 2 * math.pi)) / (2 * math.log(1e4)))
    for i in range(64):
        r = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        assert w[i] == pytest.approx(plain[i] * (1 - r) + plain[i] / 8 * r, rel=1e-13)
    assert w[0] == plain[0] and w[-1] == pytest.approx(plain[-1] / 8, rel=1e-14)


def test_rope_frequency_refusals(lib):
    for bad in (dict(rot=4), dict(rot=132), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5),
                dict(factor=float("inf")), dict(scaling=4), dict(scaling=-1), dict(scaling=3, factor=2.0, orig=0),
                dict(scaling=3, factor=2.0, orig=10, fast=1.0, slow=2.0), dict(scaling=3, orig=10, slow=0.0),
                dict(scaling=3, orig=10, fast=float("nan"))):
        assert _freq(lib, **bad)[0] == INV, bad
    assert lib.aq_rope_frequencies(128, 1e4, 0, 1.0, 0, 32.0, 1.0, None, None) == INV


# ----------------------------------------------------------- 8-bit cache ----
def _cache(fn, c=None, fmt=0, Bn=2, T=2, H=2, kv=FAKE, pages=FAKE, scales=FAKE, NP=8, bt=FAKE, mp=4, lens=FAKE, cu=None):
    return fn(cfg() if c is None else c, fmt, Bn, T, H, kv, pages, scales, NP, bt, mp, lens, cu, None, None)


@pytest.mark.parametrize("name", ["aq_q8_append", "aq_q8_load"])
def test_q8_cache_refusals(lib, name):
    fn = getattr(lib, name)
    assert _cache(fn, c=cfg(D=64)) == UNS and _cache(fn, c=cfg(P=32)) == UNS and _cache(fn, c=cfg(D=0)) == INV
    assert fn(None, 0, 2, 2, 2, FAKE, FAKE, FAKE, 8, FAKE, 4, FAKE, None, None, None) == INV
    for bad in (dict(fmt=2), dict(fmt=-1), dict(Bn=-1), dict(T=-1), dict(H=0), dict(NP=-1), dict(mp=-1),
                dict(T=3), dict(kv=None), dict(pages=None), dict(scales=None), dict(bt=None), dict(lens=None),
                dict(kv=ODD), dict(pages=ODD), dict(scales=ODD)):
        assert _cache(fn, **bad) == INV, bad
    assert _cache(fn, H=70000) == UNS and _cache(fn, Bn=70000, T=70000) == UNS
    assert _cache(fn, Bn=0, T=0, kv=None) == 0
    assert _cache(fn, T=0, cu=FAKE, kv=None) == 0


def _attend(lib, c=None, fmt=0, Bn=2, Hq=4, Hkv=2, q=FAKE, pages=FAKE, scales=FAKE, NP=8, bt=FAKE, mp=8, lens=FAKE,
            most=100, scale=0.1, splits=0, out=FAKE, ws=None, wsb=0):
    return lib.aq_q8_decode_attention(cfg() if c is None else c, fmt, Bn, Hq, Hkv, q, pages, scales, NP, bt, mp, lens,
                                      most, scale, splits, out, ws, wsb, None, None)


def test_q8_attention_refusals(lib):
    assert _attend(lib, c=cfg(D=64)) == UNS and _attend(lib, c=cfg(P=32)) == UNS
    for bad in (dict(fmt=3), dict(Bn=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(NP=-1), dict(mp=-1), dict(most=-1),
                dict(most=129), dict(scale=float("nan")), dict(splits=-1), dict(q=None), dict(pages=None),
                dict(scales=None), dict(bt=None), dict(lens=None), dict(out=None), dict(q=ODD), dict(pages=ODD),
                dict(scales=ODD), dict(out=ODD), dict(ws=ODD, wsb=1 << 20)):
        assert _attend(lib, **bad) == INV, bad
    assert _attend(lib, Bn=70000) == UNS and _attend(lib, Hq=70000, Hkv=70000) == UNS
    # up to 8 splits merge in a cluster; more need a workspace
    assert _attend(lib, mp=64, most=1000, splits=9) == WS
    assert _attend(lib, mp=64, most=1000, splits=9, ws=FAKE, wsb=64) == WS
    assert _attend(lib, NP=1 << 31) == UNS              # a page copy's coordinate
    assert _attend(lib, Bn=0, q=None) == 0


def test_q8_plans(lib):
    def plan(Bn, Hq, Hkv, L, req=0):
        s, w = ctypes.c_int32(), ctypes.c_size_t()
        assert lib.aq_q8_decode_plan(cfg(), Bn, Hq, Hkv, L, req, ctypes.byref(s), ctypes.byref(w)) == 0
        return s.value, w.value
    assert plan(1, 2, 2, 0) == (1, 0) and plan(1, 2, 2, 1) == (1, 0)
    assert plan(2, 4, 4, 100, 3)[0] == 3 and plan(2, 4, 4, 100, 50)[0] == 7       # no empty split
    for Bn, Hq, Hkv, L in [(1, 2, 2, 512), (8, 64, 8, 1000), (4, 32, 32, 2048), (1, 32, 32, 131072),
                           (256, 32, 32, 4096), (1, 1, 1, 2**31 - 1), (65535, 8, 1, 100)]:
        s, w = plan(Bn, Hq, Hkv, L)
        assert 1 <= s <= 4096 and w == (Bn * Hq * s * 130 * 4 if s > 8 else 0)


# ------------------------------------------------------------------ pages ----
def _pool(data=0x10000, nbytes=64):
    return (_lib.PagePool * 1)(_lib.PagePool(data, nbytes))


def test_pages_refusals(lib):
    def ext(n=2, rows=FAKE, lens=FAKE, bt=FAKE, R=4, mp=8, sl=FAKE, rc=FAKE, NP=100, pools=None, k=0, ws=FAKE, wsb=1 << 20):
        return lib.aq_pages_extend(n, rows, lens, bt, R, mp, sl, rc, NP, pools, k, ws, wsb, None, None)

    def fork(n=2, src=FAKE, dst=FAKE, bt=FAKE, R=4, mp=8, sl=FAKE, rc=FAKE, NP=100):
        return lib.aq_pages_fork(n, src, dst, bt, R, mp, sl, rc, NP, None, None)

    def free(n=2, rows=FAKE, keep=None, bt=FAKE, R=4, mp=8, sl=FAKE, rc=FAKE, NP=100):
        return lib.aq_pages_free(n, rows, keep, bt, R, mp, sl, rc, NP, None, None)

    def compact(bt=FAKE, R=4, mp=8, sl=FAKE, rc=FAKE, NP=100, pools=None, k=0, ws=FAKE, wsb=1 << 20):
        return lib.aq_pages_compact(bt, R, mp, sl, rc, NP, pools, k, ws, wsb, None, None)

    for f in (ext, fork):
        for bad in (dict(n=-1), dict(n=5), dict(R=-1), dict(mp=-1), dict(NP=-1), dict(bt=None), dict(sl=None),
                    dict(rc=None), dict(rc=ODD)):
            assert f(**bad) == INV, (f, bad)
        assert f(NP=1 << 31) == UNS and f(mp=1 << 28) == UNS
        assert f(n=0) == 0
    assert ext(ws=None) == WS and ext(wsb=16) == WS and ext(ws=ODD) == INV
    assert ext(rows=None) == INV and ext(lens=None) == INV and fork(src=None) == INV and fork(dst=None) == INV
    for bad in (dict(n=-1), dict(R=-1), dict(mp=-1), dict(rows=None), dict(bt=None), dict(sl=None), dict(rc=None), dict(rc=ODD)):
        assert free(**bad) == INV, bad
    assert free(n=0, rows=None) == 0
    for bad in (dict(R=-1), dict(mp=-1), dict(NP=-1), dict(bt=None), dict(sl=None), dict(rc=None), dict(rc=ODD), dict(ws=ODD)):
        assert compact(**bad) == INV, bad
    assert compact(ws=None) == WS and compact(wsb=16) == WS and compact(NP=0) == 0
    for f in (ext, compact):
        assert f(k=1) == INV and f(k=-1) == INV
        assert f(k=257, pools=(_lib.PagePool * 257)()) == UNS
        for pool in (_pool(0), _pool(0x10008), _pool(nbytes=0), _pool(nbytes=6)):
            assert f(k=1, pools=pool) == INV
    w = ctypes.c_size_t()
    assert lib.aq_pages_workspace(4, 100, ctypes.byref(w)) == 0 and w.value >= 3 * 400
    assert lib.aq_pages_workspace(-1, 100, ctypes.byref(w)) == INV and lib.aq_pages_workspace(4, 100, None) == INV


# --------------------------------------------------------------- wrappers ----
def test_wrappers_refuse_host_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    from decode_attention_product_gb300 import api
    i = torch.zeros(2, dtype=torch.int32)
    bt = torch.zeros(2, 4, dtype=torch.int32)
    pages, scales = torch.zeros(4, 2, 2, 16, 128, dtype=torch.int8), torch.zeros(4, 2, 2)
    kv, q = torch.zeros(2, 2, 2, 128, dtype=torch.float16), torch.zeros(2, 4, 128)
    with pytest.raises(ValueError, match="CUDA"):
        api.rope(i, torch.ones(64, dtype=torch.float64), q)
    with pytest.raises(ValueError, match="CUDA"):
        api.q8_append(kv, pages, scales, bt, i)
    with pytest.raises(TypeError, match="int8"):
        api.q8_append(kv, pages.half(), scales, bt, i)
    with pytest.raises(ValueError, match="num_tokens"):
        api.q8_load(pages, scales, bt, i, cu_tokens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.q8_decode_attention(q, pages, scales, bt, i, 16)
    with pytest.raises(ValueError, match="CUDA"):
        api.pages_free(i, bt, i, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="scaling"):
        api.rope_frequencies(scaling="cubic", device="cpu")
    with pytest.raises(ValueError, match="pool"):
        api.PageTable(4, 4, [])
