"""The 8-bit block-scaled cache on the GPU: append and read-back against a plain
sequential model (codes and scales bit for bit), decode attention against softmax
attention in 64 bits over the values that the codes stand for.

Attention's bound, per (request, head), from the arithmetic: a score is a sum of
128 products of a query split to 22 bits (2^-22 relative) with exact codes,
accumulated in fp32 (at most 130 roundings of 2^-24), times two 32-bit factors:
its error is under (2^-22 + 134 * 2^-24) * A, A = scale * sum |q_d k_d| at its
largest over the tokens.  A weight then moves by that, plus the exponential's
2^-22 and the exponent's own rounding 2^-24 * A * 3; the weights enter the value
product split to 22 bits, its sums are fp32 over at most 16 tokens a tile with one
rounding per page and one per merge (2^-24 each, under 2^10 of them in a row, and
random in sign: 2^-16 covers them).  Numerator and denominator both move, so the
output is off by at most 2 * (err_s + 2^-16) * max |v|.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

P, D = 16, 128


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_product_gb300 import build
    build.build()
    from decode_attention_product_gb300 import api
    return api


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


E4M3 = np.zeros(256)
for _c in range(256):
    _e, _f = (_c >> 3) & 15, _c & 7
    _v = _f * 2.0 ** -9 if _e == 0 else (1 + _f / 8) * 2.0 ** (_e - 7)
    E4M3[_c] = (-1.0 if _c >> 7 else 1.0) * (math.nan if _c & 0x7f == 0x7f else _v)


def values(codes, fmt):
    return codes.astype(np.float64) if fmt == "int8" else E4M3[codes]


def nearest(x, fmt):
    """codes nearest to x (float64), ties to even"""
    if fmt == "int8":
        return np.rint(x).astype(np.int8)
    grid = E4M3[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return c | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)


def model_append(pages, scales, bt, start, x, fmt):
    """One request's tokens x [n][H][2][D] fp16 at positions start .. in place."""
    n, t = len(x), start
    while t < start + n:
        e = min(start + n, t // P * P + P)
        pg, s0 = bt[t // P], t % P
        y = x[t - start:e - start].astype(np.float64)
        amax = np.abs(y).max(axis=(0, 3))                                  # [H][2]
        with np.errstate(invalid="ignore", divide="ignore"):
            if fmt == "int8":
                want = (amax.astype(np.float32) / np.float32(127)).astype(np.float32)
            else:
                want = np.where(amax > 0, 2.0 ** np.ceil(np.log2(np.where(amax > 0, amax, 1) / 448)), 0)
                want = np.where((want > 0) & (amax <= 448 * want / 2), want / 2, want).astype(np.float32)
            want[~np.isfinite(amax)] = np.nan
            old = scales[pg].copy() if s0 else np.zeros_like(want)
            new = np.where(np.isnan(old) | np.isnan(want), np.float32(np.nan), np.fmax(old, want)).astype(np.float32)
            for h in range(new.shape[0]):
                for w in range(2):
                    s, o = float(new[h, w]), float(old[h, w])
                    if s0 and not math.isnan(o) and s != o:
                        kept = values(pages[pg, h, w, :s0], fmt)
                        pages[pg, h, w, :s0] = nearest(kept * o / s, fmt) if s > 0 and o > 0 else 0
                    pages[pg, h, w, s0:s0 + e - t] = nearest(y[:, h, w] / s, fmt) if s > 0 else 0
            scales[pg] = new
        t = e


def same_values(a, b, fmt):
    """Codes equal as values (E4M3 has two zeros)."""
    return np.array_equal(a, b) or (fmt == "e4m3" and np.array_equal(E4M3[a], E4M3[b], equal_nan=True))


def draw_kv(g, T, H, wide=False):
    x = g.standard_normal((T, H, 2, D)) * g.uniform(0.5, 2.0, (H, 2, D))
    if wide:
        x *= 2.0 ** g.integers(-16, 8, (T, 1, 1, 1))
    return np.clip(x, -65504, 65504).astype(np.float16)


def empty(g, NP, H, fmt):
    """A pool full of what other requests left behind."""
    codes = g.integers(0, 256, (NP, H, 2, P, D)).astype(np.uint8)
    return codes.view(np.int8) if fmt == "int8" else codes, g.uniform(0.001, 1.0, (NP, H, 2)).astype(np.float32)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H", [1, 3, 9])
@pytest.mark.parametrize("wide", [False, True], ids=["normal", "growing"])
def test_append_matches_sequential_model(A, fmt, H, wide):
    """Requests growing by uneven chunks, single tokens among them, some calls
    adding nothing to a request: every slot and scale of the pool after every call."""
    g = np.random.default_rng(H * 10 + wide)
    B, mp = 5, 9
    pages, scales = empty(g, B * mp + 4, H, fmt)
    bt = g.permutation(B * mp + 4)[:B * mp].reshape(B, mp).astype(np.int32)
    dp, ds, dbt = dev(pages), dev(scales), dev(bt)
    lens = np.zeros(B, np.int32)
    for call in range(14):
        room = mp * P - lens
        n = np.ones(B, np.int32) if call % 3 == 0 else np.minimum(room, g.choice([0, 1, 2, 15, 16, 17, 33, 40], B)).astype(np.int32)
        n = room.astype(np.int32) if call == 13 else np.minimum(n, room)
        one = call % 3 == 0 and np.all(n == 1)
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(cu[-1]) + (0 if one else 3)                                # rows behind the last sequence
        kv = draw_kv(g, T, H, wide)
        if not one:
            kv[cu[-1]:] = np.nan
        lens = lens + n
        status = A.new_status()
        A.q8_append(dev(kv), dp, ds, dbt, dev(lens), None if one else dev(cu), status)
        for b in range(B):
            model_append(pages, scales, bt[b], lens[b] - n[b], kv[cu[b]:cu[b + 1]], fmt)
        assert int(status.item()) == 0
        assert np.array_equal(ds.cpu().numpy(), scales), f"scales after call {call}"
        assert same_values(dp.cpu().numpy(), pages, fmt), f"codes after call {call}"
        # the same tokens read back
        back = A.q8_load(dp, ds, dbt, dev(lens), None if one else dev(cu), T).cpu().numpy()
        for b in range(B):
            for i in range(n[b]):
                t = lens[b] - n[b] + i
                pg, s = bt[b, t // P], t % P
                want = values(pages[pg, :, :, s], fmt) * scales[pg].astype(np.float64)[..., None]
                # code * scale in fp32, then fp16: half a step of each
                err = np.abs(back[cu[b] + i].astype(np.float64) - want)
                assert np.all(err <= (2.0 ** -11 + 2.0 ** -23) * np.abs(want) + 2.0 ** -25)
    assert lens.max() == mp * P


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_prompt_over_many_requests(A, fmt):
    """More requests than one step of the 32-way search, and long prompts."""
    g = np.random.default_rng(7)
    H, B = 2, 75
    n = np.where(g.random(B) < 0.1, g.integers(200, 400, B), g.integers(0, 40, B)).astype(np.int32)
    kept = g.integers(0, 40, B).astype(np.int32)
    lens = kept + n
    mp = -(-int(lens.max()) // P)
    pages, scales = empty(g, B * mp, H, fmt)
    bt = g.permutation(B * mp).reshape(B, mp).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    kv = draw_kv(g, int(cu[-1]), H)
    dp, ds = dev(pages), dev(scales)
    A.q8_append(dev(kv), dp, ds, dev(bt), dev(lens), dev(cu))
    if fmt == "e4m3":                       # the stale codes of earlier slots may be NaN: as values they stay NaN
        pages[(pages & 0x7f) == 0x7f] = 0x7f
    for b in range(B):
        model_append(pages, scales, bt[b], kept[b], kv[cu[b]:cu[b + 1]], fmt) if fmt == "int8" else None
    if fmt == "int8":
        assert np.array_equal(ds.cpu().numpy(), scales) and np.array_equal(dp.cpu().numpy(), pages)
    else:                                   # new slots and scales (earlier slots hold no valid codes here)
        fresh = [(bt[b, t // P], t % P, cu[b] + t - kept[b]) for b in range(B) for t in range(kept[b], lens[b])]
        p, s, i = (np.array(x) for x in zip(*fresh))
        sc = ds.cpu().numpy()[p]
        with np.errstate(invalid="ignore"):
            want = nearest(kv[i].astype(np.float64) / sc.astype(np.float64)[..., None], fmt)
        assert np.array_equal(E4M3[dp.cpu().numpy()[p, :, :, s]], E4M3[want])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_rounds_to_the_nearest_code(A, fmt):
    """Values at and one step beside every midpoint between codes."""
    g = np.random.default_rng(11)
    for top in (127.0, 126.9375, 1.0, 65504.0, 2.0 ** -24, 448.0, 7.0, 449.0):
        top = float(np.float16(top))
        scale = np.float32(top) / np.float32(127)
        mid = (np.arange(0, 127) + 0.5) * float(scale)
        x = np.float16(mid)
        x = np.concatenate([x, np.nextafter(x, np.float16(0)), np.nextafter(x, np.float16(65504)), -x])
        x = np.clip(x, -top, top).astype(np.float16)
        x = np.concatenate([x, g.uniform(-top, top, 16 * D - len(x) - 1).astype(np.float16), [np.float16(top)]])
        kv = np.stack([x.reshape(16, 1, D), x[::-1].reshape(16, 1, D)], 2)
        pages, scales = empty(g, 1, 1, fmt)
        dp, ds = dev(pages), dev(scales)
        bt, lens, cu = np.zeros((1, 1), np.int32), np.array([16], np.int32), np.array([0, 16], np.int32)
        A.q8_append(dev(kv), dp, ds, dev(bt), dev(lens), dev(cu))
        model_append(pages, scales, bt[0], 0, kv, fmt)
        assert np.array_equal(ds.cpu().numpy(), scales)
        assert same_values(dp.cpu().numpy(), pages, fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_zero_and_non_finite_blocks(A, fmt):
    """All-zero blocks have scale 0 and grow from it; a block that met an
    infinity or a NaN is NaN from then on, its neighbours are not."""
    g = np.random.default_rng(12)
    H = 2
    pages, scales = empty(g, 3, H, fmt)
    dp, ds, bt = dev(pages), dev(scales), np.array([[2, 0]], np.int32)
    steps = [np.zeros((1, H, 2, D)), np.zeros((2, H, 2, D)), g.standard_normal((1, H, 2, D)), np.zeros((1, H, 2, D)),
             g.standard_normal((3, H, 2, D)), g.standard_normal((2, H, 2, D)), g.standard_normal((9, H, 2, D))]
    steps[4][1, 0, 0, 5] = np.inf
    steps[5][0, 1, 1, 99] = np.nan
    L = 0
    for x in steps:
        x = x.astype(np.float16)
        lens, cu = np.array([L + len(x)], np.int32), np.array([0, len(x)], np.int32)
        A.q8_append(dev(x), dp, ds, dev(bt), dev(lens), dev(cu))
        model_append(pages, scales, bt[0], L, x, fmt)
        L += len(x)
        assert np.array_equal(ds.cpu().numpy(), scales, equal_nan=True)
        assert same_values(dp.cpu().numpy(), pages, fmt)
    assert np.isnan(scales[2, 0, 0]) and np.isnan(scales[2, 1, 1]) and not np.isnan(scales[2, 0, 1])
    assert not np.isnan(scales[0]).any()
    back = A.q8_load(dp, ds, dev(bt), dev(np.array([L], np.int32)), dev(np.array([0, L], np.int32)), L).cpu().numpy()
    assert np.isnan(back[:16, 0, 0]).all() and np.isnan(back[:16, 1, 1]).all()
    assert np.isfinite(back[:16, 0, 1]).all() and np.isfinite(back[16:]).all()


def test_append_and_load_data_errors(A):
    """Requests that do not fit are flagged and skipped, the others served; a
    read-back of what does not exist is NaN."""
    g = np.random.default_rng(13)
    H, B = 2, 6
    pages, scales = empty(g, 8, H, "int8")
    dp, ds = dev(pages), dev(scales)
    bt = np.array([[0, 1], [2, 99], [-1, 3], [4, 5], [6, 7], [0, 0]], np.int32)
    lens = np.array([20, 20, 20, 3, 33, -5], np.int32)                     # 3: more new tokens than length; 4: beyond the table
    n = np.array([20, 20, 20, 5, 2, 1], np.int32)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    kv = draw_kv(g, int(cu[-1]), H)
    st = A.new_status()
    A.q8_append(dev(kv), dp, ds, dev(bt), dev(lens), dev(cu), st)
    assert int(st.item()) == 1 | 2
    model_append(pages, scales, bt[0], 0, kv[:20], "int8")
    model_append(pages, scales, bt[1][:1], 0, kv[20:36], "int8")
    model_append(pages, scales, [0, 3], 16, kv[56:60], "int8")
    assert np.array_equal(dp.cpu().numpy(), pages) and np.array_equal(ds.cpu().numpy(), scales)
    st.zero_()
    back = A.q8_load(dp, ds, dev(bt), dev(lens), dev(cu), len(kv), status=st).cpu().numpy()
    assert int(st.item()) == 1 | 2
    bad = np.isnan(back).all(axis=(1, 2, 3))
    assert bad.tolist() == [False] * 20 + [False] * 16 + [True] * 4 + [True] * 16 + [False] * 4 + [True] * 8
    assert np.isfinite(back[~bad]).all()
    # cu_tokens that runs backwards or past the rows
    for cu2 in ([0, 20, 10, 30, 40, 50, 60], [0, 20, 40, 60, 65, 1000, 1000], [-4, 20, 40, 60, 65, 67, 68]):
        st.zero_()
        before = dp.clone()
        A.q8_append(dev(kv), before, ds.clone(), dev(bt), dev(lens), dev(np.array(cu2, np.int32)), st)
        assert int(st.item()) & 2


# ------------------------------------------------------------- attention ----
def problem(g, B, Hkv, G, lens, fmt, spare=3, scales=(0.005, 0.04)):
    lens = np.asarray(lens, np.int32)
    mp = max(1, -(-int(lens.max()) // P)) + 1
    need = [-(-int(x) // P) for x in lens]
    NP = sum(need) + spare
    perm = g.permutation(NP)
    bt = g.integers(-5, NP + 5, (B, mp)).astype(np.int32)                  # entries past the length mean nothing
    i = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[i:i + n]
        i += n
    if fmt == "int8":
        pages = np.clip(np.rint(g.standard_normal((NP, Hkv, 2, P, D)) * 40), -127, 127).astype(np.int8)
        sc = g.uniform(*scales, (NP, Hkv, 2)).astype(np.float32)
    else:
        pages = nearest(g.standard_normal((NP, Hkv, 2, P, D)) * 100, fmt)
        sc = 2.0 ** np.rint(np.log2(g.uniform(*scales, (NP, Hkv, 2)) / 4)).astype(np.float32)
    used = np.zeros((NP, P), bool)
    for b, L in enumerate(lens):
        t = np.arange(L)
        used[bt[b, t // P], t % P] = True
    # stale slots: anything, NaN codes among them
    stale = ~used
    pages = pages.copy()
    np.moveaxis(pages, 3, 1)[stale] = np.uint8(0x7f).view(pages.dtype) if fmt == "e4m3" else 127
    q = g.standard_normal((B, Hkv * G, D)).astype(np.float32)
    return dict(q=q, pages=pages, scales=sc.astype(np.float32), bt=bt, lens=lens, fmt=fmt, G=G)


def reference(p, scale=D ** -0.5):
    """(out, bound) in float64"""
    B, Hq, _ = p["q"].shape
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, 1))
    for b, L in enumerate(p["lens"]):
        if L <= 0:
            continue
        t = np.arange(L)
        pg, s = p["bt"][b, t // P], t % P
        for h in range(p["pages"].shape[1]):
            k = values(p["pages"][pg, h, 0, s], p["fmt"]) * p["scales"][pg, h, 0].astype(np.float64)[:, None]
            v = values(p["pages"][pg, h, 1, s], p["fmt"]) * p["scales"][pg, h, 1].astype(np.float64)[:, None]
            for j in range(h * p["G"], (h + 1) * p["G"]):
                q = p["q"][b, j].astype(np.float64)
                x = k @ q * scale
                w = np.exp(x - x.max())
                out[b, j] = w @ v / w.sum()
                a = abs(scale) * (np.abs(k) @ np.abs(q)).max()
                err = (2.0 ** -22 + 137 * 2.0 ** -24) * a + 2.0 ** -22
                tol[b, j] = 2 * (err + 2.0 ** -16) * np.abs(v).max()
    return out, tol


def attend(A, p, splits=0, most=None, scale=None, **kw):
    st = A.new_status()
    most = int(max(p["lens"].max(), 0)) if most is None else most
    out = A.q8_decode_attention(dev(p["q"]), dev(p["pages"]), dev(p["scales"]), dev(p["bt"]), dev(p["lens"]), most,
                                scale, splits, status=st, **kw)
    torch.cuda.synchronize()
    return out.cpu().numpy(), int(st.item())


def close(got, want, tol):
    assert np.all(np.isfinite(got)), "non-finite output"
    err = np.abs(got.astype(np.float64) - want)
    assert np.all(err <= tol), f"{np.max(err - tol):.3e} past the bound, worst {np.max(err):.3e}"


CASES = [
    # (B, Hkv, G, lens)
    (1, 1, 1, [1]), (1, 2, 1, [512]), (5, 3, 1, [0, 1, 15, 16, 17]), (3, 2, 2, [33, 128, 129]),
    (2, 1, 3, [700, 45]), (2, 2, 4, [1000, 257]), (1, 1, 5, [100]), (2, 1, 7, [300, 64]), (8, 8, 8, [300, 1, 77, 160, 999, 64, 5, 410]),
    (1, 2, 9, [130]), (2, 1, 12, [511, 2]), (1, 1, 16, [2049]), (1, 2, 17, [50]), (1, 1, 2, [9001]), (40, 4, 1, list(range(0, 800, 20))),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}H{c[1]}G{c[2]}L{max(c[3])}" for c in CASES])
@pytest.mark.parametrize("splits", [0, 1, 2, 7, 11])
def test_attention_matches_reference(A, case, fmt, splits):
    B, Hkv, G, lens = case
    p = problem(np.random.default_rng(B * 1000 + G * 10 + len(fmt)), B, Hkv, G, lens, fmt)
    got, st = attend(A, p, splits)
    assert st == 0
    close(got, *reference(p))
    for b, L in enumerate(lens):
        if L == 0:
            assert np.all(got[b] == 0.0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_planned_longer_than_the_requests(A, fmt):
    """max_seq_len far above the lengths: whole splits are empty."""
    p = problem(np.random.default_rng(5), 3, 2, 4, [40, 0, 3], fmt)
    p["bt"] = np.concatenate([p["bt"], np.full((3, 500), -7, np.int32)], 1)
    for splits in (0, 5, 13):
        got, st = attend(A, p, splits, most=8000)
        assert st == 0
        close(got, *reference(p))


@pytest.mark.parametrize("splits", [1, 3])
def test_attention_scales_of_every_size(A, splits):
    """Blocks whose scales differ by 2^40, zero among them; a peaked softmax; and
    queries from 2^-100 to 2^60 (their keys scaled to match)."""
    g = np.random.default_rng(6)
    p = problem(g, 2, 3, 4, [400, 163], "int8")
    p["scales"][..., 1] *= 2.0 ** g.integers(-30, 11, p["scales"].shape[:2])
    p["scales"][::5, 0, 1] = 0.0
    p["scales"][::7, 1, 0] = 0.0
    p["scales"][3::4, 2, 0] *= 30.0
    close(attend(A, p, splits)[0], *reference(p))
    for e in (-100, -20, 60):
        p2 = problem(g, 2, 2, 2, [100, 37], "int8")
        p2["q"] *= np.float32(2.0 ** e)
        p2["scales"][..., 0] *= np.float32(2.0 ** -e)
        close(attend(A, p2, splits)[0], *reference(p2))
    p3 = problem(g, 1, 1, 2, [64], "e4m3")
    p3["q"][0, 1] = 0.0                                                     # equal weights
    close(attend(A, p3, splits)[0], *reference(p3))
    p4 = problem(g, 1, 2, 3, [90], "int8")
    for s in (0.0, -0.3):
        close(attend(A, p4, splits, scale=s)[0], *reference(p4, s))


@pytest.mark.parametrize("splits", [1, 2])
def test_attention_long_flat_softmax(A, splits):
    """Many tokens far below the largest: their small weights count together."""
    g = np.random.default_rng(8)
    p = problem(g, 1, 1, 1, [20000], "int8")
    p["pages"][:, :, 0] = 0
    p["pages"][:, :, 1] = 100
    p["scales"][..., 0], p["scales"][..., 1] = 1.0, 0.01
    pg = p["bt"][0, 0]
    p["pages"][pg, 0, 0, 0] = 1                                             # one key with a score of 11.5
    p["pages"][pg, 0, 1, 0] = -100
    p["q"][:] = 11.5 / D * D ** 0.5
    close(attend(A, p, splits)[0], *reference(p))


@pytest.mark.parametrize("splits", [1, 3])
def test_attention_nan_blocks_and_data_errors(A, splits):
    g = np.random.default_rng(9)
    p = problem(g, 4, 2, 2, [100, 50, 70, 20], "int8")
    want, tol = reference(p)
    q = dict(p, scales=p["scales"].copy())
    q["scales"][p["bt"][0, 2], 0, 0] = np.nan                               # a key block of request 0, head 0
    q["scales"][p["bt"][1, 3], 1, 1] = np.nan                               # a value block, one token of it in use... or none
    q["scales"][-3:] = np.where(np.isin(np.arange(len(p["scales"]))[-3:, None, None], p["bt"][:, :7]), q["scales"][-3:], np.nan)
    got, st = attend(A, q, splits)
    assert st == 0
    assert np.isnan(got[0, :2]).all() and np.isnan(got[1, 2:]).all()
    keep = np.ones((4, 4), bool)
    keep[0, :2] = keep[1, 2:] = False
    close(got[keep], want[keep], tol[keep])
    for j, bad in ((1, 10**6), (0, -1)):
        r = dict(p, bt=p["bt"].copy())
        r["bt"][2, j] = bad
        got, st = attend(A, r, splits)
        assert st == 1 and np.isnan(got[2]).all()
        close(got[[0, 1, 3]], want[[0, 1, 3]], tol[[0, 1, 3]])
    for L, most in ((-1, 100), (10**6, 100), (80, 79)):
        r = dict(p, lens=p["lens"].copy())
        r["lens"][3], r["lens"][0] = L, min(100, most)
        got, st = attend(A, r, splits, most=most)
        w, t = reference(dict(r, lens=np.where(np.arange(4) == 3, 0, r["lens"]).astype(np.int32)))
        assert st == 2 and np.isnan(got[3]).all()
        close(got[:3], w[:3], t[:3])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_writes_only_its_outputs(A, fmt):
    p = problem(np.random.default_rng(10), 3, 2, 3, [200, 0, 77], fmt)
    n = p["q"].size
    for splits in (1, 3, 12):
        need = A.q8_decode_plan(3, 6, 2, 200, splits)[1]
        buf = torch.full((n + 2048,), 7.0, device="cuda")
        ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out = buf[1024:1024 + n].view(3, 6, D)
        got, st = attend(A, p, splits, out=out, workspace=ws[2048:2048 + need] if need else None)
        close(got, *reference(p))
        assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all())
        assert bool((ws[:2048] == 0xA5).all()) and bool((ws[2048 + need:] == 0xA5).all())


def test_attention_in_two_streams_and_graphs(A):
    """Calls on two streams at once, and captured ones that share no workspace,
    equal the plain call."""
    p = problem(np.random.default_rng(14), 4, 4, 4, [900, 30, 500, 411], "int8")
    t = [dev(p[k]) for k in ("q", "pages", "scales", "bt", "lens")]
    want = A.q8_decode_attention(*t, 900, num_splits=12)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([A.q8_decode_attention(*t, 900, num_splits=12) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for x in outs for o in x)
    graphs, outs = [], [torch.zeros_like(want) for _ in range(2)]
    for o in outs:
        g = torch.cuda.CUDAGraph()
        ws = torch.empty(A.q8_decode_plan(4, 16, 4, 900, 12)[1], dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(g):
            A.q8_decode_attention(*t, 900, num_splits=12, out=o, workspace=ws)
        graphs.append((g, ws))
    for s, (g, _) in zip(streams, graphs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_cache_past_32_bits(A):
    """Pages whose byte offset passes 2^32, appended to, read back and attended over."""
    H, NP = 32, 36000                                                       # 4.7 GB of codes
    pages, scales = torch.zeros((NP, H, 2, P, D), dtype=torch.int8, device="cuda"), torch.zeros((NP, H, 2), device="cuda")
    g = np.random.default_rng(15)
    bt = np.array([[NP - 1, 33000, 2]], np.int32)
    kv = draw_kv(g, 40, H)
    lens, cu = dev(np.array([40], np.int32)), dev(np.array([0, 40], np.int32))
    st = A.new_status()
    A.q8_append(dev(kv), pages, scales, dev(bt), lens, cu, st)
    small, ssc = np.zeros((3, H, 2, P, D), np.int8), np.zeros((3, H, 2), np.float32)
    model_append(small, ssc, [0, 1, 2], 0, kv, "int8")
    sel = torch.from_numpy(bt[0].astype(np.int64)).cuda()
    assert np.array_equal(pages[sel].cpu().numpy(), small) and np.array_equal(scales[sel].cpu().numpy(), ssc)
    assert int(pages.count_nonzero()) == int(np.count_nonzero(small))
    q = g.standard_normal((1, H, D)).astype(np.float32)
    got = A.q8_decode_attention(dev(q), pages, scales, dev(bt), lens, 40, status=st)
    assert int(st.item()) == 0
    p = dict(q=q, pages=small, scales=ssc, bt=np.array([[0, 1, 2]]), lens=np.array([40]), fmt="int8", G=1)
    close(got.cpu().numpy(), *reference(p))


def test_wrappers_refuse(A):
    p = problem(np.random.default_rng(16), 2, 2, 2, [20, 30], "int8")
    q, pages, sc, bt, lens = (dev(p[k]) for k in ("q", "pages", "scales", "bt", "lens"))
    kv = torch.zeros(2, 2, 2, D, dtype=torch.float16, device="cuda")
    for bad in ((kv.float(), pages, sc, bt, lens), (kv, pages.half(), sc, bt, lens), (kv, pages, sc[:1], bt, lens),
                (kv, pages, sc, bt[:1], lens), (kv, pages, sc, bt, lens.long()), (kv[:1], pages, sc, bt, lens),
                (kv[:, :1], pages, sc, bt, lens), (kv, pages, sc, bt, lens, torch.zeros(2, dtype=torch.int32, device="cuda")),
                (kv, pages[:, :, :1].contiguous(), sc, bt, lens), (kv, pages.transpose(0, 1), sc, bt, lens)):
        with pytest.raises((ValueError, TypeError)):
            A.q8_append(*bad)
    for bad in ((q.half(), pages, sc, bt, lens), (q[:1], pages, sc, bt, lens), (q[..., :64].contiguous(), pages, sc, bt, lens)):
        with pytest.raises((ValueError, TypeError)):
            A.q8_decode_attention(*bad, 30)
    with pytest.raises(A._lib.AQError):
        A.q8_decode_attention(q[:, :3].contiguous(), pages, sc, bt, lens, 30)           # 3 heads over 2
    with pytest.raises(A._lib.AQError):
        A.q8_decode_attention(q, pages, sc, bt, lens, 10**6)                            # beyond the table
    wide = torch.zeros(2, 20, dtype=torch.int32, device="cuda")
    with pytest.raises(A._lib.AQError):
        A.q8_decode_attention(q, pages, sc, wide, lens, 300, num_splits=9, workspace=torch.zeros(64, device="cuda"))


def test_attention_wait_limit(A):
    """With no time to wait for its copies a call ends all the same: every output
    is NaN or right, NaN only with the timeout bit, and the next call is right.
    (A cold cache of 100 MB, so that copies queue behind one another.)"""
    g = np.random.default_rng(17)
    p = problem(g, 26, 8, 1, [0, 16] + [int(x) for x in g.integers(1500, 2001, 24)], "int8")
    want, tol = reference(p)
    lib = A._lib.load()
    t = [dev(p[k]) for k in ("q", "pages", "scales", "bt", "lens")]
    flush = torch.zeros(300 << 20, dtype=torch.uint8, device="cuda")
    for splits in (1, 4, 12):
        seen, st = 0, A.new_status()
        for limit in (0, 0, 0, None):
            flush += 1
            st.zero_()
            prev = lib.aq_set_wait_limit_ns(limit) if limit is not None else None
            try:
                got = A.q8_decode_attention(*t, int(p["lens"].max()), num_splits=splits, status=st)
                torch.cuda.synchronize()
            finally:
                if prev is not None:
                    lib.aq_set_wait_limit_ns(prev)
            got, flag = got.cpu().numpy(), int(st.item())
            assert flag in ((0, 8) if limit is not None else (0,))
            bad = np.isnan(got)
            assert np.array_equal(bad.any(-1), bad.all(-1)) and (flag == 8) == bool(bad.any())
            close(got[~bad.any(-1)], want[~bad.any(-1)], tol[~bad.any(-1)])
            seen |= flag
        assert seen == 8, splits


@pytest.mark.parametrize("splits", [1, 4, 12])
def test_attention_non_finite_queries_stay_in_their_heads(A, splits):
    """An infinite or NaN query makes its own head's output NaN, no other's."""
    g = np.random.default_rng(18)
    for fmt in ("int8", "e4m3"):
        p = problem(g, 2, 2, 8, [300, 17], fmt)
        want, tol = reference(p)
        p["q"][0, 3, 5], p["q"][0, 12, 100], p["q"][1, 0, 0] = np.inf, np.nan, -np.inf
        got, st = attend(A, p, splits)
        bad = np.zeros((2, 16), bool)
        bad[0, 3] = bad[0, 12] = bad[1, 0] = True
        assert st == 0 and np.isnan(got[bad]).all()
        close(got[~bad], want[~bad], tol[~bad])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_step_in_a_graph(A, fmt):
    """Q8DecodeStep captured once and replayed while the requests grow equals the
    calls made one by one."""
    g = np.random.default_rng(19)
    B, H, G, mp = 3, 2, 4, 6
    rope = A.Rope(128, 1e4)
    bt = dev(g.permutation(B * mp).reshape(B, mp).astype(np.int32))
    caches = [A.new_q8_cache(B * mp, H, e4m3=fmt == "e4m3") for _ in range(2)]
    lens = dev(np.array([30, 1, 15], np.int32))
    kv0 = dev(draw_kv(g, 46, H))
    cu = dev(np.array([0, 30, 31, 46], np.int32))
    for pages, scales in caches:
        A.q8_append(kv0, pages, scales, bt, lens, cu)
    q, kv = torch.zeros(B, H * G, D, device="cuda"), torch.zeros(B, H, 2, D, dtype=torch.float16, device="cuda")
    steps = [A.Q8DecodeStep(pages, scales, bt, lens, mp * P, H * G, rope=rope, num_splits=s) for (pages, scales), s in zip(caches, (0, 0))]
    keep = [c.clone() for c in caches[0]]
    lens += 1
    steps[0].run(q, kv)                                                     # (loads the kernels)
    lens -= 1
    for c, k in zip(caches[0], keep):
        c.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        steps[0].run(q, kv)
    for _ in range(20):
        q.copy_(dev(g.standard_normal((B, H * G, D)).astype(np.float32)))
        kv.copy_(dev(draw_kv(g, B, H)))
        graph.replay()
        want = steps[1].run(q, kv)
        assert torch.equal(steps[0].out, want)
        assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    for s in steps:
        s.check_status()
    assert lens.tolist() == [50, 21, 35]


def test_rows_past_32_bits(A):
    """Appends and read-backs whose element offsets pass 2^31."""
    T, H = 70001, 128                                                       # 2.3e9 halves
    g = np.random.default_rng(20)
    kv = torch.zeros((T, H, 2, D), dtype=torch.float16, device="cuda")
    tail = draw_kv(g, 33, H)
    kv[-33:] = dev(tail)
    NP = -(-T // P)
    pages, scales = A.new_q8_cache(NP, H)
    bt, lens = dev(np.arange(NP, dtype=np.int32)[None]), dev(np.array([T], np.int32))
    cu = dev(np.array([0, T], np.int32))
    st = A.new_status()
    A.q8_append(kv, pages, scales, bt, lens, cu, st)
    back = A.q8_load(pages, scales, bt, lens, cu, T, status=st)
    assert int(st.item()) == 0
    small, ssc = np.zeros((4, H, 2, P, D), np.int8), np.zeros((4, H, 2), np.float32)
    first = (T - 33) // P * P
    x = np.concatenate([np.zeros((T - 33 - first, H, 2, D), np.float16), tail])
    model_append(small, ssc, [0, 1, 2, 3], 0, x, "int8")
    n = -(-len(x) // P)
    assert np.array_equal(pages[-n:, :, :].cpu().numpy()[:-1], small[:n - 1])
    assert np.array_equal(pages[-1, :, :, :(T - 1) % P + 1].cpu().numpy(), small[n - 1, :, :, :(T - 1) % P + 1])
    assert np.array_equal(scales[-n:].cpu().numpy(), ssc[:n])
    err = (back[-33:].float() - dev(tail).float()).abs()
    assert float((err - 0.51 * scales[-n:].max()).max()) <= 0 and int(back[:first].count_nonzero()) == 0


@pytest.mark.parametrize("splits", [1, 4, 12])
def test_nan_block_of_no_weight_is_not_lost(A, splits):
    """A NaN value block whose tokens' weights vanish still makes its outputs NaN."""
    g = np.random.default_rng(21)
    p = problem(g, 1, 2, 2, [900], "int8")
    p["pages"][:, 0, 0] = 0
    pg = p["bt"][0, 5]
    p["pages"][p["bt"][0, 40], 0, 0, 3] = 127                               # one key far ahead of all others
    p["scales"][:, 0, 0] = 10.0
    p["q"][0, :2] = 10.0
    p["scales"][pg, 0, 1] = np.nan
    got, st = attend(A, p, splits)
    assert st == 0 and np.isnan(got[0, :2]).all() and np.isfinite(got[0, 2:]).all()
