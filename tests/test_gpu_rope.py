"""Rotary positions on the GPU against the formula in 64 bits.

Error of a rotated element: the 32-bit fraction of a half turn is off by 2^-25
(pi * 2^-25 = 9.4e-8 in the angle), sine and cosine by 2^-23, their product with
mscale 2^-24, the two products and the sum 3 * 2^-24: together under 5e-7 *
mscale * (|x1| + |x2|).  The angle itself holds a frequency of 53 bits on both
sides: the kernel's turns per position are off by 1.5 * 2^-53 relative, the
reference's product by 2^-53, so position * w * 2.5 * 2^-53 comes on top (6e-7 at
position 2^31, w = 1).  A key is then rounded to fp16, half a step: 2^-11 of its
value (2^-25 below fp16's normal range).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_product_gb300 import build
    build.build()
    from decode_attention_product_gb300 import api
    return api


def reference(x, pos, w, interleaved, m, transpose):
    """(rotated x, error bound) in float64; x [T][H][D]"""
    x = np.asarray(x, np.float64)
    r = 2 * len(w)
    i = np.arange(r).reshape(-1, 2) if interleaved else np.arange(r).reshape(2, -1).T
    a = np.maximum(pos, 0).astype(np.float64)[:, None] * w[None]
    c, s = np.cos(a)[:, None] * m, np.sin(a)[:, None] * (-m if transpose else m)
    y, tol = x.copy(), np.zeros_like(x)
    x1, x2 = x[..., i[:, 0]], x[..., i[:, 1]]
    y[..., i[:, 0]], y[..., i[:, 1]] = x1 * c - x2 * s, x1 * s + x2 * c
    tol[..., i[:, 0]] = tol[..., i[:, 1]] = (5e-7 + a[:, None] * 2.5 * 2.0 ** -53) * m * (np.abs(x1) + np.abs(x2))
    pad = pos < 0
    y[pad], tol[pad] = x[pad], 0.0
    return y, tol


def check(A, T, Hq, Hkv, rot, interleaved, far, transpose=False, m=1.0, seed=0, in_place=False):
    g = np.random.default_rng(seed)
    pos = g.integers(0, far + 1, T).astype(np.int32)
    pos[0] = far
    if T > 2:
        pos[1], pos[-1] = 0, -1
    w = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    q = g.standard_normal((T, Hq, 128), np.float32) if Hq else None
    kv = g.standard_normal((T, Hkv, 2, 128), np.float32).astype(np.float16) if Hkv else None
    dq, dkv = (torch.from_numpy(t).cuda() if t is not None else None for t in (q, kv))
    kw = dict(q_out=dq, kv_out=dkv) if in_place else {}
    qo, kvo = A.rope(torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(), dq, dkv, interleaved=interleaved,
                     mscale=m, transpose=transpose, **kw)
    torch.cuda.synchronize()
    if Hq:
        want, tol = reference(q, pos, w, interleaved, m, transpose)
        err = np.abs(qo.cpu().numpy() - want)
        assert np.all(err <= tol), f"q: {np.max(err - tol):.3e} past the bound"
        assert (qo.data_ptr() == dq.data_ptr()) == in_place
        if not in_place:
            assert np.array_equal(dq.cpu().numpy(), q)
    if Hkv:
        got = kvo.cpu().numpy()
        want, tol = reference(kv[:, :, 0], pos, w, interleaved, m, transpose)
        turned = tol > 0
        tol = tol + np.where(turned, 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -25, 0.0)
        assert np.all(np.abs(got[:, :, 0].astype(np.float64) - want) <= tol)
        assert np.array_equal(got[:, :, 1], kv[:, :, 1])


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [8, 24, 64, 96, 120, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (3, 5, 3), (17, 64, 8), (300, 9, 0), (300, 0, 9), (5, 1, 33)])
def test_rope_matches_formula(A, T, Hq, Hkv, rot, interleaved):
    check(A, T, Hq, Hkv, rot, interleaved, 5000, m=1.25)
    check(A, T, Hq, Hkv, rot, interleaved, 131072, transpose=True, in_place=True)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("far", [0, 1, 2**20 + 1, 2**31 - 1])
def test_rope_far_positions(A, far, interleaved):
    check(A, 40, 4, 4, 128, interleaved, far)


def test_rope_prompt_size(A):
    check(A, 2049, 32, 32, 64, True, 131072, m=1.1)


def test_rope_gradient(A):
    """The map is linear, so the gradient of sum(g * rope(x)) is rope^T(g):
    against the formula's, and against central differences of the kernel
    itself.  Step h = 2^-4: the difference quotient's rounding is the two outputs'
    2 * 5e-7 (|x1| + |x2|) m over 2 h, times |g|, for both outputs of the pair; x + h
    is rounded too (2^-22 over 2 h).  With |x|, |g| <= 5: under 5e-7 * 10 * 1.5 * 16 *
    5 * 2 + 2^-22 * 8 * 1.5 * 5 * 2 = 1.3e-3."""
    g = np.random.default_rng(3)
    T, H, rot = 7, 3, 96
    pos = torch.from_numpy(g.integers(0, 9000, T).astype(np.int32)).cuda()
    w = torch.from_numpy(10000.0 ** (-np.arange(0, rot, 2) / rot)).cuda()
    x = torch.from_numpy(g.standard_normal((T, H, 128), np.float32)).cuda()
    up = torch.from_numpy(g.standard_normal((T, H, 128), np.float32)).cuda()
    for inter in (False, True):
        grad = A.rope(pos, w, up, interleaved=inter, mscale=1.5, transpose=True)[0].double()
        want, tol = reference(up.cpu().numpy(), pos.cpu().numpy(), w.cpu().numpy(), inter, 1.5, True)
        assert np.all(np.abs(grad.cpu().numpy() - want) <= tol)
        h = 2.0 ** -4
        for d in (0, 1, 47, 48, 95, 96, 127):
            e = torch.zeros_like(x)
            e[:, :, d] = h
            hi = A.rope(pos, w, x + e, interleaved=inter, mscale=1.5)[0].double()
            lo = A.rope(pos, w, x - e, interleaved=inter, mscale=1.5)[0].double()
            diff = ((hi - lo) / (2 * h) * up.double()).sum(-1)
            assert float((diff - grad[:, :, d]).abs().max()) <= 1.3e-3


def test_rope_lengths_and_nothing(A):
    """lengths=True stands token t at length - 1 (length 0: padding); no tokens: no output."""
    r = A.Rope(64, 5e5, interleaved=True, scaling="yarn", factor=4.0, original_len=2048)
    q = torch.randn(4, 3, 128, device="cuda")
    lens = torch.tensor([1, 0, 77, 2**31 - 1], dtype=torch.int32, device="cuda")
    a, none = r(lens, q, lengths=True)
    assert none is None and torch.equal(a, r(lens - 1, q)[0])
    assert torch.equal(a[1], q[1])
    assert torch.equal(a[0, :, 64:], q[0, :, 64:])
    low = torch.tensor([-2**31] * 4, dtype=torch.int32, device="cuda")
    assert torch.equal(r(low, q, lengths=True)[0], q)
    e = r(lens[:0], q[:0])[0]
    assert e.shape == (0, 3, 128)


def test_rope_non_finite_values_stay_in_their_pairs(A):
    q = torch.ones(2, 2, 128, device="cuda")
    q[0, 0, 3], q[1, 1, 100] = math.inf, math.nan
    w = torch.full((32,), 0.3, dtype=torch.float64, device="cuda")
    y = A.rope(torch.tensor([5, 6], dtype=torch.int32, device="cuda"), w, q)[0]
    bad = ~torch.isfinite(y)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 35]
    assert bad[1, 1].nonzero().flatten().tolist() == [100]              # an unturned dim
    assert int(bad.sum()) == 3


def test_rope_refuses(A):
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones(64, dtype=torch.float64, device="cuda")
    q, kv = torch.zeros(4, 2, 128, device="cuda"), torch.zeros(4, 2, 2, 128, dtype=torch.float16, device="cuda")
    for bad in (dict(), dict(q=q[:3]), dict(q=q.half()), dict(q=q.transpose(0, 1)), dict(kv=kv.float()),
                dict(q=q, q_out=q[:2]), dict(kv=kv[:, :, :1].contiguous()), dict(q_out=q, kv=kv), dict(kv_out=kv, q=q)):
        with pytest.raises((ValueError, TypeError)):
            A.rope(pos, w, **bad)
    long = torch.zeros(5, 2, 128, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        A.rope(pos, w, q=long[:4], q_out=long[1:])
    with pytest.raises(RuntimeError):
        A.rope(pos, w[:3], q=q)                                          # 6 dims
    with pytest.raises(RuntimeError):
        A.rope(pos, w, q=torch.zeros(4, 2, 64, device="cuda"))           # head_dim


def test_rope_on_a_stream_and_in_a_graph(A):
    r = A.Rope(128, 1e4)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    q, kv = torch.randn(6, 4, 128, device="cuda"), torch.randn(6, 2, 2, 128, device="cuda").half()
    want = r(pos, q, kv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = r(pos, q, kv)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qo, kvo = torch.empty_like(q), torch.empty_like(kv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r(pos, q, kv, q_out=qo, kv_out=kvo)
    pos += 1000
    graph.replay()
    want = r(pos, q, kv)
    torch.cuda.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(kvo, want[1])


def test_decode_step_with_rope(A):
    """DecodeStep(rope=...) is the rotation followed by the step without one."""
    import workloads as W
    p = W.paged_codes_problem(5, 2, 4, 2, 4, [40, 17], num_sets=2)
    d = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in p.items() if k != "num_pages"}
    kv = torch.randn(2, 2, 2, 128, device="cuda").half()
    rope = A.Rope(128, 1e4)

    def step(r, pages):
        return A.DecodeStep(pages, d["codebooks"], d["req_set"], d["block_table"], d["seq_lens"], 40, None, None, 4, rope=r)
    p1, p2 = d["code_pages"].clone(), d["code_pages"].clone()
    s1 = step(rope, p1)
    got = s1.run(d["q"], kv)
    q2, kv2 = rope(d["seq_lens"] - 1, d["q"], kv)
    want = step(None, p2).run(q2, kv2)
    torch.cuda.synchronize()
    s1.check_status()
    assert torch.equal(got, want) and torch.equal(p1, p2) and not torch.equal(p1, d["code_pages"])


def test_rope_past_32_bits(A):
    """Rows whose element offset passes 2^31."""
    T, H = 70001, 256                                                       # 2.3e9 elements
    q = torch.zeros(T, H, 128, device="cuda")
    g = np.random.default_rng(7)
    tail = g.standard_normal((3, H, 128), np.float32)
    q[-3:] = torch.from_numpy(tail).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    w = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    A.rope(pos, torch.from_numpy(w).cuda(), q, q_out=q)
    want, tol = reference(tail, np.arange(T - 3, T), w, False, 1.0, False)
    assert np.all(np.abs(q[-3:].cpu().numpy() - want) <= tol)
    assert int(q[:-3].count_nonzero()) == 0
