"""Page management on the GPU against a plain sequential model of a block table
with reference counts, every array compared after every call; and the operators
together, as a decode server runs them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

P = 16
BAD_PAGE, BAD_LENGTH, NO_PAGE, BAD_ROW = 1, 2, 32, 64


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_attention_product_gb300 import build
    build.build()
    from decode_attention_product_gb300 import api
    return api


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).cuda()


def pages_of(n):
    return -(-n // P)


class Model:
    def __init__(self, R, mp, NP, widths, seed=0):
        g = np.random.default_rng(seed)
        self.bt = np.full((R, mp), -1, np.int32)
        self.lens, self.rc, self.status = np.zeros(R, np.int32), np.zeros(NP, np.int32), 0
        self.pools = [g.integers(0, 256, (NP, w)).astype(np.uint8) for w in widths]

    def ok(self, r):
        return 0 <= r < len(self.lens)

    def extend(self, rows, lens):
        cap, free = self.bt.shape[1] * P, np.nonzero(self.rc == 0)[0]
        rc0, pools0 = self.rc.copy(), [p.copy() for p in self.pools]
        used, seen, plan = 0, set(), []
        for r, n in zip(rows, lens):
            if not self.ok(r) or r in seen:
                self.status |= BAD_ROW
                continue
            seen.add(r)
            L = int(self.lens[r])
            if not 0 <= L <= cap or not L <= n <= cap:
                self.status |= BAD_LENGTH
                continue
            have, want, copy = pages_of(L), pages_of(n), False
            if n > L and L % P:
                pg = self.bt[r, have - 1]
                if not 0 <= pg < len(self.rc):
                    self.status |= BAD_PAGE
                    continue
                copy = rc0[pg] > 1
            plan.append((r, n, have, want, copy, used))
            used += want - have + copy
        for r, n, have, want, copy, at in plan:
            need = want - have + copy
            if need and at + need > len(free):
                self.status |= NO_PAGE
                continue
            new = free[at:at + need]
            self.rc[new] = 1
            if copy:
                old = self.bt[r, have - 1]
                self.rc[old] -= 1
                for p, p0 in zip(self.pools, pools0):
                    p[new[0]] = p0[old]
            self.bt[r, have - copy:want] = new
            self.lens[r] = n

    def fork(self, src, dst):
        lens0, seen = self.lens.copy(), set()
        for s, d in zip(src, dst):
            first = d not in seen
            seen.add(d)
            if not self.ok(s) or not self.ok(d) or not first or lens0[d] != 0 or s in dst:
                self.status |= BAD_ROW
                continue
            n = pages_of(int(lens0[s]))
            self.bt[d, :n] = self.bt[s, :n]
            for pg in self.bt[s, :n]:
                self.rc[pg] += 1
            self.lens[d] = lens0[s]

    def free(self, rows, keep=None):
        for r, k in zip(rows, np.zeros(len(rows), int) if keep is None else keep):
            if not self.ok(r):
                self.status |= BAD_ROW
                continue
            if k < 0:
                self.status |= BAD_LENGTH
                continue
            for j in range(pages_of(int(k)), pages_of(int(self.lens[r]))):
                self.rc[self.bt[r, j]] -= 1
                self.bt[r, j] = -1
            self.lens[r] = min(self.lens[r], k)

    def compact(self):
        live = self.rc > 0
        n, ids = int(live.sum()), np.arange(len(self.rc))
        movers, holes = ids[live & (ids >= n)], ids[~live & (ids < n)]
        to = ids.copy()
        to[movers] = holes
        for p in self.pools:
            p[holes] = p[movers]
        self.rc[holes] = self.rc[movers]
        self.rc[movers] = 0
        for r, L in enumerate(self.lens):
            self.bt[r, :pages_of(int(L))] = to[self.bt[r, :pages_of(int(L))]]


class Both:
    """The model and the device side by side."""

    def __init__(self, A, R, mp, NP, widths=(64, 4, 20, 4112), seed=0):
        self.A, self.m = A, Model(R, mp, NP, widths, seed)
        self.t = A.PageTable(R, mp, [torch.from_numpy(p).cuda() for p in self.m.pools])

    def same(self):
        for name, a, b in (("block_table", self.t.block_table, self.m.bt), ("seq_lens", self.t.seq_lens, self.m.lens),
                           ("refcount", self.t.refcount, self.m.rc)):
            assert np.array_equal(a.cpu().numpy(), b), name
        for i, (a, b) in enumerate(zip(self.t.pools, self.m.pools)):
            assert np.array_equal(a.cpu().numpy(), b), f"pool {i}"
        assert int(self.t.status.item()) == self.m.status

    def do(self, op, *args):
        getattr(self.m, op)(*[None if a is None else np.asarray(a) for a in args])
        getattr(self.t, op)(*[None if a is None else dev(a) for a in args])
        self.same()


@pytest.mark.parametrize("seed,R,mp,NP", [(0, 12, 9, 60), (1, 40, 5, 150), (2, 3, 40, 64), (3, 200, 12, 5000), (4, 8, 3, 4096),
                                          (5, 6, 4, 4097), (6, 1500, 3, 6 * 4096), (7, 30, 6, 6 * 4096 + 1)])
def test_random_runs_match_the_model(A, seed, R, mp, NP):
    """Random forks, growth, truncation, endings and compactions; pools run out
    now and then; rows repeat, lie outside, or break the rules."""
    g = np.random.default_rng(seed)
    b = Both(A, R, mp, NP, (64, 4, 20) if NP > 20000 else (64, 4, 20, 4112), seed=seed)
    for _ in range(30):
        lens, n = b.m.lens, int(g.integers(1, R + 1))
        op = g.choice(["extend", "extend", "fork", "free", "truncate", "compact"])
        rows = g.permutation(R)[:n] if g.random() < 0.7 else g.integers(-1, R + 1, n)
        if op == "extend":
            old = np.array([lens[r] if 0 <= r < R else 0 for r in rows])
            new = np.minimum(old + g.choice([0, 1, 3, 16, 17, 50], n), mp * P + int(g.random() < 0.2))
            new = np.where(g.random(n) < 0.05, old - 1, new)
            b.do("extend", rows, new)
        elif op == "fork":
            empty = np.nonzero(lens == 0)[0]
            dst = g.choice(empty, n) if len(empty) and g.random() < 0.8 else g.integers(-1, R + 1, n)
            b.do("fork", rows, dst)
        elif op == "free":
            b.do("free", rows[:max(1, n // 3)], None)
        elif op == "truncate":
            b.do("free", rows, g.integers(-1 if g.random() < 0.2 else 0, mp * P + 1, n))
        else:
            b.do("compact")


def test_fork_shares_and_growth_copies(A):
    b = Both(A, 6, 4, 20)
    b.do("extend", [0], [40])
    b.do("fork", [0, 0, 0], [1, 2, 3])
    assert b.m.rc[:3].tolist() == [4, 4, 4]
    b.do("extend", [2], [41])                   # a copy of page 2 for row 2 alone
    assert b.m.bt[2, :3].tolist() == [0, 1, 3] and b.m.rc[:4].tolist() == [4, 4, 3, 1]
    b.do("extend", [0, 1, 3], [48, 49, 40])     # row 3 does not grow: it keeps the shared page
    assert b.m.rc[2] == 1 and b.m.bt[3, 2] == 2
    b.do("free", [1], [20])                     # mid-page: page 1 stays shared
    b.do("extend", [1], [33])                   # ... and is copied before it is written again
    assert b.m.bt[1, 1] != 1 and b.m.rc[1] == 3
    b.do("free", [0, 1, 2, 3, 0], None)
    assert not b.m.rc.any() and not b.m.lens.any()
    b.do("extend", [5, 4], [64, 1])
    assert b.m.bt[5].tolist() == [0, 1, 2, 3] and b.m.bt[4, 0] == 4


def test_pool_runs_out(A):
    """Rows are served in order; one that does not fit changes nothing."""
    b = Both(A, 4, 8, 10)
    b.do("extend", [0], [50])
    b.do("fork", [0], [1])
    b.do("extend", [0, 1, 2], [51, 100, 16])    # 1 copy, then 1 copy + 3 pages, then 1
    assert b.m.status == 0
    b.do("extend", [3, 2], [17, 20])            # 2 pages, one left
    assert b.m.status == NO_PAGE and b.m.lens[3] == 0 and b.m.lens[2] == 16
    b.do("extend", [2], [16])                   # no growth needs no page
    b.do("free", [1], [10])
    b.do("extend", [3], [17])


def test_needs_beyond_32_bits_do_not_wrap(A):
    """Rows that ask for far more pages than there are, together past 2^32."""
    R, mp = 520, 1 << 23
    bt = torch.full((R, 8), -1, dtype=torch.int32, device="cuda")
    lens, rc = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
    st = A.new_status()
    A.pages_extend(dev(np.arange(R)), dev(np.full(R, 8 * P)), bt, lens, rc, [], status=st)
    assert int(st.item()) == NO_PAGE and not int(lens.any()) and not int(rc.any())
    wide = torch.full((R, mp), -1, dtype=torch.int32, device="cuda")        # 17 GB
    rows = [3] + [r for r in range(R) if r != 3]
    st.zero_()
    A.pages_extend(dev(rows), dev([P] + [mp * P - 1] * (R - 1)), wide, lens, rc, [], status=st)
    assert int(st.item()) == NO_PAGE and lens.nonzero().flatten().tolist() == [3] and int(lens[3]) == P
    assert rc.tolist() == [1, 0, 0, 0, 0] and int(wide[3, 0]) == 0 and int((wide[:8] != -1).sum()) == 1


def test_large_pool_and_pages(A):
    """More tiles than one CTA has threads would sum in a step; pages of 1 MB."""
    g = np.random.default_rng(3)
    NP, R, mp = 4096 * 1100 + 5, 64, 100
    rc = np.zeros(NP, np.int32)
    busy = g.random(NP) < 0.5
    rc[busy] = g.integers(1, 5, int(busy.sum()))
    d, bt, lens = dev(rc), torch.full((R, mp), -1, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    A.pages_extend(dev(np.arange(R)), dev(np.full(R, mp * P)), bt, lens, d, [])
    free = np.nonzero(rc == 0)[0][:R * mp]
    assert np.array_equal(bt.cpu().numpy().reshape(-1), free)
    rc[free] = 1
    assert np.array_equal(d.cpu().numpy(), rc)
    A.pages_compact(bt, lens, d, [])
    n = int((rc > 0).sum())
    got = d.cpu().numpy()
    assert (got[:n] > 0).all() and not got[n:].any() and int(got.sum()) == int(rc.sum())
    assert int(bt.max()) < n and len(np.unique(bt.cpu().numpy())) == R * mp
    b = Both(A, 3, 4, 9, widths=(1 << 20, 4))
    b.do("extend", [0, 1], [60, 30])
    b.do("fork", [1], [2])
    b.do("extend", [2, 1], [31, 32])
    b.do("free", [0], None)
    b.do("compact")


def test_damaged_tables_are_flagged(A):
    """Pages outside the pool or without references: a status bit, and nothing is
    read or written outside the arrays."""
    b = Both(A, 4, 4, 10)
    b.do("extend", [0, 1], [40, 20])
    t = b.t
    t.block_table[0, 1] = 99
    t.block_table[1, 1] = 7                                                 # not allocated
    t.fork(dev([0, 1]), dev([2, 3]))
    assert int(t.status.item()) == BAD_PAGE
    t.status.zero_()
    t.free(dev([0]))
    assert int(t.status.item()) == BAD_PAGE and t.refcount[:8].tolist() == [1, 1, 1, 2, 1, 0, 0, 1]
    t.status.zero_()
    t.seq_lens[3] = 1000
    t.compact()
    assert int(t.status.item()) & BAD_LENGTH
    t.status.zero_()
    t.extend(dev([3]), dev([1001]))
    t.fork(dev([3]), dev([0]))
    t.free(dev([3]))
    assert int(t.status.item()) == BAD_LENGTH


def test_calls_of_nothing_and_without_pools(A):
    bt, lens, rc = torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), dev([0, 0]), dev([0] * 5)
    none = dev([])
    A.pages_extend(none, none, bt, lens, rc, [])
    A.pages_fork(none, none, bt, lens, rc)
    A.pages_free(none, bt, lens, rc)
    A.pages_compact(bt, lens, rc, [])
    A.pages_extend(dev([1]), dev([17]), bt, lens, rc, [])
    assert bt.tolist() == [[-1] * 3, [0, 1, -1]] and lens.tolist() == [0, 17] and rc.tolist() == [1, 1, 0, 0, 0]
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    st = A.new_status()
    A.pages_extend(dev([0]), dev([1]), bt.clone(), dev([0, 0]), empty, [], status=st)
    assert int(st.item()) == NO_PAGE
    with pytest.raises(ValueError):
        A.pages_extend(dev([1]), dev([17, 3]), bt, lens, rc, [])
    with pytest.raises(ValueError):
        A.pages_extend(dev([1]), dev([18]), bt, lens, rc, [torch.zeros(4, 16, device="cuda")])     # 4 pages, not 5
    with pytest.raises(A._lib.AQError):
        A.pages_extend(dev([1]), dev([18]), bt, lens, rc, [torch.zeros(5, 6, dtype=torch.uint8, device="cuda")])
    with pytest.raises(A._lib.AQError):
        A.pages_extend(dev([0, 1, 0]), dev([1, 1, 1]), bt, lens, rc, [])    # more entries than rows
    with pytest.raises(A._lib.AQError):
        A.pages_extend(dev([0]), dev([1]), bt, lens, rc, [], workspace=torch.zeros(4, device="cuda"))


def test_captured_calls(A):
    """Fork, growth and truncation in a graph, replayed on new rows."""
    b = Both(A, 8, 4, 30)
    b.do("extend", [0, 1], [20, 35])
    src, dst, rows, lens = dev([0, 1]), dev([2, 3]), dev([2, 3]), dev([21, 36])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.t.fork(src, dst)
        b.t.extend(rows, lens)
        b.t.compact()
    for d in ([2, 3], [4, 5]):
        dst.copy_(dev(d))
        rows.copy_(dev(d))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.m.fork([0, 1], d)
        b.m.extend(d, [21, 36])
        b.m.compact()
        b.same()


# ------------------------------------------------------------- together ----
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_serving_run(A, fmt):
    """Prompts are appended in chunks, forked into samples, decoded step by step
    (rotary positions, append, attention), some end, the pool is compacted, new
    prompts take the freed pages.  Each step's output is compared with softmax
    attention in 64 bits over the tokens read back from the cache, and the tokens
    read back with the turned vectors that went in."""
    g = np.random.default_rng(4)
    R, mp, NP, Hkv, G = 8, 12, 60, 2, 3
    rope = A.Rope(64, 1e4, interleaved=True)
    pages, scales = A.new_q8_cache(NP, Hkv, e4m3=fmt == "e4m3")
    t = A.PageTable(R, mp, [pages, scales])
    raw = [np.zeros((0, Hkv, 2, 128)) for _ in range(R)]

    def vectors(n):
        return g.standard_normal((n, Hkv, 2, 128)).astype(np.float16)

    def prefill(rows, ns):
        lens = [len(raw[r]) + n for r, n in zip(rows, ns)]
        t.extend(dev(rows), dev(lens))
        kv = vectors(sum(ns))
        pos = np.concatenate([np.arange(len(raw[r]), L) for r, L in zip(rows, lens)])
        turned = rope(dev(pos), kv=torch.from_numpy(kv).cuda())[1]
        cu = np.concatenate([[0], np.cumsum(ns)])
        sel = dev(rows).long()
        A.q8_append(turned, pages, scales, t.block_table[sel], t.seq_lens[sel], dev(cu), t.status)
        for i, r in enumerate(rows):
            raw[r] = np.concatenate([raw[r], turned[cu[i]:cu[i + 1]].cpu().numpy().astype(np.float64)])

    def step(rows):
        lens = [len(raw[r]) + 1 for r in rows]
        t.extend(dev(rows), dev(lens))
        sel = dev(rows).long()
        bt, sl = t.block_table[sel], t.seq_lens[sel]
        kv = torch.from_numpy(vectors(len(rows))).cuda()
        q = torch.from_numpy(g.standard_normal((len(rows), Hkv * G, 128)).astype(np.float32)).cuda()
        s = A.Q8DecodeStep(pages, scales, bt, sl, max(lens), Hkv * G, rope=rope)
        out = s.run(q, kv).cpu().numpy()
        s.check_status()
        qt, kvt = rope(sl - 1, q, kv)
        cu = np.concatenate([[0], np.cumsum(lens)])
        back = A.q8_load(pages, scales, bt, sl, dev(cu), int(cu[-1]), status=t.status).cpu().numpy().astype(np.float64)
        for i, r in enumerate(rows):
            raw[r] = np.concatenate([raw[r], kvt[i:i + 1].cpu().numpy().astype(np.float64)])
            got = back[cu[i]:cu[i + 1]]
            # at most half a code per rounding; the 16 slots of a block grow its scale at most 15 times
            for p0 in range(0, lens[i], P):
                x = raw[r][p0:p0 + P]
                amax = np.abs(x).max(axis=(0, 3), keepdims=True)
                half = amax / 254 if fmt == "int8" else np.abs(x) * 2.0 ** -4 + amax * 2.0 ** -17
                assert np.all(np.abs(got[p0:p0 + P] - x) <= 16 * half + 2.0 ** -10 * amax)
            k, v = got[:, :, 0], got[:, :, 1]
            for h in range(Hkv):
                for j in range(h * G, (h + 1) * G):
                    w = k[:, h] @ qt[i, j].cpu().numpy().astype(np.float64) / 128 ** 0.5
                    w = np.exp(w - w.max())
                    want = w @ v[:, h] / w.sum()
                    # the read-back rounds keys and values to fp16 (2^-11): scores by 2^-11 * scale * sum |q k|
                    a = (np.abs(k[:, h]) @ np.abs(qt[i, j].cpu().numpy())).max() / 128 ** 0.5
                    assert np.all(np.abs(out[i, j] - want) <= (2 * 2.0 ** -11 * (a + 1) + 1e-4) * np.abs(v[:, h]).max())

    prefill([0, 1, 2], [37, 5, 64])
    prefill([1, 2], [30, 3])
    t.fork(dev([0, 0, 2]), dev([3, 4, 5]))
    for s, d in ((0, 3), (0, 4), (2, 5)):
        raw[d] = raw[s].copy()
    for _ in range(3):
        step([0, 1, 2, 3, 4, 5])
    t.free(dev([0, 2]))
    raw[0], raw[2] = raw[0][:0], raw[2][:0]
    t.compact()
    live = int((t.refcount > 0).sum())
    assert bool((t.refcount[:live] > 0).all())
    step([3, 4, 1, 5])
    prefill([7, 0], [50, 1])
    t.free(dev([4]), dev([36]))                     # back to a point inside the prompt it shares
    raw[4] = raw[4][:36]
    for _ in range(18):
        step([0, 1, 3, 4, 5, 7])
    t.check_status()
    lens = t.seq_lens.cpu().numpy()
    assert lens.tolist() == [len(x) for x in raw]
    assert int(t.refcount.sum()) == sum(pages_of(int(x)) for x in lens)
