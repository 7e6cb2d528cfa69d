"""The decode server's operators around the paged caches: rotary positions, the
8-bit block-scaled cache (append, read back, decode attention) and page
management (fork, extend with copy on write, free, compact).

A case names one operator and its sizes; `run` is one call as a decode server
makes it.  Shapes follow the package's own workloads (head_dim 128, pages of 16
tokens): tiny (2 heads, 512 tokens), page1 (4 requests, 32 heads, 2048 tokens),
qwen_gqa (8 requests, 64 query heads over 8 kv heads, 1000 tokens), long (131072
tokens, 32 heads) and ragged (256 requests of 64 to 4096 tokens, 32 heads).
"""
import math
import random

import torch

own = False

P, D = 16, 128            # tokens of a page, head_dim
INT8_MAX, E4M3_MAX = 127.0, 448.0


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one decode step of a GQA model: the smallest rotary call, latency counts
        {"name": "rope_step_gqa", "op": "rope", "tokens": 8, "q_heads": 64, "kv_heads": 8, "rot": 128,
         "interleaved": False, "far": 1000, "base": 1e6, "factor": 1.0, "transpose": False},
        # a prompt batch at long-context positions: partial, interleaved, frequencies stretched 4x
        {"name": "rope_prompt", "op": "rope", "tokens": 8192, "q_heads": 32, "kv_heads": 32, "rot": 64,
         "interleaved": True, "far": 131072, "base": 1e4, "factor": 4.0, "transpose": False},
        # every request of the ragged batch appends its current token
        {"name": "append_step_ragged", "op": "append", "batch": 256, "heads": 32, "fmt": "int8", "new_min": 1,
         "new_max": 1, "kept_max": 4095, "lens": 5},
        # prompts of uneven length behind uneven prefixes (prefill in chunks)
        {"name": "append_prompt_int8", "op": "append", "batch": 5, "heads": 32, "fmt": "int8", "new_min": 1000,
         "new_max": 2300, "kept_max": 700, "lens": 6},
        {"name": "append_prompt_e4m3", "op": "append", "batch": 4, "heads": 8, "fmt": "e4m3", "new_min": 2048,
         "new_max": 2048, "kept_max": 0, "lens": 7},
        # attention of one decode step: the tiny, qwen_gqa, page1, long and ragged shapes
        {"name": "attend_tiny", "op": "attend", "batch": 1, "q_heads": 2, "kv_heads": 2, "min_len": 512,
         "max_len": 512, "fmt": "int8", "lens": 1},
        {"name": "attend_gqa", "op": "attend", "batch": 8, "q_heads": 64, "kv_heads": 8, "min_len": 1000,
         "max_len": 1000, "fmt": "e4m3", "lens": 2},
        {"name": "attend_page1", "op": "attend", "batch": 4, "q_heads": 32, "kv_heads": 32, "min_len": 2048,
         "max_len": 2048, "fmt": "int8", "lens": 3},
        {"name": "attend_long", "op": "attend", "batch": 1, "q_heads": 32, "kv_heads": 32, "min_len": 131072,
         "max_len": 131072, "fmt": "int8", "lens": 4},
        {"name": "attend_ragged", "op": "attend", "batch": 256, "q_heads": 32, "kv_heads": 32, "min_len": 64,
         "max_len": 4096, "fmt": "int8", "lens": 8},
        # parallel samples: each prompt forked several times, then every row grows by a token
        # (shared partial pages are copied), over fp16 pages of page1's size
        {"name": "fork_samples", "op": "fork", "rows": 4, "forks": 7, "min_len": 1500, "max_len": 2047, "grow": 1,
         "page_halfs": 131072, "spare": 64, "lens": 9},
        # a third of a ragged batch ends; its pages are freed and the pool is compacted
        {"name": "compact_ragged", "op": "compact", "rows": 256, "freed": 85, "min_len": 64, "max_len": 4096,
         "page_halfs": 2048, "spare": 1000, "lens": 10},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "fork", "compact"])
    if op == "rope":
        kv = _log(rng, 1, 32)
        return {"op": op, "tokens": _log(rng, 1, 8192), "q_heads": kv * rng.choice([1, 1, 2, 3, 8]) if kv <= 8 else kv,
                "kv_heads": kv, "rot": 8 * rng.randint(1, 16), "interleaved": rng.random() < 0.5,
                "far": _log(rng, 1, 2000000), "base": rng.choice([1e4, 5e5, 1e6]), "factor": rng.choice([1.0, 2.0, 8.0]),
                "transpose": rng.random() < 0.3}
    if op == "append":
        batch, top = (_log(rng, 1, 256), 1) if rng.random() < 0.5 else (_log(rng, 1, 8), _log(rng, 2, 1000))
        return {"op": op, "batch": batch, "heads": _log(rng, 1, 32), "fmt": rng.choice(["int8", "e4m3"]),
                "new_min": rng.randint(0 if top > 1 else 1, top), "new_max": top, "kept_max": _log(rng, 1, 2000),
                "lens": rng.randrange(1 << 30)}
    if op == "attend":
        kv = _log(rng, 1, 32)
        batch = _log(rng, 1, 64)
        top = min(_log(rng, 1, 131072), 2000000 // (kv * batch) + 1)
        return {"op": op, "batch": batch, "q_heads": kv * rng.choice([1, 1, 2, 3, 4, 7, 8, 12]), "kv_heads": kv,
                "min_len": rng.randint(0, top), "max_len": top, "fmt": rng.choice(["int8", "e4m3"]),
                "lens": rng.randrange(1 << 30)}
    if op == "fork":
        rows = _log(rng, 1, 16)
        top = _log(rng, 1, 4000)
        return {"op": op, "rows": rows, "forks": rng.randint(1, 8), "min_len": rng.randint(1, top), "max_len": top,
                "grow": _log(rng, 1, 60), "page_halfs": 8 * _log(rng, 16, 4000), "spare": rng.randint(0, 100),
                "lens": rng.randrange(1 << 30)}
    rows = _log(rng, 2, 200)
    top = _log(rng, 16, 4000)
    return {"op": op, "rows": rows, "freed": rng.randint(1, rows - 1), "min_len": rng.randint(0, top), "max_len": top,
            "page_halfs": 8 * _log(rng, 16, 500), "spare": rng.randint(0, 500), "lens": rng.randrange(1 << 30)}


# ------------------------------------------------- sizes that a case implies ----
def _attend_lens(case):
    r, lo, hi = random.Random(case["lens"]), case["min_len"], case["max_len"]
    if case["batch"] > 128 and hi >= 4096:        # the ragged batch: 30 % at the top, the others short
        return [hi if r.random() < 0.3 else r.randint(lo, 512) for _ in range(case["batch"])]
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _append_lens(case):
    """[(tokens kept, tokens appended)] of the requests"""
    r = random.Random(case["lens"])
    got = [[r.randint(0, case["kept_max"]), r.randint(case["new_min"], case["new_max"])] for _ in range(case["batch"])]
    if not any(n for _, n in got):
        got[0][1] = 1
    return got


def _page_lens(case):
    r = random.Random(case["lens"])
    got = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["rows"])]
    if not any(got):
        got[0] = 1
    return got


def _pages(n):
    return -(-n // P)


# ---------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _tables(lens, rows, width, pages, g):
    """A table of pages in random order over a pool; entries not in use are 0."""
    perm = torch.randperm(pages, device="cuda", generator=g).int()
    n = torch.tensor([_pages(x) for x in lens] + [0] * (rows - len(lens)))
    used = torch.arange(width)[None, :] < n[:, None]
    bt = torch.zeros((rows, width), dtype=torch.int32, device="cuda")
    bt[used.cuda()] = perm[:int(n.sum())]
    return bt


def _codes(shape, fmt, g):
    """8-bit codes of vectors with uneven channels, as a cache holds them."""
    x = torch.randn(shape, device="cuda", generator=g, dtype=torch.float16)
    x *= 0.5 + 1.5 * torch.rand((shape[1], 2, 1, D), device="cuda", generator=g).half()
    if fmt == "int8":
        return (x * 24).round_().clamp_(-127, 127).to(torch.int8)
    return (x * 80).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "rope":
        T, r = case["tokens"], case["rot"]
        # frequencies base^(-2i/rot), positions squeezed by the context's stretch
        w = case["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r) / case["factor"]
        pos = torch.randint(0, case["far"] + 1, (T,), device="cuda", generator=g).int()
        if T > 4:
            pos[-1] = -1                                 # a padding row at the end of the batch
        return {"op": op, "case": case, "pos": pos, "w": w, "m": 1.0 + 0.1 * math.log(case["factor"]),
                "q": torch.randn((T, case["q_heads"], D), device="cuda", generator=g),
                "kv": torch.randn((T, case["kv_heads"], 2, D), device="cuda", generator=g).half()}
    if op == "append":
        kept, new = zip(*_append_lens(case))
        H = case["heads"]
        lens = [a + b for a, b in zip(kept, new)]
        pages = sum(_pages(x) for x in lens) + 3
        cu = [0]
        back = [0]                                       # read back: the whole blocks that the call changes
        for a, b in zip(kept, new):
            cu.append(cu[-1] + b)
            back.append(back[-1] + (a % P + b if b else 0))
        kv = torch.randn((cu[-1], H, 2, D), device="cuda", generator=g)
        kv *= 0.5 + 1.5 * torch.rand((H, 2, D), device="cuda", generator=g)
        pool = _codes((pages, H, 2, P, D), case["fmt"], g)
        scales = 0.005 + 0.03 * torch.rand((pages, H, 2), device="cuda", generator=g)
        if case["fmt"] == "e4m3":
            scales = torch.exp2(torch.randint(-9, -6, (pages, H, 2), device="cuda", generator=g).float())
        return {"op": op, "case": case, "kv": kv.half(), "pool": pool, "scales": scales, "cu": _ints(cu),
                "back": _ints(back), "back_tokens": back[-1], "lens": _ints(lens), "one": case["new_max"] == 1,
                "bt": _tables(lens, len(lens), max(1, max(_pages(x) for x in lens)), pages, g)}
    if op == "attend":
        lens = _attend_lens(case)
        H = case["kv_heads"]
        pages = sum(_pages(x) for x in lens) + 3
        scales = 0.01 + 0.03 * torch.rand((pages, H, 2), device="cuda", generator=g)
        if case["fmt"] == "e4m3":
            scales = torch.exp2(torch.randint(-8, -5, (pages, H, 2), device="cuda", generator=g).float())
        return {"op": op, "case": case, "q": torch.randn((len(lens), case["q_heads"], D), device="cuda", generator=g),
                "pool": _codes((pages, H, 2, P, D), case["fmt"], g), "scales": scales, "lens": _ints(lens),
                "max_len": max(lens), "bt": _tables(lens, len(lens), max(1, _pages(max(lens))), pages, g)}
    lens = _page_lens(case)
    if op == "fork":
        rows = case["rows"] * (1 + case["forks"])
        grown = [x + case["grow"] for x in lens] * (1 + case["forks"])
        pages = sum(_pages(x) for x in lens) + rows * (_pages(case["grow"]) + 1) + case["spare"]
        width = _pages(max(grown))
    else:
        rows, grown, pages, width = case["rows"], None, sum(_pages(x) for x in lens) + case["spare"], max(1, _pages(max(lens)))
    bt = _tables(lens, rows, width, pages, g)
    rc = torch.zeros(pages, dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda")[None, :] < _ints([_pages(x) for x in lens] + [0] * (rows - len(lens)))[:, None]
    rc[bt[used].long()] = 1
    s = {"op": op, "case": case, "bt": bt, "rc": rc, "lens": _ints(lens + [0] * (rows - len(lens))),
         "pool": torch.randn((pages, case["page_halfs"]), device="cuda", generator=g).half()}
    if op == "fork":
        s["src"] = _ints([i % case["rows"] for i in range(case["rows"] * case["forks"])])
        s["dst"] = _ints(list(range(case["rows"], rows)))
        s["all"], s["grown"] = _ints(list(range(rows))), _ints(grown)
    else:
        s["gone"] = torch.randperm(rows, device="cuda", generator=g)[:case["freed"]].int()
    return s


# ------------------------------------------------------------- one pass ----
def run(s):
    if s["op"] == "rope":
        return _rope_own(s) if own else _rope(s)
    if s["op"] == "append":
        return _append_own(s) if own else _append(s)
    if s["op"] == "attend":
        return _attend_own(s) if own else _attend(s)
    # the page operators change tables in place: each pass starts from the scheduler's snapshot
    bt, lens, rc = s["bt"].clone(), s["lens"].clone(), s["rc"].clone()
    if s["op"] == "fork":
        return _fork_own(s, bt, lens, rc) if own else _fork(s, bt, lens, rc)
    return _compact_own(s, bt, lens, rc) if own else _compact(s, bt, lens, rc)


def _rope_own(s):
    from decode_attention_product_gb300 import api
    c = s["case"]
    return list(api.rope(s["pos"], s["w"], q=s["q"], kv=s["kv"], interleaved=c["interleaved"], mscale=s["m"],
                         transpose=c["transpose"]))


def _append_own(s):
    from decode_attention_product_gb300 import api
    api.q8_append(s["kv"], s["pool"], s["scales"], s["bt"], s["lens"], cu_tokens=None if s["one"] else s["cu"])
    back = api.q8_load(s["pool"], s["scales"], s["bt"], s["lens"], s["back"], s["back_tokens"])
    return [back, s["scales"]]


def _attend_own(s):
    from decode_attention_product_gb300 import api
    return api.q8_decode_attention(s["q"], s["pool"], s["scales"], s["bt"], s["lens"], s["max_len"])


def _fork_own(s, bt, lens, rc):
    from decode_attention_product_gb300 import api
    api.pages_fork(s["src"], s["dst"], bt, lens, rc)
    api.pages_extend(s["all"], s["grown"], bt, lens, rc, [s["pool"]])
    return [s["pool"], bt, lens, rc]


def _compact_own(s, bt, lens, rc):
    from decode_attention_product_gb300 import api
    api.pages_free(s["gone"], bt, lens, rc)
    api.pages_compact(bt, lens, rc, [s["pool"]])
    return [s["pool"], bt, lens, rc]


# ---- plain forms: elementary torch operations in 32 bits (64 for far angles
# ---- and for the decision of a code)
def _turned(x, cos, sin, r, interleaved):
    """x [T][heads][D] fp32 with its first r dims rotated"""
    a, rest = x[..., :r], x[..., r:]
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if interleaved else (a[..., :r // 2], a[..., r // 2:])
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return torch.cat((y, rest), -1)


def _rope(s):
    c, pos = s["case"], s["pos"]
    a = pos.clamp(min=0).double()[:, None, None] * s["w"]
    sign = -1.0 if c["transpose"] else 1.0
    cos, sin = (s["m"] * a.cos()).float(), (sign * s["m"] * a.sin()).float()
    pad = (pos < 0)[:, None, None]
    q = torch.where(pad, s["q"], _turned(s["q"], cos, sin, c["rot"], c["interleaved"]))
    k = _turned(s["kv"][:, :, 0].float(), cos, sin, c["rot"], c["interleaved"]).half()
    k = torch.where(pad, s["kv"][:, :, 0], k)
    return [q, torch.stack((k, s["kv"][:, :, 1]), 2)]


def _values(codes, fmt):
    return codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()


def _places(cu, tokens, lens, bt):
    """page and slot of the last cu[b+1]-cu[b] tokens of each request, in order"""
    i = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), i.int(), right=True)
    pos = lens[b].long() - (cu[b + 1].long() - i)
    return bt[b, pos // P].long(), pos % P


def _append(s):
    fmt, pool, scales = s["case"]["fmt"], s["pool"], s["scales"]
    x = s["kv"].float()
    page, slot = _places(s["cu"], x.shape[0], s["lens"], s["bt"])
    amax = torch.zeros_like(scales)
    amax.index_reduce_(0, page, x.abs().amax(-1), "amax")
    first = torch.full((pool.shape[0],), P, dtype=torch.long, device="cuda")
    first.index_reduce_(0, page, slot, "amin")
    hit = torch.unique(page)
    old = torch.where((first[hit] > 0)[:, None, None], scales[hit], torch.zeros_like(scales[hit]))
    if fmt == "int8":
        want = amax[hit] / INT8_MAX
    else:                                                # the least power of two that keeps amax within 448
        f, e = torch.frexp(amax[hit])
        want = torch.ldexp(torch.ones_like(f), e - torch.where(f <= 0.875, 9, 8))
        want = torch.where(amax[hit] > 0, want, torch.zeros_like(want))
    new = torch.maximum(old, want)
    # codes already in the block, rounded again where its scale grew
    kept = _values(pool[hit], fmt).double() * (old.double() / torch.where(new > 0, new, torch.ones_like(new)).double())[..., None, None]
    mine = torch.arange(P, device="cuda")[None, :] < first[hit][:, None]
    grew = (new > old) & (old > 0)
    pool[hit] = torch.where(mine[:, None, None, :, None] & grew[..., None, None], _coded(kept, fmt), pool[hit])
    scales[hit] = new
    at = scales[page]
    quot = torch.where(at > 0, x.double().movedim(-1, 0) / at.double(), torch.zeros_like(at, dtype=torch.float64)).movedim(0, -1)
    pool[page, :, :, slot] = _coded(quot, fmt)
    page, slot = _places(s["back"], s["back_tokens"], s["lens"], s["bt"])
    return [(_values(pool[page, :, :, slot], fmt) * scales[page][..., None]).half(), scales]


def _coded(x, fmt):
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _attend(s):
    fmt = s["case"]["fmt"]
    q, bt, lens = s["q"], s["bt"].long(), s["lens"]
    B, Hq, H = q.shape[0], q.shape[1], s["pool"].shape[1]
    L = bt.shape[1] * P
    k = (_values(s["pool"][bt, :, 0], fmt) * s["scales"][bt, :, 0][..., None, None]).transpose(1, 2).reshape(B, H, L, D)
    w = torch.matmul(q.view(B, H, Hq // H, D), k.transpose(2, 3)) * D ** -0.5
    seen = (torch.arange(L, device="cuda")[None, :] < lens[:, None])[:, None, None, :]
    w = torch.where(seen, w, torch.full_like(w, -math.inf))
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = w.sum(-1, keepdim=True)
    v = (_values(s["pool"][bt, :, 1], fmt) * s["scales"][bt, :, 1][..., None, None]).transpose(1, 2).reshape(B, H, L, D)
    o = torch.matmul(w, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, Hq, D)


def _fork(s, bt, lens, rc):
    src, dst, pool = s["src"].long(), s["dst"].long(), s["pool"]
    col = torch.arange(bt.shape[1], device="cuda")[None, :]
    used = col < ((lens[src] + P - 1) // P)[:, None]
    bt[dst] = torch.where(used, bt[src], bt[dst])
    lens[dst] = lens[src]
    rc.index_add_(0, bt[src][used].long(), torch.ones_like(bt[src][used]))
    # growth: new pages from the lowest free ids; a shared partial page is copied first
    row, grown = s["all"].long(), s["grown"]
    have, want = ((lens[row] + P - 1) // P)[:, None], ((grown + P - 1) // P)[:, None]
    last = bt[row].gather(1, (have - 1).clamp(min=0).long()).long()
    copy = (lens[row] % P > 0)[:, None] & (rc[last] > 1)
    need = want - have + copy
    fresh = (col >= have) & (col < want) | copy & (col == have - 1)
    rank = need.cumsum(0) - need + col - have + copy
    free = torch.nonzero(rc == 0)[:, 0].int()
    bt[row] = torch.where(fresh, free[rank.clamp(0, free.shape[0] - 1).long()], bt[row])
    rc[bt[row][fresh].long()] = 1
    rc.index_add_(0, last[copy], torch.full_like(rc[last[copy]], -1))
    pool[bt[row].gather(1, (have - 1).clamp(min=0).long()).long()[copy]] = pool[last[copy]]
    lens[row] = grown
    return [pool, bt, lens, rc]


def _compact(s, bt, lens, rc):
    gone, pool = s["gone"].long(), s["pool"]
    col = torch.arange(bt.shape[1], device="cuda")[None, :]
    used = col < ((lens[gone] + P - 1) // P)[:, None]
    rc.index_add_(0, bt[gone][used].long(), torch.full_like(bt[gone][used], -1))
    bt[gone] = torch.where(used, torch.full_like(bt[gone], -1), bt[gone])
    lens[gone] = 0
    live = rc > 0
    ids = torch.arange(rc.shape[0], device="cuda")
    top = live.sum()
    movers, holes = torch.nonzero(live & (ids >= top))[:, 0], torch.nonzero(~live & (ids < top))[:, 0]
    pool[holes] = pool[movers]
    to = ids.int()
    to[movers] = holes.int()
    rc[holes] = rc[movers]
    rc[movers] = 0
    used = col < ((lens + P - 1) // P)[:, None]
    bt.copy_(torch.where(used, to[bt.clamp(min=0).long()], bt))
    return [pool, bt, lens, rc]


# ------------------------------------------------------------------ work ----
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * D * (case["q_heads"] * 4 + case["kv_heads"] * 2 * 2)
        return {"bytes": 2 * n + 4 * case["tokens"] + 4 * case["rot"],
                "flops": 3 * case["tokens"] * case["rot"] * (case["q_heads"] + case["kv_heads"])}
    if op == "append":
        lens = _append_lens(case)
        new = sum(n for _, n in lens)
        back = sum(a % P + n for a, n in lens if n)
        blocks = sum(_pages(a % P + n) for a, n in lens if n)
        per = case["heads"] * 2
        # fp16 in, codes out; codes in again and fp16 out; scales of the blocks
        return {"bytes": per * (new * D * 3 + back * D * 3 + blocks * 4 * 3) + 4 * len(lens) * 3,
                "flops": per * D * (3 * new + back)}
    if op == "attend":
        lens = _attend_lens(case)
        pages = sum(_pages(x) for x in lens)
        return {"bytes": case["kv_heads"] * (sum(lens) * 2 * D + pages * 8) + 2 * case["batch"] * case["q_heads"] * D * 4
                + 4 * (pages + case["batch"]), "flops": 4 * D * case["q_heads"] * sum(lens)}
    lens = _page_lens(case)
    per = case["page_halfs"] * 2
    total = sum(_pages(x) for x in lens)
    if op == "fork":
        f, n = case["forks"], case["rows"]
        pages = total + n * (1 + f) * (_pages(case["grow"]) + 1) + case["spare"]
        copies = sum(1 + f for x in lens if x % P)       # every row that shares its partial page copies it
        return {"bytes": copies * 2 * per + 4 * (3 * total * (1 + f) + 3 * pages), "flops": 0}
    # which rows go is the seed's: freed pages on average, and the share of them that lies below the live pages
    pages = total + case["spare"]
    live = total * (1 - case["freed"] / case["rows"])
    return {"bytes": 2 * per * live * (1 - live / pages) + 4 * (3 * total + 3 * pages), "flops": 0}


# --------------------------------------- the definitions in 64 bits, apart ----
def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None                                      # pages moved and counted: nothing is computed
    s = prepare(case, seed)
    if op == "rope":
        return _rope_64(s)
    if op == "append":
        return _append_64(s)
    return _attend_64(s)


def _rope_64(s):
    c, r = s["case"], s["case"]["rot"]
    z = torch.polar(torch.full_like(s["w"], s["m"])[None] * (s["pos"] >= 0).double()[:, None]
                    + (s["pos"] < 0).double()[:, None], s["pos"].clamp(min=0).double()[:, None] * s["w"][None])
    if c["transpose"]:
        z = z.conj()

    def turn(x):
        x = x.double()
        idx = torch.arange(r, device="cuda").view(-1, 2) if c["interleaved"] else torch.arange(r, device="cuda").view(2, -1).t()
        y = torch.complex(x[..., idx[:, 0]], x[..., idx[:, 1]]) * z[:, None]
        out = x.clone()
        out[..., idx[:, 0]], out[..., idx[:, 1]] = y.real, y.imag
        return out
    kv = s["kv"].double()
    kv[:, :, 0] = turn(s["kv"][:, :, 0])
    return [turn(s["q"]), kv]


def _append_64(s):
    fmt = s["case"]["fmt"]
    grid = None
    if fmt == "e4m3":
        grid = torch.arange(127, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn).double()
        two = torch.tensor([2.0 ** k for k in range(-40, 20)], dtype=torch.float64, device="cuda")

    def nearest(x):
        """codes' values nearest to x (ties to the even code)"""
        if fmt == "int8":
            return x.round()
        a = x.abs()
        hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)
        lo = hi - 1
        dl, dh = a - grid[lo], grid[hi] - a
        pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        return grid[pick] * x.sign()
    lens, cu, back = s["lens"].tolist(), s["cu"].tolist(), s["back"].tolist()
    scales, bt = s["scales"].clone(), s["bt"].tolist()
    out = torch.zeros((s["back_tokens"],) + tuple(s["kv"].shape[1:]), dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        t, o = L - n, back[b]
        while t < L:
            e = min(L, t // P * P + P)
            pg, s0 = bt[b][t // P], t % P
            x = s["kv"][cu[b] + t - (L - n):cu[b] + e - (L - n)].double()          # [n][H][2][D]
            a = x.abs().amax((0, 3))
            if fmt == "int8":
                want = (a / 127).float()
            else:
                want = two[torch.searchsorted(448 * two, a)] * (a > 0)
                want = want.float()
            old = scales[pg].clone() if s0 else torch.zeros_like(want)
            new = torch.maximum(old, want)
            d = torch.where(new > 0, new, torch.ones_like(new)).double()
            if s0:                                        # what the block held, rounded again where its scale grew
                c = s["pool"][pg, :, :, :s0]
                c = c.double() if fmt == "int8" else c.contiguous().view(torch.float8_e4m3fn).double()
                c = torch.where((new > old)[..., None, None], nearest(c * (old.double() / d)[..., None, None]), c)
                out[o:o + s0] = (c * new.double()[..., None, None]).permute(2, 0, 1, 3)
            out[o + s0:o + s0 + e - t] = nearest(x / d[None, ..., None]) * new.double()[None, ..., None]
            scales[pg] = new
            o += s0 + e - t
            t = e
    return [out, scales.double()]


def _attend_64(s):
    fmt, q = s["case"]["fmt"], s["q"].double()
    out = torch.zeros_like(q)
    H = s["pool"].shape[1]
    G = q.shape[1] // H
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        pg = s["bt"][b, :_pages(L)].long()
        for h in range(0, H, 4):                          # a few heads at a time: the values fill memory in 64 bits
            c, e = s["pool"][pg, h:h + 4], s["scales"][pg, h:h + 4].double()
            c = c.double() if fmt == "int8" else c.view(torch.float8_e4m3fn).double()
            c = (c * e[..., None, None]).permute(2, 1, 0, 3, 4).flatten(2, 3)[:, :, :L]           # [2][h][L][D]
            x = q[b, h * G:(h + 4) * G].view(-1, G, D)
            p = torch.softmax(x @ c[0].mT / math.sqrt(D), -1)
            out[b, h * G:(h + 4) * G] = (p @ c[1]).flatten(0, 1)
    return out
