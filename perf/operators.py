"""Timed cases of the paged key-value cache: planning a step's pages and slots,
appending new keys and values, attention of one new token per request, and the
same attention over the pages that a cheap score selects.

Each case is a dict of plain values.  `prepare` makes what a serving program
has in hand before the call, `run` makes one pass (plain torch in 32 bits, or
the library's entry points where `own` is true), `exact` evaluates the
definition in 64 bits, request by request.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.uint8}
BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}
# plan: a request's verdict bits
SHORT, BAD_LENGTH, CAPACITY, BAD_STATE = 1, 2, 4, 8


def listed():
    return [
        # one decoding step of a small batch: every request gets one token
        dict(name="plan_step", op="plan", R=16, lo=100, hi=8192, page=64, new_lo=1, new_hi=1, drop=0),
        # a continuous batch: prefills of every length, tokens taken back, requests that end
        dict(name="plan_mixed", op="plan", R=512, lo=1, hi=32768, page=64, new_lo=1, new_hi=1501, drop=3),
        # the step's new rows of a batch of 64 requests, with the bounds the page selection reads
        dict(name="append_step", op="append", R=64, lo=1, hi=2048, page=64, hkv=8, d=128, dtype="bf16",
             new_lo=1, new_hi=1, bounds=True, heads_first=False),
        # K and V of an 8192-token prefill as the attention layer saves them ([H][S][D])
        dict(name="append_prefill", op="append", R=1, lo=0, hi=0, page=64, hkv=16, d=128, dtype="bf16",
             new_lo=8192, new_hi=8192, bounds=True, heads_first=True),
        # ragged prefill chunks stored in 8 bits
        dict(name="append_e4m3", op="append", R=13, lo=0, hi=900, page=16, hkv=4, d=64, dtype="e4m3",
             new_lo=1, new_hi=1501, bounds=True, heads_first=False),
        # the smallest call: one request, a short prompt
        dict(name="decode_short", op="decode", R=1, lo=257, hi=257, page=16, hq=16, hkv=16, d=128, dtype="bf16"),
        # one request at the training length, one key head for each query head
        dict(name="decode_32768", op="decode", R=1, lo=32768, hi=32768, page=64, hq=32, hkv=32, d=128, dtype="bf16"),
        # a batch of very different lengths, shared key heads
        dict(name="decode_ragged", op="decode", R=48, lo=1, hi=16384, page=64, hq=32, hkv=8, d=128, dtype="bf16"),
        # the longest context, the cache in 8 bits
        dict(name="decode_e4m3_131072", op="decode", R=1, lo=131072, hi=131072, page=128, hq=32, hkv=8, d=128,
             dtype="e4m3"),
        # 32-bit cache, odd lengths, a group of three
        dict(name="decode_fp32", op="decode", R=7, lo=33, hi=4097, page=16, hq=6, hkv=2, d=64, dtype="fp32"),
        # one long request: 64 of 2048 pages are attended
        dict(name="sparse_131072", op="sparse", R=1, lo=131072, hi=131072, page=64, hq=32, hkv=8, d=128,
             dtype="bf16", budget=64, keep_first=1),
        # a ragged batch, some requests shorter than the budget
        dict(name="sparse_ragged", op="sparse", R=32, lo=100, hi=32768, page=32, hq=16, hkv=4, d=128, dtype="bf16",
             budget=100, keep_first=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "sparse"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return dict(op=op, R=_log(rng, 1, 512), lo=rng.choice([0, 1, 77]), hi=_log(rng, 100, 32768), page=page,
                    new_lo=1, new_hi=_log(rng, 1, 1501), drop=rng.choice([0, 2, 3, 5]))
    if op == "append":
        R = _log(rng, 1, 64)
        hkv, d = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
        top = max(1, min(8192, 8192 * 16 * 128 // (R * hkv * d)))
        return dict(op=op, R=R, lo=0, hi=_log(rng, 1, 2048), page=page, hkv=hkv, d=d,
                    dtype=rng.choice(["bf16", "bf16", "e4m3", "fp32"]), new_lo=1, new_hi=_log(rng, 1, top),
                    bounds=rng.random() < 0.7, heads_first=rng.random() < 0.5)
    hkv, d = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16] if hkv < 16 else [1, 2, 4])
    dtype = rng.choice(["bf16", "bf16", "e4m3", "fp32"] if op == "decode" else ["bf16", "bf16", "e4m3"])
    R = _log(rng, 1, 128)
    top = max(64, min(131072, (1 << 27) // (R * hkv * d * (2 if dtype == "fp32" else 1))))
    hi = _log(rng, 16, top)
    c = dict(op=op, R=R, lo=rng.choice([0, 1, hi // 2 + 1, hi]), hi=hi, page=page, hq=hkv * group, hkv=hkv, d=d,
             dtype=dtype)
    if op == "sparse":
        c.update(budget=_log(rng, 2, max(3, hi // page)), keep_first=rng.choice([0, 1]))
    return c


# ---- sizes that follow from a case alone ----

def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly spaced in their logarithm."""
    if n == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (n - 1)))) - 1 for i in range(n)]


def _deltas(c, lens):
    """What each request asks for: new tokens; of every `drop`-th, tokens taken back or its end."""
    new, drop = _spread(c["R"], c["new_lo"], c["new_hi"])[::-1], c["drop"]
    gone = [-lens[i] if i % 2 else -min(lens[i], 1 + i % 7) for i in range(c["R"])]
    return [gone[i] if drop and i % drop == 1 else new[i] for i in range(c["R"])]


def _pages(n, page):
    return -(-n // page)


def _sizes(c):
    """(lens before, new tokens, page-table width, pages in the pool)."""
    lens = _spread(c["R"], c["lo"], c["hi"])
    if c["op"] == "plan":
        new = _deltas(c, lens)
    elif c["op"] == "append":
        new = _spread(c["R"], c["new_lo"], c["new_hi"])
    else:
        new = [0] * c["R"]
    held = [_pages(n + max(d, 0), c["page"]) for n, d in zip(lens, new)]
    return lens, new, max(1, max(held)), sum(held) + 8


def work(case):
    c = case
    lens, new, width, _ = _sizes(c)
    if c["op"] == "plan":
        moved = sum(abs(_pages(n + d, c["page"]) - _pages(n, c["page"])) for n, d in zip(lens, new))
        tokens = sum(d for d in new if d > 0)
        # lens and deltas in, lens and token offsets out, a page number read and written, a slot a token
        return {"bytes": 16 * c["R"] + 8 * moved + 8 * tokens, "flops": tokens + moved}
    b = BYTES[c["dtype"]]
    if c["op"] == "append":
        tokens, row = sum(new), c["hkv"] * c["d"]
        rows_in = 4 if c["dtype"] == "fp32" else 2
        touched = sum(_pages(n + d, c["page"]) - n // c["page"] for n, d in zip(lens, new) if d)
        return {"bytes": 2 * tokens * row * (rows_in + b) + 8 * tokens + (2 * touched * row * b if c["bounds"] else 0),
                "flops": tokens * row * (2 if c["bounds"] else 1)}
    io = c["R"] * c["hq"] * (2 * c["d"] * (4 if c["dtype"] == "fp32" else 2) + 4)
    pages = [_pages(n, c["page"]) for n in lens]
    if c["op"] == "decode":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * c["hkv"] * c["d"] * b + 4 * sum(pages) + io, "flops": 4 * tokens * c["hq"] * c["d"]}
    seen = sum(min(n, c["budget"] * c["page"]) for n in lens)
    return {"bytes": 2 * seen * c["hkv"] * c["d"] * b + 2 * sum(pages) * c["hkv"] * c["d"] * b + 4 * sum(pages)
            + 4 * c["R"] * c["hkv"] * c["budget"] + io,
            "flops": 4 * seen * c["hq"] * c["d"] + 4 * sum(pages) * c["hq"] * c["d"]}


# ---- inputs ----

def _place():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _table(lens, page, width, num_pages, g):
    """A page table whose requests hold scattered pages of the pool, and the pages that are free."""
    order = torch.randperm(num_pages, generator=g)
    held = torch.tensor([_pages(n, page) for n in lens])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[torch.arange(width)[None] < held[:, None]] = order[:int(held.sum())].int()
    return table, order[int(held.sum()):]


def _quantised(x, amax):
    """e4m3 codes of x with the scale 448 / amax, as bytes."""
    return (x.float() * (448.0 / amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    c, dev = case, _place()
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=dev).manual_seed(seed)
    lens, new, width, num_pages = _sizes(c)
    who = torch.randperm(c["R"], generator=g).tolist()  # which request has which length
    lens, new = [lens[i] for i in who], [new[i] for i in who]
    page = c["page"]
    table, free = _table([n + d for n, d in zip(lens, new)] if c["op"] == "append" else lens, page, width, num_pages, g)
    s = dict(op=c["op"], page=page, block_table=table.to(dev), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if c["op"] == "plan":
        head = int(torch.randint(num_pages, (1,), generator=g))
        ring = torch.full((num_pages,), -1, dtype=torch.int32)
        ring[(head + torch.arange(len(free))) % num_pages] = free.int()
        s.update(delta=torch.tensor(new, dtype=torch.int32, device=dev), free_ring=ring.to(dev),
                 free_state=torch.tensor([head, len(free)], dtype=torch.int32, device=dev),
                 capacity=sum(d for d in new if d > 0) + 16)
        return s

    hkv, d, kind = c["hkv"], c["d"], DTYPES[c["dtype"]]
    pool = (num_pages, hkv, page, d)
    amax = torch.tensor([6.5, 6.0], dtype=torch.float32, device=dev) if c["dtype"] == "e4m3" else None

    def rows(*shape):
        return torch.randn(shape, generator=gd, device=dev, dtype=torch.float32 if kind == torch.float32 else torch.bfloat16)

    k, v = rows(*pool), rows(*pool)
    if c["op"] == "sparse":  # neighbouring keys are alike, so that pages differ
        k = k.mul_(0.6).add_(rows(num_pages, hkv, 1, d).mul_(0.8))
    if amax is not None:
        k, v = _quantised(k, 6.5), _quantised(v, 6.0)
    s.update(k_cache=k, v_cache=v, kv_amax=amax)
    if c["op"] == "append":
        r = torch.repeat_interleave(torch.arange(c["R"]), torch.tensor(new))
        pos = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, new)])
        slots = table.long()[r, pos // page] * page + pos % page
        total = sum(new)
        if c["heads_first"]:
            kn, vn = rows(hkv, total, d).transpose(0, 1), rows(hkv, total, d).transpose(0, 1)
        else:
            kn, vn = rows(total, hkv, d), rows(total, hkv, d)
        s.update(k_new=kn, v_new=vn, slots=slots.to(dev),
                 k_bounds=_bounds_of(k, s["block_table"], s["lens"]) if c["bounds"] else None)
        return s
    s.update(q=rows(c["R"], c["hq"], d), scale=d ** -0.5)
    if c["op"] == "sparse":
        s.update(k_bounds=_bounds_of(k, s["block_table"], s["lens"]), budget=c["budget"], keep_first=c["keep_first"])
    return s


def _values(x):
    """Stored rows in 32 bits (8-bit codes as the numbers they encode, unscaled)."""
    return x.view(torch.float8_e4m3fn).float() if x.dtype == torch.uint8 else x.float()


def _stored(x, dtype):
    return x.to(torch.float8_e4m3fn).view(torch.uint8) if dtype == torch.uint8 else x.to(dtype)


def _bounds_of(k, table, lens):
    """Smallest and largest key of each held page: [num_pages][Hkv][2][D], zeros elsewhere."""
    num_pages, hkv, page, d = k.shape
    out = torch.zeros((num_pages, hkv, 2, d), dtype=torch.float32, device=k.device)
    j = torch.arange(table.shape[1], device=k.device)
    left = (lens[:, None] - j[None, :] * page).clamp(0, page)  # filled rows of each page
    held = left > 0
    ids, left = table[held].long(), left[held]
    x = _values(k[ids])
    off = torch.arange(page, device=k.device)[None, None, :, None] >= left[:, None, None, None]
    out[ids] = torch.stack([x.masked_fill(off, math.inf).amin(2), x.masked_fill(off, -math.inf).amax(2)], 2)
    return _stored(out, k.dtype)


# ---- one pass ----

def run(state):
    s = state
    if own:
        from long_sequence_context_b200 import cpattn as cp
        if s["op"] == "plan":
            lens, free_state, cu, slots, verdict = cp.cache_plan(s["lens"], s["delta"], s["block_table"], s["free_ring"],
                                                                 s["free_state"], s["page"], s["capacity"])
            return lens, s["block_table"], s["free_ring"], free_state, cu, slots, verdict
        if s["op"] == "append":
            cp.cache_append_(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"], k_bounds=s["k_bounds"],
                             kv_amax=s["kv_amax"])
            return _seen(s)
        pages = None
        if s["op"] == "sparse":
            pages = cp.select_pages(s["q"], s["k_bounds"], s["block_table"], s["lens"], s["page"], s["budget"],
                                    keep_first=s["keep_first"])
        o, lse = cp.decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], pages=pages,
                           kv_amax=s["kv_amax"], scale=s["scale"])
        return (o, lse) if pages is None else (pages, o, lse)
    if s["op"] == "plan":
        return _plan(s)
    if s["op"] == "append":
        return _append(s)
    if s["op"] == "decode":
        return _decode(s, None)
    pages = _select(s)
    return (pages, *_decode(s, pages))


def _seen(s):
    """The cache after an append, 8-bit rows as numbers (a view)."""
    out = [s["k_cache"], s["v_cache"]] + ([s["k_bounds"]] if s["k_bounds"] is not None else [])
    return [x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x for x in out]


def _plan(s):
    lens, delta, table, ring, page, cap = (s[k] for k in ("lens", "delta", "block_table", "free_ring", "page", "capacity"))
    R, width = table.shape
    num_pages = ring.shape[0]
    head, count = s["free_state"].long().unbind()
    after = lens.long() + delta
    before_p, after_p = (lens.long() + page - 1) // page, (after + page - 1) // page
    new, pops, pushes = delta.long().clamp(min=0), (after_p - before_p).clamp(min=0), (before_p - after_p).clamp(min=0)
    ends, pop_ends, push_ends = new.cumsum(0), pops.cumsum(0), pushes.cumsum(0)
    books = (head < 0) | (head >= num_pages) | (count < 0) | (count > num_pages) | (count + push_ends[-1] > num_pages)
    verdict = (SHORT * (pop_ends[-1] > count) + BAD_LENGTH * ((lens < 0) | (after < 0) | (after > width * page)).any()
               + CAPACITY * (ends[-1] > cap) + BAD_STATE * books)
    ok = verdict == 0
    cells = torch.arange(width, device=lens.device)[None, :]
    # pages taken, first in first out, request by request
    taken = (cells >= before_p[:, None]) & (cells < after_p[:, None]) & ok
    from_ring = (head + (pop_ends - pops)[:, None] + cells - before_p[:, None]) % num_pages
    table.copy_(torch.where(taken, ring[from_ring.clamp(min=0)], table))
    # pages given back behind the last free one
    back = (cells >= after_p[:, None]) & (cells < before_p[:, None]) & ok
    to_ring = (head + count + (push_ends - pushes)[:, None] + cells - after_p[:, None]) % num_pages
    wide = torch.cat([ring, ring[:1]])
    wide[torch.where(back, to_ring, num_pages)] = table
    ring.copy_(wide[:num_pages])
    t = torch.arange(cap, device=lens.device)
    r = torch.searchsorted(ends, t, right=True).clamp(max=R - 1)
    pos = lens[r] + t - (ends - new)[r]
    slots = table[r, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    slots = torch.where((t < ends[-1]) & ok, slots, -1)
    cu = torch.where(ok, torch.cat([ends.new_zeros(1), ends]), 0).int()
    moved = torch.stack([(head + pop_ends[-1]) % num_pages, count - pop_ends[-1] + push_ends[-1]])
    return (torch.where(ok, after, lens).int(), table, ring, torch.where(ok, moved, s["free_state"]).int(), cu, slots,
            verdict.int().reshape(1))


def _append(s):
    k_cache, v_cache, bounds, page = s["k_cache"], s["v_cache"], s["k_bounds"], s["page"]
    at, off = s["slots"] // page, s["slots"] % page
    k, v = s["k_new"].float(), s["v_new"].float()
    if s["kv_amax"] is not None:
        scale = 448.0 / s["kv_amax"]
        k, v = ((x * scale[i]).clamp(-448.0, 448.0) for i, x in enumerate((k, v)))
    k, v = _stored(k, k_cache.dtype), _stored(v, v_cache.dtype)
    k_cache[at, :, off] = k
    v_cache[at, :, off] = v
    if bounds is not None:
        x = _values(k)
        fresh = torch.zeros(k_cache.shape[0], device=x.device).index_reduce_(0, at, (off == 0).float(), "amax")
        fresh = (fresh > 0)[:, None, None]
        old = _values(bounds)
        lo = torch.where(fresh, math.inf, old[:, :, 0]).index_reduce_(0, at, x, "amin")
        hi = torch.where(fresh, -math.inf, old[:, :, 1]).index_reduce_(0, at, x, "amax")
        bounds.copy_(_stored(torch.stack([lo, hi], 2), bounds.dtype))
    return _seen(s)


def _select(s):
    """Pages with the largest upper bound of q.k, ascending; the newest page and the first ones always."""
    q, bounds, table, lens, page, budget = (s[k] for k in ("q", "k_bounds", "block_table", "lens", "page", "budget"))
    R, hq, d = q.shape
    hkv, width = bounds.shape[1], table.shape[1]
    held = (lens.long() + page - 1) // page
    b = _values(bounds)[table.clamp(min=0).long()].permute(0, 2, 3, 4, 1).double()  # R, Hkv, 2, D, pages
    qd = q.double().view(R, hkv, hq // hkv, d)
    # the largest q.k a key inside the bounds could have, in 64 bits: near pages must not swap
    score = (qd.clamp(max=0.0) @ b[:, :, 0] + qd.clamp(min=0.0) @ b[:, :, 1]).amax(2).float() + 0.0
    j = torch.arange(width, device=q.device)
    forced = (j[None] < s["keep_first"]) | (j[None] == held[:, None] - 1)
    score = score.masked_fill(forced[:, None], math.inf).masked_fill(j >= held[:, None, None], -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    best = torch.where(best < held[:, None, None], best, width).sort(dim=-1).values
    best = torch.where(best < width, best, -1).int()
    return torch.nn.functional.pad(best, (0, budget - best.shape[-1]), value=-1)


def _decode(s, pages):
    q, k_cache, v_cache, table, lens, page = (s[k] for k in ("q", "k_cache", "v_cache", "block_table", "lens", "page"))
    R, hq, d = q.shape
    hkv = k_cache.shape[1]
    off = torch.arange(page, device=q.device)
    if pages is None:
        j = torch.arange(table.shape[1], device=q.device)
        ids = table.clamp(min=0).long()
        k, v = (_values(x[ids].transpose(1, 2)) for x in (k_cache, v_cache))  # R, Hkv, pages, page, D
        see = ((j[:, None] * page + off).reshape(1, -1) < lens[:, None])[:, None, None]
    else:
        ids = table.clamp(min=0).long().gather(1, pages.clamp(min=0).long().view(R, -1)).view(pages.shape)
        h = torch.arange(hkv, device=q.device)[None, :, None]
        k, v = (_values(x[ids, h]) for x in (k_cache, v_cache))
        see = (pages[..., None] >= 0) & (pages[..., None] * page + off < lens[:, None, None, None])
        see = see.reshape(R, hkv, 1, -1)
    k, v = k.reshape(R, hkv, -1, d), v.reshape(R, hkv, -1, d)
    if s["kv_amax"] is not None:
        scale = 448.0 / s["kv_amax"]
        k, v = k / scale[0], v / scale[1]
    score = (q.float().view(R, hkv, hq // hkv, d) @ k.transpose(2, 3)) * s["scale"]
    score = score.masked_fill(~see, -math.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    return o.reshape(R, hq, d).to(q.dtype), (m + torch.log(total)).reshape(R, hq)


# ---- the definition in 64 bits, request by request ----

def exact(case, seed):
    s = prepare(case, seed)

    def plan():
        lens, delta, table, ring = (s[k].tolist() for k in ("lens", "delta", "block_table", "free_ring"))
        head, count = s["free_state"].tolist()
        page, cap, size = s["page"], s["capacity"], len(ring)
        free = [ring[(head + i) % size] for i in range(count)]
        slots, cu, after, back, used = [], [0], [], [], 0
        for r, (n, d) in enumerate(zip(lens, delta)):
            after.append(n + d)
            for j in range(_pages(n, page), _pages(n + d, page)):
                table[r][j] = free[used]
                used += 1
            back += table[r][_pages(n + d, page):_pages(n, page)] if d < 0 else []
            slots += [table[r][p // page] * page + p % page for p in range(n, n + d)]
            cu.append(len(slots))
        for i, p in enumerate(back):
            ring[(head + count + i) % size] = p
        out = (after, table, ring, [(head + used) % size, count - used + len(back)], cu, slots + [-1] * (cap - len(slots)), [0])
        return tuple(torch.tensor(x, dtype=torch.int64 if i == 5 else torch.int32) for i, x in enumerate(out))

    def append():
        k_cache, v_cache, bounds, page = s["k_cache"], s["v_cache"], s["k_bounds"], s["page"]
        wide = []
        for cache, new, i in ((k_cache, s["k_new"], 0), (v_cache, s["v_new"], 1)):
            x = cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache
            new = new.double()
            if s["kv_amax"] is not None:
                # the format's own step: the code of x * s with s and the product in 32 bits
                new = (new.float() * (448.0 / s["kv_amax"][i])).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).double()
            x = x.double().transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])
            x[s["slots"]] = new
            wide.append(x.view(cache.shape[0], page, cache.shape[1], cache.shape[3]))
        out = [x.transpose(1, 2) for x in wide]
        if bounds is not None:
            b = (bounds.view(torch.float8_e4m3fn) if bounds.dtype == torch.uint8 else bounds).double()
            slots = s["slots"].tolist()
            fresh = {t // page for t in slots if t % page == 0}
            rows = {}
            for t in slots:
                rows.setdefault(t // page, []).append(t % page)
            for p, offs in rows.items():
                x = wide[0][p, offs[0]:offs[-1] + 1]
                lo, hi = x.amin(0), x.amax(0)
                if p not in fresh:
                    lo, hi = torch.minimum(lo, b[p, :, 0]), torch.maximum(hi, b[p, :, 1])
                b[p, :, 0], b[p, :, 1] = lo, hi
            out.append(b)
        return out

    if s["op"] == "plan":
        return plan()
    if s["op"] == "append":
        return append()
    q, table, lens, page = s["q"].double(), s["block_table"].tolist(), s["lens"].tolist(), s["page"]
    R, hq, d = q.shape
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    hkv = k_cache.shape[1]
    unit = [1.0, 1.0] if s["kv_amax"] is None else [float(a) / 448.0 for a in s["kv_amax"].tolist()]
    o = torch.zeros((R, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((R, hq), -math.inf, dtype=torch.float64, device=q.device)
    picked = torch.full((R, hkv, s["budget"]), -1, dtype=torch.int32, device=q.device) if s["op"] == "sparse" else None
    for r in range(R):
        n = lens[r]
        held = _pages(n, page)
        if not n:
            continue
        ids = torch.tensor(table[r][:held], device=q.device)
        for h in range(hkv):
            mine = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            keep = torch.arange(held, device=q.device)
            if picked is not None:
                b = s["k_bounds"][ids, h]
                b = (b.view(torch.float8_e4m3fn) if b.dtype == torch.uint8 else b).double()
                qq = q[r, mine][:, None, :]
                top = torch.maximum(qq * b[None, :, 0], qq * b[None, :, 1]).sum(-1).amax(0).float()
                top[held - 1] = math.inf
                top[:s["keep_first"]] = math.inf
                order = sorted(range(held), key=lambda j, t=top.tolist(): (-t[j], j))
                keep = torch.tensor(sorted(order[:s["budget"]]), device=q.device)
                picked[r, h, :len(keep)] = keep.int()
            k, v = (x[ids[keep], h] for x in (k_cache, v_cache))
            k, v = ((x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double() * u for x, u in zip((k, v), unit))
            there = (keep[:, None] * page + torch.arange(page, device=q.device)[None]).reshape(-1) < n
            k, v = k.reshape(-1, d)[there], v.reshape(-1, d)[there]
            x = (k @ q[r, mine].T) * s["scale"]  # keys, heads
            lse[r, mine] = torch.logsumexp(x, 0)
            o[r, mine] = torch.softmax(x, 0).T @ v
    return (o, lse) if picked is None else (picked, o, lse)
