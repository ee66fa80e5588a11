"""Plain fp64 restatement of the paged key-value cache: the books of a step,
the rows of an append, the page selection and single-token attention, request
by request and token by token (numpy, no code shared with the CUDA path).

A cache is an array [num_pages, Hkv, page_size, D] of the values its elements
stand for."""
import numpy as np

SHORT, BAD_LENGTH, CAPACITY, BAD_STATE = 1, 2, 4, 8


def pages_of(n, page_size):
    return -(-int(n) // page_size)


def plan(lens, delta, table, ring, state, page_size, capacity):
    """(lens, table, ring, state, cu_new, slots, verdict) after one step."""
    lens, delta, ring = [int(x) for x in lens], [int(x) for x in delta], [int(x) for x in ring]
    table = np.array(table, dtype=np.int64)
    head, count = (int(x) for x in state)
    R, width = table.shape
    verdict, need, back, tokens = 0, 0, 0, 0
    for n, d in zip(lens, delta):
        if not 0 <= n <= width * page_size or not 0 <= n + d <= width * page_size:
            verdict |= BAD_LENGTH
            continue
        more = pages_of(n + d, page_size) - pages_of(n, page_size)
        need, back, tokens = need + max(more, 0), back + max(-more, 0), tokens + max(d, 0)
    if need > count:
        verdict |= SHORT
    if tokens > capacity:
        verdict |= CAPACITY
    if not 0 <= head < len(ring) or not 0 <= count <= len(ring) or count + back > len(ring):
        verdict |= BAD_STATE
    if verdict:
        return lens, table, ring, [head, count], [0] * (R + 1), [-1] * capacity, verdict
    free = [ring[(head + i) % len(ring)] for i in range(count)]
    taken, returned, slots, cu = 0, [], [], [0]
    for r in range(R):
        before, after = pages_of(lens[r], page_size), pages_of(lens[r] + delta[r], page_size)
        for j in range(before, after):
            table[r, j] = free[taken]
            taken += 1
        for j in range(after, before):
            returned.append(int(table[r, j]))
        for pos in range(lens[r], lens[r] + delta[r]):
            slots.append(int(table[r, pos // page_size]) * page_size + pos % page_size)
        cu.append(len(slots))
    for i, p in enumerate(returned):
        ring[(head + count + i) % len(ring)] = p
    state = [(head + taken) % len(ring), count - taken + len(returned)]
    return ([n + d for n, d in zip(lens, delta)], table, ring, state, cu, slots + [-1] * (capacity - len(slots)), 0)


def append(cache, rows, slots):
    """A copy of `cache` with rows[i] ([Hkv, D]) in slots[i]; negative slots are skipped."""
    out = np.array(cache)
    P = cache.shape[2]
    for x, s in zip(rows, slots):
        if s >= 0:
            out[int(s) // P, :, int(s) % P] = x
    return out


def bounds(cache, table, lens):
    """{(page, kv head): (smallest, largest key)} of every held page, exact."""
    P = cache.shape[2]
    out = {}
    for r, n in enumerate(lens):
        for j in range(pages_of(n, P)):
            p = int(table[r][j])
            rows = cache[p, :, :min(P, int(n) - j * P)]
            for h in range(cache.shape[1]):
                out[p, h] = rows[h].min(0), rows[h].max(0)
    return out


def scores(q, lo, hi):
    """Upper bound of q.k over keys inside [lo, hi], the largest of the group's heads: q [group, D].
    A zero of q counts as zero beside an infinite bound; heads whose sum is NaN do not count (NaN: none does)."""
    with np.errstate(invalid="ignore"):
        seen = ~(np.isnan(lo) | np.isnan(hi))
        sums = [float(np.sum(np.where((x == 0) & seen, 0.0, np.maximum(x * lo, x * hi)))) for x in q]
    return max([s for s in sums if s == s], default=float("nan"))


def select(q, bounds_of, table, n, page_size, h, budget, keep_first):
    """Pages of one (request, kv head): q [group, D], bounds_of {(page, head): (lo, hi)}."""
    held = pages_of(n, page_size)
    s = [float(np.float32(scores(q, *bounds_of[int(table[j]), h]))) for j in range(held)]
    # the pages that are always listed, then by the score, NaN last
    rank = lambda j: (not (j < keep_first or j == held - 1), s[j] != s[j], 0.0 if s[j] != s[j] else -s[j], j)
    best = sorted(range(held), key=rank)[:budget]
    return sorted(best) + [-1] * (budget - len(best))


def gather(cache, table, n, h, pages=None):
    """Keys (or values) [m, D] of one (request, kv head) in the order of its pages."""
    P = cache.shape[2]
    listed = range(pages_of(n, P)) if pages is None else [int(j) for j in pages if j >= 0]
    rows = [cache[int(table[j]), h, :max(0, min(P, int(n) - j * P))] for j in listed]
    return np.concatenate(rows) if rows else np.zeros((0, cache.shape[3]))


def attend(q, k, v, scale):
    """One token over m keys: (o [D], lse, sum_j p_j |v_j| [D], sum_d |q_d| |k_jd| at most)."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    x = scale * (k @ q)
    m = x.max()
    e = np.exp(x - m)
    return e @ v / e.sum(), m + np.log(e.sum()), e @ np.abs(v) / e.sum(), float((np.abs(k) @ np.abs(q)).max())


def decode(q, k_cache, v_cache, table, lens, scale, pages=None):
    """(o, lse, mass, reach) of a batch: q [R, Hq, D]; mass and reach as `attend` gives them."""
    R, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    o, mass = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    lse, reach = np.full((R, Hq), -np.inf), np.zeros((R, Hq))
    for r in range(R):
        for h in range(Hkv):
            mine = None if pages is None else pages[r][h][:pages_of(lens[r], k_cache.shape[2])]
            k = gather(k_cache, table[r], lens[r], h, mine)
            v = gather(v_cache, table[r], lens[r], h, mine)
            for i in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                o[r, i], lse[r, i], mass[r, i], reach[r, i] = attend(q[r, i], k, v, scale)
    return o, lse, mass, reach
