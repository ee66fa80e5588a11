"""The paged key-value cache on the GPU at the edges of what its calls allow."""
import numpy as np
import pytest
import torch

from oracle import fp8, paged
from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from long_sequence_context_b200 import cpattn
    cpattn.set_path(0)
    return cpattn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("R", [3, 1024, 1025])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_refuses_a_length_above_its_table(cp, R, in_place):
    """A request that gives tokens back from a length its row has no pages for: nothing
    changes, and no cell of a row is taken for another row's."""
    P, width = 16, 4
    around = torch.arange((R + 2) * width, dtype=torch.int32, device="cuda").view(R + 2, width)
    table = around[1:R + 1]
    ring = torch.full((4 * R * width,), -1, dtype=torch.int32, device="cuda")
    ring[:8] = torch.arange(8, dtype=torch.int32, device="cuda") + (R + 2) * width
    state = _i32([0, 8])
    for who, n in [(0, width * P + 1), (R - 1, width * P + 40), (R // 2, 2 ** 31 - 1)]:
        for d in (-n, -(n - width * P), -(n - 5)):
            lens, delta = _i32([20] * R), _i32([0] * R)
            lens[who], delta[who] = n, d
            keep = [x.clone() for x in (around, ring, state, lens)]
            kw = dict(lens_out=lens, free_state_out=state) if in_place else {}
            out = cp.cache_plan(lens, delta, table, ring, state, P, 64, **kw)
            want = paged.plan(keep[3].tolist(), delta.tolist(), table.cpu().numpy(), ring.tolist(), [0, 8], P, 64)
            assert cp.sync_status() == cp.OK
            assert out[4].item() == want[6] == cp.PLAN_BAD_LENGTH
            assert all(torch.equal(x, y) for x, y in zip((around, ring, state, lens), keep))
            assert torch.equal(out[0], keep[3]) and torch.equal(out[1], keep[2])
            assert out[2].count_nonzero() == 0 and torch.all(out[3] == -1)


@pytest.mark.parametrize("many", [1, 300])
def test_plan_reports_pages_outside_of_the_pool_that_come_back(cp, many):
    """The books count them all the same, and the next request that takes one gets no slots in it."""
    P, width, num_pages = 16, 2 * many, 4 * many + 2
    table = torch.arange(2 * width, dtype=torch.int32).view(2, width)
    table[1, 3 % width], table[1, width - 1] = -1, num_pages
    ring, state = torch.full((num_pages,), -1, dtype=torch.int32), [0, 0]
    t, r = table.cuda(), ring.cuda()
    lens, delta = [P * width, P * width], [0, -P * width]
    out = cp.cache_plan(_i32(lens), _i32(delta), t, r, _i32(state), P, 0)
    want = paged.plan(lens, delta, table.numpy(), ring.tolist(), state, P, 0)
    assert cp.sync_status() == cp.ERR_PAGE and cp.sync_status() == cp.OK
    assert out[4].item() == want[6] == 0
    assert r.tolist() == want[2] and out[1].tolist() == want[3] and torch.equal(t.cpu(), table)
    n = P * width
    out = cp.cache_plan(out[0], _i32([0, n]), t, r, out[1], P, n)
    assert cp.sync_status() == cp.ERR_PAGE and out[4].item() == 0
    pages = table[1].long()
    slots = (pages[:, None] * P + torch.arange(P)).masked_fill(((pages < 0) | (pages >= num_pages))[:, None], -1)
    assert torch.equal(out[3].cpu(), slots.view(-1))


@pytest.mark.parametrize("width", [10, 2048])
@pytest.mark.parametrize("amax", [5.0, 0.05])
@pytest.mark.parametrize("exponent", [-133, -128, -126, -120, -110])
def test_decode_tiny_queries_at_the_ordinary_scale(cp, exponent, amax, width):
    """Scores next to 0 are a mean of V, also where the masked rows of a step stand beside them."""
    c = pu.make_cache([300, 40, 7, 64, 0], 6, 2, 128, 32, "e4m3", seed=15, width=width)
    c["q"] = (c["q"].double() * 2.0 ** exponent).to(c["q"].dtype)
    c["amax"] = torch.tensor([amax, 0.9 * amax])
    d = pu.on_gpu(c)
    o, lse = cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], kv_amax=d["amax"])
    assert cp.sync_status() == cp.OK
    pu.assert_decode(o, lse, pu.reference(c, 128 ** -0.5), 128, 128 ** -0.5, 300, "e4m3")


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("width", [10, 2048])
def test_decode_smallest_scale(cp, kind, width):
    c = pu.make_cache([300, 40, 7], 6, 2, 128, 32, kind, seed=17, width=width)
    scale = 2.0 ** -149
    d = pu.on_gpu(c)
    o, lse = cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], kv_amax=d["amax"], scale=scale)
    assert cp.sync_status() == cp.OK
    pu.assert_decode(o, lse, pu.reference(c, scale), 128, scale, 300, kind)


@pytest.mark.parametrize("width", [5, 4096])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("D,group", [(64, 1), (128, 1), (64, 9), (128, 40)])
def test_decode_values_as_large_as_their_sum_allows(cp, kind, D, group, width):
    """64 keys of weight 1 and 256 of less, |v| up to 2^122: a weighted sum stays below 2^128
    (2^122 (64 + 24)), and does so only while no weight is above 1.  Scores rise from page to
    page, by less than what makes the reference of the weights follow."""
    n, P, heads = 320, 64, 300
    c = pu.make_cache([n], group * heads, heads, D, P, kind, seed=16, width=width)
    c["q"] = torch.zeros_like(c["q"])
    c["q"][..., 0] = 1.0
    for j in range(5):
        page = c["table"][0, j].long()
        c["k"][page] = 0
        c["k"][page, :, :, 0] = 1.3 * j
        c["v"][page] = (c["v"][page].float().abs().clamp(max=8.0) * 2.0 ** 119).to(c["v"].dtype)
    d = pu.on_gpu(c)
    o, lse = cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], scale=1.0)
    assert cp.sync_status() == cp.OK
    pu.assert_decode(o, lse, pu.reference(c, 1.0), D, 1.0, n, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("Hkv,D,P", [(1, 64, 16), (3, 128, 64)])
def test_append_bounds_of_pages_whose_new_tokens_leave_gaps(cp, kind, Hkv, D, P):
    """Slots of one page with gaps, in either direction, over the blocks' 32 tokens; skipped
    tokens between pages.  Bounds start afresh with a page's first row, else go on."""
    g = torch.Generator().manual_seed(D + P)
    n_pages = 40
    amax = torch.tensor([6.0, 6.0])
    am = amax.cuda() if kind == "e4m3" else None
    k = torch.zeros((n_pages, Hkv, P, D), dtype=pu.DTYPES[kind], device="cuda")
    v, b = k.clone(), torch.zeros((n_pages, Hkv, 2, D), dtype=pu.DTYPES[kind], device="cuda")
    shadow, want = [pu.values(k), pu.values(v)], pu.values(b)
    for step in range(3):
        slots = []
        for p in torch.randperm(n_pages, generator=g).tolist():
            rows = sorted(torch.randperm(P, generator=g)[:1 + int(torch.randint(P, (1,), generator=g))].tolist())
            if step == 0 and 0 not in rows:
                rows = [0] + rows
            if p % 5 == 4:
                rows.reverse()
            slots += [p * P + i for i in rows]
            slots += [-1] * (0 if p % 3 else int(torch.randint(1, 40, (1,), generator=g)))
        rows = [torch.randn(len(slots), Hkv, D, generator=g).to(pu.rows_dtype(kind)) for _ in range(2)]
        cp.cache_append_(rows[0].cuda(), rows[1].cuda(), torch.tensor(slots, device="cuda"), k, v, k_bounds=b, kv_amax=am)
        assert cp.sync_status() == cp.OK
        put = [pu.values(pu.stored(x, kind, 6.0)) if kind != "e4m3" else fp8.decode(pu.codes_of(x, 6.0)) for x in rows]
        shadow = [paged.append(c, x, slots) for c, x in zip(shadow, put)]
        for p in {s // P for s in slots if s >= 0}:
            mine = [i for i, s in enumerate(slots) if s >= 0 and s // P == p]
            lo, hi = put[0][mine].min(0), put[0][mine].max(0)
            if not any(slots[i] % P == 0 for i in mine):
                lo, hi = np.minimum(lo, want[p, :, 0]), np.maximum(hi, want[p, :, 1])
            want[p, :, 0], want[p, :, 1] = lo, hi
        assert np.array_equal(pu.values(k), shadow[0]) and np.array_equal(pu.values(v), shadow[1])
        assert np.array_equal(pu.values(b), want)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("pages,D,Hq,budget", [(90, 64, 2, 12), (300, 64, 2, 12), (700, 128, 9, 33)])
def test_select_pages_with_infinite_bounds_by_the_definition(cp, kind, pages, D, Hq, budget):
    """One infinite key leaves the other side of its column, and zeros of q leave the column out."""
    g = torch.Generator().manual_seed(pages + D)
    x = torch.randn(pages, 1, 2, D, generator=g).sort(2).values
    inf = float("inf")
    x[5, 0, 0, 3] = -inf
    x[40, 0, 0, :5] = -inf
    x[[5, 40], 0, 1] += 0.5
    x[41, 0, 1, 7] = inf
    x[41, 0, :, 11] = -inf
    x[42, 0, :, 13] = torch.tensor([-inf, inf])
    x[43, 0, 0, 20], x[43, 0, 1, 21] = -inf, inf
    x[44, 0, 1, 30] = -inf
    x[44, 0, 0, 30] = -inf
    x[7, 0, :, 9] = float("nan")
    b = x.to(pu.DTYPES[kind])
    q = torch.randn(1, Hq, D, generator=g).abs().to(pu.rows_dtype(kind))
    q[0, :, :12] = 0
    q[0, 0, :4] = 1
    q[0, 1, 20:22] *= -1
    table = torch.randperm(pages, generator=g).int()[None]
    n = 16 * pages - 1
    got = cp.select_pages(q.cuda(), b.cuda(), table.cuda(), _i32([n]), 16, budget, keep_first=1)
    assert cp.sync_status() == cp.OK
    bv = pu.values(b)
    exact = {(p, 0): (bv[p, 0, 0], bv[p, 0, 1]) for p in range(pages)}
    assert got.cpu().tolist()[0][0] == paged.select(pu.values(q)[0], exact, table[0], n, 16, 0, budget, 1)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_append_bounds_of_columns_that_hold_nan_keys(cp, kind):
    """NaN keys are left out; where there is no other the bounds are NaN, and later keys replace them."""
    Hkv, D, P, n_pages = 2, 64, 16, 40
    am = torch.tensor([448.0, 448.0], device="cuda") if kind == "e4m3" else None
    k = torch.zeros((n_pages, Hkv, P, D), dtype=pu.DTYPES[kind], device="cuda")
    v, b = k.clone(), torch.zeros((n_pages, Hkv, 2, D), dtype=pu.DTYPES[kind], device="cuda")
    g = torch.Generator().manual_seed(19)
    x = torch.randint(-6, 7, (n_pages * P, Hkv, D), generator=g).to(pu.rows_dtype(kind))  # exact in 8 bits
    x[3 * P:3 * P + 9, 1, 5] = float("nan")
    x[7 * P + 2, 0, 50] = float("nan")
    some = torch.arange(n_pages * P).view(n_pages, P)
    first, second = some[:, :9].reshape(-1), some[:, 9:].reshape(-1)
    def bounds(y):  # numpy's fmin and fmax leave NaN out, and give it where there is nothing else
        y = y.float().numpy().reshape(n_pages, -1, Hkv, D)
        return np.stack([np.fmin.reduce(y, 1), np.fmax.reduce(y, 1)], 2)
    for part, upto in ((first, bounds(x[first])), (second, bounds(x))):
        cp.cache_append_(x[part].cuda(), x[part].cuda(), part.cuda(), k, v, k_bounds=b, kv_amax=am)
        assert cp.sync_status() == cp.OK
        assert np.array_equal(pu.values(b), upto, equal_nan=True)
        assert np.isnan(upto).sum() == (2 if part is first else 0)
        # a page whose bounds are NaN ranks last, whatever the other columns say
        q = torch.full((1, Hkv, D), 40.0).to(x.dtype)
        table = torch.arange(n_pages, dtype=torch.int32)[None].cuda()
        got = cp.select_pages(q.cuda(), b, table, _i32([n_pages * P]), P, n_pages - 1).cpu().tolist()[0]
        bv, qv = pu.values(b), pu.values(q)[0]
        exact = {(p, h): (bv[p, h, 0], bv[p, h, 1]) for p in range(n_pages) for h in range(Hkv)}
        assert got == [paged.select(qv[h:h + 1], exact, range(n_pages), n_pages * P, P, h, n_pages - 1, 0) for h in range(Hkv)]
        assert part is second or 3 not in got[1]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hq,pages,budget", [(128, 1, 3000, 700), (64, 5, 400, 150)])
def test_select_sums_that_cancel(cp, kind, D, Hq, pages, budget):
    """Terms of hundreds whose sums differ by less than fp32 sums are off: the band around the
    threshold has to hold every page that could be on either side."""
    g = torch.Generator().manual_seed(pages)
    half = torch.randint(64, 449, (pages, 1, 1, D // 2), generator=g).float()
    half = half.to(torch.float8_e4m3fn).float()
    x = torch.cat([half, -half], 3)[..., torch.randperm(D, generator=g)]
    few = torch.randint(D, (pages,), generator=g)
    x[torch.arange(pages), 0, 0, few] *= 1 + torch.randint(0, 2, (pages,), generator=g) / 8
    b = x.expand(pages, 1, 2, D).contiguous()
    b = b.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else b.bfloat16()
    q = (1 + torch.randint(0, 128, (1, Hq, D), generator=g) / 128).bfloat16()
    q[..., ::3] = 1 + 2.0 ** -7
    table = torch.randperm(pages, generator=g).int()[None]
    n = 16 * pages - 5
    got = cp.select_pages(q.cuda(), b.cuda(), table.cuda(), _i32([n]), 16, budget)
    assert cp.sync_status() == cp.OK
    bv = pu.values(b)
    exact = {(p, 0): (bv[p, 0, 0], bv[p, 0, 1]) for p in range(pages)}
    assert got.cpu().tolist()[0][0] == paged.select(pu.values(q)[0], exact, table[0], n, 16, 0, budget, 0)


@pytest.mark.parametrize("width", [3, 5000])
def test_select_largest_budget(cp, width):
    """2^31 - 1 entries (8.6 GB), of which a request of three pages fills three."""
    q, b = torch.zeros((1, 1, 64), device="cuda"), torch.zeros((3, 1, 2, 64), device="cuda")
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    table[0, :3] = torch.arange(3)
    got = cp.select_pages(q, b, table, _i32([40]), 16, 2 ** 31 - 1, keep_first=7)[0, 0]
    assert cp.sync_status() == cp.OK
    assert got[:3].tolist() == [0, 1, 2]
    assert got[3:].max().item() == got[3:].min().item() == -1


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("R,Hkv,Hq,D,width,budget", [(1, 1, 2, 64, 49152, 700), (1, 2, 18, 128, 24577, 15423),
                                                     (1, 1, 1, 64, 24576, 300), (40, 4, 4, 64, 9000, 200)])
def test_select_over_the_widest_tables(cp, kind, R, Hkv, Hq, D, width, budget):
    """Scores of up to 192 KB of a block's shared memory, with clusters of every size; near the
    threshold many pages of alike bounds."""
    g = torch.Generator().manual_seed(width + Hq)
    pool = min(R * width, 60000)
    x = torch.randn(pool, Hkv, 2, D, generator=g).sort(2).values
    x[1::2] = x[::2][:pool // 2]  # pairs of equal pages
    b = x.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else x.to(pu.DTYPES[kind])
    q = torch.randn(R, Hq, D, generator=g).to(pu.rows_dtype(kind))
    table = torch.stack([torch.randperm(pool, generator=g)[:width] for _ in range(R)]).int()
    held = [width - (r * 311) % width for r in range(R)]
    lens = [16 * n - r % 16 for r, n in enumerate(held)]
    got = cp.select_pages(q.cuda(), b.cuda(), table.cuda(), _i32(lens), 16, budget, keep_first=2).cpu()
    assert cp.sync_status() == cp.OK
    bv, qv, group = pu.values(b), pu.values(q), Hq // Hkv
    lo, hi = (torch.from_numpy(bv[:, :, i]).cuda() for i in (0, 1))
    for r in range(R):
        ids = table[r, :held[r]].long().cuda()
        for h in range(Hkv):
            # the definition in 64 bits, a head at a time
            s = torch.stack([torch.maximum(x * lo[ids, h], x * hi[ids, h]).sum(1)
                             for x in torch.from_numpy(qv[r, h * group:(h + 1) * group]).cuda()]).amax(0).float()
            s[:2] = float("inf")
            s[-1] = float("inf")
            n = min(budget, held[r])
            want = s.sort(descending=True, stable=True).indices[:n].sort().values.int().cpu()
            assert torch.equal(got[r, h, :n], want) and torch.all(got[r, h, n:] == -1), (r, h)


def test_decode_refuses_an_empty_list_of_pages(cp):
    d = pu.on_gpu(pu.make_cache([30], 2, 1, 64, 16, "bf16", seed=47))
    for kw in ({}, dict(out_dtype=torch.float32)):
        with pytest.raises(ValueError, match="pages must have room"):
            cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], pages=_i32([[[]]]), **kw)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("D,P", [(64, 256), (128, 128), (64, 16)])
def test_append_runs_of_every_length_and_start(cp, kind, D, P):
    """Consecutive rows from and to any row, with and without one gap, beside the steps of 32 and 64 tokens."""
    g = torch.Generator().manual_seed(D * P)
    am = torch.tensor([6.0, 6.0], device="cuda") if kind == "e4m3" else None
    starts = [0, 1, 15] if P == 16 else [0, 1, 31, 32, 33, 63, 64, 65, P - 2, P - 1]
    ends = [s + n for s in starts for n in (1, 31, 32, 33, 63, 64, 65, 127, 128, 129, P)]
    runs = sorted({(s, min(e, P)) for s, e in zip([s for s in starts for _ in range(11)], ends)})
    slots = []
    for p, (lo, hi) in enumerate(runs + runs):
        rows = list(range(lo, hi))
        if p >= len(runs) and len(rows) > 2:
            rows.pop(int(torch.randint(1, len(rows) - 1, (1,), generator=g)))
        slots += [p * P + i for i in rows]
    n_pages = 2 * len(runs)
    k = torch.zeros((n_pages, 2, P, D), dtype=pu.DTYPES[kind], device="cuda")
    v, b = k.clone(), torch.zeros((n_pages, 2, 2, D), dtype=pu.DTYPES[kind], device="cuda")
    rows = [torch.randn(len(slots), 2, D, generator=g).to(pu.rows_dtype(kind)) for _ in range(2)]
    for bounds in (None, b):
        k.zero_(), v.zero_()
        cp.cache_append_(rows[0].cuda(), rows[1].cuda(), torch.tensor(slots, device="cuda"), k, v, k_bounds=bounds, kv_amax=am)
        assert cp.sync_status() == cp.OK
        put = [fp8.decode(pu.codes_of(x, 6.0)) if kind == "e4m3" else pu.values(x) for x in rows]
        for got, x in ((k, put[0]), (v, put[1])):
            want = np.zeros((n_pages * P, 2, D))
            want[slots] = x
            assert np.array_equal(pu.values(got), want.reshape(n_pages, P, 2, D).transpose(0, 2, 1, 3))
    bv, page_of = pu.values(b), np.array(slots) // P
    for p in range(n_pages):
        mine = put[0][page_of == p]
        lo, hi = mine.min(0), mine.max(0)
        if p * P not in slots:  # it goes on from the zeros
            lo, hi = np.minimum(lo, 0), np.maximum(hi, 0)
        assert np.array_equal(bv[p, :, 0], lo) and np.array_equal(bv[p, :, 1], hi)
