"""The paged key-value cache on the GPU against the fp64 oracle."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from long_sequence_context_b200.inputs import make_qkv
from oracle import fp8, paged
from tests import paged_util as pu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    from long_sequence_context_b200 import cpattn
    cpattn.set_path(0)
    return cpattn


# ---- decode ----

def _decode(cp, c, scale, pages=None, **kw):
    d = pu.on_gpu(c)
    o, lse = cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], pages=pages, kv_amax=d["amax"], scale=scale, **kw)
    assert cp.sync_status() == cp.OK
    return o, lse


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", [
    ([1], 1, 1, 64, 16),
    ([17], 3, 1, 128, 16),
    ([0, 5, 0], 4, 2, 64, 32),
    ([64, 63, 65, 1, 16, 15, 300], 8, 8, 128, 64),
    ([1000, 3, 257], 8, 1, 128, 128),
    ([513, 130], 9, 1, 64, 16),
    ([200, 0, 77], 32, 2, 128, 32),
    ([90, 333], 20, 1, 128, 256),
    ([150], 34, 1, 64, 64),
    ([311, 40], 64, 1, 128, 16),
])
def test_decode_matches_oracle(cp, kind, lens, Hq, Hkv, D, P):
    c = pu.make_cache(lens, Hq, Hkv, D, P, kind, seed=sum(lens) + Hq + D)
    o, lse = _decode(cp, c, D ** -0.5)
    assert o.dtype == c["q"].dtype
    pu.assert_decode(o, lse, pu.reference(c, D ** -0.5), D, D ** -0.5, max(lens), kind)


@pytest.mark.parametrize("kind,D,P,Hkv", [("bf16", 128, 64, 2), ("e4m3", 64, 16, 1), ("fp32", 128, 32, 1)])
def test_decode_long_context_split_over_many_blocks(cp, kind, D, P, Hkv):
    lens = [20011, 1, 4096]
    c = pu.make_cache(lens, 2 * Hkv, Hkv, D, P, kind, seed=5)
    o, lse = _decode(cp, c, D ** -0.5)
    pu.assert_decode(o, lse, pu.reference(c, D ** -0.5), D, D ** -0.5, max(lens), kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("group,D", [(17, 128), (32, 64), (48, 128), (64, 64)])
def test_decode_large_groups_over_long_and_short_requests(cp, kind, group, D):
    """Warps of several head groups share the keys' ring, over many pairs and turns."""
    lens = [5003, 0, 64, 1, 900, 2048, 17]
    c = pu.make_cache(lens, 2 * group, 2, D, 64, kind, seed=group + D)
    o, lse = _decode(cp, c, D ** -0.5)
    pu.assert_decode(o, lse, pu.reference(c, D ** -0.5), D, D ** -0.5, max(lens), kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp32"])
def test_decode_many_short_requests(cp, kind):
    g = np.random.default_rng(6)
    lens = [int(x) for x in g.integers(0, 40, 700)]
    c = pu.make_cache(lens, 2, 1, 64, 16, kind, seed=6)
    o, lse = _decode(cp, c, 0.125)
    pu.assert_decode(o, lse, pu.reference(c, 0.125), 64, 0.125, 40, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
def test_decode_large_scores(cp, kind):
    """Scores of several hundred: one key takes nearly all the weight, the rest underflow."""
    c = pu.make_cache([777, 30], 4, 2, 128, 32, kind, seed=7, scale=1.0)
    o, lse = _decode(cp, c, 8.0)
    ref = pu.reference(c, 8.0)
    pu.assert_decode(o, lse, ref, 128, 8.0, 777, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P", [
    ([1], 1, 1, 64, 16),
    ([0, 5, 0], 4, 2, 64, 32),
    ([257], 16, 16, 128, 16),
    ([700, 0, 64, 333], 12, 4, 64, 16),
    ([513, 130], 9, 1, 128, 64),
    ([1024, 1023, 1, 512], 34, 2, 64, 32),
    ([2048, 77], 48, 1, 128, 256),
    ([0, 0], 128, 2, 64, 16),
    ([128] * 37, 8, 4, 128, 16),
    ([0, 300, 50, 129] * 10, 5, 5, 64, 64),
    ([4096], 24, 8, 64, 128),
])
def test_decode_with_a_table_just_wide_enough_and_with_a_wide_one(cp, kind, lens, Hq, Hkv, D, P):
    """The table's width decides how the keys are dealt to blocks: both ways, all cluster sizes."""
    refs = []
    for width in (max(1, -(-max(lens) // P)), 8192 // P, 65536 // P):
        c = pu.make_cache(lens, Hq, Hkv, D, P, kind, seed=sum(lens) + Hq, width=width)
        refs = refs or [pu.reference(c, D ** -0.5)]
        for out_dtype in (None, torch.float32):
            o, lse = _decode(cp, c, D ** -0.5, out_dtype=out_dtype)
            pu.assert_decode(o, lse, refs[0], D, D ** -0.5, max(lens), kind, str(width))


@pytest.mark.parametrize("kind,exponent", [(k, e) for k in ("bf16", "fp32", "e4m3") for e in (-100, -60, 60, 100)] +
                         [("e4m3", -133), ("e4m3", -128), ("e4m3", -126)])
def test_decode_queries_of_any_size(cp, kind, exponent):
    """A scale that brings the scores back to ordinary ones, as far as it goes; 8-bit keys
    take queries down to the subnormal ones, which they scale into half precision."""
    c = pu.make_cache([300, 40], 6, 2, 128, 32, kind, seed=14)
    c["q"] = (c["q"].double() * 2.0 ** exponent).to(c["q"].dtype)
    scale = 2.0 ** max(-124, min(124, -exponent)) * 128 ** -0.5
    ref = pu.reference(c, scale)
    o, lse = _decode(cp, c, scale)
    pu.assert_decode(o, lse, ref, 128, scale, 300, kind)


def test_a_batch_of_twenty_thousand_requests(cp):
    R, D, P = 20011, 64, 16
    g = torch.Generator().manual_seed(50)
    lens = torch.randint(0, 3, (R,), generator=g)
    k, v = torch.randn(2, R, 1, P, D, generator=g)
    q = torch.randn(R, 2, D, generator=g)
    table = torch.arange(R, dtype=torch.int32)[:, None]
    o, lse = cp.decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), lens.int().cuda(), scale=0.3)
    pages = cp.select_pages(q.cuda(), torch.zeros(R, 1, 2, D, device="cuda"), table.cuda(), lens.int().cuda(), P, 2)
    assert cp.sync_status() == cp.OK
    assert torch.equal(pages.cpu()[:, 0, 0], torch.where(lens > 0, 0, -1).int()) and torch.all(pages[:, 0, 1] == -1)
    x = 0.3 * torch.einsum("rhd,rjd->rhj", q.double(), k[:, 0, :2].double())
    x = x.masked_fill(torch.arange(2) >= lens[:, None, None], float("-inf"))
    want_lse = torch.logsumexp(x, -1)
    w = torch.exp(x - want_lse.masked_fill(want_lse.isinf(), 0.0)[..., None])
    want = torch.einsum("rhj,rjd->rhd", w, v[:, 0, :2].double())
    assert torch.equal(lse.cpu().isneginf(), want_lse.isneginf())
    seen = lens > 0
    # (D + 2) 2^-24 scale sum |q k| <= 3e-5 on a score, twice that on a weight, |v| <= 6
    assert (lse.cpu().double() - want_lse)[seen].abs().max() < 5e-5 and (o.cpu().double() - want).abs().max() < 4e-4
    assert torch.all(o.cpu()[~seen] == 0)


def test_decode_fp32_output_and_merge_of_two_halves_of_a_context(cp):
    """Each of two ranks holds half of the keys: their fp32 results merge to the whole."""
    c = pu.make_cache([1500, 1500], 8, 2, 128, 64, "bf16", seed=8)
    whole = pu.reference(c, 0.1)
    o, lse = _decode(cp, c, 0.1, out_dtype=torch.float32)
    pu.assert_decode(o, lse, whole, 128, 0.1, 1500, "bf16")
    first, second = dict(c), dict(c)
    first["lens"] = torch.tensor([640, 640], dtype=torch.int32)
    second["table"] = c["table"][:, 10:].contiguous()
    second["lens"] = torch.tensor([860, 860], dtype=torch.int32)
    oa, la = _decode(cp, first, 0.1, out_dtype=torch.float32)
    ob, lb = _decode(cp, second, 0.1, out_dtype=torch.float32)
    cp.merge_(oa, la, ob, lb)
    pu.assert_decode(oa, la, whole, 128, 0.1, 1500, "bf16", "merged")


def test_decode_is_deterministic_and_keeps_its_surroundings(cp):
    c = pu.on_gpu(pu.make_cache([3000, 0, 511], 8, 2, 64, 32, "bf16", seed=9))
    buf = torch.full((5, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lbuf = torch.full((5, 8), 7.0, dtype=torch.float32, device="cuda")
    args = (c["q"], c["k"], c["v"], c["table"], c["lens"])
    o1, l1 = cp.decode(*args, out=buf[1:4], lse=lbuf[1:4])
    o1, l1 = o1.clone(), l1.clone()
    ws = torch.full((cp.decode_workspace_bytes(3, 8, 2, 64),), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = cp.decode(*args, workspace=ws)
    assert cp.sync_status() == cp.OK
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.all(buf[0] == 7) and torch.all(buf[4] == 7) and torch.all(lbuf[0] == 7) and torch.all(lbuf[4] == 7)


def test_decode_result_of_a_request_does_not_depend_on_the_others_values(cp):
    c = pu.on_gpu(pu.make_cache([700, 900], 4, 2, 128, 32, "bf16", seed=10))
    args = lambda k: (c["q"], k, c["v"], c["table"], c["lens"])
    o1, l1 = cp.decode(*args(c["k"]))
    k2 = c["k"].clone()
    k2[c["table"][1, :29].long()] = float("nan")
    o2, l2 = cp.decode(*args(k2))
    assert torch.equal(o1[0], o2[0]) and torch.equal(l1[0], l2[0])
    assert torch.isnan(o2[1]).all()


def test_decode_bad_pages_and_lengths_are_left_out_and_reported(cp):
    c = pu.make_cache([100, 64], 2, 1, 64, 16, "fp32", seed=11, width=8)
    d = pu.on_gpu(c)
    bad = d["table"].clone()
    bad[0, 2] = 1 << 30
    bad[0, 3] = -5
    o, lse = cp.decode(d["q"], d["k"], d["v"], bad, d["lens"], scale=0.1)
    assert cp.sync_status() == cp.ERR_PAGE and cp.sync_status() == cp.OK
    keep = [[[0, 1, 4, 5, 6]], [[0, 1, 2, 3]]]
    pu.assert_decode(o, lse, pu.reference(c, 0.1, keep), 64, 0.1, 100, "fp32")
    for lens in ([-3, 64], [100, 1 << 30]):
        full = dict(d, table=torch.zeros_like(d["table"]), k=torch.zeros_like(d["k"]), v=torch.zeros_like(d["v"]))
        cp.decode(full["q"], full["k"], full["v"], full["table"], torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert cp.sync_status() == cp.ERR_PAGE


def test_decode_cache_offsets_beyond_32_bits(cp):
    """A page behind 2^32 bytes of cache (and 2^32 elements, in 8 bits)."""
    P, Hkv, D = 256, 8, 128
    n = (1 << 32) // (P * Hkv * D) + 3
    k = torch.zeros((n, Hkv, P, D), dtype=torch.uint8, device="cuda")
    c = pu.make_cache([300], 8, Hkv, D, P, "e4m3", seed=12, poison=False)
    for i, p in enumerate(c["table"][0, :2].tolist()):
        k[n - 1 - i] = c["k"][p].cuda()
    table = torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device="cuda")
    # the same codes serve as K and V: a second cache of that size adds nothing
    o, lse = cp.decode(c["q"].cuda(), k, k, table, c["lens"].cuda(), kv_amax=c["amax"].cuda())
    assert cp.sync_status() == cp.OK
    a = c["amax"].tolist()
    kk, vv = pu.values(c["k"], a[0]), pu.values(c["k"], a[1])
    ref = paged.decode(pu.values(c["q"]), kk, vv, c["table"].numpy(), [300], D ** -0.5)
    pu.assert_decode(o, lse, ref, D, D ** -0.5, 300, "e4m3")
    rows = torch.randn(2, Hkv, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([(n - 1) * P + 5, (n - 1) * P + 6], device="cuda")
    cp.cache_append_(rows, rows, slots, k, k.clone(), kv_amax=c["amax"].cuda())
    assert cp.sync_status() == cp.OK
    want = torch.from_numpy(pu.codes_of(rows.cpu(), a[0]))
    assert torch.equal(k[n - 1, :, 5:7].transpose(0, 1).cpu(), want)


# ---- selected pages ----

def _select_case(cp, lens, Hq, Hkv, D, P, kind, budget, keep, seed):
    c = pu.make_cache(lens, Hq, Hkv, D, P, kind, seed)
    kv = pu.values(c["k"])
    exact = paged.bounds(kv, c["table"].numpy(), lens)
    b = torch.zeros((c["k"].shape[0], Hkv, 2, D))
    for (p, h), (lo, hi) in exact.items():
        b[p, h, 0], b[p, h, 1] = torch.from_numpy(lo), torch.from_numpy(hi)
    c["bounds"] = b.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else b.to(c["k"].dtype)
    d = pu.on_gpu(c)
    sel = cp.select_pages(d["q"], d["bounds"], d["table"], d["lens"], P, budget, keep_first=keep)
    assert cp.sync_status() == cp.OK
    q = pu.values(c["q"])
    g = Hq // Hkv
    want = [[paged.select(q[r, h * g:(h + 1) * g], exact, c["table"][r], lens[r], P, h, budget, keep)
             for h in range(Hkv)] for r in range(len(lens))]
    assert sel.cpu().tolist() == want
    return c, d, sel, want


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,P,budget,keep", [
    ([1, 0, 40], 2, 1, 64, 16, 1, 0),
    ([700, 333, 100], 8, 2, 128, 16, 7, 1),
    ([5000], 12, 1, 64, 16, 100, 3),
    ([4097, 16], 20, 1, 128, 32, 64, 0),
    ([300] * 160, 2, 2, 64, 16, 5, 2),
])
def test_select_and_decode_selected_match_oracle(cp, kind, lens, Hq, Hkv, D, P, budget, keep):
    c, d, sel, want = _select_case(cp, lens, Hq, Hkv, D, P, kind, budget, keep, seed=len(lens) + budget)
    o, lse = _decode(cp, c, D ** -0.5, pages=sel)
    pu.assert_decode(o, lse, pu.reference(c, D ** -0.5, want), D, D ** -0.5, max(lens), kind)


def test_select_ties_go_to_the_lower_page(cp):
    P, D, n = 16, 64, 16 * 1000
    q = torch.ones((1, 1, D), device="cuda")
    b = torch.zeros((1000, 1, 2, D), device="cuda")
    b[500:, :, 1] = 1.0
    b[::7] = -0.0
    table = torch.arange(1000, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    top = [j for j in range(500, 999) if j % 7]
    for budget in (4, 100, 600):
        got = cp.select_pages(q, b, table, lens, P, budget).cpu().tolist()[0][0]
        rest = [j for j in range(999) if j < 500 or j % 7 == 0]
        assert got == sorted((top + rest)[:budget - 1] + [999])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "fp32"])
@pytest.mark.parametrize("D,Hq,pages,budget", [(64, 3, 700, 100), (128, 9, 300, 20), (128, 1, 5000, 2500)])
def test_select_near_ties_are_settled_exactly(cp, kind, D, Hq, pages, budget):
    """Pages that differ by one step of one column, some not at all: fp32 sums could swap them."""
    g = torch.Generator().manual_seed(pages + budget)
    base = torch.randn(2, D, generator=g).abs() * torch.tensor([[-1.0], [1.0]])
    b = base.expand(pages, 1, 2, D).clone()
    col, side = torch.randint(D, (pages,), generator=g), torch.randint(2, (pages,), generator=g)
    step = torch.where(torch.randint(3, (pages,), generator=g) > 0, 1 + 2.0 ** -7, 1.0)
    b[torch.arange(pages), 0, side, col] *= step
    b = b.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else b.to(pu.DTYPES[kind])
    q = torch.randn(1, Hq, D, generator=g).to(pu.rows_dtype(kind))
    table = torch.randperm(pages, generator=g).int()[None]
    n = 16 * pages - 3
    got = cp.select_pages(q.cuda(), b.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), 16, budget,
                          keep_first=1)
    assert cp.sync_status() == cp.OK
    bv = pu.values(b)
    exact = {(p, 0): (bv[p, 0, 0], bv[p, 0, 1]) for p in range(pages)}
    # the definition's sums in 64 bits, rounded to fp32: as the oracle forms them
    assert got.cpu().tolist()[0][0] == paged.select(pu.values(q)[0], exact, table[0], n, 16, 0, budget, 1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_select_with_infinite_and_nan_bounds(cp, kind):
    pages, D, budget = 200, 64, 10
    g = torch.Generator().manual_seed(7)
    x = torch.randn(pages, 1, 2, D, generator=g).sort(2).values
    if kind == "bf16":
        x[5, 0, 1, 3] = float("inf")
        x[6, 0, 0, 3] = float("-inf")
    x[7, 0, :, 9] = float("nan")
    x[8, 0, 0, 9] = float("nan")
    b = x.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else x.to(torch.bfloat16)
    q = torch.randn(1, 2, D, generator=g).bfloat16()
    q[q == 0] = 1
    q[0, 0] = q[0, 0].abs()
    q[0, 1] = -q[0, 1].abs()
    table = torch.arange(pages, dtype=torch.int32)[None]
    lens = torch.tensor([16 * pages], dtype=torch.int32)
    got = cp.select_pages(q.cuda(), b.cuda(), table.cuda(), lens.cuda(), 16, budget).cpu().tolist()[0][0]
    assert cp.sync_status() == cp.OK
    bv = pu.values(b)
    score = []
    for j in range(pages):
        # as the kernel writes it: min(q, 0) lo + max(q, 0) hi; a head whose sum is NaN does not count
        heads = [np.sum(np.minimum(h, 0) * bv[j, 0, 0] + np.maximum(h, 0) * bv[j, 0, 1]) for h in pu.values(q)[0]]
        heads = [h for h in heads if not np.isnan(h)]
        score.append(float(np.float32(max(heads))) if heads else -np.inf)
    score[-1] = np.inf
    assert got == sorted(sorted(range(pages), key=lambda j: (-score[j], j))[:budget])


def test_decode_reads_lists_with_gaps_and_pages_behind_the_length(cp):
    c = pu.make_cache([200, 70], 4, 2, 64, 16, "bf16", seed=13)
    lists = [[[-1, 3, 12, -1, 5], [12, 0, 1, 2, 3]], [[4, -1, -1, 0, 9], [9, -1, -1, -1, 2]]]
    pages = torch.tensor(lists, dtype=torch.int32, device="cuda")
    o, lse = _decode(cp, c, 0.125, pages=pages)
    keep = [[[j for j in x if 0 <= j < paged.pages_of(n, 16)] for x in l] for l, n in zip(lists, [200, 70])]
    a = pu.values(c["q"]), pu.values(c["k"]), pu.values(c["v"])
    ref = paged.decode(*a, c["table"].numpy(), [200, 70], 0.125, keep)
    pu.assert_decode(o, lse, ref, 64, 0.125, 200, "bf16")


# ---- the books ----

def _plan(cp, s, delta, P, cap, **kw):
    t = lambda x, n=torch.int32: torch.tensor(x, dtype=n, device="cuda")
    table, ring = s["table"].clone(), s["ring"].clone()
    out = cp.cache_plan(s["lens"], t(delta), table, ring, s["state"], P, cap, **kw)
    want = paged.plan(s["lens"].tolist(), delta, s["table"].cpu().numpy(), s["ring"].tolist(), s["state"].tolist(), P, cap)
    lens, state, cu, slots, verdict = out
    assert verdict.item() == want[6]
    assert lens.tolist() == want[0] and state.tolist() == want[3] and cu.tolist() == want[4]
    assert slots.tolist() == want[5]
    assert np.array_equal(table.cpu().numpy(), want[1]) and ring.tolist() == want[2]
    assert cp.sync_status() == cp.OK
    return dict(lens=lens, state=state, table=table, ring=ring), cu, slots, want[6]


def _books(R, width, num_pages, head=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return dict(lens=torch.zeros(R, dtype=torch.int32, device="cuda"),
                table=torch.full((R, width), -1, dtype=torch.int32, device="cuda"),
                ring=torch.randperm(num_pages, generator=g).int().cuda(),
                state=torch.tensor([head, num_pages], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("R,width,P,num_pages,most,cap", [
    (1, 3, 16, 3, 48, 48), (5, 9, 16, 31, 90, 300), (70, 40, 32, 900, 700, 40000), (1500, 5, 64, 3500, 200, 100000),
    (20011, 2, 16, 30000, 30, 300000)])
def test_plan_steps_match_oracle(cp, R, width, P, num_pages, most, cap):
    g = np.random.default_rng(R)
    s = _books(R, width, num_pages, head=num_pages // 2, seed=R)
    for _ in range(8):
        lens = s["lens"].tolist()
        delta = []
        for n in lens:
            what = g.integers(4)
            delta.append(-n if what == 0 else -int(g.integers(0, min(n, 5) + 1)) if what == 1
                         else int(g.integers(0, min(most, width * P - n) + 1)))
        s, _, _, _ = _plan(cp, s, delta, P, cap)


def test_plan_returns_and_takes_thousands_of_pages_in_a_small_step(cp):
    """One token for one request while another returns 5000 pages and a third takes 900."""
    P, width = 16, 5200
    s = _books(3, width, 7000, head=6990, seed=8)
    s, _, _, v = _plan(cp, s, [80000, 100, 3], P, 80103)
    assert v == 0
    s, _, slots, v = _plan(cp, s, [-80000, 1, 1000], P, 1001)
    assert v == 0 and slots[:1001].min() >= 0
    s, _, _, v = _plan(cp, s, [1, -101, -1003], P, 1)
    assert v == 0 and s["state"][1].item() == 6999


def test_plan_refusals_change_nothing(cp):
    s, _, _, v = _plan(cp, _books(3, 4, 9), [20, 33, 5], 16, 64)
    assert v == 0
    for delta, cap, bits in [([40, 30, 30], 200, paged.SHORT), ([1, 1, 1], 2, paged.CAPACITY),
                             ([-21, 0, 0], 9, paged.BAD_LENGTH), ([45, 0, 0], 99, paged.BAD_LENGTH),
                             ([44, 31, 59], 9, paged.SHORT | paged.CAPACITY)]:
        after, cu, slots, v = _plan(cp, s, delta, 16, cap)
        assert v == bits
        assert all(torch.equal(after[k], s[k]) for k in s)
    for state in ([9, 1], [-1, 2], [0, 10], [0, -1], [3, 9]):
        broken = dict(s, state=torch.tensor(state, dtype=torch.int32, device="cuda"))
        _, _, _, v = _plan(cp, broken, [-20, 0, 0], 16, 9)
        assert v & paged.BAD_STATE


def test_plan_in_place_and_again(cp):
    s = _books(4, 8, 20)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    keep = {k: x.clone() for k, x in s.items()}
    once = cp.cache_plan(s["lens"], t([30, 0, 1, 17]), s["table"], s["ring"], s["state"], 16, 50)
    again = cp.cache_plan(s["lens"], t([30, 0, 1, 17]), s["table"], s["ring"], s["state"], 16, 50)
    assert all(torch.equal(a, b) for a, b in zip(once, again))
    assert torch.equal(s["lens"], keep["lens"]) and torch.equal(s["state"], keep["state"])
    got = cp.cache_plan(s["lens"], t([30, 0, 1, 17]), s["table"], s["ring"], s["state"], 16, 50, lens_out=s["lens"],
                        free_state_out=s["state"])
    assert got[0] is s["lens"] and torch.equal(s["lens"], once[0]) and torch.equal(s["state"], once[1])
    assert torch.equal(got[3], once[3])


@pytest.mark.parametrize("which", ["lens", "state", "both"])
@pytest.mark.parametrize("R,cap", [(7, 600), (1000, 2048), (7, 2049), (1024, 70000), (1025, 70000)])
def test_plan_in_place_matches_oracle(cp, R, cap, which):
    """Lengths, state or both updated where they are, at sizes on both sides of every limit of the launches."""
    P, width = 16, 8
    g = np.random.default_rng(R + cap)
    s = _books(R, width, R * width, head=R, seed=cap)
    most = min(60, cap // R)
    for step in range(4):
        lens = s["lens"].tolist()
        delta = [-n if g.integers(5) == 0 else int(g.integers(-min(n, 40), min(most, width * P - n) + 1)) for n in lens]
        want = paged.plan(lens, delta, s["table"].cpu().numpy(), s["ring"].tolist(), s["state"].tolist(), P, cap)
        kw = {}
        if which != "state":
            kw["lens_out"] = s["lens"]
        if which != "lens":
            kw["free_state_out"] = s["state"]
        out = cp.cache_plan(s["lens"], torch.tensor(delta, dtype=torch.int32, device="cuda"), s["table"], s["ring"],
                            s["state"], P, cap, **kw)
        assert out[4].item() == want[6] == 0
        s["lens"], s["state"] = out[0], out[1]
        assert out[0].tolist() == want[0] and out[1].tolist() == want[3]
        assert out[2].tolist() == want[4] and out[3].tolist() == want[5]
        assert np.array_equal(s["table"].cpu().numpy(), want[1]) and s["ring"].tolist() == want[2]
        assert cp.sync_status() == cp.OK


# ---- rows ----

@pytest.mark.parametrize("kind", ["bf16", "fp32", "e4m3"])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("Hkv,D,P", [(1, 64, 16), (3, 128, 16), (2, 64, 128)])
def test_append_matches_oracle_bit_for_bit(cp, kind, heads_first, Hkv, D, P):
    g = torch.Generator().manual_seed(Hkv + D + P)
    amax = torch.tensor([3.0, 2.5])  # some rows saturate
    am = amax.cuda() if kind == "e4m3" else None
    s = _books(4, 300 // P + 2, 4 * (300 // P + 2), seed=3)
    n_pages = s["ring"].shape[0]
    k = torch.full((n_pages, Hkv, P, D), 0, dtype=pu.DTYPES[kind], device="cuda")
    v, b = k.clone(), torch.zeros((n_pages, Hkv, 2, D), dtype=pu.DTYPES[kind], device="cuda")
    shadow = pu.values(k), pu.values(v)
    for delta in ([1, 0, 100, 17], [1, 30, 1, 64], [-2, -30, 150, 1], [5, 33, 1, 0]):
        s, cu, slots, verdict = _plan(cp, s, delta, P, 300)
        assert verdict == 0
        rows = [torch.randn(300, Hkv, D, generator=g).to(pu.rows_dtype(kind)) for _ in range(2)]
        if heads_first:
            dev = [x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in rows]
        else:
            dev = [torch.cat([x, x], 2).cuda()[:, :, :D] for x in rows]  # heads 2 D apart
        cp.cache_append_(dev[0], dev[1], slots, k, v, k_bounds=b, kv_amax=am)
        assert cp.sync_status() == cp.OK
        put = []
        for i, x in enumerate(rows):
            if kind == "e4m3":
                put.append(fp8.decode(pu.codes_of(x, amax[i].item())))
            else:
                put.append(pu.values(x))
        shadow = tuple(paged.append(c, x, slots.tolist()) for c, x in zip(shadow, put))
        assert np.array_equal(pu.values(k), shadow[0]) and np.array_equal(pu.values(v), shadow[1])
        bv = pu.values(b)
        for (p, h), (lo, hi) in paged.bounds(shadow[0], s["table"].cpu().numpy(), s["lens"].tolist()).items():
            # rows taken back may still be covered: the bounds hold, and are exact until then
            assert np.all(bv[p, h, 0] <= lo) and np.all(bv[p, h, 1] >= hi)
            if min(delta) >= 0 and delta[0] == 1:
                assert np.array_equal(bv[p, h, 0], lo) and np.array_equal(bv[p, h, 1], hi)


def test_append_skips_negative_slots_and_reports_slots_behind_the_cache(cp):
    k = torch.zeros((4, 2, 16, 64), device="cuda")
    v = torch.zeros_like(k)
    x = torch.ones((5, 2, 64), device="cuda")
    slots = torch.tensor([3, -1, 17, 64, -(1 << 40)], device="cuda")
    cp.cache_append_(x, x, slots, k, v)
    assert cp.sync_status() == cp.ERR_PAGE and cp.sync_status() == cp.OK
    want = torch.zeros_like(k)
    want[0, :, 3] = 1
    want[1, :, 1] = 1
    assert torch.equal(k, want) and torch.equal(v, want)
    cp.cache_append_(x[:0], x[:0], slots[:0], k, v)
    assert torch.equal(k, want)


# ---- together ----

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prefill_by_the_ring_then_decode_token_by_token(cp, kind):
    """K and V of a causal forward fill the cache (all but the last tokens at once,
    the rest one by one); each decoded row is the forward's row."""
    B, H, S, D, P = 2, 4, 512, 128, 64
    q, k, v, _ = make_qkv(B, H, S, D, torch.bfloat16, seed=21, with_dout=False)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    o_ring, lse_ring = cp.fwd(qd, kd, vd, 2, True)
    amax = torch.cat([cp.amax(kd), cp.amax(vd)]) if kind == "e4m3" else None
    s = _books(B, S // P, B * S // P + 1, seed=4)
    shape = (B * S // P + 1, H, P, D)
    kc = torch.zeros(shape, dtype=pu.DTYPES[kind], device="cuda")
    vc, kb = torch.zeros_like(kc), torch.zeros((shape[0], H, 2, D), dtype=kc.dtype, device="cuda")
    start = S - 3
    for at, n in [(0, start), (start, 1), (start + 1, 1), (start + 2, 1)]:
        s, cu, slots, verdict = _plan(cp, s, [n] * B, P, B * n)
        assert verdict == 0
        for r in range(B):
            cp.cache_append_(kd[r, :, at:at + n].transpose(0, 1), vd[r, :, at:at + n].transpose(0, 1),
                             slots[r * n:(r + 1) * n], kc, vc, k_bounds=kb, kv_amax=amax)
        row = qd[:, :, at + n - 1].contiguous()
        o, lse = cp.decode(row, kc, vc, s["table"], s["lens"], kv_amax=amax)
        pages = cp.select_pages(row, kb, s["table"], s["lens"], P, S // P)
        os_, ls_ = cp.decode(row, kc, vc, s["table"], s["lens"], pages=pages, kv_amax=amax)
        assert cp.sync_status() == cp.OK
        assert torch.equal(o, os_) and torch.equal(lse, ls_)  # the budget covers every page
        c = dict(q=row, k=kc, v=vc, table=s["table"].cpu(), lens=s["lens"].cpu(), amax=amax.cpu() if amax is not None else None)
        pu.assert_decode(o, lse, pu.reference(c, D ** -0.5), D, D ** -0.5, S, kind)
        if kind == "bf16":
            # the forward's own bound: one bf16 rounding of P (2^-8) and of O each side
            err = (o.float() - o_ring[:, :, at + n - 1].float()).abs().max().item()
            assert err <= 2e-2 and (lse - lse_ring[:, :, at + n - 1]).abs().max().item() <= 1e-3


def test_a_captured_step_replayed_as_the_context_grows(cp):
    """plan in place, append, select and decode in one CUDA graph, replayed thirty times."""
    R, Hq, Hkv, D, P, width = 3, 4, 2, 64, 16, 8
    s = _books(R, width, R * width, seed=5)
    kc = torch.zeros((R * width, Hkv, P, D), dtype=torch.bfloat16, device="cuda")
    vc, kb = torch.zeros_like(kc), torch.zeros((R * width, Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    delta = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
    kn = torch.zeros((4, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vn, q = torch.zeros_like(kn), torch.zeros((R, Hq, D), dtype=torch.bfloat16, device="cuda")

    def step():
        lens, state, cu, slots, verdict = cp.cache_plan(s["lens"], delta, s["table"], s["ring"], s["state"], P, 4,
                                                        lens_out=s["lens"], free_state_out=s["state"])
        cp.cache_append_(kn, vn, slots, kc, vc, k_bounds=kb)
        pages = cp.select_pages(q, kb, s["table"], s["lens"], P, 2)
        return verdict, *cp.decode(q, kc, vc, s["table"], s["lens"]), *cp.decode(q, kc, vc, s["table"], s["lens"], pages=pages)

    keep = {k: x.clone() for k, x in s.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in ((s[k], keep[k]) for k in s):
        x.copy_(y)
    for x in (kc, vc, kb):
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        verdict, o, lse, o2, lse2 = step()
    g = torch.Generator().manual_seed(6)
    rows = [[], [], []]
    for i in range(30):
        x = torch.randn(2, 4, Hkv, D, generator=g).bfloat16()
        qq = torch.randn(R, Hq, D, generator=g).bfloat16()
        kn.copy_(x[0])
        vn.copy_(x[1])
        q.copy_(qq)
        graph.replay()
        assert cp.sync_status() == cp.OK and verdict.item() == 0
        rows[0].append(x[:, 0])
        rows[2] += [x[:, 1], x[:, 2]]
        assert s["lens"].tolist() == [i + 1, 0, 2 * i + 2]
        c = dict(q=qq, k=kc, v=vc, table=s["table"].cpu(), lens=s["lens"].cpu(), amax=None)
        ref = pu.reference(c, D ** -0.5)
        for r in (0, 2):  # the cache holds the rows in order
            got = paged.gather(pu.values(kc), c["table"][r], s["lens"][r].item(), 1)
            assert np.array_equal(got, np.stack([pu.values(y[0, 1]) for y in rows[r]]))
        pu.assert_decode(o, lse, ref, D, D ** -0.5, 64, "bf16", f"step {i}")
        if 2 * i + 2 <= 2 * P:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_streams_with_their_own_workspaces(cp):
    cs = [pu.make_cache([2000 + i, 90], 8, 2, 128, 64, "bf16", seed=30 + i) for i in range(2)]
    ds = [pu.on_gpu(c) for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            d = ds[i]
            got[i].append(cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], stream=streams[i]))
    torch.cuda.synchronize()
    assert cp.sync_status() == cp.OK
    for i in range(2):
        ref = pu.reference(cs[i], 128 ** -0.5)
        for o, lse in got[i]:
            pu.assert_decode(o, lse, ref, 128, 128 ** -0.5, 2001, "bf16")


def test_ordinary_calls_and_calls_through_ctypes_agree(cp, monkeypatch):
    c = pu.on_gpu(pu.make_cache([300, 0, 41], 6, 2, 64, 16, "e4m3", seed=40))
    g = torch.Generator().manual_seed(41)
    rows = torch.randn(5, 2, 64, generator=g).bfloat16().cuda()
    slots = torch.tensor([3, 4, -1, 20, 21], device="cuda")
    bounds = torch.randn(c["k"].shape[0], 2, 2, 64, generator=g).sort(2).values.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    s = _books(3, 4, 9)
    delta = torch.tensor([20, 0, 33], dtype=torch.int32, device="cuda")

    def all_four():
        k, v, b = c["k"].clone(), c["v"].clone(), bounds.clone()
        table, ring = s["table"].clone(), s["ring"].clone()
        out = list(cp.cache_plan(s["lens"], delta, table, ring, s["state"], 16, 60)) + [table, ring]
        cp.cache_append_(rows, rows, slots, k, v, k_bounds=b, kv_amax=c["amax"])
        pages = cp.select_pages(c["q"], b, c["table"], c["lens"], 16, 5, keep_first=1)
        out += [k, v, b, pages, *cp.decode(c["q"], k, v, c["table"], c["lens"], pages=pages, kv_amax=c["amax"], scale=0.2)]
        return out

    first = all_four()
    for name in ("cache_plan", "cache_append", "select_pages", "decode"):
        monkeypatch.setattr(cp._calls, name, lambda *a: None)
    second = all_four()
    assert cp.sync_status() == cp.OK
    assert len(first) == len(second) and all(torch.equal(x, y) for x, y in zip(first, second))


def test_ordinary_calls_raise_the_library_s_errors(cp):
    c = pu.on_gpu(pu.make_cache([30], 2, 1, 64, 16, "bf16", seed=42))
    args = (c["q"], c["k"], c["v"], c["table"], c["lens"])
    with pytest.raises(cp.CpattnError) as e:
        cp.decode(*args, scale=-1.0)
    assert e.value.status == cp.ERR_ARG
    with pytest.raises(cp.CpattnError) as e:  # a page of 24 rows
        cp.decode(c["q"], c["k"].new_zeros(2, 1, 24, 64), c["k"].new_zeros(2, 1, 24, 64), c["table"], c["lens"])
    assert e.value.status == cp.ERR_SHAPE
    x = torch.zeros(3 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    off = x[4:].view(3, 1, 64)  # 8 bytes behind an aligned address
    with pytest.raises(cp.CpattnError) as e:
        cp.cache_append_(off, off, torch.arange(3, device="cuda"), c["k"], c["v"])
    assert e.value.status == cp.ERR_ALIGN
    assert cp.sync_status() == cp.OK


def test_append_of_one_token_with_any_stride_of_the_token_axis(cp):
    k = torch.zeros((2, 3, 16, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    x = torch.randn(3, 64, 1, device="cuda").bfloat16().permute(2, 0, 1)
    assert x.stride(0) == 1
    cp.cache_append_(x, x, torch.tensor([19], device="cuda"), k, v)
    assert cp.sync_status() == cp.OK and torch.equal(k[1, :, 3], x[0])
    assert k.count_nonzero() == x.count_nonzero()


@pytest.mark.parametrize("heads", [4, 64])
def test_decode_wait_that_runs_out_is_reported_and_the_device_stays_usable(cp, heads):
    """One block's load is left out: its wait gives up after its limit, the call ends."""
    c = pu.make_cache([900, 70], heads, 2, 64, 32, "bf16", seed=43)
    assert cp.sync_status() == cp.OK
    cp.debug_stall(1)
    try:
        d = pu.on_gpu(c)
        cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"])
        st = cp.sync_status()
    finally:
        cp.debug_stall(0)
    assert st == cp.ERR_TIMEOUT, cp.status_str(st)
    o, lse = _decode(cp, c, 0.125)
    pu.assert_decode(o, lse, pu.reference(c, 0.125), 64, 0.125, 900, "bf16", "after it")


@pytest.mark.parametrize("kind,group", [("bf16", 2), ("e4m3", 20), ("fp32", 2)])
def test_decode_wait_that_runs_out_in_a_wide_table(cp, kind, group):
    c = pu.make_cache([900, 70], 2 * group, 2, 64, 32, kind, seed=45, width=2000)
    assert cp.sync_status() == cp.OK
    cp.debug_stall(1)
    try:
        d = pu.on_gpu(c)
        cp.decode(d["q"], d["k"], d["v"], d["table"], d["lens"], kv_amax=d["amax"])
        st = cp.sync_status()
    finally:
        cp.debug_stall(0)
    assert st == cp.ERR_TIMEOUT, cp.status_str(st)
    o, lse = _decode(cp, c, 0.125)
    pu.assert_decode(o, lse, pu.reference(c, 0.125), 64, 0.125, 900, kind, "after it")


@pytest.mark.parametrize("width", [8, 4000])
def test_decode_bad_pages_in_narrow_and_wide_tables(cp, width):
    c = pu.make_cache([100, 64], 2, 1, 64, 16, "bf16", seed=46, width=width)
    d = pu.on_gpu(c)
    bad = d["table"].clone()
    bad[0, 1], bad[1, 3] = c["k"].shape[0], -1
    o, lse = cp.decode(d["q"], d["k"], d["v"], bad, d["lens"], scale=0.1)
    assert cp.sync_status() == cp.ERR_PAGE and cp.sync_status() == cp.OK
    keep = [[[0, 2, 3, 4, 5, 6]], [[0, 1, 2]]]
    pu.assert_decode(o, lse, pu.reference(c, 0.1, keep), 64, 0.1, 100, "bf16")


def test_select_with_operands_below_the_normal_range(cp):
    pages, D = 100, 64
    g = torch.Generator().manual_seed(44)
    b = (torch.randn(pages, 1, 2, D, generator=g).sort(2).values).bfloat16()
    q = (torch.randn(1, 1, D, generator=g) * 1e-39).bfloat16()
    table = torch.arange(pages, dtype=torch.int32)[None]
    got = cp.select_pages(q.cuda(), b.cuda(), table.cuda(), torch.tensor([16 * pages], dtype=torch.int32, device="cuda"), 16, 9)
    bv = pu.values(b)
    want = paged.select(pu.values(q)[0], {(p, 0): (bv[p, 0, 0], bv[p, 0, 1]) for p in range(pages)}, table[0], 16 * pages, 16, 0, 9, 0)
    assert got.cpu().tolist()[0][0] == want


def test_first_calls_of_a_process_can_be_captured():
    """No call has gone before in the child: module loading and attributes fall into the capture."""
    code = (
        "import torch\n"
        "from long_sequence_context_b200 import cpattn as cp\n"
        "z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device='cuda')\n"
        "k, q = z(4, 1, 16, 64, t=torch.bfloat16), z(1, 2, 64, t=torch.bfloat16)\n"
        "b, lens, table, ring = z(4, 1, 2, 64, t=torch.bfloat16), z(1), z(1, 3), torch.arange(4, dtype=torch.int32, device='cuda')\n"
        "state, delta, x = torch.tensor([0, 4], dtype=torch.int32, device='cuda'), z(1) + 40, z(40, 1, 64, t=torch.bfloat16) + 1\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    n, _, cu, slots, verdict = cp.cache_plan(lens, delta, table, ring, state, 16, 40)\n"
        "    cp.cache_append_(x, x, slots, k, k, k_bounds=b)\n"
        "    pages = cp.select_pages(q, b, table, n, 16, 2)\n"
        "    o, lse = cp.decode(q, k, k, table, n, pages=pages)\n"
        "g.replay()\n"
        "cp.check_device_status()\n"
        "assert verdict.item() == 0 and n.item() == 40 and pages.tolist() == [[[0, 2]]], (verdict, n, pages)\n"
        "assert torch.all(o == 1) and abs(lse[0, 0].item() - __import__('math').log(24)) < 1e-6\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stdout + r.stderr
