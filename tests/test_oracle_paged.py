"""The paged cache's oracle against independent statements: full attention's last
row, invariants of the books, and a selection that covers everything."""
import numpy as np
import torch

from oracle import oracle as orc
from oracle import paged
from tests import paged_util as pu


def test_decode_is_the_last_row_of_causal_attention():
    n, H, D, P = 37, 2, 64, 16
    c = pu.make_cache([n], H, H, D, P, "fp32", 1)
    k = np.stack([paged.gather(pu.values(c["k"]), c["table"][0], n, h) for h in range(H)])
    v = np.stack([paged.gather(pu.values(c["v"]), c["table"][0], n, h) for h in range(H)])
    q = np.zeros((1, H, n, D))
    q[0, :, -1] = pu.values(c["q"])[0]
    o, lse = orc.attn_fwd(q, k[None], v[None], True, D ** -0.5)
    ro, rl, _, _ = pu.reference(c, D ** -0.5)
    assert np.abs(ro[0] - o[0, :, -1]).max() < 1e-12 and np.abs(rl[0] - lse[0, :, -1]).max() < 1e-12


def test_decode_matches_torch_attention_with_shared_heads():
    c = pu.make_cache([50, 0, 1], 6, 2, 64, 16, "fp32", 2)
    ro, rl, _, _ = pu.reference(c, 0.2)
    assert np.all(ro[1] == 0) and np.all(np.isneginf(rl[1]))
    for r in (0, 2):
        n = int(c["lens"][r])
        for i in range(6):
            k, v = (torch.from_numpy(paged.gather(pu.values(c[x]), c["table"][r], n, i // 3)) for x in ("k", "v"))
            w = torch.softmax(0.2 * (k @ c["q"][r, i].double()), 0)
            assert np.abs((w @ v).numpy() - ro[r, i]).max() < 1e-12


def test_plan_keeps_every_page_owned_once():
    g = np.random.default_rng(3)
    R, width, P, num_pages = 5, 6, 16, 20
    lens, table = [0] * R, np.full((R, width), -1)
    ring, state = list(range(num_pages)), [7, num_pages]
    for _ in range(60):
        delta = [int(g.integers(-n, min(40, width * P - n) + 1)) for n in lens]
        out = paged.plan(lens, delta, table, ring, state, P, 400)
        if out[6]:
            assert out[6] == paged.SHORT and out[0] == lens and list(out[3]) == state
        lens, table, ring, state = out[:4]
        owned = [int(table[r, j]) for r in range(R) for j in range(paged.pages_of(lens[r], P))]
        free = [ring[(state[0] + i) % num_pages] for i in range(state[1])]
        assert sorted(owned + free) == list(range(num_pages))
        slots = [s for s in out[5] if s >= 0]
        assert len(set(slots)) == len(slots) == out[4][-1]


def test_selection_lists_every_page_within_the_budget_and_breaks_ties_low():
    c = pu.make_cache([70], 2, 1, 64, 16, "fp32", 4)
    b = paged.bounds(pu.values(c["k"]), c["table"].numpy(), [70])
    q = pu.values(c["q"])[0]
    assert paged.select(q, b, c["table"][0], 70, 16, 0, 5, 0) == [0, 1, 2, 3, 4]
    assert paged.select(0 * q, b, c["table"][0], 70, 16, 0, 3, 0) == [0, 1, 4]
    assert paged.select(0 * q, b, c["table"][0], 70, 16, 0, 7, 0) == [0, 1, 2, 3, 4, -1, -1]
    # a bound is never below a key's own product
    for (p, h), (lo, hi) in b.items():
        j = [int(x) for x in c["table"][0][:5]].index(p)
        rows = pu.values(c["k"])[p, 0, :min(16, 70 - 16 * j)]
        assert paged.scores(q, lo, hi) >= (rows @ q.T).max() - 1e-12


def test_plan_refuses_a_length_above_its_table():
    table, ring = np.array([[0, 1], [2, 3]]), [4, 5, 6, 7]
    for lens, delta in [([32, 70], [0, -70]), ([33, 5], [-33, 0]), ([32, 2 ** 31 - 1], [0, -(2 ** 31 - 33)])]:
        out = paged.plan(lens, delta, table, ring, [0, 2], 16, 4)
        assert out[6] == paged.BAD_LENGTH and out[0] == lens and out[2] == ring and np.array_equal(out[1], table)
    assert paged.plan([32, 32], [0, -32], table, ring + [0] * 4, [0, 2], 16, 4)[6] == 0


def test_scores_beside_infinite_and_nan_bounds():
    inf, nan = np.inf, np.nan
    lo, hi = np.array([-inf, -1.0, 0.5]), np.array([2.0, 1.0, 0.75])
    assert paged.scores(np.array([[1.0, 1.0, 1.0]]), lo, hi) == 3.75
    assert paged.scores(np.array([[0.0, 1.0, 1.0]]), lo, hi) == 1.75
    assert paged.scores(np.array([[-1.0, 1.0, 1.0]]), lo, hi) == inf
    bad = np.array([nan, 1.0, 1.0])
    assert np.isnan(paged.scores(np.array([[0.0, 1.0, 1.0]]), lo, bad))
    # a NaN page ranks behind one of -inf, and an infinite score does not take a forced page's place
    bounds = {(0, 0): (np.array([-inf]), np.array([-inf])), (1, 0): (np.array([nan]), np.array([nan])),
              (2, 0): (np.array([inf]), np.array([inf])), (3, 0): (np.array([0.0]), np.array([0.0]))}
    one = np.array([[1.0]])
    assert paged.select(one, bounds, [1, 0, 2, 3], 64, 16, 0, 3, 0) == [1, 2, 3]
    assert paged.select(one, bounds, [2, 1, 0, 3], 64, 16, 0, 1, 0) == [3]
