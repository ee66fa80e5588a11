"""The paged key-value cache on the GPU at the edges of what its calls allow."""
import numpy as np
import pytest
import torch

from oracle import paged
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
