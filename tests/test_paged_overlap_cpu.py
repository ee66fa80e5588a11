"""cache_plan's blocks read while others write: memory that overlaps is refused by the C ABI, on the CPU."""
import ctypes
import itertools

import pytest

from long_sequence_context_b200 import cpattn as cp

R, WIDTH, PAGES, CAP = 6, 4, 32, 5000
WS = cp.cache_plan_workspace_bytes(R, CAP)
BYTES = dict(lens=4 * R, delta=4 * R, table=4 * R * WIDTH, ring=4 * PAGES, state=8, lens_out=4 * R, state_out=8,
             cu=4 * (R + 1), slots=8 * CAP, verdict=4, ws=WS)
WRITTEN = ["table", "ring", "lens_out", "state_out", "cu", "slots", "verdict", "ws"]


def _apart():
    at, out = 1 << 20, {}
    for name, n in BYTES.items():
        out[name] = at
        at += (n + 15) // 16 * 16
    return out


def _call(p):
    v = {n: ctypes.c_void_p(x) for n, x in p.items()}
    return cp.lib.cpattn_cache_plan(v["lens"], v["delta"], v["table"], R, WIDTH, 16, v["ring"], v["state"], PAGES,
                                    v["lens_out"], v["state_out"], v["cu"], v["slots"], CAP, v["verdict"], v["ws"], WS, None)


@pytest.fixture(autouse=True)
def nowhere(has_gpu):
    if has_gpu:
        pytest.skip("made-up addresses: only where no kernel can start")


@pytest.mark.parametrize("written", WRITTEN)
def test_what_is_written_may_not_overlap_anything_else(written):
    for other in BYTES:
        if other == written:
            continue
        step = 16 if "ws" in (written, other) else 8 if "slots" in (written, other) else 4
        for shift in {0, step, BYTES[other] - step, step - BYTES[written]}:
            p = _apart()
            at = p[other] + shift
            if at % step or not p[other] - BYTES[written] < at < p[other] + BYTES[other]:
                continue
            p[written] = at
            if shift == 0 and (written, other) in (("lens_out", "lens"), ("state_out", "state")):
                assert _call(p) == cp.ERR_CUDA  # in place: all checks passed, and no GPU is here
            else:
                assert _call(p) == cp.ERR_ARG, (written, other, shift)


def test_neighbours_and_updates_in_place_are_taken():
    assert _call(_apart()) == cp.ERR_CUDA
    p = _apart()
    p["lens_out"], p["state_out"] = p["lens"], p["state"]
    assert _call(p) == cp.ERR_CUDA
    names = ["lens_out", "state_out", "cu", "verdict"]
    for order in itertools.permutations(names):  # one behind another without a gap
        p, at = _apart(), 1 << 24
        for n in order:
            p[n] = at
            at += BYTES[n]
        assert _call(p) == cp.ERR_CUDA, order
