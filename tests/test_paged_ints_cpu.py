"""Sizes that do not fit into the C ABI's int are refused on the CPU: their low bits are other sizes."""
import pytest
import torch

from long_sequence_context_b200 import cpattn as cp
from tests.test_paged_cpu import P, _decode_args, _plan_args, _select_args


@pytest.mark.parametrize("fn,args,name,good", [(cp.cache_plan, _plan_args, "page_size", P), (cp.cache_plan, _plan_args, "capacity", 4),
                                               (cp.select_pages, _select_args, "page_size", P),
                                               (cp.select_pages, _select_args, "budget", 2),
                                               (cp.select_pages, _select_args, "keep_first", 0)])
def test_whole_numbers_are_not_cut_to_their_low_bits(fn, args, name, good):
    n0 = cp.launch_count()
    for high in (1 << 32, 1 << 64, -(1 << 32), 1 << 31):
        with pytest.raises(ValueError, match=f"{name} is out of range"):
            fn(**{**args(), name: good + high})
    for wrong in (float(good), str(good), torch.tensor(good)):
        with pytest.raises(TypeError, match=f"{name} must be an int"):
            fn(**{**args(), name: wrong})
    assert cp.launch_count() == n0


def test_sizes_asked_of_the_workspaces():
    assert cp.decode_workspace_bytes(2, 4, 2, 128) > 0
    for bad in ((2 + (1 << 32), 4, 2, 128), (2, 4 + (1 << 32), 2, 128), (2, 4, 2, 128 + (1 << 32))):
        with pytest.raises(ValueError, match="out of range"):
            cp.decode_workspace_bytes(*bad)
    with pytest.raises(ValueError, match="out of range"):
        cp.cache_plan_workspace_bytes(2 + (1 << 32), 5000)


def test_sizes_of_tensors_are_held_to_the_same_limits():
    cp._ints(R=0, Hq=(1 << 31) - 1)
    with pytest.raises(ValueError, match="num_pages"):
        cp._ints(R=3, num_pages=1 << 31)


def test_an_empty_list_of_pages_is_not_every_page():
    a = _decode_args()
    a["pages"] = torch.zeros((a["q"].shape[0], a["k_cache"].shape[1], 0), dtype=torch.int32)
    with pytest.raises(ValueError, match="pages must have room"):
        cp.decode(**a)
