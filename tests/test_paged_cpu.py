"""Refusals of the paged cache's entry points, on the CPU: the binding names the
wrong argument, the C ABI returns a status, and nothing is launched."""
import ctypes

import pytest
import torch

from long_sequence_context_b200 import cpattn as cp

N, R, HQ, HKV, D, P, PAGES, WIDTH = 5, 3, 4, 2, 64, 16, 7, 4


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _cache(dtype=torch.bfloat16):
    return torch.zeros((PAGES, HKV, P, D), dtype=dtype)


def _decode_args(dtype=torch.bfloat16):
    return dict(q=torch.zeros((R, HQ, D), dtype=torch.bfloat16), k_cache=_cache(dtype), v_cache=_cache(dtype),
                block_table=_i32(R, WIDTH), lens=_i32(R), pages=_i32(R, HKV, 2),
                out=torch.zeros((R, HQ, D), dtype=torch.bfloat16), lse=torch.zeros((R, HQ)))


def _plan_args():
    return dict(lens=_i32(R), delta=_i32(R), block_table=_i32(R, WIDTH), free_ring=_i32(PAGES), free_state=_i32(2),
                page_size=P, capacity=4, lens_out=_i32(R), free_state_out=_i32(2))


def _append_args(dtype=torch.bfloat16):
    return dict(k_new=torch.zeros((N, HKV, D), dtype=torch.bfloat16), v_new=torch.zeros((N, HKV, D), dtype=torch.bfloat16),
                slots=torch.zeros(N, dtype=torch.int64), k_cache=_cache(dtype), v_cache=_cache(dtype),
                k_bounds=torch.zeros((PAGES, HKV, 2, D), dtype=dtype))


def _select_args():
    return dict(q=torch.zeros((R, HQ, D), dtype=torch.bfloat16), k_bounds=torch.zeros((PAGES, HKV, 2, D), dtype=torch.bfloat16),
                block_table=_i32(R, WIDTH), lens=_i32(R), page_size=P, budget=2)


CALLS = [(cp.decode, _decode_args, ["q", "k_cache", "v_cache", "block_table", "lens", "pages", "out", "lse"]),
         (cp.cache_plan, _plan_args, ["lens", "delta", "free_ring", "free_state", "lens_out", "free_state_out"]),
         (cp.cache_append_, _append_args, ["k_new", "v_new", "slots", "v_cache", "k_bounds"]),
         (cp.select_pages, _select_args, ["q", "k_bounds", "lens"])]


@pytest.mark.parametrize("fn,args,name", [(f, a, n) for f, a, names in CALLS for n in names],
                         ids=[f"{f.__name__}-{n}" for f, _, names in CALLS for n in names])
def test_each_tensor_argument_is_checked(fn, args, name):
    n0 = cp.launch_count()
    for change in (lambda t: t.to(torch.float64), lambda t: torch.zeros((*t.shape, 2), dtype=t.dtype), lambda t: None):
        a = args()
        wrong = change(a[name])
        if wrong is None and name in ("pages", "out", "lse", "lens_out", "free_state_out", "k_bounds"):
            continue
        a[name] = wrong
        with pytest.raises((ValueError, TypeError)) as e:
            fn(**a)
        text = str(e.value)
        assert "CUDA tensor" not in text, text
        assert name in text or "dtype" in text, text
    assert cp.launch_count() == n0


@pytest.mark.parametrize("fn,args", [(f, a) for f, a, _ in CALLS], ids=[f.__name__ for f, _, _ in CALLS])
def test_with_everything_right_only_the_device_is_left_to_refuse(fn, args):
    with pytest.raises(ValueError, match="CUDA tensor"):
        fn(**args())


def test_shapes_that_do_not_belong_together():
    def refuse(fn, a, text, **change):
        a.update(change)
        with pytest.raises((ValueError, TypeError), match=text):
            fn(**a)

    refuse(cp.decode, _decode_args(), "not a multiple", q=torch.zeros((R, 5, D), dtype=torch.bfloat16), out=None, lse=None)
    refuse(cp.decode, _decode_args(), "q must have shape", q=torch.zeros((R, HQ, 128), dtype=torch.bfloat16))
    refuse(cp.decode, _decode_args(), "q must be", q=torch.zeros((R, HQ, D)))
    refuse(cp.decode, _decode_args(torch.uint8), "kv_amax must be given")
    refuse(cp.decode, _decode_args(), "kv_amax is for", kv_amax=torch.ones(2))
    refuse(cp.decode, _decode_args(torch.uint8), "kv_amax must have shape", kv_amax=torch.ones(3))
    refuse(cp.decode, _decode_args(), "contiguous", k_cache=_cache().transpose(0, 1).contiguous().transpose(0, 1))
    refuse(cp.decode, _decode_args(), "unsupported dtype", out_dtype=torch.float16, out=None)
    refuse(cp.decode, _decode_args(), "out must be", out_dtype=torch.float32)
    refuse(cp.decode, _decode_args(), "pages must have shape", pages=_i32(R, HKV + 1, 2))
    refuse(cp.cache_append_, _append_args(), "contiguous columns",
           k_new=torch.zeros((N, D, HKV), dtype=torch.bfloat16).transpose(1, 2))
    refuse(cp.cache_append_, _append_args(), "k_new must be", k_new=torch.zeros((N, HKV, D)))
    refuse(cp.select_pages, _select_args(), "budget", budget=0)
    refuse(cp.select_pages, _select_args(), "budget", budget=2, keep_first=2)
    refuse(cp.select_pages, _select_args(), "keep_first", keep_first=-1)


VP = ctypes.c_void_p(256)


def _c_decode(R=2, Hq=4, Hkv=2, D=128, P=64, width=8, pages=16, budget=0, scale=0.1, dtype=0, cache=0, out=0, ptr=VP,
              lists=None, amax=None, ws=VP, ws_bytes=1 << 40):
    return cp.lib.cpattn_decode(ptr, VP, VP, VP, VP, lists, VP, VP, R, Hq, Hkv, D, P, width, pages, budget, scale, amax, ws,
                                ws_bytes, dtype, cache, out, None)


def test_decode_status_codes():
    n0 = cp.launch_count()
    for kw in (dict(R=0), dict(Hq=5), dict(Hq=130, Hkv=2), dict(D=96), dict(P=8), dict(P=48), dict(P=512), dict(width=0),
               dict(pages=0), dict(width=1 << 25), dict(lists=VP, budget=0)):
        assert _c_decode(**kw) == cp.ERR_SHAPE, kw
    for kw in (dict(dtype=7), dict(cache=1), dict(dtype=1, cache=2), dict(dtype=1), dict(out=2), dict(cache=3)):
        assert _c_decode(**kw) == cp.ERR_DTYPE, kw
    for kw in (dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=-1.0), dict(ptr=None), dict(cache=2)):
        assert _c_decode(**kw) == cp.ERR_ARG, kw
    assert _c_decode(ptr=ctypes.c_void_p(264)) == cp.ERR_ALIGN
    assert _c_decode(ws=ctypes.c_void_p(16)) == cp.ERR_ALIGN
    need = cp.decode_workspace_bytes(2, 4, 2, 128)
    assert need > 0 and _c_decode(ws_bytes=need - 1) == cp.ERR_WORKSPACE and _c_decode(ws=None) == cp.ERR_WORKSPACE
    assert cp.decode_workspace_bytes(2, 5, 2, 128) == 0 and cp.decode_workspace_bytes(2, 4, 2, 100) == 0
    assert cp.launch_count() == n0


def test_select_status_codes():
    def call(R=2, Hq=4, Hkv=2, D=128, P=64, width=8, pages=16, budget=4, keep=1, dtype=0, cache=0, ptr=VP):
        return cp.lib.cpattn_select_pages(ptr, VP, VP, VP, VP, R, Hq, Hkv, D, P, width, pages, budget, keep, dtype, cache, None)

    for kw in (dict(R=0), dict(Hq=5), dict(Hq=130), dict(D=32), dict(P=24), dict(width=0), dict(width=49153), dict(budget=0),
               dict(budget=1), dict(keep=-1), dict(pages=0), dict(budget=2147483647, keep=2147483647)):
        assert call(**kw) == cp.ERR_SHAPE, kw
    assert call(dtype=3) == cp.ERR_DTYPE and call(dtype=1, cache=2) == cp.ERR_DTYPE
    assert call(ptr=None) == cp.ERR_ARG and call(ptr=ctypes.c_void_p(8)) == cp.ERR_ALIGN


def test_plan_status_codes():
    def call(R=2, width=8, P=64, pages=16, cap=4, ptr=VP, slots=VP, ws=VP, ws_bytes=1 << 30):
        return cp.lib.cpattn_cache_plan(ptr, VP, VP, R, width, P, VP, VP, pages, VP, VP, VP, slots, cap, VP, ws, ws_bytes, None)

    for kw in (dict(R=0), dict(width=0), dict(P=65), dict(pages=0), dict(cap=-1), dict(cap=1 << 31), dict(width=1 << 25)):
        assert call(**kw) == cp.ERR_SHAPE, kw
    assert call(ptr=None) == cp.ERR_ARG and call(slots=None) == cp.ERR_ARG
    assert call(ptr=ctypes.c_void_p(2)) == cp.ERR_ALIGN and call(slots=ctypes.c_void_p(4)) == cp.ERR_ALIGN
    need = cp.cache_plan_workspace_bytes(2, 5000)
    assert need > 0 and cp.cache_plan_workspace_bytes(0, 5000) == 0 and cp.cache_plan_workspace_bytes(2, 4) == 0
    assert call(cap=5000, ws=None) == cp.ERR_WORKSPACE and call(cap=5000, ws_bytes=need - 1) == cp.ERR_WORKSPACE
    assert call(ws=ctypes.c_void_p(8)) == cp.ERR_ALIGN


def test_append_status_codes():
    def call(st=(256, 128, 256, 128), N=4, Hkv=2, D=128, P=64, pages=16, dtype=0, cache=0, ptr=VP, slots=VP, amax=None):
        return cp.lib.cpattn_cache_append(ptr, VP, *st, slots, N, VP, VP, None, Hkv, D, P, pages, amax, dtype, cache, None)

    for kw in (dict(N=-1), dict(Hkv=0), dict(D=80), dict(P=1), dict(pages=0), dict(st=(255, 128, 256, 128)),
               dict(st=(256, 128, 256, -8)), dict(st=(256, 4, 256, 128)), dict(N=1 << 31)):
        assert call(**kw) == cp.ERR_SHAPE, kw
    assert call(N=0) == cp.OK
    assert call(cache=1) == cp.ERR_DTYPE and call(dtype=1, cache=2) == cp.ERR_DTYPE and call(dtype=2, cache=2) == cp.ERR_DTYPE
    assert call(ptr=None) == cp.ERR_ARG and call(cache=2) == cp.ERR_ARG
    assert call(ptr=ctypes.c_void_p(8)) == cp.ERR_ALIGN and call(slots=ctypes.c_void_p(4)) == cp.ERR_ALIGN


def test_status_string_of_a_page_error():
    assert "page" in cp.status_str(cp.ERR_PAGE)
