"""Refusals of the layer in parts, through the C ABI on the CPU: every bad argument is answered before a device is
touched.  Addresses are made up and never dereferenced."""
import ctypes

import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm

INVALID, NULL, MISALIGNED, WORKSPACE = -1, -2, -3, -4
NO_DEVICE = (-5, -6)
MB = 1 << 20


def _accepted(st):
    assert (st in NO_DEVICE) if not torch.cuda.is_available() else st == 0, st


cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses would be launched on")


# ------------------------------------------------------------------------------------ sort
def _sp(T=4, H=256, E=8, k=2, **kw):
    return mm.SortProblem.make(T, H, E, k, **kw)


def _sort(p, x=1 * MB, x_sf=None, idx=2 * MB, rows=3 * MB, rows_sf=None, src=4 * MB, pos=5 * MB, offset=6 * MB, ws=None,
          ws_bytes=0):
    return mm.library().mega_moe_sort_tokens(ctypes.byref(p), x, x_sf, idx, rows, rows_sf, src, pos, offset, ws, ws_bytes,
                                             None)


BAD_SORT = [dict(T=-1), dict(T=1 << 30), dict(T=1 << 29, k=2), dict(H=0), dict(H=100), dict(H=16512), dict(E=0),
            dict(E=8193), dict(k=0), dict(k=65), dict(dtype=3), dict(dtype=-1), dict(recipe=3), dict(flags=1),
            dict(x_stride=248), dict(x_stride=260), dict(x_stride=-256), dict(x_stride=1 << 40),
            dict(dtype=mm.DTYPE_F32, x_stride=258), dict(dtype=mm.DTYPE_E4M3, x_stride=264)]


@pytest.mark.parametrize("kw", BAD_SORT)
def test_sort_refuses_bad_problems(kw):
    assert _sort(_sp(**kw)) == INVALID
    with pytest.raises(mm.MegaMoEError) as e:
        mm.mega_moe_sort_workspace_size(_sp(**kw))
    assert e.value.status == INVALID


def test_sort_refuses_bad_pointers():
    for name in ("x", "idx", "rows", "src", "pos", "offset"):
        assert _sort(_sp(), **{name: None}) == NULL, name
    for name in ("x", "idx", "rows", "src", "pos", "offset", "ws"):
        assert _sort(_sp(), **{name: 8 * MB + 8}) == MISALIGNED, name
    e4 = _sp(dtype=mm.DTYPE_E4M3)
    assert _sort(e4) == NULL and _sort(e4, x_sf=7 * MB) == NULL and _sort(e4, rows_sf=7 * MB) == NULL
    assert _sort(_sp(), x_sf=7 * MB) == INVALID and _sort(_sp(), rows_sf=7 * MB) == INVALID    # scales of no 8-bit rows
    assert _sort(e4, x=None, rows=None, x_sf=7 * MB, rows_sf=8 * MB) == INVALID
    lib = mm.library()
    assert lib.mega_moe_sort_tokens(None, *[MB] * 9, 0, None) == NULL
    assert lib.mega_moe_sort_workspace_size(None, None) == NULL
    assert lib.mega_moe_sort_workspace_size(ctypes.byref(_sp()), None) == NULL
    assert _sort(_sp(T=0), offset=None) == NULL                            # the offsets are written even then


def test_sort_refuses_overlapping_buffers():
    assert _sort(_sp(), rows=1 * MB + 4 * 512 - 16) == INVALID              # on x
    assert _sort(_sp(), pos=2 * MB + 16) == INVALID                         # on the ids
    assert _sort(_sp(), offset=3 * MB + 8 * 512 - 16) == INVALID            # two outputs
    assert _sort(_sp(x_stride=512), rows=1 * MB + 3 * 1024) == INVALID      # the last of x's strided rows
    big = _sp(T=4096)
    need = mm.mega_moe_sort_workspace_size(big)
    at = dict(x=16 * MB, rows=64 * MB)
    assert _sort(big, **at, ws=2 * MB, ws_bytes=need) == INVALID            # the workspace on the ids


def test_sort_workspace():
    assert mm.mega_moe_sort_workspace_size(_sp(T=2048)) == 0                # 4096 pairs
    need = mm.mega_moe_sort_workspace_size(_sp(T=2049))
    assert need >= 5 * 8 * 4
    assert mm.mega_moe_sort_workspace_size(_sp(T=1 << 20, E=8192)) <= (1024 + 1) * 8192 * 4 + 512
    p, at = _sp(T=2049), dict(x=16 * MB, rows=64 * MB)
    assert _sort(p, **at, ws=8 * MB, ws_bytes=need - 1) == WORKSPACE
    assert _sort(p, **at, ws=None, ws_bytes=need) == WORKSPACE


@cpu_only
def test_sort_accepts():
    _accepted(_sort(_sp()))
    _accepted(_sort(_sp(x_stride=264)))
    _accepted(_sort(_sp(dtype=mm.DTYPE_E4M3, recipe=2, x_stride=272), x_sf=7 * MB, rows_sf=8 * MB))
    _accepted(_sort(_sp(), x=None, rows=None))
    _accepted(_sort(_sp(dtype=mm.DTYPE_E4M3), x=None, rows=None))
    _accepted(_sort(_sp(T=0), x=None, idx=None, rows=None, src=None, pos=None))
    p = _sp(T=2049)
    _accepted(_sort(p, x=16 * MB, rows=64 * MB, ws=8 * MB, ws_bytes=mm.mega_moe_sort_workspace_size(p)))


# ------------------------------------------------------------------------------------ back
def _up(T=4, H=256, k=2, **kw):
    return mm.UnsortProblem.make(T, H, k, **kw)


def _unsort(p, rows=1 * MB, pos=2 * MB, w=3 * MB, y=4 * MB):
    return mm.library().mega_moe_unsort_tokens(ctypes.byref(p), rows, pos, w, y, None)


def _back(p, dy=1 * MB, rows=2 * MB, pos=3 * MB, w=4 * MB, d_rows=5 * MB, d_w=6 * MB):
    return mm.library().mega_moe_unsort_backward(ctypes.byref(p), dy, rows, pos, w, d_rows, d_w, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 30), dict(T=1 << 29), dict(H=0), dict(H=200), dict(H=16512),
                                dict(k=0), dict(k=65), dict(dtype=2), dict(dtype=-1), dict(flags=1), dict(num_rows=-1),
                                dict(num_rows=(1 << 30) + 1), dict(stride=255), dict(stride=260), dict(stride=-256),
                                dict(stride=1 << 40), dict(dtype=1, stride=258)])
def test_back_refuses_bad_problems(kw):
    assert _unsort(_up(**kw)) == INVALID and _back(_up(**kw)) == INVALID


def test_back_refuses_bad_pointers():
    for name in ("rows", "pos", "y"):
        assert _unsort(_up(), **{name: None}) == NULL
    for name in ("rows", "pos", "w", "y"):
        assert _unsort(_up(), **{name: 8 * MB + 8}) == MISALIGNED
    for name in ("dy", "rows", "pos"):
        assert _back(_up(), **{name: None}) == NULL
    for name in ("dy", "rows", "pos", "w", "d_rows", "d_w"):
        assert _back(_up(), **{name: 8 * MB + 8}) == MISALIGNED
    assert _back(_up(), d_rows=None, d_w=None) == INVALID
    assert _unsort(_up(), y=1 * MB + 8 * 512 - 16) == INVALID
    assert _unsort(_up(num_rows=100), y=1 * MB + 100 * 512 - 16) == INVALID
    assert _back(_up(), d_rows=2 * MB + 16) == INVALID                      # not quite in place
    assert _back(_up(), d_w=4 * MB) == INVALID
    assert _back(_up(), d_w=5 * MB) == INVALID
    lib = mm.library()
    assert lib.mega_moe_unsort_tokens(None, MB, MB, MB, MB, None) == NULL
    assert lib.mega_moe_unsort_backward(None, *[MB] * 6, None) == NULL
    assert _unsort(_up(T=0), rows=None, pos=None, y=None) == 0 and _back(_up(T=0), dy=None, pos=None) == 0


@cpu_only
def test_back_accepts():
    _accepted(_unsort(_up(stride=264, num_rows=3), w=None))
    _accepted(_back(_up(), d_rows=2 * MB))                                  # in place over the rows
    _accepted(_back(_up(), rows=None, d_w=None))
    _accepted(_back(_up(dtype=1), w=None, d_rows=None))


# --------------------------------------------------------------------------------- product
def _pp(M=4, N=256, K=256, G=1, **kw):
    return mm.ProductProblem.make(M, N, K, G, **kw)


def _product(p, x=1 * MB, x_sf=2 * MB, w=3 * MB, w_sf=4 * MB, offset=5 * MB + 4, y=6 * MB):
    return mm.library().mega_moe_block_product(ctypes.byref(p), x, x_sf, w, w_sf, offset, y, None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(M=1 << 30), dict(N=0), dict(N=12), dict(N=(1 << 20) + 8), dict(K=0),
                                dict(K=192), dict(K=16512), dict(G=0), dict(G=8193), dict(flags=1), dict(x_stride=240),
                                dict(x_stride=264), dict(x_stride=-256), dict(x_stride=(1 << 22) + 16),
                                dict(y_stride=248), dict(y_stride=260), dict(y_stride=1 << 40)])
def test_product_refuses_bad_problems(kw):
    assert _product(_pp(**kw)) == INVALID


def test_product_refuses_bad_pointers():
    for name in ("x", "x_sf", "w", "w_sf", "y"):
        assert _product(_pp(), **{name: None}) == NULL
        assert _product(_pp(), **{name: 8 * MB + 8}) == MISALIGNED
    assert _product(_pp(G=2), offset=None) == NULL
    assert _product(_pp(), offset=5 * MB + 2) == MISALIGNED
    assert _product(_pp(), y=1 * MB + 4 * 256 - 16) == INVALID              # on x
    assert _product(_pp(G=2), y=3 * MB + 2 * 256 * 256 - 16) == INVALID     # on the last group's weights
    assert _product(_pp(), y=5 * MB) == INVALID                             # on the offsets
    assert _product(_pp(N=136), y=4 * MB + 2 * 2 * 4 - 16) == INVALID       # on the scales of a part of a block
    assert mm.library().mega_moe_block_product(None, *[MB] * 6, None) == NULL
    assert _product(_pp(M=0, G=2), x=None, x_sf=None, w=None, w_sf=None, offset=None, y=None) == 0


@cpu_only
def test_product_accepts():
    _accepted(_product(_pp()))
    _accepted(_product(_pp(N=8, x_stride=272, y_stride=16), offset=None))
    _accepted(_product(_pp(G=3, x_stride=1 << 22, M=1)))


# ------------------------------------------------------------------------------ activation
def _ap(M=4, I=256, **kw):
    return mm.ActProblem.make(M, I, **kw)


def _act(p, x=1 * MB, num_valid=2 * MB + 4, q=3 * MB, q_sf=4 * MB, out=5 * MB):
    return mm.library().mega_moe_act_quant(ctypes.byref(p), x, num_valid, q, q_sf, out, None)


def _act_back(p, x=1 * MB, d_out=2 * MB, num_valid=3 * MB + 4, d_x=4 * MB):
    return mm.library().mega_moe_act_backward(ctypes.byref(p), x, d_out, num_valid, d_x, None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(M=1 << 30), dict(I=0), dict(I=96), dict(I=16512), dict(act=2),
                                dict(act=-1), dict(recipe=3), dict(x_dtype=2), dict(swiglu_clamp=-1.0),
                                dict(swiglu_clamp=float("nan")), dict(flags=1), dict(flags=8), dict(x_stride=256),
                                dict(x_stride=516), dict(x_stride=1 << 40), dict(x_dtype=1, x_stride=514),
                                dict(act=0, swiglu_clamp=1.0), dict(act=0, flags=4), dict(act=0, x_stride=248)])
def test_activation_refuses_bad_problems(kw):
    assert _act(_ap(**kw)) == INVALID and _act_back(_ap(**kw)) == INVALID


def test_activation_refuses_bad_pointers():
    assert _act(_ap(), x=None) == NULL and _act(_ap(), q=None) == NULL and _act(_ap(), q_sf=None) == NULL
    assert _act(_ap(), q=None, q_sf=None, out=None) == INVALID
    for name in ("x", "q", "q_sf", "out"):
        assert _act(_ap(), **{name: 8 * MB + 8}) == MISALIGNED
    assert _act(_ap(), num_valid=2 * MB + 2) == MISALIGNED
    assert _act(_ap(), q=1 * MB + 4 * 1024 - 16) == INVALID and _act(_ap(), out=3 * MB) == INVALID
    assert _act(_ap(), q_sf=2 * MB) == INVALID                              # on num_valid
    for name in ("x", "d_out", "d_x"):
        assert _act_back(_ap(), **{name: None}) == NULL
        assert _act_back(_ap(), **{name: 8 * MB + 8}) == MISALIGNED
    assert _act_back(_ap(), num_valid=2) == MISALIGNED
    assert _act_back(_ap(), d_x=1 * MB + 16) == INVALID and _act_back(_ap(), d_x=2 * MB) == INVALID
    assert _act_back(_ap(act=0)) == INVALID
    lib = mm.library()
    assert lib.mega_moe_act_quant(None, *[MB] * 5, None) == NULL
    assert lib.mega_moe_act_backward(None, *[MB] * 4, None) == NULL
    assert _act(_ap(M=0), x=None, q=None, q_sf=None, out=None) == 0 and _act_back(_ap(M=0), x=None) == 0


@cpu_only
def test_activation_accepts():
    _accepted(_act(_ap(swiglu_clamp=float("inf"), flags=4, x_stride=520), num_valid=None))
    _accepted(_act(_ap(act=0, recipe=2, x_dtype=1, x_stride=260), out=None))
    _accepted(_act(_ap(), q=None, q_sf=None))
    _accepted(_act_back(_ap(swiglu_clamp=1.0), d_x=1 * MB))                 # in place over x
    _accepted(_act_back(_ap(x_dtype=1), num_valid=None))
