"""Refusals of the operators in front of the expert layer, through the C ABI on the CPU: every bad
argument is answered before a device is touched.  Addresses are made up and never dereferenced."""
import ctypes

import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm

INVALID, NULL, MISALIGNED = -1, -2, -3
NO_DEVICE = (-5, -6)
MB = 1 << 20


def _norm(p, x=1 * MB, residual=2 * MB, weight=3 * MB, residual_out=4 * MB, normed=5 * MB, q=6 * MB, q_sf=7 * MB):
    return mm.library().mega_moe_norm_quant(ctypes.byref(p), x, residual, weight, residual_out, normed, q, q_sf, None)


def _np(T=4, H=256, **kw):
    return mm.NormProblem.make(T, H, **kw)


def _accepted(st):
    assert (st in NO_DEVICE) if not torch.cuda.is_available() else st == 0, st


cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses would be launched on")


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 30), dict(H=0), dict(H=100), dict(H=16512), dict(recipe=3),
                                dict(recipe=-1), dict(x_dtype=2), dict(weight_dtype=-1), dict(eps=0.0),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(flags=1),
                                dict(x_stride=255), dict(x_stride=260), dict(x_stride=-256), dict(x_stride=1 << 40),
                                dict(residual_stride=128), dict(x_dtype=1, residual_stride=258)])
def test_norm_refuses_bad_problems(kw):
    assert _norm(_np(**kw)) == INVALID


def test_norm_refuses_bad_pointers():
    for name in ("x", "weight"):
        assert _norm(_np(), **{name: None}) == NULL
    assert _norm(_np(), q=None) == NULL and _norm(_np(), q_sf=None) == NULL
    assert _norm(_np(), normed=None, q=None, q_sf=None) == INVALID
    for name in ("x", "residual", "weight", "residual_out", "normed", "q", "q_sf"):
        assert _norm(_np(), **{name: 8 * MB + 8}) == MISALIGNED
    assert mm.library().mega_moe_norm_quant(None, *[MB] * 7, None) == NULL
    assert _norm(_np(T=0), x=None, weight=None, q=None) == 0


def test_norm_refuses_overlapping_buffers():
    n = 4 * 256 * 2
    assert _norm(_np(), normed=1 * MB + n - 16) == INVALID                  # on x
    assert _norm(_np(), q=3 * MB) == INVALID                                # on the weight
    assert _norm(_np(), q_sf=5 * MB + n - 16) == INVALID                    # two outputs
    assert _norm(_np(), residual_out=2 * MB + 16) == INVALID                # not quite in place
    assert _norm(_np(x_stride=512), residual_out=1 * MB) == INVALID         # in place over x with another stride


@cpu_only
def test_norm_accepts_in_place_and_partial_outputs():
    _accepted(_norm(_np(), residual_out=2 * MB))
    _accepted(_norm(_np(x_stride=512, residual_stride=512), residual_out=1 * MB))
    _accepted(_norm(_np(), residual=None, residual_out=None, normed=None))
    _accepted(_norm(_np(recipe=2, x_dtype=1, weight_dtype=1, x_stride=260), q=None, q_sf=None))


def _gate(p, x=1 * MB, w=2 * MB, logits=3 * MB):
    return mm.library().mega_moe_gate_logits(ctypes.byref(p), x, w, logits, None)


def _gp(T=4, H=256, E=8, **kw):
    return mm.GateProblem.make(T, H, E, **kw)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 30), dict(H=0), dict(H=200), dict(H=16512), dict(E=0),
                                dict(E=8193), dict(weight_dtype=2), dict(flags=1), dict(x_stride=248),
                                dict(x_stride=260), dict(x_stride=-8), dict(x_stride=(1 << 22) + 8)])
def test_gate_refuses_bad_problems(kw):
    assert _gate(_gp(**kw)) == INVALID


def test_gate_refuses_bad_pointers():
    for name in ("x", "w", "logits"):
        assert _gate(_gp(), **{name: None}) == NULL
        assert _gate(_gp(), **{name: 4 * MB + 4}) == MISALIGNED
    assert _gate(_gp(), logits=1 * MB + 16) == INVALID
    assert _gate(_gp(), logits=2 * MB + 8 * 256 * 2 - 16) == INVALID
    assert _gate(_gp(weight_dtype=1), logits=2 * MB + 8 * 256 * 4 - 16) == INVALID
    assert mm.library().mega_moe_gate_logits(None, MB, MB, MB, None) == NULL
    assert _gate(_gp(T=0), x=None, w=None, logits=None) == 0


@cpu_only
def test_gate_accepts():
    _accepted(_gate(_gp(E=3, x_stride=264)))
    _accepted(_gate(_gp(T=1, x_stride=1 << 22)))


def _topk(p, logits=1 * MB, bias=2 * MB, num_valid=3 * MB + 4, idx=4 * MB, w=5 * MB):
    return mm.library().mega_moe_gate_topk(ctypes.byref(p), logits, bias, num_valid, idx, w, None)


def _tp(T=4, E=16, k=4, **kw):
    return mm.TopkProblem.make(T, E, k, **kw)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=1 << 30), dict(T=1 << 28), dict(E=0), dict(E=8193),
                                dict(E=8192, num_shared=1), dict(k=0), dict(k=17), dict(E=256, k=65),
                                dict(E=256, k=60, num_shared=5), dict(num_shared=-1), dict(score=2), dict(score=-1),
                                dict(logits_dtype=2), dict(flags=2), dict(num_groups=0), dict(num_groups=3),
                                dict(num_groups=128, E=256), dict(num_groups=4, topk_groups=0),
                                dict(num_groups=4, topk_groups=5), dict(num_groups=8, topk_groups=1), dict(group_top=0),
                                dict(group_top=3), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(shared_weight=float("nan")), dict(logits_stride=15), dict(logits_stride=-16),
                                dict(logits_stride=1 << 40)])
def test_topk_refuses_bad_problems(kw):
    assert _topk(_tp(**kw)) == INVALID


def test_topk_refuses_bad_pointers():
    for name in ("logits", "idx", "w"):
        assert _topk(_tp(), **{name: None}) == NULL
    for name in ("logits", "bias", "idx", "w"):
        assert _topk(_tp(), **{name: 6 * MB + 4}) == MISALIGNED
    assert _topk(_tp(), num_valid=3 * MB + 2) == MISALIGNED
    assert _topk(_tp(), w=4 * MB + 48) == INVALID                 # the two outputs
    assert _topk(_tp(), idx=1 * MB) == INVALID                    # on the logits
    assert _topk(_tp(), w=2 * MB) == INVALID                      # on the bias
    assert _topk(_tp(), num_valid=5 * MB) == INVALID              # num_valid inside an output
    assert mm.library().mega_moe_gate_topk(None, *[MB] * 5, None) == NULL
    assert _topk(_tp(T=0), logits=None, idx=None, w=None) == 0


@cpu_only
def test_topk_accepts():
    _accepted(_topk(_tp(num_groups=8, topk_groups=2, group_top=2, num_shared=60, logits_stride=17), bias=None,
                    num_valid=None))


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        mm.mega_moe_norm_quant(_np(), x, x[0], normed=x)
    with pytest.raises(ValueError, match="device tensors"):
        mm.mega_moe_gate_logits(_gp(), x, x, x)
    with pytest.raises(ValueError, match="device tensors"):
        mm.mega_moe_gate_topk(_tp(), x, x, x)
    with pytest.raises(ValueError, match="must be a tensor"):
        mm.mega_moe_norm_quant(_np(), x, None, normed=x)
    with pytest.raises(ValueError, match="problem structure"):
        mm.mega_moe_norm_quant(_gp(), x, x[0], normed=x)
    with pytest.raises(ValueError, match="problem structure"):
        mm.mega_moe_gate_topk(None, x, x, x)
