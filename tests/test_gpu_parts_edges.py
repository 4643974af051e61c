"""Values of the layer in parts that few batches hold, on an MI355X: gradients where the clamp drops a value that is not
finite, and rows of every width.
"""
import numpy as np
import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm
from oracle import parts

pytestmark = pytest.mark.gpu

DT = {"bf16": (mm.DTYPE_BF16, torch.bfloat16), "f32": (mm.DTYPE_F32, torch.float32)}
INF = float("inf")


def _say(*a):
    print("[edges]", *a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _backward(x, d, clamp=0.0, inputs=False):
    kind = mm.DTYPE_BF16 if x.dtype == torch.bfloat16 else mm.DTYPE_F32
    d_x = torch.full_like(x, 7.0)
    p = mm.ActProblem.make(x.shape[0], x.shape[1] // 2, x_dtype=kind, swiglu_clamp=clamp,
                           flags=mm.FLAG_CLAMP_INPUTS if inputs else 0)
    mm.mega_moe_act_backward(p, x, d, d_x)
    return d_x


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradients_of_what_the_clamp_drops_are_zero(kind):
    """silu(g) u outside [-c, c]: both gradients are 0, whatever g, u and d are; a neighbour's are what they were."""
    _say("dropped", kind)
    I, c = 128, 2.0
    pairs = [(INF, 1.0), (INF, -1.0), (1.0, INF), (3.0, -INF), (-1.0, INF), (INF, INF), (INF, -INF), (1e3, 1e38), (5.0, 5.0)]
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(2, 2 * I, generator=g) * 0.5).to(DT[kind][1]).cuda()
    d = torch.randn(2, I, generator=g).to(DT[kind][1]).cuda()
    ref = _backward(x, d, c)
    for i, (gate, up) in enumerate(pairs):
        x[0, 3 * i], x[0, I + 3 * i] = gate, up
    x[1, 7], x[1, I + 7], d[1, 7] = 9.0, 9.0, INF
    got = _backward(x, d, c)
    at = [3 * i for i in range(len(pairs))]
    assert (got[0, at] == 0).all() and (got[0, [I + i for i in at]] == 0).all()
    assert got[1, 7] == 0 and got[1, I + 7] == 0
    same = torch.ones_like(got, dtype=torch.bool)
    same[0, at], same[0, [I + i for i in at]], same[1, [7, I + 7]] = False, False, False
    assert torch.equal(got[same], ref[same])
    with np.errstate(invalid="ignore"):
        want, _ = parts.act_backward(_f64(x), _f64(d), c)
    assert (want[0, at] == 0).all() and np.isfinite(want).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradients_of_clamped_inputs_that_are_not_finite(kind):
    """Each input outside its clamp has the gradient 0, the other one the clamped input's."""
    _say("inputs", kind)
    I, c = 128, 2.0
    x = torch.ones(1, 2 * I, dtype=DT[kind][1], device="cuda")
    d = torch.ones(1, I, dtype=DT[kind][1], device="cuda")
    for i, (gate, up) in enumerate([(INF, 1.0), (-INF, 1.0), (1.0, INF), (1.0, -INF), (INF, -INF)]):
        x[0, i], x[0, I + i] = gate, up
    got = _backward(x, d, c, True)
    capped = x.clamp(-c, c)
    ref = _backward(capped, d)                                      # within the clamp there is none
    outside = x.abs() > c
    assert (got[outside] == 0).all() and torch.equal(got[~outside], ref[~outside])


def _copied(M, I):
    x = torch.randn(M, I, device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(x)
    mm.mega_moe_act_quant(mm.ActProblem.make(M, I, mm.ACT_NONE), x, out=out)
    return torch.equal(out.view(torch.int16), x.view(torch.int16))


def test_every_width_finds_its_rows():
    """Without an activation the BF16 output is the input: each piece of eight columns has to find its row and place."""
    assert [j for j in range(1, 129) if not _copied(67, 128 * j)] == []


@pytest.mark.parametrize("M,I", [(3000001, 128), (1400003, 384), (70001, 128 * 127), (524309, 128 * 13)])
def test_many_rows_of_a_width_find_theirs(M, I):
    _say("rows", M, I)
    assert _copied(M, I)


@pytest.mark.parametrize("clamp", [3.4028234663852886e38, 2.0 ** -120, 2.0 ** -126, 2.0 ** -134])
def test_gradients_next_to_clamps_at_either_end_of_float32(clamp):
    """silu(g) u within float32 steps of a clamp near the largest and the smallest numbers, where the float32 product
    overflows or has few bits left: kept or dropped as the float64 value says."""
    _say("clamp", clamp)
    M, I = 32, 1024
    rng = np.random.default_rng(5)
    g = np.where(rng.random((M, I)) < 0.5, rng.uniform(0.2, 6, (M, I)), rng.uniform(-12, -3, (M, I))).astype(np.float32)
    g64 = g.astype(np.float64)
    if clamp < 1:
        g = np.where(rng.random((M, I)) < 0.5, g, rng.uniform(-100, -87, (M, I)).astype(np.float32))
        g64 = g.astype(np.float64)
    else:
        g = np.abs(g) + np.float32(2)                                # silu(g) above 1: `up` is a float32 number
        g64 = g.astype(np.float64)
    silu = g64 / (1 + np.exp(-g64))
    u = (clamp / silu).astype(np.float32)
    for _ in range(3):
        u = np.where(rng.random((M, I)) < 0.5, np.nextafter(u, np.copysign(np.float32(np.inf), u)), np.nextafter(u, np.float32(0)))
    assert np.isfinite(u).all()
    x = torch.from_numpy(np.concatenate([g, u], axis=1)).cuda()
    d = torch.full((M, I), 1e8 if clamp < 1 else 1e-8, device="cuda")
    got = _f64(_backward(x, d, clamp))
    outside = np.abs(silu * u.astype(np.float64)) > clamp
    assert outside.any() and not outside.all()
    assert np.array_equal(got[:, I:] == 0, outside)
