"""How exact the activation and its gradient are in float32, on an MI355X, over the whole range of gates.

In half steps, 2^-24 of a value: exp(-|g|) is the hardware's power of two, good to one unit in the last place (2), and the
part of its argument that the first one leaves out, a multiply-add (1) or an argument rounded to 2^-26 (0.2): 3.  For g < 0,
s = e / (1 + e) moves by 1 / (1 + e) of e's error at most: 3, and the sum, the reciprocal with a step of Newton (1.1) and the
product e r: 6.1; for g >= 0, s = r: half of e's error and two roundings.  v = g s u: 8.1.  The scale v / 448 is a division more:
9.1, asserted 10.  d_u is v with d for u: 8.1, asserted 9.  d_g = (d u) s (1 + g rest): 1 + 6.1 + 1, the bracket, relative
to 1 + |g rest|, rest's 6.1 and one rounding, a product: 16.2, asserted 18.  Beyond |g| 86 a factor is multiplied by a power of
two first, which is exact, or the result is below 2^-119 and off by less than 2^-141.
"""
import numpy as np
import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm
from oracle import parts

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24
GATES = np.concatenate([np.linspace(-103, -87, 4001), np.linspace(-87, 87, 60001), np.linspace(-3, 3, 20001),
                        [1e-30, -1e-30, 1e-6, -1e-6, 120.0, 3e38]]).astype(np.float32)
GATES = GATES[GATES != 0]


def _f64(t):
    return t.double().cpu().numpy()


def _say(*a):
    print("[precision]", *a, flush=True)


def _pairs(seed):
    """Every gate with an `up` of any sign and some size; larger where silu(g) is tiny, so that the product is not."""
    rng = np.random.default_rng(seed)
    u = (rng.uniform(0.5, 2.0, GATES.size) * np.where(rng.random(GATES.size) < 0.5, 1, -1)).astype(np.float32)
    u = np.where(GATES < -60, u * np.float32(1e30), u)
    return GATES, np.where(GATES > 1e30, np.sign(u) * 0.5, u).astype(np.float32)


def test_values_are_within_ten_half_steps():
    """One value a group of 128: its float scale is that value / 448."""
    g, u = _pairs(1)
    n, I = g.size, 128
    x = torch.zeros(n, 2 * I, device="cuda")
    x[:, 3], x[:, I + 3] = torch.from_numpy(g).cuda(), torch.from_numpy(u).cuda()
    q, q_sf = torch.zeros(n, I, dtype=torch.uint8, device="cuda"), torch.zeros(n, 1, device="cuda")
    mm.mega_moe_act_quant(mm.ActProblem.make(n, I, x_dtype=mm.DTYPE_F32), x, q, q_sf)
    with np.errstate(over="ignore"):
        v = np.abs(g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64))) * u)
    got = _f64(q_sf)[:, 0] * 448
    off = np.abs(got - v) / v / HALF
    _say("values: worst", off.max(), "half steps at g", g[off.argmax()], "rms", np.sqrt((off ** 2).mean()))
    assert off.max() <= 10


def test_gradients_are_within_their_half_steps():
    g, u = _pairs(2)
    n = g.size // 128 * 128
    g, u = g[-n:], u[-n:]
    d = np.random.default_rng(3).uniform(0.5, 2.0, n).astype(np.float32)
    d = np.where(g < -60, d * np.float32(1e7), d).astype(np.float32)
    x = torch.from_numpy(np.concatenate([g.reshape(-1, 128), u.reshape(-1, 128)], axis=1)).cuda()
    dt = torch.from_numpy(d.reshape(-1, 128)).cuda()
    d_x = torch.empty_like(x)
    mm.mega_moe_act_backward(mm.ActProblem.make(n // 128, 128, x_dtype=mm.DTYPE_F32), x, dt, d_x)
    ref, mag = parts.act_backward(_f64(x), _f64(dt))
    got = _f64(d_x)
    tiny = 2.0 ** -141
    off_g = np.maximum(np.abs(got - ref)[:, :128] - tiny, 0) / mag[:, :128] / HALF
    off_u = np.maximum(np.abs(got - ref)[:, 128:] - tiny, 0) / np.abs(ref[:, 128:]) / HALF
    for name, off in (("d_g", off_g), ("d_u", off_u)):
        at = np.unravel_index(off.argmax(), off.shape)
        _say(name, "worst", off.max(), "half steps at g", g.reshape(-1, 128)[at], "rms", np.sqrt((off ** 2).mean()))
    assert off_u.max() <= 9 and off_g.max() <= 18


@pytest.mark.parametrize("clamp", [0.0, 4.0])
def test_gates_below_the_normal_exponentials(clamp):
    """g below -87.3 and `up` so large that silu(g) up is an ordinary number: values, codes and what the clamp drops."""
    rng = np.random.default_rng(4)
    M, I = 16, 512
    g = rng.uniform(-102, -87.4, (M, I)).astype(np.float32)
    silu = g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64)))
    v = np.exp(rng.uniform(-3, 3, (M, I)))
    u = np.minimum(-v / silu, 3e38).astype(np.float32)
    x = torch.from_numpy(np.concatenate([g, u], axis=1)).cuda()
    v = np.clip(silu * u, -clamp, clamp) if clamp else silu * u
    q, q_sf = torch.zeros(M, I, dtype=torch.uint8, device="cuda"), torch.zeros(M, I // 32, dtype=torch.uint8, device="cuda")
    out = torch.zeros(M, I, dtype=torch.bfloat16, device="cuda")
    p = mm.ActProblem.make(M, I, recipe=2, x_dtype=mm.DTYPE_F32, swiglu_clamp=clamp)
    mm.mega_moe_act_quant(p, x, q, q_sf, out)
    assert np.array_equal(q_sf.cpu().numpy(), parts.scales(v, 2)[1])
    assert (np.abs(_f64(out) - v) <= (2.0 ** -8 + 10 * HALF) * np.abs(v)).all()
    d = torch.ones(M, I, device="cuda")
    d_x = torch.empty_like(x)
    mm.mega_moe_act_backward(p, x, d, d_x)
    ref, mag = parts.act_backward(_f64(x), _f64(d), clamp)
    got = _f64(d_x)
    assert np.array_equal(got[:, :I] == 0, ref[:, :I] == 0)
    assert (np.abs(got - ref)[:, :I] <= 19 * HALF * mag[:, :I]).all()
