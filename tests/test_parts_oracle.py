"""The float64 oracle of the layer in parts, pinned by hand-worked values, by torch and by differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import parts


def test_sort_plan_by_hand():
    # pairs 0..7: experts 2, 0 | -1, 2 | 5 (none), 0 | 1, 2
    offset, src, pos = parts.sort_plan(np.array([[2, 0], [-1, 2], [5, 0], [1, 2]]), 4)
    assert offset.tolist() == [0, 2, 3, 6, 6]
    assert src.tolist() == [1, 5, 6, 0, 3, 7]
    assert pos.tolist() == [[3, 0], [-1, 4], [-1, 1], [2, 5]]


def test_sort_plan_is_the_layers_dispatch():
    rng = np.random.default_rng(1)
    idx = rng.integers(-1, 12, size=(50, 3)).astype(np.int32)
    offset, src, pos = parts.sort_plan(idx, 11)
    d = oracle.route(idx, 11)
    assert np.array_equal(offset, d["offset"]) and np.array_equal(pos.reshape(-1), d["pos"])
    assert np.array_equal(src, d["src"][:len(src)])


def test_back_and_its_gradient_against_autograd():
    rng = np.random.default_rng(2)
    idx = rng.integers(-1, 6, size=(20, 4)).astype(np.int32)
    offset, src, pos = parts.sort_plan(idx, 6)
    rows, w, dy = rng.standard_normal((80, 8)), rng.standard_normal((20, 4)), rng.standard_normal((20, 8))
    r, tw = torch.tensor(rows, requires_grad=True), torch.tensor(w, requires_grad=True)
    used = torch.tensor(pos >= 0)[..., None]
    y = (torch.where(used, r[torch.tensor(pos).long().clamp_min(0)], 0.0) * tw[..., None]).sum(1)
    y.backward(torch.tensor(dy))
    got, _ = parts.unsort(rows, pos, w)
    d_rows, d_w, _ = parts.unsort_backward(dy, rows, pos, w)
    n = int(offset[-1])
    assert np.allclose(got, y.detach().numpy(), atol=1e-12)
    assert np.allclose(d_rows[:n], r.grad.numpy()[:n], atol=1e-12) and np.isnan(d_rows[n:]).all()
    assert np.allclose(d_w, tw.grad.numpy(), atol=1e-12)


def test_gradient_of_the_sort_is_the_unweighted_way_back():
    """<d, sort(x)> differentiated by x along a direction."""
    rng = np.random.default_rng(3)
    idx = rng.integers(-1, 5, size=(9, 3)).astype(np.int32)
    offset, src, pos = parts.sort_plan(idx, 5)
    x, v, d = rng.standard_normal((9, 4)), rng.standard_normal((9, 4)), rng.standard_normal((27, 4))
    n = len(src)
    f = lambda z: (z[src // 3] * d[:n]).sum()                              # noqa: E731
    h = 1e-6
    assert abs((f(x + h * v) - f(x - h * v)) / (2 * h) - (parts.unsort(d, pos)[0] * v).sum()) < 1e-7


def test_block_product_of_powers_of_two_by_hand():
    # one block: codes 0x38 = 1, 0x40 = 2; scales move the result by their product
    x = np.zeros((3, 256), dtype=np.uint8)
    w = np.zeros((2, 8, 256), dtype=np.uint8)
    x[:, 0], x[:, 200] = 0x38, 0x40
    w[0, 5, 0], w[1, 5, 200] = 0x40, 0x40
    x_sf = np.array([[1.0, 8.0], [0.5, 4.0], [2.0, 1.0]])
    y, mag = parts.block_product(x, x_sf, w, np.array([[[3.0, 1.0]], [[1.0, 0.25]]]), np.array([0, 1, 2]))
    assert y[0, 5] == 1 * 2 * 3 and y[1, 5] == 2 * 2 * 4 * 0.25 and np.isnan(y[2]).all()
    assert np.array_equal(np.delete(y[:2], 5, axis=1), np.zeros((2, 7))) and mag[1, 5] == 4


@pytest.mark.parametrize("clamp,inputs", [(0.0, False), (0.7, False), (0.7, True)])
def test_activation_and_its_gradient_against_differences(clamp, inputs):
    rng = np.random.default_rng(4)
    x, d, v = (rng.standard_normal(s) * 1.5 for s in ((6, 256), (6, 128), (6, 256)))
    h = 1e-7
    f = lambda z: parts.activation(z, clamp=clamp, inputs=inputs)          # noqa: E731
    want = ((f(x + h * v) - f(x - h * v)) / (2 * h) * d).sum()
    got = (parts.act_backward(x, d, clamp, inputs)[0] * v).sum()
    assert abs(got - want) < 1e-5 * max(1.0, abs(want))
    g, u = torch.tensor(x).chunk(2, dim=1)
    if clamp and inputs:
        g, u = g.clamp(-clamp, clamp), u.clamp(-clamp, clamp)
    ref = torch.nn.functional.silu(g) * u
    assert np.allclose(f(x), (ref.clamp(-clamp, clamp) if clamp and not inputs else ref).numpy(), atol=1e-12)


def test_scales_are_the_smallest_that_hold_the_group():
    v = np.zeros((1, 128))
    v[0, :4], v[0, 40] = [1, -448, 3, 0], 448.0000001
    sf, code = parts.scales(v, 1)
    assert code.tolist() == [[127, 128, 0, 0]] and sf[0, :2].tolist() == [1.0, 2.0]
    assert parts.scales(v, 0)[0][0, 0] == 448.0000001 / 448
