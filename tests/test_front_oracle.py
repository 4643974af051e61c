"""The float64 oracle of the operators in front of the expert layer, against values worked by hand."""
import numpy as np

from oracle import front


def test_norm_quant_by_hand():
    # 128 columns of +-3 with residual 1: h = 4 or -2, mean square = (16 + 4) / 2 = 10
    x = np.where(np.arange(128) % 2 == 0, 3.0, -3.0)[None]
    r = front.norm_quant(x, np.ones((1, 128)), np.full(128, 2.0), 0.0, 0)
    assert np.array_equal(r["h"][0, :2], [4.0, -2.0])
    assert np.allclose(r["v"][0, :2], [8 / np.sqrt(10), -4 / np.sqrt(10)], rtol=1e-15)
    assert np.allclose(r["sf"], 8 / np.sqrt(10) / 448, rtol=1e-15)
    assert np.allclose(r["scaled"][0, :2], [448.0, -224.0], rtol=1e-14)


def test_norm_quant_power_of_two_scales():
    x = np.zeros((1, 128))
    x[0, :4] = 1.0                                # mean square 1/32, v = sqrt(32) = 5.657 times the weight
    w = np.ones(128)
    r = front.norm_quant(x, None, w, 0.0, 1)
    assert r["code"][0].tolist() == [127 - 6, 0, 0, 0]           # 5.657/448 = 0.0126 in (2^-7, 2^-6]
    x = np.full((1, 128), 2.0)                    # v = weight exactly; 7/448 = 2^-6 exactly
    r = front.norm_quant(x, None, np.full(128, 7.0), 0.0, 1)
    assert r["code"][0].tolist() == [121] * 4
    r = front.norm_quant(x, None, np.full(128, np.nextafter(7.0, 8.0)), 0.0, 1)
    assert r["code"][0].tolist() == [122] * 4


def test_topk_groups_bias_and_ties():
    l = np.array([[0.0, 1.0, 1.0, -1.0, 2.0, -np.inf, np.nan, 0.0]])
    idx, w = front.gate_topk(l, None, 3, score="sigmoid")
    assert idx.tolist() == [[4, 1, 2]]                           # equal logits: the lower id first
    assert np.allclose(w[0], 1 / (1 + np.exp(-np.array([2.0, 1.0, 1.0]))))
    # groups of two: best experts 1.0, 1.0, 2.0, 0.0 -> groups 2 and 0
    idx, _ = front.gate_topk(l, None, 3, score="sigmoid", num_groups=4, topk_groups=2)
    assert idx.tolist() == [[4, 1, 0]]
    # a bias moves the order and not the weights
    bias = np.array([0.9, 0, 0, 0, -5.0, 0, 0, 0.0])
    idx, w = front.gate_topk(l, bias, 2, score="sigmoid", renorm=True, scale=2.0)
    assert idx.tolist() == [[0, 1]]
    s = 1 / (1 + np.exp(-np.array([0.0, 1.0])))
    assert np.allclose(w[0], 2 * s / s.sum())


def test_topk_too_few_candidates_shared_and_padding():
    l = np.full((3, 4), -np.inf)
    l[0, 2] = 0.5
    idx, w = front.gate_topk(l, None, 2, num_shared=1, shared_weight=0.5, num_valid=2, renorm=True)
    assert idx.tolist() == [[2, -1, 4], [-1, -1, 4], [-1, -1, -1]]
    assert np.allclose(w, [[1, 0, 0.5], [0, 0, 0.5], [0, 0, 0]])


def test_topk_infinite_logits_share_the_softmax():
    idx, w = front.gate_topk(np.array([[np.inf, 3.0, np.inf]]), None, 3)
    assert idx.tolist() == [[0, 2, 1]] and np.allclose(w, [[0.5, 0.5, 0.0]])
