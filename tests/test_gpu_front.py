"""The operators in front of the expert layer on an MI355X, against their float64 oracle.

Tolerances, from the arithmetic.  An output is rounded once from float32: half a step, 2^-8 of the
value for BF16, 2^-24 for float32, half the distance of neighbouring codes for E4M3.  Before that the norm
makes five float32 roundings (the sum x + residual, the reciprocal root, two products, one division
for the scales): below 2^-21.  UE8M0 codes and chosen experts are decided as in float64 and must be
equal.  The gate's sums of H exact products round at most once a product, by at most 2^-23 of a partial sum,
which is at most the sum of the products' magnitudes.  Weights of chosen experts: a float32 exponential's
argument may be rounded by 2^-24 of itself (magnitudes up to 32 here, 2^-19) and a few results by 2^-23.
"""
import numpy as np
import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm
import oracle
import synth
from harness import assert_y_close, e4m3_spacing, run_oracle
from oracle import front

pytestmark = pytest.mark.gpu

DT = {"bf16": (mm.DTYPE_BF16, torch.bfloat16), "f32": (mm.DTYPE_F32, torch.float32)}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
E4M3 = oracle.e4m3_decode_table()


def _say(*a):
    print("[front]", *a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _rows(values, pad):
    """The values as the rows of a wider buffer (its other columns NaN)."""
    wide = torch.full((values.shape[0], values.shape[1] + pad), float("nan"), dtype=values.dtype, device="cuda")
    wide[:, :values.shape[1]] = values
    return wide[:, :values.shape[1]]


# ------------------------------------------------------------------------------------ norm
def _norm_inputs(T, H, x="bf16", w="bf16", residual=True, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    channel = torch.exp(0.5 * torch.randn(H, generator=g))
    r = (torch.randn(T, H, generator=g) * channel).to(DT[x][1]).cuda() if residual else None
    return (_rows((0.3 * torch.randn(T, H, generator=g) * channel).to(DT[x][1]).cuda(), pad), r,
            (1 + 0.2 * torch.randn(H, generator=g)).to(DT[w][1]).cuda())


def _norm(x, residual, weight, recipe, eps=1e-6, residual_out="new", stream=None):
    T, H = x.shape
    code = {v[1]: v[0] for v in DT.values()}
    if isinstance(residual_out, str):
        residual_out = None if residual is None else torch.full((T, H), float("nan"), dtype=x.dtype, device="cuda")
    stride = lambda t: 0 if t is None or t.is_contiguous() else t.stride(0)  # noqa: E731
    p = mm.NormProblem.make(T, H, recipe, code[x.dtype], code[weight.dtype], eps, x_stride=stride(x),
                            residual_stride=stride(residual if residual is not None else residual_out))
    normed = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda")
    q_sf = (torch.full((T, H // 128), float("nan"), device="cuda") if recipe == 0 else
            torch.full((T, H // 32), 0x55, dtype=torch.uint8, device="cuda"))
    mm.mega_moe_norm_quant(p, x, weight, residual, residual_out, normed, q, q_sf, stream)
    return dict(residual_out=residual_out, normed=normed, q=q, q_sf=q_sf)


def _check_norm(got, x, residual, weight, recipe, eps=1e-6, rows=None):
    kind = "f32" if x.dtype == torch.float32 else "bf16"
    eps32 = float(np.float32(eps))
    rows = slice(None) if rows is None else rows
    ref = front.norm_quant(_f64(x)[rows], None if residual is None else _f64(residual)[rows], _f64(weight), eps32, recipe)
    if got["residual_out"] is not None:
        out = _f64(got["residual_out"])[rows]
        assert (np.abs(out - ref["h"]) <= (HALF[kind] + 2.0 ** -23) * np.abs(ref["h"])).all()
    tiny = 2.0 ** -133                                       # half a step of BF16 below its normal numbers
    assert (np.abs(_f64(got["normed"])[rows] - ref["v"]) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(ref["v"]) + tiny).all()
    g = 128 if recipe == 0 else 32
    if recipe == 0:
        sf = _f64(got["q_sf"])[rows]
        assert (np.abs(sf - ref["sf"]) <= 2.0 ** -21 * ref["sf"]).all()
    else:
        code = got["q_sf"].cpu().numpy().astype(np.int64)[rows]
        assert np.array_equal(code, ref["code"]), f"{int((code != ref['code']).sum())} codes differ"
        sf = np.where(code > 0, np.ldexp(1.0, code - 127), 2.0 ** -127)
    q = E4M3[got["q"].cpu().numpy()[rows]]
    sf = np.repeat(sf, g, axis=1)
    scaled = np.divide(ref["v"], sf, out=np.zeros_like(ref["v"]), where=sf > 0)
    # to the nearest code: at most half the spacing of the codes at the value
    allowed = e4m3_spacing(scaled) / 2 * (1 + 2.0 ** -20) + np.abs(scaled) * 2.0 ** -20
    assert (np.abs(q - scaled) <= allowed).all()


@pytest.mark.parametrize("recipe", [0, 1, 2])
@pytest.mark.parametrize("T,H,x,w,residual,pad", [
    (1, 7168, "bf16", "bf16", True, 0), (1, 128, "bf16", "f32", False, 0), (3, 256, "f32", "bf16", True, 4),
    (37, 3712, "f32", "f32", True, 64), (5, 16384, "bf16", "bf16", True, 8), (2, 16384, "f32", "f32", True, 0),
    (300, 1152, "bf16", "f32", True, 0), (2500, 640, "bf16", "bf16", False, 8), (130, 8192, "f32", "bf16", True, 0),
    (129, 8320, "bf16", "bf16", True, 16), (700, 4096, "bf16", "bf16", True, 0), (67, 512, "f32", "f32", False, 0)])
def test_norm_quant(T, H, x, w, residual, pad, recipe):
    _say("norm", T, H, x, w, residual, pad, recipe)
    X, R, W = _norm_inputs(T, H, x, w, residual, pad, seed=T + H)
    got = _norm(X, R, W, recipe)
    torch.cuda.synchronize()
    _check_norm(got, X, R, W, recipe)


@pytest.mark.parametrize("recipe", [0, 1, 2])
@pytest.mark.parametrize("T,H,x,w,pad", [(3, 8320, "bf16", "f32", 8), (40, 16384, "bf16", "f32", 0),
                                         (5, 9088, "f32", "bf16", 4), (3, 16384, "f32", "bf16", 0)])
def test_norm_quant_of_long_rows_with_mixed_types(T, H, x, w, pad, recipe):
    """More than 8192 columns: two chunks a thread."""
    X, R, W = _norm_inputs(T, H, x, w, True, pad, seed=T + H)
    _check_norm(_norm(X, R, W, recipe), X, R, W, recipe)


@pytest.mark.parametrize("H", [128, 7168, 16384])
@pytest.mark.parametrize("steps", [0, 1, 2, 5])
def test_norm_power_of_two_scales_at_their_borders(H, steps):
    """One large value a group whose weight brings amax/448 within `steps` float32 steps of a power of two, from
    either side: the codes must be those of the float64 values."""
    _say("norm border", H, steps)
    g = torch.Generator().manual_seed(H + steps)
    X = torch.randn(1, H, generator=g)
    h = X.double().numpy()[0]
    r = 1 / np.sqrt((h * h).mean() + float(np.float32(1e-6)))
    W = np.full(H, 1e-3, dtype=np.float32)
    n = H // 32
    at = np.arange(n) * 32 + np.arange(n) % 32
    target = 448.0 * np.exp2(np.arange(n) % 9 - 4.0)
    W[at] = (target / (np.abs(h[at]) * r)).astype(np.float32)
    for _ in range(steps):
        W[at] = np.nextafter(W[at], np.where(np.arange(n) % 2, np.float32(np.inf), np.float32(0)))
    X, W = X.cuda(), torch.from_numpy(W).cuda()
    got = _norm(X, None, W, 1)
    _check_norm(got, X, None, W, 1)


@pytest.mark.parametrize("recipe", [0, 2])
@pytest.mark.parametrize("pad", [0, 24])
def test_norm_in_place(recipe, pad):
    X, R, W = _norm_inputs(33, 1280, seed=9)
    R0 = R.clone()
    ref = _norm(X, R, W, recipe)
    Rw = _rows(R, pad)
    got = _norm(X, Rw, W, recipe, residual_out=Rw)
    for k in ref:
        assert torch.equal(got[k].contiguous().view(torch.uint8), ref[k].view(torch.uint8)), k
    if pad:
        wide = Rw._base if Rw._base is not None else Rw
        assert torch.isnan(wide[:, 1280:]).all()              # the columns beside the rows stay as they were
    # over x, and x as its own residual
    X1 = X.contiguous().clone()
    _norm(X1, R0, W, recipe, residual_out=X1)
    assert torch.equal(X1, ref["residual_out"])
    X2 = X.contiguous().clone()
    twice = _norm(X2, X2, W, recipe, residual_out=X2)
    assert torch.equal(twice["residual_out"], (X.float() * 2).to(X.dtype))


def test_norm_outputs_that_are_not_asked_for():
    X, R, W = _norm_inputs(6, 384, seed=3)
    full = _norm(X, R, W, 1)
    p = mm.NormProblem.make(6, 384, 1)
    normed = torch.empty_like(full["normed"])
    mm.mega_moe_norm_quant(p, X, W, residual=R, normed=normed)
    assert torch.equal(normed, full["normed"])
    q, q_sf = torch.empty_like(full["q"]), torch.empty_like(full["q_sf"])
    mm.mega_moe_norm_quant(p, X, W, residual=R, q=q, q_sf=q_sf)
    assert torch.equal(q, full["q"]) and torch.equal(q_sf, full["q_sf"])
    copy = torch.empty_like(X)                                # residual_out without a residual: x itself
    mm.mega_moe_norm_quant(p, X, W, residual_out=copy, normed=normed)
    assert torch.equal(copy, X)


@pytest.mark.parametrize("recipe", [0, 1])
def test_norm_zeros_infinities_and_large_values(recipe):
    X, _, W = _norm_inputs(8, 512, x="f32", w="f32", residual=False, seed=4)
    X[1] = 0
    X[2, :] = 1e-30
    X[3, 7] = float("inf")
    X[4, 300] = float("nan")
    X[5] *= 1e30                                              # squares beyond float32
    X[6, 128:256] = 0
    got = _norm(X, None, W, recipe)
    fine = [0, 1, 2, 5, 6, 7]
    _check_norm(got, X, None, W, recipe, rows=fine)
    assert (got["q"][1] == 0).all() and (got["q"][6, 128:256] == 0).all() and (got["normed"][1] == 0).all()
    sf = got["q_sf"]
    assert (sf[1] == 0).all() and (sf[6, 1:2] == 0).all() if recipe == 0 else (sf[1] == 0).all()
    for t in (3, 4):
        assert torch.isnan(got["normed"][t]).all() and ((got["q"][t] & 0x7F) == 0x7F).all()
        assert torch.isnan(sf[t]).all() if recipe == 0 else (sf[t] == 255).all()
    W2 = W.clone()
    W2[200] = float("inf")                                    # one group of each row
    got2 = _norm(X, None, W2, recipe)
    g = 128 if recipe == 0 else 32
    q = (got2["q"][0].view(-1, g) & 0x7F) == 0x7F
    assert q[200 // g].all() and q.sum() == g
    keep = torch.arange(512 // g, device="cuda") != 200 // g
    assert torch.equal(got2["q"][0].view(-1, g)[keep], got["q"][0].view(-1, g)[keep])
    assert torch.equal(got2["q_sf"][0][keep], got["q_sf"][0][keep])


def test_norm_values_below_float32s_normal_numbers():
    X = torch.randn(3, 256, generator=torch.Generator().manual_seed(8)).cuda()
    X[:, 5] = 0
    for size in (1e-38, 1e-41, 1e-44, 0.0):
        W = torch.full((256,), size, device="cuda")
        got = _norm(X, None, W, 0)
        q = E4M3[got["q"].cpu().numpy()]
        assert np.isfinite(q).all() and (q[:, 5] == 0).all() and torch.isfinite(got["q_sf"]).all()
        assert (got["q"].view(3, 2, 128)[got["q_sf"] == 0] == 0).all()
        got = _norm(X, None, W, 1)
        assert np.isfinite(E4M3[got["q"].cpu().numpy()]).all()
        # half a code's step at the smallest scale, and what the values themselves have lost
        v = _f64(X) / np.sqrt((_f64(X) ** 2).mean(axis=1, keepdims=True) + 1e-6) * _f64(W)
        scale = np.ldexp(1.0, np.repeat(got["q_sf"].cpu().numpy().astype(int), 32, axis=1) - 127)
        err = np.abs(E4M3[got["q"].cpu().numpy()] * scale - v)
        assert (err <= np.abs(v) * 2.0 ** -4 * 1.01 + 2.0 ** -10 * scale + 2.0 ** -148).all()


def test_norm_more_rows_than_workgroups():
    T = (1 << 20) + 3
    X = torch.ones(T, 128, dtype=torch.bfloat16, device="cuda")
    X[1 << 20:] = torch.randn(3, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    W = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    got = _norm(X, None, W, 1)
    tail = slice(T - 5, T)
    _check_norm({k: None if v is None else v[tail] for k, v in got.items()}, X[tail], None, W, 1)
    assert (got["normed"][:1 << 20] == got["normed"][0, 0]).all() and (got["q_sf"][:1 << 20] == got["q_sf"][0, 0]).all()


def test_norm_no_tokens():
    for recipe in (0, 1):
        _norm(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), None,
              torch.ones(256, dtype=torch.bfloat16, device="cuda"), recipe)
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------ gate
def _gate(x, w, stream=None):
    T, H = x.shape
    E = w.shape[0]
    p = mm.GateProblem.make(T, H, E, mm.DTYPE_F32 if w.dtype == torch.float32 else mm.DTYPE_BF16,
                            x_stride=0 if x.is_contiguous() else x.stride(0))
    guard = torch.full((T * E + 64,), float("nan"), device="cuda")      # what lies behind stays as it was
    logits = guard[:T * E].view(T, E)
    mm.mega_moe_gate_logits(p, x, w, logits, stream)
    assert torch.isnan(guard[T * E:]).all()
    return logits


GATE_SHAPES = [(1, 128, 1), (1, 7168, 256), (2, 256, 7), (3, 1024, 60), (5, 7168, 256), (16, 2048, 64),
               (17, 384, 33), (31, 896, 130), (64, 4096, 128), (65, 640, 257), (100, 7168, 8), (128, 7168, 256),
               (200, 16384, 40), (257, 1280, 384), (513, 512, 160), (1021, 4096, 128), (1500, 256, 17),
               (2050, 768, 256), (4099, 384, 192), (3, 256, 2051), (5000, 256, 200), (8197, 128, 131), (8, 640, 8),
               (9, 1024, 9), (7, 128, 200), (130, 1152, 255), (40, 16384, 129)]


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", GATE_SHAPES)
def test_gate_logits(T, H, E, w):
    _say("gate", T, H, E, w)
    g = torch.Generator().manual_seed(T * 7 + E)
    x = _rows(torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), 8 * (E % 3))
    W = (torch.randn(E, H, generator=g) * 0.02).to(DT[w][1]).cuda()
    got = _f64(_gate(x, W))
    ref, mag = front.gate_logits(_f64(x), _f64(W))
    assert (np.abs(got - ref) <= (H * (3 if w == "f32" else 1) + 8) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", GATE_SHAPES)
def test_gate_logits_whole_numbers_are_exact(T, H, E, w):
    """Small whole numbers: every partial sum is a whole number below 2^24, so the result is exact."""
    g = torch.Generator().manual_seed(T + E)
    x = torch.randint(-4, 5, (T, H), generator=g).to(torch.bfloat16).cuda()
    W = torch.randint(-8, 9, (E, H), generator=g).to(DT[w][1]).cuda()
    assert torch.equal(_gate(x, W).double(), (x.cpu().double() @ W.cpu().double().t()).cuda())


def test_gate_float32_weights_keep_all_their_bits():
    g = torch.Generator().manual_seed(5)
    T = H = 256
    W = (1 + torch.rand(31, H, generator=g)) * torch.exp2(torch.randint(-102, 100, (31, H), generator=g).float())
    W = torch.where(torch.rand(31, H, generator=g) < 0.5, W, -W).cuda()
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(T), torch.arange(T)] = 1.0
    for rows in (T, 3):
        assert torch.equal(_gate(x[:rows].contiguous(), W), W.t()[:rows])


# both sides of the sizes at which few logits are taken as dot products of rows: 64 tokens, 2048 logits, one
# or two tokens a workgroup (512 logits), rows of one pass of 8192 columns and of more
GATE_EDGES = [(64, 512, 32), (65, 512, 31), (64, 384, 33), (1, 256, 2048), (1, 256, 2049), (2, 640, 256),
              (2, 640, 257), (2, 512, 1024), (2, 512, 1025), (3, 8192, 255), (3, 8320, 171), (7, 16384, 256),
              (1, 16384, 3), (5, 128, 1), (63, 8064, 1), (33, 1152, 62), (33, 1152, 63)]


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", GATE_EDGES)
def test_gate_logits_of_few_rows(T, H, E, w):
    """Each term (three of them with weights in three parts) is added to a sum that the terms' magnitudes
    bound, with an error of at most a step of it, 2^-23 (matrix instructions need not round to nearest); a few
    more additions join the parts."""
    _say("gate rows", T, H, E, w)
    g = torch.Generator().manual_seed(T * 11 + E)
    x = _rows(torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), 8 * (T % 4))
    W = (torch.randn(E, H, generator=g) * 0.02).to(DT[w][1]).cuda()
    got = _f64(_gate(x, W))
    ref, mag = front.gate_logits(_f64(x), _f64(W))
    assert (np.abs(got - ref) <= (H * (3 if w == "f32" else 1) + 8) * 2.0 ** -23 * mag).all()
    xi = torch.randint(-4, 5, (T, H), generator=g).to(torch.bfloat16).cuda()
    Wi = torch.randint(-8, 9, (E, H), generator=g).to(DT[w][1]).cuda()
    assert torch.equal(_gate(xi, Wi).double(), (xi.cpu().double() @ Wi.cpu().double().t()).cuda())


# every tile of both types of weights (test_gate_policy.py sees to that), ragged, with fewer steps of 64 columns than a
# workgroup has waves and with steps that the waves do not share evenly
GATE_TILES = [(31, 128, 130), (45, 1152, 130), (100, 1152, 200), (127, 128, 253), (65, 2176, 257), (140, 128, 255), (150, 1664, 250),
              (300, 128, 250), (513, 1152, 161), (700, 128, 250), (1021, 7168, 255), (1000, 1664, 254), (1537, 128, 254),
              (2047, 1152, 255), (1800, 7168, 256), (2050, 128, 253), (3001, 1152, 250), (4100, 128, 250),
              (6001, 1152, 255), (8197, 128, 131), (9000, 1152, 130)]


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,E", GATE_TILES)
def test_gate_logits_of_every_tile(T, H, E, w):
    """Whole numbers exactly, random values within test_gate_logits_of_few_rows' bound."""
    _say("gate tiles", T, H, E, w)
    g = torch.Generator().manual_seed(T * 5 + E)
    xi = _rows(torch.randint(-4, 5, (T, H), generator=g).to(torch.bfloat16).cuda(), 8 * (T % 3))
    Wi = torch.randint(-8, 9, (E, H), generator=g).to(DT[w][1]).cuda()
    assert torch.equal(_gate(xi, Wi).double(), (xi.cpu().double() @ Wi.cpu().double().t()).cuda())
    x = _rows(torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), 8 * (E % 3))
    W = (torch.randn(E, H, generator=g) * 0.02).to(DT[w][1]).cuda()
    got = _f64(_gate(x, W))
    ref, mag = front.gate_logits(_f64(x), _f64(W))
    assert (np.abs(got - ref) <= (H * (3 if w == "f32" else 1) + 8) * 2.0 ** -23 * mag).all()


GATE_BITS = [(31, 130), (127, 253), (140, 255), (300, 250), (700, 250), (1537, 254), (4100, 250)]


@pytest.mark.parametrize("T,E", GATE_BITS)
def test_gate_float32_weights_keep_all_their_bits_in_every_tile(T, E):
    g = torch.Generator().manual_seed(T)
    H = 384
    W = (1 + torch.rand(E, H, generator=g)) * torch.exp2(torch.randint(-102, 100, (E, H), generator=g).float())
    W = torch.where(torch.rand(E, H, generator=g) < 0.5, W, -W).cuda()
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(T, device="cuda") % H
    x[torch.arange(T, device="cuda"), at] = 1.0
    assert torch.equal(_gate(x, W), W.t()[at])


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 6, 700])
def test_gate_infinities_give_no_finite_logits(T, w):
    g = torch.Generator().manual_seed(8)
    x = (1 + torch.rand(T, 640, generator=g)).to(torch.bfloat16).cuda()
    W = (1 + torch.rand(50, 640, generator=g)).to(DT[w][1]).cuda()
    clean = _gate(x, W).clone()
    x[T - 1, 639] = float("inf")
    W[49, 5] = -float("inf")
    got = _gate(x, W)
    assert not torch.isfinite(got[T - 1]).any() and not torch.isfinite(got[:, 49]).any()
    assert torch.isnan(got[T - 1, 49])
    assert torch.equal(got[:T - 1, :49], clean[:T - 1, :49])


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 4])
def test_gate_weights_below_the_normal_range_of_few_rows(T, w):
    """One term a logit, x = 1: the weight itself, subnormal or not."""
    e = torch.arange(-140 if w == "f32" else -133, -100)
    W = torch.zeros(len(e), 128)
    W[torch.arange(len(e)), torch.arange(len(e)) % 128] = torch.exp2(e.double()).float()
    assert (W.sum(1) > 0).all()
    x = torch.ones(T, 128, dtype=torch.bfloat16, device="cuda")
    got = _gate(x, W.to(DT[w][1]).cuda())
    assert torch.equal(got, W.sum(1).cuda().expand(T, -1))


@pytest.mark.parametrize("E", [1, 9])
def test_gate_logits_of_more_tokens_than_one_launch_takes(E):
    T, H = (1 << 23) + 77, 128
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, 4095, (1 << 23) - 1, 1 << 23, (1 << 23) + 63, T - 1], device="cuda")
    x[rows] = torch.randint(-4, 5, (len(rows), H), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    W = torch.randint(-8, 9, (E, H), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    logits = _gate(x, W)
    assert torch.equal(logits[rows], (x[rows].float().cpu() @ W.float().cpu().t()).cuda())
    logits[rows] = 0
    assert not logits.any()


@pytest.mark.parametrize("T", [1, 40, 700])
@pytest.mark.parametrize("w", ["bf16", "f32"])
def test_gate_values_that_are_not_finite_stay_in_their_row(T, w):
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, 512, generator=g).to(torch.bfloat16).cuda()
    W = torch.randn(50, 512, generator=g).to(DT[w][1]).cuda()
    clean = _gate(x, W).clone()
    x[T // 2, 17] = float("nan")
    W[20, 400] = float("nan")
    got = _gate(x, W)
    assert torch.isnan(got[T // 2]).all() and torch.isnan(got[:, 20]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[T // 2], keep[:, 20] = False, False
    assert torch.equal(got[keep], clean[keep])


# ------------------------------------------------------------------------------------ topk
def _topk(logits, k, bias=None, num_valid=None, stream=None, **kw):
    T, E = logits.shape
    renorm = kw.pop("renorm", False)
    score = kw.pop("score", "softmax")
    p = mm.TopkProblem.make(T, E, k, score=mm.SCORE_SIGMOID if score == "sigmoid" else mm.SCORE_SOFTMAX,
                            logits_dtype=mm.DTYPE_BF16 if logits.dtype == torch.bfloat16 else mm.DTYPE_F32,
                            flags=mm.FLAG_TOPK_RENORM if renorm else 0,
                            logits_stride=0 if logits.is_contiguous() else logits.stride(0), **kw)
    cols = k + kw.get("num_shared", 0)
    idx = torch.full((T * cols + 64,), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T * cols + 64,), float("nan"), device="cuda")
    mm.mega_moe_gate_topk(p, logits, idx[:T * cols].view(T, cols), w[:T * cols].view(T, cols), bias, num_valid, stream)
    assert (idx[T * cols:] == -77).all() and torch.isnan(w[T * cols:]).all()
    return idx[:T * cols].view(T, cols), w[:T * cols].view(T, cols)


def _check_topk(logits, k, bias=None, num_valid=None, times=1, **kw):
    """times: the rows that many times over (large batches take another kernel)."""
    idx, w = _topk(logits.repeat(times, 1) if times > 1 else logits, k, bias, num_valid, **dict(kw))
    ref_i, ref_w = front.gate_topk(_f64(logits), None if bias is None else _f64(bias), k,
                                   num_valid=None if num_valid is None else int(num_valid.item()), **kw)
    ref_i, ref_w = np.tile(ref_i, (times, 1)), np.tile(ref_w, (times, 1))
    got_i = idx.cpu().numpy()
    assert np.array_equal(got_i, ref_i), f"rows {np.unique(np.argwhere(got_i != ref_i)[:, 0])[:8]} differ"
    got_w = _f64(w)
    assert np.isfinite(got_w).all()
    # below float32's normal numbers (times the scale) a weight may be flushed
    assert (np.abs(got_w - ref_w) <= 2.0 ** -18 * np.abs(ref_w) + 2.0 ** -120).all()


CONFIGS = {
    "softmax": dict(),
    "softmax_renorm_scaled": dict(renorm=True, scale=2.5),
    "sigmoid_renorm": dict(score="sigmoid", renorm=True),
    "sigmoid_shared": dict(score="sigmoid", num_shared=2, shared_weight=0.75),
}


@pytest.mark.parametrize("name", list(CONFIGS))
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k,dtype,pad", [
    (1, 1, 1, "f32", 0), (1, 256, 8, "f32", 0), (3, 7, 7, "bf16", 1), (40, 60, 4, "f32", 4), (33, 128, 8, "bf16", 0),
    (65, 256, 8, "f32", 3), (20, 257, 6, "bf16", 0), (17, 384, 12, "f32", 0), (9, 513, 10, "f32", 0),
    (5, 1030, 33, "bf16", 0), (2, 8190, 62, "f32", 0), (130, 16, 2, "f32", 0), (300, 64, 62, "f32", 0)])
def test_topk(T, E, k, dtype, pad, biased, name):
    _say("topk", T, E, k, dtype, pad, biased, name)
    g = torch.Generator().manual_seed(T * 31 + E)
    logits = _rows((torch.randn(T, E, generator=g) * 1.5).to(DT[dtype][1]).cuda(), pad)
    bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
    _check_topk(logits, k, bias, **CONFIGS[name])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("T,E,k,G,KG", [(1, 256, 8, 8, 4), (50, 256, 8, 8, 4), (33, 64, 6, 64, 6), (21, 128, 8, 2, 1),
                                        (40, 160, 6, 8, 3), (9, 48, 5, 3, 2), (7, 1024, 8, 16, 4), (10, 60, 8, 4, 4),
                                        (6, 4096, 20, 64, 10), (31, 24, 12, 8, 4)])
def test_topk_groups(T, E, k, G, KG, group_top, biased, score):
    _say("topk groups", T, E, k, G, KG, group_top, biased, score)
    g = torch.Generator().manual_seed(T + E + G)
    logits = (torch.randn(T, E, generator=g) * 1.5).cuda()
    bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
    _check_topk(logits, k, bias, score=score, num_groups=G, topk_groups=KG, group_top=group_top, renorm=True)


LARGE = [(8201, 256, 8, 8, 4, 2), (8192, 256, 8, 1, 1, 1), (4099, 64, 6, 1, 1, 1), (4100, 128, 14, 16, 5, 2),
         (9000, 200, 3, 5, 2, 1), (4097, 24, 1, 8, 1, 2), (4096, 96, 15, 3, 2, 1), (4500, 7, 7, 1, 1, 1),
         (5000, 130, 12, 13, 4, 2)]


@pytest.mark.parametrize("dtype,pad", [("f32", 0), ("bf16", 1)])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("T,E,k,G,KG,group_top", LARGE)
def test_topk_large_batches(T, E, k, G, KG, group_top, score, biased, dtype, pad):
    _say("topk large", T, E, k, G, KG, group_top, score, biased, dtype)
    g = torch.Generator().manual_seed(T + E)
    rows = 331                                                # different ones; the oracle goes row by row
    logits = (torch.randn(rows, E, generator=g) * 1.5).to(DT[dtype][1])
    bias = (torch.randn(E, generator=g) * 0.1).cuda() if biased else None
    big = _rows(logits.repeat(T // rows + 1, 1)[:T].cuda(), pad)
    kw = dict(score=score, num_groups=G, topk_groups=KG, group_top=group_top, renorm=True)
    n = T - 9
    idx, w = _topk(big, k, bias, torch.tensor([n], dtype=torch.int32, device="cuda"),
                   num_shared=1 if k < 14 else 0, **dict(kw))
    ref_i, ref_w = front.gate_topk(_f64(logits), None if bias is None else _f64(bias), k,
                                   num_shared=1 if k < 14 else 0, **kw)
    of = np.arange(n) % rows
    assert np.array_equal(idx[:n].cpu().numpy(), ref_i[of])
    assert (np.abs(_f64(w[:n]) - ref_w[of]) <= 2.0 ** -18 * ref_w[of] + 2.0 ** -120).all()
    assert (idx[n:] == -1).all() and (w[n:] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,KG,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
@pytest.mark.parametrize("times", [1, 65])
def test_topk_ties_and_close_scores(times, G, KG, group_top, biased, score):
    """Equal logits, logits one float32 step apart and scores that round to the same float32."""
    g = torch.Generator().manual_seed(11)
    T, E, k = 64, 64, 9
    logits = torch.randint(-2, 3, (T, E), generator=g).float()
    one = torch.ones(T, E)
    steps = torch.randint(0, 3, (T, E), generator=g)
    logits[16:32] = torch.where(steps[16:32] > 0, torch.nextafter(one, 2 * one)[16:32], one[16:32])
    logits[32:48] = 20 + steps[32:48].float()                 # sigmoid within 2^-28 of 1
    logits[48:] = 0
    bias = (torch.randint(0, 2, (E,), generator=g).float() * 0.25).cuda() if biased else None
    _check_topk(logits.cuda(), k, bias, times=times, score=score, num_groups=G, topk_groups=KG, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,KG,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("E,times", [(32, 1), (32, 21), (256, 1), (256, 41)])
def test_topk_scores_a_rounding_apart(E, times, G, KG, group_top, biased, score):
    """Scores that differ by less than a float32 exponential is off: logits spread over a few hundred
    steps around one value, with biases that nearly cancel the difference of two levels."""
    g = torch.Generator().manual_seed(12)
    T, k = 200, 8
    step = torch.randint(-300, 300, (T, E), generator=g).double() * 2.0 ** -24
    logits = (0.7 + step).float()
    bias = None
    if biased:
        high = torch.arange(E) % 2 == 0
        s = torch.sigmoid(torch.tensor([0.7, 0.2], dtype=torch.float64)) if score == "sigmoid" else None
        if s is not None:
            logits = torch.where(high, logits, logits - 0.5)
            bias = torch.where(high, torch.zeros(()), (s[0] - s[1]).float()).cuda()
        else:
            bias = (torch.randint(0, 2, (E,), generator=g).float() * 2.0 ** -26).cuda()
    _check_topk(logits.cuda(), k, bias, times=times, score=score, num_groups=G, topk_groups=KG, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2.0 ** 20, 3.0e37])
@pytest.mark.parametrize("times", [1, 21])
def test_topk_group_sums_whose_terms_cancel(times, size, score):
    """Two experts a group with biases of opposite sign: the sums are of the order of the scores while their
    terms round by far more."""
    g = torch.Generator().manual_seed(15)
    logits = torch.randn(200, 64, generator=g)
    bias = torch.full((64,), -float("inf"))
    bias[0::8], bias[3::8] = size, -size
    _check_topk(logits.cuda(), 6, bias.cuda(), times=times, score=score, num_groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [4096.0, 2.0 ** 20, 1.0e9, 2.0 ** 30])
@pytest.mark.parametrize("E,G,KG,times", [(16, 4, 1, 1), (16, 4, 1, 41), (64, 8, 3, 1), (64, 8, 3, 41), (24, 3, 2, 1),
                                          (24, 3, 2, 41), (256, 8, 4, 1), (256, 8, 4, 82), (1024, 8, 4, 1)])
def test_topk_one_group_whose_terms_cancel_among_ordinary_ones(E, G, KG, times, size, score):
    """One group has two experts with biases of opposite sign, so that its float32 sum is off by far more than
    the sums of the other groups are apart, and may stand anywhere in their order."""
    g = torch.Generator().manual_seed(E + G)
    n = E // G
    spread = min(1.5, size * 2.0 ** -23 * (E / 2 if score == "softmax" else 4))
    logits = torch.randn(100, E, generator=g) * spread
    for group in (0, G // 2, G - 1):
        bias = torch.zeros(E)
        bias[group * n:(group + 1) * n] = -float("inf")
        bias[group * n], bias[group * n + 2] = size, -size
        _check_topk(logits.cuda(), 3, bias.cuda(), times=times, score=score, num_groups=G, topk_groups=KG, group_top=2)


@pytest.mark.parametrize("times", [1, 4096])
def test_topk_cancelling_group_worked_by_hand(times):
    """Two sigmoid scores of 0.952574 with biases of +-2^30: their sum is 1.905 and in float32 0, the best of the
    other groups' is 1.32.  The other groups' experts are far apart, so that nothing else asks for 64 bits."""
    logits = torch.tensor([0.0, 0.3, 0.2, 0.1] * 4)[None].clone()
    logits[0, 0] = logits[0, 2] = 3.0
    bias = torch.zeros(16)
    bias[0], bias[2], bias[1], bias[3] = 2.0 ** 30, -2.0 ** 30, -float("inf"), -float("inf")
    bias[4:8], bias[8:12] = 0.1, 0.05
    idx, _ = _topk(logits.repeat(times, 1).cuda(), 2, bias.cuda(), score="sigmoid", num_groups=4, topk_groups=1, group_top=2)
    assert torch.equal(idx.cpu(), torch.tensor([[0, 2]], dtype=torch.int32).expand(times, -1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,KG,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,times", [(32, 1), (32, 342), (256, 1), (256, 683), (1024, 1)])
def test_topk_masked_experts(E, times, dtype, G, KG, group_top, score):
    g = torch.Generator().manual_seed(13)
    k = 6
    logits = torch.randn(12, E, generator=g)
    low = torch.finfo(DT[dtype][1]).min
    logits[1] = -float("inf")                                  # nothing to choose
    logits[2] = float("nan")
    logits[3, 3:] = -float("inf")                              # three left, in one group
    logits[4, ::2] = float("nan")
    logits[5] = low                                            # the type's lowest value is a number
    logits[6, 1:] = low
    logits[7, 5], logits[7, 21] = float("inf"), float("inf")
    logits[8, 8:16] = -float("inf")                            # a whole group
    logits[9] = -200.0                                         # scores beyond float32's range
    logits[9, 4], logits[9, 20] = -199.0, -150.0
    logits[10, :E - 1] = -float("inf")
    logits = logits.to(DT[dtype][1]).cuda()
    bias = torch.zeros(E)
    bias[2], bias[17], bias[30], bias[9] = float("nan"), -float("inf"), float("inf"), 0.5
    for b in (None, bias.cuda()):
        for renorm in (False, True):
            _check_topk(logits, k, b, times=times, score=score, num_groups=G, topk_groups=KG, group_top=group_top,
                        renorm=renorm, num_shared=1)


@pytest.mark.parametrize("T,E,k,dtype", [((1 << 24) + 5, 2, 1, "f32"), ((1 << 22) + 5, 16, 15, "bf16"),
                                         ((1 << 20) + 3, 520, 2, "bf16")])
def test_topk_more_rows_than_one_pass_of_the_workgroups(T, E, k, dtype):
    logits = torch.zeros(T, E, dtype=DT[dtype][1], device="cuda")
    logits[:, E - 1] = 1                                      # the last expert, then from the first on
    tail = torch.randn(9, E, generator=torch.Generator().manual_seed(3)).to(DT[dtype][1]).cuda()
    logits[T - 9:] = tail
    idx, w = _topk(logits, k, renorm=True)
    ref_i, ref_w = front.gate_topk(_f64(tail), None, k, renorm=True)
    assert np.array_equal(idx[T - 9:].cpu().numpy(), ref_i)
    assert (np.abs(_f64(w[T - 9:]) - ref_w) <= 2.0 ** -18 * ref_w).all()
    first = torch.tensor([E - 1, *range(k - 1)], dtype=torch.int32, device="cuda")
    assert (idx[:T - 9] == first).all() and (w[:T - 9] == w[0]).all()


@pytest.mark.parametrize("n", [-3, 0, 1, 30, 37, 100])
def test_topk_padded_rows(n):
    g = torch.Generator().manual_seed(14)
    logits = torch.randn(37, 64, generator=g).cuda()
    if 0 <= n < 37:
        logits[n:] = float("nan")                             # padding holds anything
    num_valid = torch.tensor([n], dtype=torch.int32, device="cuda")
    _check_topk(logits, 4, None, num_valid, num_shared=1, renorm=True)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,G,KG,group_top", [(64, 1, 1, 1), (96, 4, 2, 2), (256, 8, 4, 2)])
def test_topk_rows_are_independent_of_their_neighbours_and_of_the_padding(E, G, KG, group_top, score, biased, renorm):
    """A row's experts and weights, bit for bit, whatever lies in the other rows and behind the last valid one."""
    g = torch.Generator().manual_seed(E + KG)
    T, k, n = 8195, 6, 8190                                   # four rows a wave: 8188 and 8189 share theirs with padding
    kw = dict(score=score, num_groups=G, topk_groups=KG, group_top=group_top, renorm=renorm)
    logits = torch.randn(T, E, generator=g).cuda()
    bias = (0.1 * torch.randn(E, generator=g)).cuda() if biased else None
    num_valid = torch.tensor([n], dtype=torch.int32, device="cuda")
    idx, w = _topk(logits, k, bias, num_valid, **dict(kw))
    assert (idx[n:] == -1).all() and (w[n:] == 0).all()
    for value in (-200.0, float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).max):
        other = logits.clone()
        other[n:] = value
        got_i, got_w = _topk(other, k, bias, num_valid, **dict(kw))
        assert torch.equal(got_i, idx) and torch.equal(got_w.view(torch.int32), w.view(torch.int32)), f"padding of {value}"
        other[1::4], other[2::4] = value, value               # every row's neighbours but these rows' own
        keep = torch.arange(0, n, 4, device="cuda")
        got_i, got_w = _topk(other, k, bias, num_valid, **dict(kw))
        for r in (keep, keep[:-1] + 3):
            assert torch.equal(got_i[r], idx[r]) and torch.equal(got_w[r].view(torch.int32), w[r].view(torch.int32)), \
                f"neighbours of {value}"


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("E,k,G,KG,group_top,times", [
    (16, 2, 1, 1, 1, 1), (64, 6, 1, 1, 1, 1), (64, 6, 1, 1, 1, 21), (96, 8, 4, 2, 2, 1), (96, 8, 4, 2, 2, 21),
    (256, 8, 8, 4, 2, 1), (256, 8, 8, 4, 2, 41), (384, 8, 1, 1, 1, 1), (600, 8, 1, 1, 1, 1)])
def test_topk_weights_are_rounded_once(E, k, G, KG, group_top, times, score, biased, renorm):
    """One rounding to float32, 2^-24 of the weight (half of 2^-149 below the normal numbers), of values in float64: a
    series for the exponential to 2^-33, sums and reciprocals to 2^-46, so 2^-30 with room.  Without the
    renormalisation the softmax's sum has float32 terms e^x: x is rounded as a difference and times log2 e, which is
    2 |x| 2^-24 of the term, and the exponential by 2^-23; the terms' mean of |x| is at most the entropy, ln 600; up to
    16 of them are added in float32, in four levels of 2^-24: at most (7.4 + 2) 2^-23 < 2^-19.  The same sum weighs the renormalisation's 1e-20, which counts where biases
    push the chosen experts as low as in the last rows."""
    g = torch.Generator().manual_seed(E + k)
    logits = torch.randn(200, E, generator=g) * 3
    logits[150:175] *= 12                                     # scores down to 1e-40
    logits[175:, E // 2:] -= 40 + torch.arange(25)[:, None].float()
    kw = dict(score=score, num_groups=G, topk_groups=KG, group_top=group_top, renorm=renorm, scale=2.5)
    for low in (False, True) if biased else (False,):
        bias = (torch.randn(E, generator=g) * 0.1) if biased else None
        if low:
            bias[E // 2:] += 2.0
        idx, w = _topk((logits.repeat(times, 1)).cuda(), k, None if bias is None else bias.cuda(), **dict(kw))
        ref_i, ref_w = front.gate_topk(_f64(logits), None if bias is None else _f64(bias), k, **kw)
        assert np.array_equal(idx.cpu().numpy(), np.tile(ref_i, (times, 1)))
        ref_w = np.tile(ref_w, (times, 1))
        off = 2.0 ** -19 if score == "softmax" and (low or not renorm) else 2.0 ** -30
        err = np.abs(_f64(w) - ref_w) - ((2.0 ** -24 + off) * np.abs(ref_w) + 2.0 ** -150)
        assert (err <= 0).all(), f"{int((err > 0).sum())} of {err.size} weights"


# ------------------------------------------------------------------------------------ together
class Chain:
    """norm -> gate -> topk -> expert layer -> norm of the next layer, on buffers made once."""

    def __init__(self, T, H, I, E, k, recipe, seed=0, num_valid=None):
        self.spec = synth.Spec(T, H, I, E + 1, k + 1, recipe=recipe, seed=900 + seed, weight_set=900)
        g = torch.Generator().manual_seed(seed)
        self.weights = synth.make_weights(self.spec, "cuda")
        self.w_norm = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
        self.w_gate = (torch.randn(E, H, generator=g) / H ** 0.5).cuda()
        self.bias = (0.05 * torch.randn(E, generator=g)).cuda()
        self.x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        self.residual = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        self.num_valid = num_valid
        self.norm = mm.NormProblem.make(T, H, recipe)
        self.gate = mm.GateProblem.make(T, H, E, mm.DTYPE_F32)
        self.topk = mm.TopkProblem.make(T, E, k, score=mm.SCORE_SIGMOID, num_groups=4, topk_groups=2, group_top=2,
                                        num_shared=1, flags=mm.FLAG_TOPK_RENORM)
        self.layer = mm.MegaMoE(mm.Problem.make(T, H, I, E + 1, k + 1, recipe), "cuda")
        new = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.residual_out, self.normed, self.y, self.normed2 = (new(T, H) for _ in range(4))
        self.residual2 = new(T, H)
        self.q = new(T, H, dtype=torch.uint8)
        self.q_sf = new(T, H // 128, dtype=torch.float32) if recipe == 0 else new(T, H // 32, dtype=torch.uint8)
        self.logits = new(T, E, dtype=torch.float32)
        self.idx, self.w = new(T, k + 1, dtype=torch.int32), new(T, k + 1, dtype=torch.float32)

    def outputs(self):
        return [self.residual_out, self.normed, self.q, self.q_sf, self.logits, self.idx, self.w, self.y,
                self.normed2, self.residual2]

    def __call__(self):
        W = self.weights
        mm.mega_moe_norm_quant(self.norm, self.x, self.w_norm, residual=self.residual, residual_out=self.residual_out,
                               normed=self.normed, q=self.q, q_sf=self.q_sf)
        mm.mega_moe_gate_logits(self.gate, self.normed, self.w_gate, self.logits)
        mm.mega_moe_gate_topk(self.topk, self.logits, self.idx, self.w, bias=self.bias, num_valid=self.num_valid)
        self.layer(self.q, self.q_sf, self.idx, self.w, W["l1_w"], W["l1_sf"], W["l2_w"], W["l2_sf"], y=self.y)
        mm.mega_moe_norm_quant(self.norm, self.y, self.w_norm, residual=self.residual_out,
                               residual_out=self.residual2, normed=self.normed2)


@pytest.mark.parametrize("recipe", [0, 1, 2])
@pytest.mark.parametrize("T", [1, 45])
def test_chain_with_the_expert_layer(T, recipe):
    _say("chain", T, recipe)
    c = Chain(T, 512, 256, 16, 3, recipe)
    c()
    torch.cuda.synchronize()
    _check_norm(dict(residual_out=c.residual_out, normed=c.normed, q=c.q, q_sf=c.q_sf), c.x, c.residual, c.w_norm, recipe)
    ref, mag = front.gate_logits(_f64(c.normed), _f64(c.w_gate))
    assert (np.abs(_f64(c.logits) - ref) <= (512 * 3 + 8) * 2.0 ** -23 * mag).all()
    ref_i, ref_w = front.gate_topk(_f64(c.logits), _f64(c.bias), 3, score="sigmoid", num_groups=4, topk_groups=2,
                                   group_top=2, num_shared=1, renorm=True)
    assert np.array_equal(c.idx.cpu().numpy(), ref_i)
    P = dict(c.weights, x=c.q, x_sf=c.q_sf, topk_idx=c.idx, topk_w=c.w)
    assert_y_close(c.y.view(torch.int16).cpu().numpy(), run_oracle(c.spec, P)["y"], f"chain {recipe}")
    total = (c.y.float() + c.residual_out.float()).to(torch.bfloat16)
    assert torch.equal(c.residual2, total)


def test_chain_padded_batch():
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    c = Chain(32, 512, 256, 16, 3, 1, num_valid=n)
    c.x[20:] = float("nan")
    c()
    assert (c.idx[20:] == -1).all() and (c.y[20:] == 0).all() and torch.isfinite(c.y[:20].float()).all()
    d = Chain(32, 512, 256, 16, 3, 1)
    d()
    for a, b in zip(c.outputs(), d.outputs()):
        assert torch.equal(a[:20].view(torch.uint8), b[:20].view(torch.uint8))


def test_chain_captured_and_replayed():
    """Two chains captured in two graphs, replayed with eager work and new inputs between."""
    chains = [Chain(24, 512, 256, 16, 3, r, seed=r) for r in (0, 2)]
    for c in chains:
        c()
    torch.cuda.synchronize()
    graphs = []
    for c in chains:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for rep in range(3):
        expected = []
        for c in chains:
            c.x.copy_(torch.randn(24, 512, generator=torch.Generator().manual_seed(50 + rep)).to(torch.bfloat16))
            c()
            torch.cuda.synchronize()
            expected.append([t.clone() for t in c.outputs()])
            for t in c.outputs():
                t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, ref in zip(chains, expected):
            for a, b in zip(c.outputs(), ref):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep


def test_side_streams_at_the_same_time():
    """The operators on two streams at once, given as an argument and as the current one."""
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    X, R, W = _norm_inputs(400, 2048, seed=1)
    G = torch.randn(96, 2048, generator=torch.Generator().manual_seed(2)).cuda()
    ref = _norm(X, R, W, 0)
    ref_l = _gate(ref["normed"], G)
    ref_i, ref_w = _topk(ref_l, 6)
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s in (s1, s2):
            with torch.cuda.stream(s):
                n = _norm(X, R, W, 0, stream=s)
                lg = _gate(n["normed"], G)
                got.append((n, lg, *_topk(lg, 6, stream=s.cuda_stream)))
        torch.cuda.synchronize()
        for n, lg, i, w in got:
            for k in ref:
                assert torch.equal(n[k].view(torch.uint8), ref[k].view(torch.uint8))
            assert torch.equal(lg, ref_l) and torch.equal(i, ref_i) and torch.equal(w, ref_w)


def test_binding_refusals_on_the_device():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(256, dtype=torch.bfloat16, device="cuda")
    p = mm.NormProblem.make(4, 256)
    for bad in (dict(normed=x.float()), dict(normed=x[:3]), dict(residual=x.t()), dict(normed=x.cpu()),
                dict(q=torch.zeros(4, 256, device="cuda")), dict(normed=torch.zeros(4, 512, device="cuda").bfloat16()[:, :256])):
        with pytest.raises(ValueError):
            mm.mega_moe_norm_quant(p, x, w, **bad)
    with pytest.raises(mm.MegaMoEError) as ei:
        mm.mega_moe_norm_quant(p, x, w)                        # no output
    assert ei.value.status == -1
    with pytest.raises(mm.MegaMoEError) as ei:
        mm.mega_moe_norm_quant(p, x, w, normed=x)              # output on its input
    assert ei.value.status == -1
    with pytest.raises(ValueError):
        mm.mega_moe_gate_logits(mm.GateProblem.make(4, 256, 8), x, x, torch.zeros(4, 8, device="cuda"))
    with pytest.raises(ValueError):
        mm.mega_moe_gate_topk(mm.TopkProblem.make(4, 256, 8), x, torch.zeros(4, 8, device="cuda"),
                              torch.zeros(4, 8, device="cuda"))


def test_binding_refuses_other_strides_than_the_problems():
    """Rows as far apart as the problem says, whatever the tensor's shape; a single row has no stride."""
    T, H, E = 4, 256, 40
    wide = torch.zeros(T, H + 16, dtype=torch.bfloat16, device="cuda")
    x, tight = wide[:, :H], torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    w, normed = torch.ones(H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def norm(x, residual=None, residual_out=None, **strides):
        mm.mega_moe_norm_quant(mm.NormProblem.make(T, H, **strides), x, w, residual=residual, residual_out=residual_out,
                               normed=normed)

    norm(x, x_stride=H + 16)
    norm(tight, x, x, residual_stride=H + 16)
    for args, strides in (((x,), {}), ((tight,), dict(x_stride=H + 16)), ((x,), dict(x_stride=H + 8)),
                          ((tight, x), {}), ((tight, tight, x), {}), ((tight, x, tight), dict(residual_stride=H + 16)),
                          ((wide.t().contiguous().t()[:, :H],), dict(x_stride=H + 16))):
        with pytest.raises(ValueError, match="expected"):
            norm(*args, **strides)
    mm.mega_moe_norm_quant(mm.NormProblem.make(1, H), x[:1], w, normed=normed[:1])

    gate, logits = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, E, device="cuda")
    mm.mega_moe_gate_logits(mm.GateProblem.make(T, H, E, x_stride=H + 16), x, gate, logits)
    for x_bad, weight, stride in ((x, gate, 0), (tight, gate, H + 16), (x, gate, H + 8),
                                  (tight, torch.zeros(E, H + 8, dtype=torch.bfloat16, device="cuda")[:, :H], 0)):
        with pytest.raises(ValueError, match="expected"):
            mm.mega_moe_gate_logits(mm.GateProblem.make(T, H, E, x_stride=stride), x_bad, weight, logits)
    with pytest.raises(ValueError, match="expected"):
        mm.mega_moe_gate_logits(mm.GateProblem.make(T, H, E), tight, gate, torch.empty(T, E + 4, device="cuda")[:, :E])

    far = torch.zeros(T, E + 3, device="cuda")[:, :E]
    idx, tw = torch.empty(T, 2, dtype=torch.int32, device="cuda"), torch.empty(T, 2, device="cuda")
    mm.mega_moe_gate_topk(mm.TopkProblem.make(T, E, 2, logits_stride=E + 3), far, idx, tw)
    for l_bad, stride in ((far, 0), (logits, E + 3), (far, E + 4), (logits.t().contiguous().t(), 0)):
        with pytest.raises(ValueError, match="expected"):
            mm.mega_moe_gate_topk(mm.TopkProblem.make(T, E, 2, logits_stride=stride), l_bad, idx, tw)
    with pytest.raises(ValueError, match="expected"):
        mm.mega_moe_gate_topk(mm.TopkProblem.make(T, E, 2), logits, idx, torch.empty(2, T, device="cuda").t())
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,E", [(37, 64), (8195, 64), (40, 600)])
def test_topk_captured_batch_with_other_valid_rows_at_each_replay(T, E):
    g = torch.Generator().manual_seed(T)
    logits, bias = torch.randn(T, E, generator=g).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    p = mm.TopkProblem.make(T, E, 6, score=mm.SCORE_SIGMOID, num_groups=4, topk_groups=2, group_top=2, num_shared=1,
                            flags=mm.FLAG_TOPK_RENORM)
    idx, w = torch.empty(T, 7, dtype=torch.int32, device="cuda"), torch.empty(T, 7, device="cuda")
    mm.mega_moe_gate_topk(p, logits, idx, w, bias=bias, num_valid=n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mm.mega_moe_gate_topk(p, logits, idx, w, bias=bias, num_valid=n)
    for valid in (T, T - 1, 0, T // 2, 1, T + 5):
        logits.copy_(torch.randn(T, E, generator=g))
        logits[max(valid, 0):] = float("nan")
        n.fill_(valid)
        eager_i, eager_w = _topk(logits, 6, bias, n, score="sigmoid", num_groups=4, topk_groups=2, group_top=2,
                                 num_shared=1, renorm=True)
        idx.fill_(-77)
        w.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, eager_i) and torch.equal(w, eager_w), valid
        assert (idx[min(valid, T):] == -1).all() and (w[min(valid, T):] == 0).all()
        assert (idx[:min(valid, T), 6] == E).all() and (idx[:min(valid, T)] >= 0).all()
