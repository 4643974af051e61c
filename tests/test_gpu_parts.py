"""The layer in parts on an MI355X, against its float64 oracle.

Tolerances, from the arithmetic.  Sorting moves bytes: equal.  Back: a float32 multiply-add a pair, each off by at most
2^-24 of a partial sum, which is at most the sum of the terms' magnitudes; d_rows is one product; d_w adds eight products in
float32 (8 roundings of partial sums), the rest in float64, and is rounded to float32.  Product: the layer's bound on the
hardware's block sums (EPS_MFMA of the sum of magnitudes), a float32 rounding for the scales' product, the scaled block
and each addition: 2^-23 (K/128 + 2) of the magnitudes is more than that.  Activation: the exponential's argument
|g| log2(e) is rounded (with the constant: 1.5 2^-24 |g| of the exponential), hardware exponential and reciprocal are good to
one unit in the last place (2^-23), and five more roundings of 2^-24: 2^-21 + 1.5 2^-24 |g| in all, twice that where two
such factors meet.  An exponential below the normal numbers (|g| above 87.3) may be 0: that is off by at most 2^-126, and
silu(g) by |g| 2^-126, for |g| up to 104 (beyond, the exponential is below 2^-150 itself and |g| exp(-|g|) falls): less than
2^-119, times |u|.  Last, each output is rounded by half a step: 2^-8 of the value for BF16, 2^-24 for float32, half the
distance of neighbouring codes for E4M3.
"""
import numpy as np
import pytest
import torch

import dispatch_fp8_grouped_topk_amd as mm
import oracle
import synth
from harness import EPS_MFMA, assert_y_close, e4m3_spacing, run_oracle
from oracle import parts

pytestmark = pytest.mark.gpu

DT = {"bf16": (mm.DTYPE_BF16, torch.bfloat16), "f32": (mm.DTYPE_F32, torch.float32), "e4m3": (mm.DTYPE_E4M3, torch.uint8)}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -126}     # below the normal numbers (float32: may be flushed)
E4M3 = oracle.e4m3_decode_table()


def _say(*a):
    print("[parts]", *a, flush=True)


def _f64(t):
    return t.double().cpu().numpy()


def _rows(values, pad):
    """The values as the rows of a wider buffer."""
    wide = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device="cuda")
    wide[:, :values.shape[1]] = values
    return wide[:, :values.shape[1]]


def _stride(t):
    return 0 if t.is_contiguous() else t.stride(0)


# ------------------------------------------------------------------------------------ sort
def _ids(T, E, k, masked=0.1, seed=0, beyond=True):
    rng = np.random.default_rng(seed)
    idx = rng.integers(0, E, size=(T, k))
    idx = np.where(rng.random((T, k)) < 0.5, idx, rng.integers(0, max(1, E // 5), size=(T, k)))     # uneven
    idx = np.where(rng.random((T, k)) < masked, rng.choice([-1, -7, E, E + 3] if beyond else [-1], size=(T, k)), idx)
    return torch.from_numpy(idx.astype(np.int32)).cuda()


def _row_values(T, H, kind, recipe, seed):
    g = torch.Generator().manual_seed(seed)
    if kind != "e4m3":
        return torch.randn(T, H, generator=g).to(DT[kind][1]).cuda(), None
    x = torch.randint(0, 256, (T, H), generator=g, dtype=torch.int16).to(torch.uint8).cuda()
    sf = torch.rand(T, H // 128, generator=g) if recipe == 0 else torch.randint(0, 256, (T, H // 32), generator=g).to(torch.uint8)
    return x, sf.cuda()


FILL = 0x5A


def _filled(*shape, dtype):
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    return torch.full((n,), FILL, dtype=torch.uint8, device="cuda").view(dtype).view(*shape)


def _sort(idx, E, x=None, x_sf=None, kind="bf16", recipe=0, H=128, stream=None, out=None):
    T, k = idx.shape
    if x is not None:
        H = x.shape[1]
    p = mm.SortProblem.make(T, H, E, k, DT[kind][0], recipe, x_stride=0 if x is None else _stride(x))
    i32 = dict(dtype=torch.int32)
    if out is None:
        out = dict(src=_filled(T * k, **i32), pos=_filled(T, k, **i32), offset=_filled(E + 1, **i32), rows=None, rows_sf=None,
                   ws=_filled(mm.mega_moe_sort_workspace_size(p), dtype=torch.uint8))
        if x is not None:
            out["rows"] = _filled(T * k, H, dtype=x.dtype)
        if x_sf is not None:
            out["rows_sf"] = _filled(T * k, x_sf.shape[1], dtype=x_sf.dtype)
    mm.mega_moe_sort_tokens(p, x, idx, out["rows"], out["src"], out["pos"], out["offset"], x_sf=x_sf,
                            rows_sf=out["rows_sf"], workspace=out["ws"], stream=stream)
    return out


def _bytes(t):
    """The bytes of a tensor's rows, of a copy (whose start is aligned)."""
    n = t.shape[0] if t.dim() else 1
    return t.clone(memory_format=torch.contiguous_format).view(-1).view(torch.uint8).view(n, -1) if t.numel() else torch.empty(0, 1, dtype=torch.uint8, device=t.device)


def _check_sort(got, idx, E, x=None, x_sf=None):
    offset, src, pos = parts.sort_plan(idx.cpu().numpy(), E)
    n = len(src)
    assert np.array_equal(got["offset"].cpu().numpy(), offset)
    assert np.array_equal(got["pos"].cpu().numpy(), pos)
    assert np.array_equal(got["src"][:n].cpu().numpy(), src)
    assert (_bytes(got["src"][n:, None]) == FILL).all()
    token = torch.from_numpy(src // idx.shape[1]).long().cuda()
    for t, rows in ((x, got["rows"]), (x_sf, got["rows_sf"])):
        if t is None:
            continue
        assert torch.equal(_bytes(rows[:n]), _bytes(t[token]))
        assert n == len(rows) or (_bytes(rows[n:]) == FILL).all()


@pytest.mark.parametrize("kind,recipe", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("e4m3", 2)])
@pytest.mark.parametrize("T,H,E,k,pad", [
    (1, 7168, 256, 8, 0), (1, 128, 1, 1, 0), (2, 16384, 8192, 64, 16), (3, 384, 7, 5, 32), (128, 2048, 256, 8, 0),
    (511, 256, 33, 8, 0), (512, 256, 33, 8, 16), (513, 256, 33, 8, 16),              # either side of 4096 pairs
    (4096, 128, 3, 1, 0), (4097, 128, 3, 1, 0), (700, 4224, 256, 9, 0), (300, 640, 8192, 64, 0), (9000, 128, 1, 2, 0),
    (130, 16384, 100, 33, 16)])
def test_sort(T, H, E, k, pad, kind, recipe):
    _say("sort", T, H, E, k, pad, kind, recipe)
    idx = _ids(T, E, k, seed=T + E)
    x, sf = _row_values(T, H, kind, recipe, T + H)
    x = _rows(x, pad)
    _check_sort(_sort(idx, E, x, sf, kind, recipe), idx, E, x, sf)


@pytest.mark.parametrize("T", [100, 3000])
def test_sort_without_any_pair_and_with_one_expert_for_all(T):
    x, _ = _row_values(T, 256, "bf16", 0, 1)
    for value in (-1, 9, 4):
        idx = torch.full((T, 3), value, dtype=torch.int32, device="cuda")
        _check_sort(_sort(idx, 9, x), idx, 9, x)


@pytest.mark.parametrize("T,E,k", [(300, 50, 4), (5000, 50, 4), (20000, 8192, 60), (1050000, 17, 1), (4500000, 5, 1)])
def test_sort_plan_alone(T, E, k):
    """The last three have more than 1024 blocks of 1024 pairs, the last more tokens than one pass of the workgroups."""
    _say("plan", T, E, k)
    idx = _ids(T, E, k, seed=T)
    _check_sort(_sort(idx, E), idx, E)


@pytest.mark.parametrize("E", [1, 256, 8192])
def test_sort_of_no_tokens_zeroes_the_offsets(E):
    got = _sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), E)
    assert (got["offset"] == 0).all()


def test_sort_past_32_bits():
    """Rows of 4.3 GB in all: the last places lie beyond 2^32 bytes."""
    T, H, E, k = 16500, 16384, 5, 16
    idx = _ids(T, E, k, masked=0.0, seed=3)
    x, sf = _row_values(T, H, "e4m3", 0, 3)
    got = _sort(idx, E, x, sf, "e4m3", 0)
    offset, src, pos = parts.sort_plan(idx.cpu().numpy(), E)
    assert np.array_equal(got["pos"].cpu().numpy(), pos)
    token = torch.from_numpy(src // k).long().cuda()
    for lo in range(0, T * k, 16384):
        hi = min(T * k, lo + 16384)
        assert torch.equal(got["rows"][lo:hi], x[token[lo:hi]]) and torch.equal(got["rows_sf"][lo:hi], sf[token[lo:hi]])


def test_sort_workspaces_need_no_initialisation_and_results_repeat():
    idx = _ids(2500, 64, 4, seed=8)
    x, _ = _row_values(2500, 128, "f32", 0, 8)
    first = _sort(idx, 64, x, kind="f32")
    for fill in (0, 0x7F, 0xFF):
        first["ws"].fill_(fill)
        again = _sort(idx, 64, x, kind="f32", out={k: v.clone() if v is not None else None for k, v in first.items()})
        for k in ("src", "pos", "offset", "rows"):
            assert torch.equal(again[k], first[k])


# ------------------------------------------------------------------------------------ back
def _places(T, E, k, R, masked, seed):
    """pair_pos as the sort makes it, or with places out of range where R is smaller."""
    idx = _ids(T, E, k, masked, seed)
    return torch.from_numpy(parts.sort_plan(idx.cpu().numpy(), E)[2]).cuda()


def _unsort_problem(T, H, k, dtype, num_rows=0, stride=0):
    return mm.UnsortProblem.make(T, H, k, mm.DTYPE_BF16 if dtype == torch.bfloat16 else mm.DTYPE_F32, num_rows=num_rows,
                                 stride=stride)


BACK = [(1, 7168, 256, 8, 0, 0.0), (1, 128, 1, 1, 0, 0.0), (2, 16384, 9, 64, 8, 0.2), (37, 384, 7, 5, 24, 0.3),
        (128, 7168, 256, 8, 0, 0.0), (513, 1152, 33, 9, 0, 0.5), (70, 8192, 16, 12, 16, 0.1), (33, 8320, 16, 17, 0, 0.1),
        (2000, 128, 4, 3, 0, 0.9), (511, 256, 8, 6, 0, 0.1), (512, 256, 8, 6, 8, 0.1), (600, 8320, 8, 3, 8, 0.1)]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,E,k,pad,masked", BACK)
def test_back_and_its_gradient(T, H, E, k, pad, masked, dtype, weights):
    _say("back", T, H, E, k, pad, masked, dtype, weights)
    g = torch.Generator().manual_seed(T + H + k)
    pos = _places(T, E, k, T * k, masked, T + k)
    used = int(pos.max()) + 1
    rows = torch.randn(T * k, H, generator=g).to(dtype).cuda()
    rows[used:] = float("nan")                                     # no pair's places
    w = torch.randn(T, k, generator=g).cuda() if weights else None
    if weights:
        w[pos < 0] = float("nan")                                  # masked pairs' weights
    dy = _rows(torch.randn(T, H, generator=g).to(dtype).cuda(), pad)
    y = _rows(torch.full((T, H), float("nan"), dtype=dtype, device="cuda"), pad)
    d_rows, d_w = _filled(T * k, H, dtype=dtype), _filled(T, k, dtype=torch.float32)
    p = _unsort_problem(T, H, k, dtype, stride=_stride(y))
    mm.mega_moe_unsort_tokens(p, rows, pos, y, topk_w=w)
    mm.mega_moe_unsort_backward(p, dy, pos, rows=rows, topk_w=w, d_rows=d_rows, d_w=d_w)
    np_pos, np_rows, np_w = pos.cpu().numpy(), _f64(rows), None if w is None else _f64(w)
    ref, mag = parts.unsort(np_rows, np_pos, np_w)
    assert (np.abs(_f64(y) - ref) <= k * 2.0 ** -24 * mag + HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -10) + HALF[dtype] * k * 2.0 ** -24 * mag + TINY[dtype]).all()
    r_rows, r_w, mag = parts.unsort_backward(_f64(dy), np_rows, np_pos, np_w)
    got = _f64(d_rows)
    at = np.zeros(T * k, dtype=bool)
    at[np_pos[np_pos >= 0]] = True
    assert (np.abs(got[at] - r_rows[at]) <= (HALF[dtype] + 2.0 ** -23) * np.abs(r_rows[at]) + TINY[dtype]).all()
    assert at.all() or (_bytes(d_rows)[torch.from_numpy(~at).cuda()] == FILL).all()
    assert (np.abs(_f64(d_w) - r_w) <= 8 * 2.0 ** -24 * mag + 2.0 ** -23 * np.abs(r_w) + 2.0 ** -126).all()
    assert (d_w[pos < 0] == 0).all()
    if pad:
        assert (y._base[:, H:] == 0).all()
    # each gradient alone, and the rows' in place
    only, alone = torch.full_like(d_w, 7.0), _filled(T * k, H, dtype=dtype)
    mm.mega_moe_unsort_backward(p, dy, pos, rows=rows, topk_w=w, d_w=only)
    mm.mega_moe_unsort_backward(p, dy, pos, topk_w=w, d_rows=alone)
    assert torch.equal(only, d_w) and torch.equal(_bytes(alone), _bytes(d_rows))
    mm.mega_moe_unsort_backward(p, dy, pos, rows=rows, topk_w=w, d_rows=rows, d_w=only)
    assert torch.equal(only, d_w) and torch.equal(_bytes(rows[:used]), _bytes(d_rows[:used]))


def test_back_takes_no_place_out_of_range():
    """Places at and past num_rows, and any negative one, are pairs without a row."""
    T, H, k, R = 50, 256, 4, 30
    rng = np.random.default_rng(5)
    pos = np.full((T, k), -1, dtype=np.int32)
    pos.reshape(-1)[rng.permutation(T * k)[:R]] = rng.permutation(R)
    bad = rng.random((T, k)) < 0.5
    pos[(pos < 0) & bad] = rng.choice([R, R + 1, 2 ** 31 - 1, -2 ** 31, -5], size=int(((pos < 0) & bad).sum()))
    pos = torch.from_numpy(pos).cuda()
    rows, dy, w = torch.randn(R, H, device="cuda"), torch.randn(T, H, device="cuda"), torch.rand(T, k, device="cuda")
    y, d_rows, d_w = torch.empty(T, H, device="cuda"), torch.zeros(R, H, device="cuda"), torch.ones(T, k, device="cuda")
    p = _unsort_problem(T, H, k, torch.float32, num_rows=R)
    mm.mega_moe_unsort_tokens(p, rows, pos, y, topk_w=w)
    mm.mega_moe_unsort_backward(p, dy, pos, rows=rows, topk_w=w, d_rows=d_rows, d_w=d_w)
    ref, mag = parts.unsort(_f64(rows), pos.cpu().numpy(), _f64(w))
    assert (np.abs(_f64(y) - ref) <= (k + 1) * 2.0 ** -24 * mag).all()
    r_rows, r_w, mag = parts.unsort_backward(_f64(dy), _f64(rows), pos.cpu().numpy(), _f64(w))
    assert (np.abs(_f64(d_rows) - r_rows) <= 2.0 ** -23 * np.abs(r_rows)).all()
    assert (np.abs(_f64(d_w) - r_w) <= 9 * 2.0 ** -24 * mag).all()
    assert (d_w[(pos < 0) | (pos >= R)] == 0).all()


def test_back_past_32_bits():
    """Rows whose elements and bytes pass 2^31 and 2^32."""
    T, H, k, R = 64, 16384, 2, 270000
    pos = torch.stack([torch.arange(T) * 7, R - 1 - torch.arange(T) * 5], dim=1).to(torch.int32).cuda()
    rows = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    rows[pos.reshape(-1).long()] = torch.randn(2 * T, H, device="cuda").to(torch.bfloat16)
    taken = rows[pos.reshape(-1).long()].view(T, k, H)
    y, dy = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.randn(T, H, device="cuda").to(torch.bfloat16)
    d_w = torch.empty(T, k, device="cuda")
    p = _unsort_problem(T, H, k, torch.bfloat16, num_rows=R)
    mm.mega_moe_unsort_tokens(p, rows, pos, y)
    assert torch.equal(y, (taken[:, 0].float() + taken[:, 1].float()).to(torch.bfloat16))
    mm.mega_moe_unsort_backward(p, dy, pos, rows=rows, d_rows=rows, d_w=d_w)
    assert torch.equal(rows[pos[:, 1].long()], dy) and torch.equal(rows[pos[:, 0].long()], dy)
    want = (taken.double() * dy.double()[:, None]).sum(2)
    mag = (taken.double() * dy.double()[:, None]).abs().sum(2)
    assert ((d_w.double() - want).abs() <= 8 * 2.0 ** -24 * mag + 2.0 ** -23 * want.abs()).all()


def test_back_of_more_rows_than_one_pass_of_the_workgroups():
    T, H = 131200, 16384
    rows = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_()
    pos = torch.randperm(T, device="cuda").to(torch.int32).view(T, 1)
    y = torch.empty_like(rows)
    mm.mega_moe_unsort_tokens(_unsort_problem(T, H, 1, torch.bfloat16), rows, pos, y)
    for lo in range(0, T, 16384):
        assert torch.equal(y[lo:lo + 16384], rows[pos[lo:lo + 16384, 0].long()])


@pytest.mark.parametrize("T", [40, 600])
def test_a_captured_sort_with_other_ids_at_each_replay(T):
    """Both the one launch and the three; ids, the number of pairs and the rows change."""
    E, k, H = 20, 8, 256
    idx, (x, _) = _ids(T, E, k, seed=1), _row_values(T, H, "bf16", 0, 1)
    out = _sort(idx, E, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _sort(idx, E, x, out=out)
    for seed in range(2, 6):
        idx.copy_(_ids(T, E, k, masked=0.2 * (seed - 2), seed=seed))
        x.copy_(_row_values(T, H, "bf16", 0, seed)[0])
        for name in ("src", "pos", "offset", "rows", "ws"):
            out[name].view(torch.uint8).fill_(FILL)
        graph.replay()
        torch.cuda.synchronize()
        _check_sort(out, idx, E, x)


@pytest.mark.parametrize("T", [200, 1500])
def test_the_way_back_without_weights_is_the_sorts_gradient(T):
    """<d, sort(x)> moved along a direction: its slope is <unsort(d), direction>, exactly where every value is a small
    whole number."""
    H, E, k = 256, 12, 4
    g = torch.Generator().manual_seed(T)
    idx = _ids(T, E, k, seed=T)
    x, v = (torch.randint(-4, 5, (T, H), generator=g).float().cuda() for _ in range(2))
    d = torch.randint(-4, 5, (T * k, H), generator=g).float().cuda()
    one, two = _sort(idx, E, x, kind="f32"), _sort(idx, E, x + v, kind="f32")
    n = int(one["offset"][-1])
    slope = ((two["rows"][:n] - one["rows"][:n]).double() * d[:n].double()).sum()
    y = torch.empty(T, H, device="cuda")
    mm.mega_moe_unsort_tokens(_unsort_problem(T, H, k, torch.float32), d, one["pos"], y)
    assert float((y.double() * v.double()).sum()) == float(slope)


# --------------------------------------------------------------------------------- product
def _codes(rows, cols, g):
    q = torch.randn(rows, cols, generator=g).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8)


def _product_inputs(M, N, K, G, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x, w = _codes(M, K, g).cuda(), _codes(G * N, K, g).view(G, N, K).cuda()
    x_sf = torch.exp(torch.randn(M, K // 128, generator=g) * 0.5).mul_(0.01).cuda()
    w_sf = torch.exp(torch.randn(G, (N + 127) // 128, K // 128, generator=g) * 0.5).mul_(0.001).cuda()
    return _rows(x, pad), x_sf, w, w_sf


def _offsets(M, G, seed, behind=0):
    rng = np.random.default_rng(seed)
    share = rng.dirichlet(np.full(G, 0.5))
    count = rng.multinomial(M - behind, share)
    return torch.from_numpy(np.concatenate([[0], np.cumsum(count)]).astype(np.int32)).cuda()


def _product(x, x_sf, w, w_sf, offset=None, pad=0, stream=None, y=None):
    (M, K), (G, N, _) = x.shape, w.shape
    if y is None:
        y = _filled(M, N + pad, dtype=torch.bfloat16)[:, :N]      # beside its columns: as filled
    p = mm.ProductProblem.make(M, N, K, G, x_stride=_stride(x), y_stride=_stride(y))
    mm.mega_moe_block_product(p, x, x_sf, w, w_sf, y, group_offset=offset, stream=stream)
    return y


def _product_bound(ref, mag, K):
    eps = EPS_MFMA + (K // 128 + 2) * 2.0 ** -23
    return eps * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + TINY[torch.bfloat16]


def _check_product(y, x, x_sf, w, w_sf, offset=None):
    off = None if offset is None else offset.cpu().numpy()
    ref, mag = parts.block_product(x.cpu().numpy(), x_sf.cpu().numpy(), w.cpu().numpy(), w_sf.cpu().numpy(), off)
    got = _f64(y)
    inside = ~np.isnan(ref[:, 0])
    K = x.shape[1]
    err = np.abs(got[inside] - ref[inside])
    bound = _product_bound(ref, mag, K)[inside]
    assert (err <= bound).all(), (int((~(err <= bound)).sum()), float(np.nanmax(err / bound)))
    if not inside.all():
        assert (_bytes(y[torch.from_numpy(~inside).cuda()]) == FILL).all()
    # the typical error is far below that bound: a dropped block or a swapped scale is not
    rms = np.sqrt((ref[inside] ** 2).mean(axis=1, keepdims=True)) + 1e-300
    assert not inside.any() or np.abs(err / rms).mean() < 4e-3


DENSE = [(1, 8, 128), (1, 4096, 7168), (2, 24, 256), (5, 520, 1152), (16, 128, 128), (17, 256, 384), (33, 2120, 1024),
         (64, 136, 16384), (65, 256, 512), (100, 1024, 2048), (128, 4096, 512), (129, 392, 3712), (200, 2048, 128),
         (255, 512, 640), (257, 264, 768), (513, 1016, 1408), (777, 2120, 896), (1500, 384, 256), (2049, 640, 384),
         (4100, 256, 256), (17, 2120, 1152), (1, 4104, 1152), (33, 4104, 1152), (33, 4104, 128), (8200, 24, 1152),
         (8200, 24, 384), (6001, 136, 1152), (8200, 136, 1152), (8200, 136, 128), (50, 40008, 128), (50, 40008, 1152),
         (8200, 392, 1152), (8200, 392, 128), (2049, 4104, 1152), (8200, 776, 128), (130, 2056, 16384), (777, 2120, 3712),
         (300, 4104, 5120), (700, 2120, 5248)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense_product(M, N, K):
    _say("product", M, N, K)
    args = _product_inputs(M, N, K, 1, M + N + K)
    _check_product(_product(*args), *args)


@pytest.mark.parametrize("M,N,K,pad", [(3, 40, 256, 16), (70, 264, 384, 48), (300, 520, 640, 16), (1030, 136, 256, 144)])
def test_dense_product_of_rows_in_wider_buffers(M, N, K, pad):
    args = _product_inputs(M, N, K, 1, M, pad)
    wide = _filled(M, N + pad, dtype=torch.bfloat16)
    _check_product(_product(*args, y=wide[:, :N]), *args)
    assert (_bytes(wide[:, N:]) == FILL).all()


GROUPED = [(1, 256, 256, 5, 0), (7, 64, 384, 9, 2), (64, 520, 512, 256, 0), (128, 256, 256, 3, 7), (300, 1032, 640, 17, 33),
           (1024, 512, 1152, 128, 16), (1000, 264, 256, 2, 0), (2000, 384, 512, 8, 100), (4096, 128, 128, 40, 0),
           (3000, 512, 384, 1, 11), (7, 24, 1152, 2, 0), (300, 24, 128, 128, 0), (7, 2120, 384, 3, 0), (1000, 264, 1152, 40, 9),
           (2000, 520, 128, 40, 0), (2000, 1032, 384, 40, 9), (4096, 1032, 128, 40, 5), (3000, 520, 1152, 20, 0), (300, 1032, 3712, 17, 0), (600, 2120, 3712, 3, 9), (600, 2120, 5120, 3, 9)]


@pytest.mark.parametrize("M,N,K,G,behind", GROUPED)
def test_product_by_group(M, N, K, G, behind):
    _say("product", M, N, K, G, behind)
    args = _product_inputs(M, N, K, G, M + N + K)
    offset = _offsets(M, G, M + G, behind)
    if G == 1:
        offset = torch.tensor([behind, M - behind], dtype=torch.int32, device="cuda")
    _check_product(_product(*args, offset=offset), *args, offset)


@pytest.mark.parametrize("M,G", [(900, 12), (40, 12)])
def test_product_with_every_row_in_one_group_or_in_none(M, G):
    args = _product_inputs(M, 256, 384, G, 9)
    for g in (0, 5, G - 1):
        offset = torch.tensor([0] * (g + 1) + [M] * (G - g), dtype=torch.int32, device="cuda")
        _check_product(_product(*args, offset=offset), *args, offset)
    none = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    assert (_bytes(_product(*args, offset=none)) == FILL).all()


def test_product_takes_offsets_out_of_range_as_the_nearest_that_are():
    M, G = 100, 6
    args = _product_inputs(M, 128, 256, G, 10)
    offset = torch.tensor([-5, 20, 30, 90, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    _check_product(_product(*args, offset=offset), *args, offset)


def test_product_of_descending_offsets_stays_within_its_buffers():
    """Rows of one group alone are right, rows behind every group as they were."""
    M, G = 120, 4
    x, x_sf, w, w_sf = _product_inputs(M, 264, 256, G, 11)
    offset = torch.tensor([0, 50, 20, 100, 90], dtype=torch.int32, device="cuda")
    y = _product(x, x_sf, w, w_sf, offset)
    for g, lo, hi in ((0, 0, 20), (2, 50, 100)):
        _check_product(y[lo:hi], x[lo:hi], x_sf[lo:hi], w[g:g + 1], w_sf[g:g + 1])
    assert (_bytes(y[100:]) == FILL).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_of_groups_beyond_2_to_the_32_bytes_of_weights(M):
    """The last groups' weights lie past 4 GiB."""
    N, K, G = 4096, 4096, 260
    w = torch.zeros(G, N, K, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(M)
    w[-1] = _codes(N, K, g).cuda()
    x, x_sf, _, _ = _product_inputs(M, 8, K, 1, M)
    w_sf = torch.full((G, N // 128, K // 128), 0.001, device="cuda")
    offset = torch.tensor([0] * G + [M], dtype=torch.int32, device="cuda")
    y = _product(x, x_sf, w, w_sf, offset)
    _check_product(y, x, x_sf, w[-1:], w_sf[-1:])


def test_product_of_rows_past_2_to_the_32_bytes():
    M, K, N, stride = 1100, 256, 128, 1 << 22
    args = _product_inputs(M, N, K, 1, 12)
    wide = torch.empty((M - 1) * stride + K, dtype=torch.uint8, device="cuda")
    x = torch.as_strided(wide, (M, K), (stride, 1))
    x.copy_(args[0])
    _check_product(_product(x, *args[1:]), x, *args[1:])


@pytest.mark.parametrize("M,G", [(30, 1), (500, 1), (500, 7)])
def test_what_is_not_finite_stays_in_its_row_and_column(M, G):
    N, K = 384, 512
    x, x_sf, w, w_sf = _product_inputs(M, N, K, G, 13)
    offset = None if G == 1 else _offsets(M, G, 13)
    ref = _product(x, x_sf, w, w_sf, offset)
    x[3, 200], x_sf[7, 1], x_sf[9, 3] = 0x7F, float("inf"), float("nan")
    w[:, 50, 300], w_sf[:, 2, 0] = 0xFF, float("nan")
    got = _product(x, x_sf, w, w_sf, offset)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3], bad[9], bad[:, 50], bad[:, 256:384] = True, True, True, True
    assert torch.isnan(got[bad]).all()
    assert not torch.isfinite(got[7]).any()
    bad[7] = True
    assert torch.equal(got[~bad], ref[~bad])


@pytest.mark.parametrize("M,N,K,G", [(8192, 4096, 1024, 1), (4096, 2048, 7168, 1), (16384, 1024, 512, 16)])
def test_large_products_on_sampled_rows(M, N, K, G):
    _say("product", M, N, K, G)
    args = _product_inputs(M, N, K, G, 14)
    x, x_sf, w, w_sf = args
    offset = None if G == 1 else _offsets(M, G, 14)
    y = _product(*args, offset=offset)
    assert torch.isfinite(y).all()
    ends = [0, M] if G == 1 else offset.cpu().tolist()
    for g in range(G):
        rows = sorted({r for r in (ends[g], ends[g] + 1, (ends[g] + ends[g + 1]) // 2, ends[g + 1] - 1,
                                   ends[g] + 255, ends[g] + 256) if ends[g] <= r < ends[g + 1]})
        if rows:
            _check_product(y[rows], x[rows], x_sf[rows], w[g:g + 1], w_sf[g:g + 1])
    assert torch.equal(y.view(torch.int16), _product(*args, offset=offset).view(torch.int16))


# ------------------------------------------------------------------------------ activation
def _act_inputs(M, I, kind, wide, pad, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, wide * I, generator=g) * scale * torch.exp(torch.randn(M, 1, generator=g) * 0.5)
    return _rows(x.to(DT[kind][1]).cuda(), pad), torch.randn(M, I, generator=g).to(DT[kind][1]).cuda()


def _act(x, I, act="swiglu", recipe=0, clamp=0.0, inputs=False, num_valid=None, q=True, out=True, stream=None):
    M = x.shape[0]
    p = mm.ActProblem.make(M, I, mm.ACT_SWIGLU if act == "swiglu" else mm.ACT_NONE, recipe,
                           mm.DTYPE_BF16 if x.dtype == torch.bfloat16 else mm.DTYPE_F32, clamp,
                           mm.FLAG_CLAMP_INPUTS if inputs else 0, _stride(x))
    r = dict(q=_filled(M, I, dtype=torch.uint8) if q else None, out=_filled(M, I, dtype=torch.bfloat16) if out else None)
    r["q_sf"] = None if not q else _filled(M, I // 128, dtype=torch.float32) if recipe == 0 else _filled(M, I // 32, dtype=torch.uint8)
    mm.mega_moe_act_quant(p, x, r["q"], r["q_sf"], r["out"], num_valid, stream)
    return r


def _act_eps(x, I, act):
    """Bound of v's relative error before its rounding."""
    if act == "none":
        return np.zeros((len(x), I))
    return 2.0 ** -21 + 1.5 * 2.0 ** -24 * np.minimum(np.abs(_f64(x)[:, :I]), 90)


def _check_act(got, x, I, act, recipe, clamp, inputs, rows=None):
    rows = slice(0, x.shape[0]) if rows is None else rows
    X = x[rows]
    v = parts.activation(_f64(X), act, clamp, inputs)
    dv = _act_eps(X, I, act) * np.abs(v) + (0 if act == "none" else 2.0 ** -119 * np.nan_to_num(np.abs(_f64(X)[:, I:])))
    sf, code = parts.scales(v, recipe)
    g = 128 if recipe == 0 else 32
    if got["out"] is not None:
        assert (np.abs(_f64(got["out"][rows]) - v) <= dv * 1.01 + 2.0 ** -8 * np.abs(v) + TINY[torch.bfloat16]).all()
    if got["q"] is None:
        return
    if recipe == 0:
        got_sf = _f64(got["q_sf"][rows])
        most = dv.reshape(len(v), -1, g).max(axis=2) / 448
        assert (np.abs(got_sf - sf) <= most * 1.01 + 2.0 ** -22 * sf + 2.0 ** -149).all()
        sf = got_sf
    else:
        assert np.array_equal(got["q_sf"][rows].cpu().numpy().astype(np.int64), code)
    sf = np.repeat(sf, g, axis=1)
    scaled = np.divide(v, sf, out=np.zeros_like(v), where=sf > 0)
    off = np.divide(dv, sf, out=np.zeros_like(v), where=sf > 0)
    q = E4M3[got["q"][rows].cpu().numpy()]
    scaled = np.clip(scaled, -448, 448)
    assert (np.abs(q - scaled) <= e4m3_spacing(scaled) / 2 * (1 + 2.0 ** -18) + 1.1 * off + np.abs(scaled) * 2.0 ** -20).all()


ACT = [(1, 2048, 0), (1, 128, 0), (3, 256, 16), (37, 1152, 24), (300, 640, 0), (5, 16384, 8), (1030, 512, 0)]


@pytest.mark.parametrize("act,clamp,inputs", [("swiglu", 0.0, False), ("swiglu", 0.5, False), ("swiglu", 1.0, True), ("none", 0.0, False)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M,I,pad", ACT)
def test_activation(M, I, pad, kind, act, clamp, inputs):
    _say("activation", M, I, pad, kind, act, clamp, inputs)
    x, d = _act_inputs(M, I, kind, 2 if act == "swiglu" else 1, pad, M + I)
    x[0, :128] = 0                                                   # a group without values
    for recipe in (0, 1, 2):
        got = _act(x, I, act, recipe, clamp, inputs)
        _check_act(got, x, I, act, recipe, clamp, inputs)
        for kw in (dict(q=False), dict(out=False)):
            part = _act(x, I, act, recipe, clamp, inputs, **kw)
            for k, t in part.items():
                assert t is None or torch.equal(_bytes(t), _bytes(got[k]))
    if act == "swiglu":
        p = mm.ActProblem.make(M, I, x_dtype=DT[kind][0], swiglu_clamp=clamp, flags=mm.FLAG_CLAMP_INPUTS if inputs else 0,
                               x_stride=_stride(x))
        d_x = _rows(torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda"), pad)
        mm.mega_moe_act_backward(p, x, d, d_x)
        ref, mag = parts.act_backward(_f64(x), _f64(d), clamp, inputs)
        eps = 2 * np.concatenate([_act_eps(x, I, act)] * 2, axis=1)
        assert (np.abs(_f64(d_x) - ref) <= eps * mag * 1.01 + HALF[x.dtype] * np.abs(ref) + TINY[x.dtype]).all()
        if pad:
            assert (d_x._base[:, 2 * I:] == 0).all()
        base = x.clone() if not pad else _rows(x, pad)
        mm.mega_moe_act_backward(p, base, d, base)                   # in place
        assert torch.equal(_bytes(base), _bytes(d_x))


@pytest.mark.parametrize("valid", [0, 1, 57, 100, 1000, -3])
def test_activation_leaves_rows_behind_the_last_valid_one(valid):
    M, I = 100, 256
    x, d = _act_inputs(M, I, "bf16", 2, 0, valid + 5)
    n = min(max(valid, 0), M)
    x[n:] = float("nan")
    num = torch.tensor([valid], dtype=torch.int32, device="cuda")
    for recipe in (0, 2):
        got = _act(x, I, recipe=recipe, num_valid=num)
        if n:
            _check_act(got, x, I, "swiglu", recipe, 0.0, False, rows=slice(0, n))
        for t in got.values():
            assert n == M or (_bytes(t[n:]) == FILL).all()
    d_x = _filled(M, 2 * I, dtype=torch.bfloat16)
    mm.mega_moe_act_backward(mm.ActProblem.make(M, I), x, d, d_x, num_valid=num)
    assert n == M or (_bytes(d_x[n:]) == FILL).all()
    assert torch.isfinite(d_x[:n]).all()


def test_activation_of_more_rows_than_one_pass_of_the_workgroups():
    """More than 2^31 values; the last rows against the oracle, the valid ones end among them."""
    M, I, n = 131200, 16384, 131190
    x = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda").normal_()
    num = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = _act(x, I, recipe=2, num_valid=num)
    for rows in (slice(0, 3), slice(n - 3, n)):
        _check_act(got, x, I, "swiglu", 2, 0.0, False, rows=rows)
    for t in got.values():
        assert (_bytes(t[n:]) == FILL).all()
    del got
    d = torch.empty(M, I, dtype=torch.bfloat16, device="cuda").normal_()
    before = x[n - 3:].clone()
    mm.mega_moe_act_backward(mm.ActProblem.make(M, I), x, d, x, num_valid=num)         # in place
    ref, mag = parts.act_backward(_f64(before[:3]), _f64(d[n - 3:n]))
    eps = 2 * np.concatenate([_act_eps(before[:3], I, "swiglu")] * 2, axis=1)
    assert (np.abs(_f64(x[n - 3:n]) - ref) <= eps * mag * 1.01 + 2.0 ** -8 * np.abs(ref) + TINY[torch.bfloat16]).all()
    assert torch.equal(x[n:], before[3:])


@pytest.mark.parametrize("steps", [0, 1, 3, 60, 127, 129])
def test_power_of_two_scales_at_their_borders(steps):
    """A group's largest value within some float32 steps of 448 times a power of two, from either side: the codes must be
    those of the float64 values, without an activation and with one."""
    M, I = 4, 1024
    n = M * I // 32
    rng = np.random.default_rng(steps)
    v = rng.uniform(-1, 1, (n, 32)).astype(np.float32) * 0.1
    target = (448.0 * np.exp2(np.arange(n) % 9 - 4.0)).astype(np.float32)
    v *= target[:, None]
    side = np.where(np.arange(n) % 2, np.float32(np.inf), np.float32(0))
    big = target.copy()
    for _ in range(steps):
        big = np.nextafter(big, side)
    v[np.arange(n), np.arange(n) % 32] = big
    x = torch.from_numpy(v.reshape(M, I)).cuda()
    _check_act(_act(x, I, "none", 1), x, I, "none", 1, 0.0, False)
    g = rng.uniform(-6, 6, (n, 32)).astype(np.float32)
    silu = g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64)))
    u = (v / silu).astype(np.float32)                                # silu(g) u is v up to float32's rounding of u
    u[~np.isfinite(u) | (np.abs(u) > 1e6)] = 0
    x = torch.from_numpy(np.concatenate([g.reshape(M, I), u.reshape(M, I)], axis=1)).cuda()
    _check_act(_act(x, I, "swiglu", 1), x, I, "swiglu", 1, 0.0, False)


def test_activation_of_extreme_values():
    """Gates far out on either side, values below float32's range after scaling, values that are not finite."""
    I = 512
    x = torch.zeros(6, 2 * I, device="cuda")
    x[0, :I], x[0, I:] = torch.linspace(-120, 120, I), 1.5
    x[1, :I], x[1, I:] = -95.0, 1e30                                 # silu(g) below the normal numbers: 0
    x[2, :I], x[2, I:] = 1e-20, 1e-20
    x[3, :I], x[3, I:] = 1.0, 1e38
    x[4, 5], x[4, 200], x[4, I + 300] = float("nan"), float("inf"), float("-inf")
    x[4, 300] = 1.0
    x[4, I + 200] = 1.0
    x[5, :I], x[5, I:] = 1e3, torch.linspace(-1e30, 1e30, I)
    for recipe in (0, 1):
        got = _act(x, I, "swiglu", recipe)
        rows = [0, 2, 3, 5]       # row 2: v = 5e-41, whose scale v / 448 = 1.1e-43 is still 80 of float32's smallest steps
        _check_act({k: t[rows] for k, t in got.items()}, x[rows], I, "swiglu", recipe, 0.0, False)
        sf = got["q_sf"][4]
        per = 128 if recipe == 0 else 32
        nan = torch.isnan(sf) if recipe == 0 else sf == 255
        assert nan.nonzero()[:, 0].tolist() == [5 // per, 200 // per, 300 // per]
        codes = got["q"][4].view(-1, per)
        assert ((codes[nan] & 0x7F) == 0x7F).all() and (codes[~nan] == 0).all()
        clamped = _act(x, I, "swiglu", recipe, clamp=2.0)
        assert (clamped["q_sf"][4].isnan() if recipe == 0 else clamped["q_sf"][4] == 255).nonzero()[:, 0].tolist() == [5 // per]


def test_gradients_next_to_the_clamp():
    """silu(g) u within float32 steps of the clamp, on either side: kept or dropped as the float64 value says."""
    M, I, c = 8, 1024, 2.0
    rng = np.random.default_rng(3)
    g = rng.uniform(0.1, 6, (M, I)).astype(np.float32)
    silu = g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64)))
    u = (c / silu).astype(np.float32)
    for _ in range(3):
        u = np.where(rng.random((M, I)) < 0.5, np.nextafter(u, np.float32(np.inf)), np.nextafter(u, np.float32(0)))
    x = torch.from_numpy(np.concatenate([g, u], axis=1)).cuda()
    d = torch.ones(M, I, device="cuda")
    d_x = torch.empty_like(x)
    mm.mega_moe_act_backward(mm.ActProblem.make(M, I, x_dtype=mm.DTYPE_F32, swiglu_clamp=c), x, d, d_x)
    ref, _ = parts.act_backward(_f64(x), _f64(d), c)
    got = _f64(d_x)
    assert np.array_equal(got[:, I:] == 0, ref[:, I:] == 0) and (ref[:, I:] == 0).any() and (ref[:, I:] != 0).any()


def test_activation_gradient_against_differences():
    M, I = 16, 256
    x, d = _act_inputs(M, I, "f32", 2, 0, 6)
    for clamp, inputs in ((0.0, False), (1.0, False), (1.0, True)):
        d_x = torch.empty_like(x)
        mm.mega_moe_act_backward(mm.ActProblem.make(M, I, x_dtype=mm.DTYPE_F32, swiglu_clamp=clamp,
                                                    flags=mm.FLAG_CLAMP_INPUTS if inputs else 0), x, d, d_x)
        v = np.random.default_rng(7).standard_normal((M, 2 * I))
        h, X = 1e-7, _f64(x)
        slope = (parts.activation(X + h * v, "swiglu", clamp, inputs) - parts.activation(X - h * v, "swiglu", clamp, inputs)) / (2 * h)
        want, got = (slope * _f64(d)).sum(), (_f64(d_x) * v).sum()
        assert abs(want - got) <= 1e-5 * np.abs(slope * _f64(d)).sum()


# ------------------------------------------------------------------------- the parts together
def _layer(spec, D, stream=None):
    """The layer of the FP8 recipe from its parts: sort, product, activation, product, back."""
    T, H, I, E, k = spec.T, spec.H, spec.I, spec.E, spec.k
    s = _sort(D["topk_idx"], E, D["x"], D["x_sf"], "e4m3", 0, stream=stream)
    hidden = _product(s["rows"], s["rows_sf"], D["l1_w"], D["l1_sf"], s["offset"], stream=stream)
    a = _act(hidden, I, "swiglu", 0, spec.swiglu_clamp, num_valid=s["offset"][E:], out=False, stream=stream)
    rows = _product(a["q"], a["q_sf"], D["l2_w"], D["l2_sf"], s["offset"], stream=stream)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mm.mega_moe_unsort_tokens(_unsort_problem(T, H, k, torch.bfloat16), rows, s["pos"], y, topk_w=D["topk_w"],
                              stream=stream)
    return dict(s=s, hidden=hidden, a=a, rows=rows, y=y)


def _device(P):
    return {k: v.cuda().contiguous() for k, v in P.items()}


SPECS = [synth.CONFIGS[0], synth.Spec(300, 512, 384, 16, 4, routing="zipf", seed=31, weight_set=31),
         synth.Spec(40, 1024, 256, 8, 3, seed=32, weight_set=32, swiglu_clamp=1.0)]


@pytest.mark.parametrize("spec", SPECS, ids=[f"T{s.T}_H{s.H}_E{s.E}" for s in SPECS])
def test_the_layer_from_its_parts(spec):
    """As close to the oracle of the whole layer as the layer itself has to be (its weights are applied before the
    8-bit rounding there and after the second product here), and as the one call."""
    P = synth.make_problem(spec)
    D = _device(P)
    got = _layer(spec, D)
    ref = run_oracle(spec, P)
    bits = got["y"].view(torch.int16).cpu().numpy().view(np.uint16)
    # two BF16 roundings more than the one call's (the hidden values; the weighted rows' sum is the same): 2^-8 of
    # a value each at most, within the stated bar of 2e-2 of the largest; their mean is below 2^-9 a rounding
    y, r = oracle.bf16_bits_to_f32(bits).astype(np.float64), oracle.bf16_bits_to_f32(ref["y"]).astype(np.float64)
    assert np.abs(y - r).max() <= 4e-2 * np.abs(r).max()
    assert np.abs(y - r).sum() <= 4e-2 * np.abs(r).sum()
    one = torch.empty_like(got["y"])
    prob = mm.Problem.make(spec.T, spec.H, spec.I, spec.E, spec.k, spec.recipe, spec.swiglu_clamp)
    ws = torch.empty(mm.mega_moe_workspace_size(prob), dtype=torch.uint8, device="cuda")
    mm.mega_moe_forward(prob, D["x"], D["x_sf"], D["topk_idx"], D["topk_w"], D["l1_w"], D["l1_sf"], D["l2_w"], D["l2_sf"],
                        one, ws)
    views = mm.mega_moe_workspace_views(prob, ws)
    n = int(got["s"]["offset"][-1])
    assert torch.equal(views["expert_offset"], got["s"]["offset"]) and torch.equal(views["pair_pos"].view(-1), got["s"]["pos"].view(-1))
    assert torch.equal(views["pool_src"][:n], got["s"]["src"][:n])
    # every step against its own inputs
    s, a = got["s"], got["a"]
    _check_product(got["hidden"], s["rows"], s["rows_sf"], D["l1_w"], D["l1_sf"], s["offset"])
    _check_act(a | {"out": None}, got["hidden"], spec.I, "swiglu", 0, spec.swiglu_clamp, False, rows=slice(0, n))
    _check_product(got["rows"], a["q"], a["q_sf"], D["l2_w"], D["l2_sf"], s["offset"])


def test_the_layers_gradient_from_its_parts():
    """From y's gradient to x's and the weights', every step against its own inputs: the products take the gradients in 8
    bits and the weights transposed."""
    spec = synth.Spec(200, 512, 256, 8, 3, routing="zipf", seed=33, weight_set=33)
    T, H, I, E, k = spec.T, spec.H, spec.I, spec.E, spec.k
    D = _device(synth.make_problem(spec))
    f = _layer(spec, D)
    s, P = f["s"], T * k
    n, tail = int(s["offset"][-1]), s["offset"][E:]
    w1t, s1t = D["l1_w"].transpose(1, 2).contiguous(), D["l1_sf"].transpose(1, 2).contiguous()      # [E, H, 2I]
    w2t, s2t = D["l2_w"].transpose(1, 2).contiguous(), D["l2_sf"].transpose(1, 2).contiguous()      # [E, I, H]
    dy = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    d_rows, d_w = _filled(P, H, dtype=torch.bfloat16), torch.empty(T, k, device="cuda")
    mm.mega_moe_unsort_backward(_unsort_problem(T, H, k, torch.bfloat16), dy, s["pos"], rows=f["rows"], topk_w=D["topk_w"],
                                d_rows=d_rows, d_w=d_w)
    q2 = _act(d_rows, H, "none", 0, num_valid=tail, out=False)
    d_act = _product(q2["q"], q2["q_sf"], w2t, s2t, s["offset"])
    d_hidden = _filled(P, 2 * I, dtype=torch.bfloat16)
    mm.mega_moe_act_backward(mm.ActProblem.make(P, I), f["hidden"], d_act, d_hidden, num_valid=tail)
    q1 = _act(d_hidden, 2 * I, "none", 0, num_valid=tail, out=False)
    d_sorted = _product(q1["q"], q1["q_sf"], w1t, s1t, s["offset"])
    d_x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mm.mega_moe_unsort_tokens(_unsort_problem(T, H, k, torch.bfloat16), d_sorted, s["pos"], d_x)
    _check_product(d_act, q2["q"], q2["q_sf"], w2t, s2t, s["offset"])
    _check_product(d_sorted, q1["q"], q1["q_sf"], w1t, s1t, s["offset"])
    # the whole against float64 autograd through the same weights without the 8-bit roundings: four E4M3 roundings of
    # at most 2^-4 of a value each (in the mean square below 2^-5) stand between them
    off = s["offset"].tolist()

    def wide(w, sf):
        return E4M3_T[w.long()] * sf.double().repeat_interleave(128, 1).repeat_interleave(128, 2)

    E4M3_T = torch.tensor(E4M3, device="cuda")
    x = (E4M3_T[D["x"].long()] * D["x_sf"].double().repeat_interleave(128, 1)).requires_grad_()
    tw = D["topk_w"].double().requires_grad_()
    W1, W2 = wide(D["l1_w"], D["l1_sf"]), wide(D["l2_w"], D["l2_sf"])
    src = s["src"][:n].long()
    rows = []
    for e in range(E):
        part = x[src[off[e]:off[e + 1]] // k] @ W1[e].t()
        g, u = part.chunk(2, dim=1)
        rows.append((torch.nn.functional.silu(g) * u) @ W2[e].t())
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add(0, src // k, torch.cat(rows) * tw.view(-1)[src, None])
    y.backward(dy.double())
    for got, want in ((d_x, x.grad), (d_w, tw.grad)):
        assert (got.double() - want).norm() <= 4 * 2.0 ** -5 * want.norm()


def test_the_chain_captured_and_replayed():
    """Two layers in two graphs, replayed in turn with new inputs and eager work on buffers of their own between; every
    replay equals the eager result."""
    spec = synth.Spec(1400, 256, 128, 8, 3, routing="zipf", seed=34, weight_set=34)       # more than 4096 pairs
    T, H, I, E, k = spec.T, spec.H, spec.I, spec.E, spec.k
    D = _device(synth.make_problem(spec))
    others = [_device(synth.make_problem(synth.Spec(1400, 256, 128, 8, 3, routing="zipf", seed=35 + i, weight_set=34))) for i in range(3)]

    def make():
        P, i32 = T * k, dict(dtype=torch.int32, device="cuda")
        sp = mm.SortProblem.make(T, H, E, k, mm.DTYPE_E4M3)
        b = dict(D={n: t.clone() for n, t in D.items()}, sp=sp, rows=torch.zeros(P, H, dtype=torch.uint8, device="cuda"),
                 rows_sf=torch.zeros(P, H // 128, device="cuda"), src=torch.zeros(P, **i32), pos=torch.zeros(T, k, **i32),
                 offset=torch.zeros(E + 1, **i32), hidden=torch.zeros(P, 2 * I, dtype=torch.bfloat16, device="cuda"),
                 ws=torch.empty(mm.mega_moe_sort_workspace_size(sp), dtype=torch.uint8, device="cuda"),
                 q=torch.zeros(P, I, dtype=torch.uint8, device="cuda"), q_sf=torch.zeros(P, I // 128, device="cuda"),
                 out=torch.zeros(P, H, dtype=torch.bfloat16, device="cuda"), y=torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"),
                 d_rows=torch.zeros(P, H, dtype=torch.bfloat16, device="cuda"), d_w=torch.zeros(T, k, device="cuda"))
        return b

    def step(b):
        d, P = b["D"], T * k
        mm.mega_moe_sort_tokens(b["sp"], d["x"], d["topk_idx"], b["rows"], b["src"], b["pos"], b["offset"], x_sf=d["x_sf"],
                                rows_sf=b["rows_sf"], workspace=b["ws"])
        _product(b["rows"], b["rows_sf"], d["l1_w"], d["l1_sf"], b["offset"], y=b["hidden"])
        mm.mega_moe_act_quant(mm.ActProblem.make(P, I), b["hidden"], b["q"], b["q_sf"], num_valid=b["offset"][E:])
        _product(b["q"], b["q_sf"], d["l2_w"], d["l2_sf"], b["offset"], y=b["out"])
        p = _unsort_problem(T, H, k, torch.bfloat16)
        mm.mega_moe_unsort_tokens(p, b["out"], b["pos"], b["y"], topk_w=d["topk_w"])
        mm.mega_moe_unsort_backward(p, b["y"], b["pos"], rows=b["out"], topk_w=d["topk_w"], d_rows=b["d_rows"], d_w=b["d_w"])

    names = ("y", "d_w", "pos", "offset")
    graphs = []
    for _ in range(2):
        b = make()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(b)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(b)
        graphs.append((graph, b))
    for o in others:
        eager = make()
        for n in o:
            eager["D"][n].copy_(o[n])
        step(eager)
        torch.cuda.synchronize()
        for graph, b in graphs:
            for n in o:
                b["D"][n].copy_(o[n])
            for n in names:
                b[n].zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, b in graphs:
            for n in names:
                assert torch.equal(b[n], eager[n]), n


def test_two_streams_at_the_same_time():
    """Given as an argument and as the current stream; each with buffers of its own."""
    spec = SPECS[1]
    D = _device(synth.make_problem(spec))
    want = _layer(spec, D)["y"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):                              # so that its buffers are made and freed in its order
                got[i].append(_layer(spec, D, stream=s if i else None)["y"])
    torch.cuda.synchronize()
    for ys in got:
        for y in ys:
            assert torch.equal(y, want)


def test_the_binding_refuses_what_does_not_fit():
    x, idx = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    p = mm.SortProblem.make(4, 256, 8, 2)
    ok = dict(rows=torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda"), pool_src=torch.zeros(8, **i32),
              pair_pos=torch.zeros(4, 2, **i32), expert_offset=torch.zeros(9, **i32))
    mm.mega_moe_sort_tokens(p, x, idx, **ok)
    for name, bad in (("rows", ok["rows"][:7]), ("rows", ok["rows"].float()), ("pool_src", ok["pool_src"][:7]),
                      ("pair_pos", ok["pair_pos"].t()), ("expert_offset", ok["expert_offset"][:8]),
                      ("pool_src", ok["pool_src"].cpu())):
        with pytest.raises(ValueError, match=name):
            mm.mega_moe_sort_tokens(p, x, idx, **(ok | {name: bad}))
    with pytest.raises(ValueError, match="x is"):
        mm.mega_moe_sort_tokens(p, x[:, ::2], idx, **ok)
    with pytest.raises(ValueError, match="problem"):
        mm.mega_moe_sort_tokens(mm.NormProblem.make(4, 256), x, idx, **ok)
    with pytest.raises(ValueError, match="device tensors"):
        mm.mega_moe_sort_tokens(p, x, idx.cpu(), **ok)
    with pytest.raises(ValueError, match="y is"):
        mm.mega_moe_unsort_tokens(mm.UnsortProblem.make(4, 256, 2), ok["rows"], ok["pair_pos"], x.float())
    a = _product_inputs(4, 16, 256, 2, 1)
    y = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 4], **i32)
    with pytest.raises(ValueError, match="group_offset"):
        mm.mega_moe_block_product(mm.ProductProblem.make(4, 16, 256, 2), *a, y, group_offset=off.long())
    with pytest.raises(ValueError, match="w_sf"):
        mm.mega_moe_block_product(mm.ProductProblem.make(4, 16, 256, 2), a[0], a[1], a[2], a[3][:1], y, group_offset=off)
    with pytest.raises(mm.MegaMoEError):
        mm.mega_moe_block_product(mm.ProductProblem.make(4, 16, 256, 2), *a, y)
    with pytest.raises(ValueError, match="q_sf"):
        mm.mega_moe_act_quant(mm.ActProblem.make(4, 128, recipe=2), x, q=torch.zeros(4, 128, dtype=torch.uint8, device="cuda"),
                              q_sf=torch.zeros(4, 1, device="cuda"))
