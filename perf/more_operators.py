"""The operators that build an expert layer from parts, as measured cases: tokens sorted by expert
(`mega_moe_sort_tokens`) and back with weights applied (`mega_moe_unsort_tokens`, its gradient
`mega_moe_unsort_backward`), the 8-bit product with a scale for each block of 128, dense or by expert
(`mega_moe_block_product`), and the activation between two products with an 8-bit output
(`mega_moe_act_quant`, its gradient `mega_moe_act_backward`).  `run` computes them in elementary torch
operations, or, with `own` set, through the library's entry points.
"""
import math

import torch

own = False

FP8_MAX = 448.0
FP8 = torch.float8_e4m3fn


# ----------------------------------------------------------------------------- cases
def _sort(T, H, E, k, rows="bf16", recipe=0, masked=0.0, padded=0, pad=0, **kw):
    return dict(kw, op="sort", T=T, H=H, E=E, k=k, rows=rows, recipe=recipe, masked=masked, padded=padded, pad=pad)


def _unsort(T, H, E, k, rows="bf16", weights=True, masked=0.0, padded=0, pad=0, **kw):
    return dict(kw, op="unsort", T=T, H=H, E=E, k=k, rows=rows, weights=weights, masked=masked, padded=padded, pad=pad)


def _grad(T, H, E, k, rows="bf16", weights=True, masked=0.0, padded=0, pad=0, **kw):
    return dict(_unsort(T, H, E, k, rows, weights, masked, padded, pad, **kw), op="unsort_grad")


def _product(M, N, K, G=1, behind=0, pad=0, **kw):
    return dict(kw, op="product", M=M, N=N, K=K, G=G, behind=behind, pad=pad)


def _act(M, I, act="swiglu", recipe=0, x="bf16", clamp=0.0, inputs=False, out=False, behind=0, pad=0, **kw):
    return dict(kw, op="act", M=M, I=I, act=act, recipe=recipe, x=x, clamp=clamp, inputs=inputs, out=out,
                behind=behind, pad=pad)


def _act_grad(M, I, x="bf16", clamp=0.0, inputs=False, behind=0, pad=0, **kw):
    return dict(kw, op="act_grad", M=M, I=I, x=x, clamp=clamp, inputs=inputs, behind=behind, pad=pad)


def listed():
    return [
        # one new token: its 8-bit row with per-32 scales to its eight experts' places; latency counts
        _sort(1, 7168, 256, 8, rows="e4m3", recipe=2, name="sort one token"),
        # a prefill batch in BF16, the last rows padding and some slots masked
        _sort(8192, 7168, 256, 8, masked=0.02, padded=129, name="sort prefill"),
        # a decode batch's expert rows back in token order, weighted
        _unsort(128, 7168, 256, 8, name="back decode"),
        # the gradient of the sort: float32 rows added up without weights, an odd batch, rows of a wider buffer
        _unsort(4091, 4096, 128, 8, rows="f32", weights=False, masked=0.1, pad=64, name="back f32 unweighted"),
        # the gradient of rows and weights at an odd mid size
        _grad(1021, 4096, 128, 8, masked=0.1, name="back gradient mid"),
        # and of a prefill batch
        _grad(8192, 7168, 256, 8, name="back gradient prefill"),
        # one token through a dense layer: the weights are read once
        _product(1, 4096, 7168, name="product one token"),
        # a decode batch's 1024 rows by 128 experts, some of them without rows
        _product(1024, 4096, 1536, G=128, behind=16, name="product experts decode"),
        # an odd dense batch, a last block of weight rows that is not whole, rows of wider buffers
        _product(777, 2120, 3712, pad=64, name="product ragged"),
        # a prefill batch through a dense layer
        _product(8192, 4096, 7168, name="product prefill"),
        # the activation of a prefill batch's expert rows, clamped, with float scales
        _act(65536, 2048, clamp=10.0, behind=1000, name="swiglu prefill"),
        # its gradient at a mid size, float32, rows of wider buffers
        _act_grad(4093, 1536, x="f32", pad=64, name="swiglu gradient mid"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = {"sort": 1.1e9, "unsort": 1.1e9, "unsort_grad": 2.0e9, "act": 7e8, "act_grad": 7e8}     # bytes of a drawn case


def _fit(case, size):
    while work(case)["bytes"] > MOST[case["op"]]:
        case[size] = case[size] // 2 + 1
        for rest in ("padded", "behind"):
            if rest in case:
                case[rest] = min(case[rest], case[size] // 4)
    return case


def draw(rng):
    op = rng.choice(("sort", "unsort", "unsort_grad", "product", "product", "act", "act_grad"))
    if op in ("sort", "unsort", "unsort_grad"):
        T, E = _log_int(rng, 1, 8192), _log_int(rng, 2, 512)
        H, k = 128 * _log_int(rng, 1, 56), rng.randint(1, min(12, E))
        masked, padded = rng.choice((0.0, 0.0, 0.05, 0.5)), rng.choice((0, 0, T // 5))
        if op == "sort":
            rows = rng.choice(("bf16", "f32", "e4m3"))
            return _fit(_sort(T, H, E, k, rows, rng.randrange(3) if rows == "e4m3" else 0, masked, padded,
                              rng.choice((0, 0, 16, 144))), "T")
        make = _unsort if op == "unsort" else _grad
        return _fit(make(T, H, E, k, rng.choice(("bf16", "f32")), rng.random() < 0.6, masked, padded,
                         rng.choice((0, 0, 16, 144))), "T")
    if op == "product":
        G = rng.choice((1, 1, 1, _log_int(rng, 2, 256)))
        M, N, K = _log_int(rng, 1, 8192), 8 * _log_int(rng, 4, 1024), 128 * _log_int(rng, 1, 56)
        while M * N * K > 8192 * 4096 * 7168:
            M = M // 2 + 1
        while G * N * K > 10 ** 9:
            G = G // 2 + 1
        return _product(M, N, K, G, rng.choice((0, M // 9)) if G > 1 else 0, rng.choice((0, 0, 64, 144)))
    M, I = _log_int(rng, 1, 65536), 128 * _log_int(rng, 1, 56)
    x, clamp = rng.choice(("bf16", "f32")), rng.choice((0.0, 0.0, 1.0, 10.0))
    behind, pad = rng.choice((0, 0, M // 7)), rng.choice((0, 0, 16, 144))
    if op == "act":
        act = rng.choice(("swiglu", "swiglu", "none"))
        return _fit(_act(M, I, act, rng.randrange(3), x, clamp if act == "swiglu" else 0.0,
                         act == "swiglu" and rng.random() < 0.4, rng.random() < 0.4, behind, pad), "M")
    return _fit(_act_grad(M, I, x, clamp, rng.random() < 0.4, behind, pad), "M")


SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


def _sf_bytes(n, recipe):
    return n // 128 * 4 if recipe == 0 else n // 32


def work(case):
    c = case
    if c["op"] in ("sort", "unsort", "unsort_grad"):
        T, H, k = c["T"], c["H"], c["k"]
        used = (T - c["padded"]) * k * (1 - c["masked"])           # pairs with a place
        row = H * SIZE[c["rows"]]
        if c["op"] == "sort":
            row += _sf_bytes(H, c["recipe"]) if c["rows"] == "e4m3" else 0
            # tokens without padding are read, ids, places and sources written once
            return {"bytes": (T - c["padded"]) * row + used * (row + 4) + T * k * 8 + 4 * c["E"], "flops": 0}
        meta = T * k * (8 if c["weights"] else 4)
        if c["op"] == "unsort":
            return {"bytes": used * row + T * row + meta, "flops": 2 * used * H}
        return {"bytes": 2 * used * row + (T - c["padded"]) * row + meta + 4 * T * k, "flops": 3 * used * H}
    if c["op"] == "product":
        M, N, K = c["M"] - c["behind"], c["N"], c["K"]
        groups = min(c["G"], M)                                   # at most that many experts have rows
        blocks = -(-N // 128) * (K // 128)
        return {"bytes": M * (K + K // 32) + groups * (N * K + 4 * blocks) + 2 * M * N, "flops": 2 * M * N * K}
    n = (c["M"] - c["behind"]) * c["I"]
    if c["op"] == "act":
        wide = 2 if c["act"] == "swiglu" else 1
        return {"bytes": n * (wide * SIZE[c["x"]] + 1 + (2 if c["out"] else 0)) + _sf_bytes(n, c["recipe"]),
                "flops": 8 * n}
    return {"bytes": n * 5 * SIZE[c["x"]], "flops": 14 * n}


# ----------------------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _wide(rows, cols, dtype, pad):
    """An empty [rows, cols] buffer; with `pad`, a part of one that is `pad` columns wider."""
    return torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _rows(values, pad):
    """The values as rows of a buffer that is `pad` columns wider."""
    if not pad:
        return values.contiguous()
    wide = _wide(values.shape[0], values.shape[1], values.dtype, pad)
    wide.copy_(values)
    return wide


def _quantise(v, group):
    """(E4M3 bytes, float scales) of rows of values, a scale for each `group` columns."""
    parts = v.view(v.shape[0], -1, group)
    sf = parts.abs().amax(dim=2).clamp_min(1e-30) / FP8_MAX
    q = (parts / sf[..., None]).clamp(-FP8_MAX, FP8_MAX).to(FP8)
    return q.view(torch.uint8).view(v.shape), sf


def _weight(g, G, N, K):
    """E4M3 weights [G, N, K] of N(0, 0.02) with a float scale for each 128 x 128 block (the last rows' block may
    be part of one)."""
    nb = -(-N // 128)
    w = torch.randn(G, nb * 128, K, generator=g, device="cuda").mul_(0.02)
    w[:, N:] = 0
    sf = w.view(G, nb, 128, K // 128, 128).abs().amax(dim=(2, 4)) / FP8_MAX
    q = w.view(G, nb, 128, K // 128, 128).div_(sf[:, :, None, :, None]).clamp_(-FP8_MAX, FP8_MAX).to(FP8)
    return q.view(torch.uint8).view(G, nb * 128, K)[:, :N].contiguous(), sf


def _choices(g, c):
    """topk_idx as a router leaves it: popular and unpopular experts, slots masked, rows of padding at the end."""
    T, E, k = c["T"], c["E"], c["k"]
    score = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    idx = score.topk(k, dim=1).indices.to(torch.int32)
    if c["masked"]:
        off = torch.rand(T, k, generator=g, device="cuda") < c["masked"]
        idx = torch.where(off, torch.tensor(-1, dtype=torch.int32, device="cuda"), idx)
    if c["padded"]:
        idx[T - c["padded"]:] = -1
    return idx.contiguous()


def _places(idx, E):
    """The row of every pair with an expert, experts after each other and a pair's order kept; -1 for the others."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(flat < 0, -1, place).to(torch.int32).view(idx.shape), order, key


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "sort":
        T, H = c["T"], c["H"]
        s["topk_idx"] = _choices(g, c)
        if c["rows"] == "e4m3":
            q, sf = _quantise(randn(T, H), 128 if c["recipe"] == 0 else 32)
            s["x"] = _rows(q, c["pad"])
            s["x_sf"] = sf if c["recipe"] == 0 else (torch.ceil(torch.log2(sf)) + 127).to(torch.uint8)
        else:
            s["x"], s["x_sf"] = _rows(randn(T, H).to(_dtype(c["rows"])), c["pad"]), None
    elif c["op"] in ("unsort", "unsort_grad"):
        T, H, P = c["T"], c["H"], c["T"] * c["k"]
        s["pair_pos"] = _places(_choices(g, c), c["E"])[0]
        s["rows"] = randn(P, H).to(_dtype(c["rows"]))
        s["rows"][s["pair_pos"].clamp_min(-1).max() + 1:] = math.nan       # places that no pair has
        s["topk_w"] = torch.softmax(randn(T, c["k"]), dim=1) * 2.5 if c["weights"] else None
        if c["op"] == "unsort_grad":
            s["dy"] = _rows(randn(T, H).to(_dtype(c["rows"])), c["pad"])
    elif c["op"] == "product":
        M, N, K, G = c["M"], c["N"], c["K"], c["G"]
        q, s["x_sf"] = _quantise(randn(M, K), 128)
        s["x"] = _rows(q, c["pad"])
        s["w"], s["w_sf"] = _weight(g, G, N, K)
        s["group_offset"], s["most"] = None, M
        if G > 1:
            share = torch.softmax(randn(G), dim=0)
            group = torch.multinomial(share, M - c["behind"], replacement=True, generator=g)
            count = torch.zeros(G, dtype=torch.int64, device="cuda").scatter_add_(0, group, torch.ones_like(group))
            s["group_offset"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
            s["most"] = max(1, int(count.max()))
    else:
        M, I = c["M"], c["I"]
        wide = 2 if c["op"] == "act_grad" or c["act"] == "swiglu" else 1
        s["x"] = _rows(randn(M, wide * I).mul_(1.5).to(_dtype(c["x"])), c["pad"])
        if c["op"] == "act_grad":
            s["d_out"] = randn(M, I).to(_dtype(c["x"]))
        s["num_valid"] = torch.tensor([M - c["behind"]], dtype=torch.int32, device="cuda") if c["behind"] else None
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"sort": _own_sort, "unsort": _own_unsort, "unsort_grad": _own_grad, "product": _own_product,
                "act": _own_act, "act_grad": _own_act_grad}[op](state)
    return {"sort": _plain_sort, "unsort": _plain_unsort, "unsort_grad": _plain_grad, "product": _plain_product,
            "act": _plain_act, "act_grad": _plain_act_grad}[op](state)


def _plain_sort(s):
    c = s["case"]
    E, k, idx = c["E"], c["k"], s["topk_idx"]
    place, order, key = _places(idx, E)
    count = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offset = torch.cat([count.new_zeros(1), count[:E].cumsum(0)])
    used = torch.arange(order.numel(), device=idx.device) < offset[E]
    token = order // k
    out = {"pair_pos": place, "pool_src": torch.where(used, order, 0).to(torch.int32),
           "expert_offset": offset.to(torch.int32)}
    rows = s["x"][token]
    rows = torch.where(used[:, None], rows, torch.zeros((), dtype=rows.dtype, device=rows.device))
    out["rows"] = rows.view(FP8) if c["rows"] == "e4m3" else rows
    if s["x_sf"] is not None:
        sf = torch.where(used[:, None], s["x_sf"][token], torch.zeros((), dtype=s["x_sf"].dtype, device=idx.device))
        out["rows_sf"] = sf if c["recipe"] == 0 else sf.view(torch.float8_e8m0fnu)
    return out


def _taken(s):
    """Each pair's row in float32 [T, k, H], zeros for pairs without one."""
    place = s["pair_pos"].long()
    rows = s["rows"][place.clamp_min(0)].float()
    return torch.where(place[..., None] >= 0, rows, 0.0)


def _plain_unsort(s):
    v = _taken(s)
    if s["topk_w"] is not None:
        v = v * s["topk_w"][..., None]
    return v.sum(dim=1).to(s["rows"].dtype)


def _plain_grad(s):
    place, dy = s["pair_pos"].long(), s["dy"].float()
    w = s["topk_w"] if s["topk_w"] is not None else torch.ones(place.shape, device=dy.device)
    # a weight's gradient is a long sum that cancels
    d_w = (_taken(s).double() * dy.double()[:, None, :]).sum(dim=2).float()
    d = (w[..., None] * dy[:, None, :]).to(s["rows"].dtype).view(place.numel(), -1)
    # pairs without a row go to one behind the last, which is cut off
    at = torch.where(place >= 0, place, place.numel()).view(-1)
    d_rows = torch.zeros(place.numel() + 1, d.shape[1], dtype=d.dtype, device=d.device).index_copy_(0, at, d)
    return {"d_rows": d_rows[:-1], "d_w": d_w}


def _plain_product(s):
    c = s["case"]
    N = c["N"]
    x = s["x"].view(FP8).float() * s["x_sf"].repeat_interleave(128, dim=1)
    scale = s["w_sf"].repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)
    w = s["w"].view(FP8).float() * scale
    if s["group_offset"] is None:
        return (x @ w[0].t()).to(torch.bfloat16)
    # the rows of every expert beside each other, as many places as the largest has
    offset = s["group_offset"].long()
    at = offset[:-1, None] + torch.arange(s["most"], device=x.device)
    y = torch.bmm(x[at.clamp_max(c["M"] - 1)], w.transpose(1, 2)).to(torch.bfloat16)
    row = torch.arange(c["M"], device=x.device)
    group = torch.searchsorted(offset[1:], row, right=True).clamp_max(c["G"] - 1)
    y = y[group, (row - offset[group]).clamp(0, s["most"] - 1)]
    return torch.where((row < offset[-1])[:, None], y, torch.zeros((), dtype=y.dtype, device=y.device))


def _halves(s, x):
    """gate and up as the activation takes them."""
    c = s["case"]
    gate, up = x[:, :c["I"]], x[:, c["I"]:]
    if c["clamp"] and c["inputs"]:
        gate, up = gate.clamp(-c["clamp"], c["clamp"]), up.clamp(-c["clamp"], c["clamp"])
    return gate, up


def _used(s):
    return torch.arange(s["x"].shape[0], device=s["x"].device)[:, None] < s["num_valid"]


def _plain_act(s):
    c = s["case"]

    def value(x):
        if c["act"] == "none":
            return x
        gate, up = _halves(s, x)
        v = gate / (1 + torch.exp(-gate)) * up
        return v.clamp(-c["clamp"], c["clamp"]) if c["clamp"] and not c["inputs"] else v

    v = value(s["x"].float())
    M, I = v.shape
    if c["recipe"] == 0:
        parts = v.view(M, I // 128, 128)
        sf = parts.abs().amax(dim=2) / FP8_MAX
        q = torch.where(sf[..., None] > 0, parts / sf[..., None], 0.0)
    else:
        # a power-of-two scale jumps where amax / 448 passes a power of two: decided in 64 bits
        amax = value(s["x"].double()).abs().view(M, I // 32, 32).amax(dim=2)
        mantissa, exponent = torch.frexp(amax / FP8_MAX)
        exponent = exponent - (mantissa == 0.5).to(exponent.dtype)
        sf = torch.where(amax > 0, (exponent + 127).clamp(0, 254), 0).to(torch.uint8)
        q = v.view(M, I // 32, 32) * torch.exp2(127.0 - sf.float())[..., None]
    q = q.clamp(-FP8_MAX, FP8_MAX).to(FP8).view(M, I)
    out = {"out": v.to(torch.bfloat16)} if c["out"] else {}
    if s["num_valid"] is not None:
        used = _used(s)
        q = torch.where(used, q.view(torch.uint8), 0).view(FP8)
        sf = torch.where(used, sf, 0)
        out = {name: torch.where(used, t, 0) for name, t in out.items()}
    out["q"], out["q_sf"] = q, sf if c["recipe"] == 0 else sf.view(torch.float8_e8m0fnu)
    return out


def _plain_act_grad(s):
    c = s["case"]
    x, d = s["x"].float(), s["d_out"].float()
    gate, up = _halves(s, x)
    sigmoid = 1 / (1 + torch.exp(-gate))
    if c["clamp"] and not c["inputs"]:
        # values next to the clamp are told apart in 64 bits
        v = gate.double() / (1 + torch.exp(-gate.double())) * up.double()
        d = torch.where(v.abs() <= c["clamp"], d, 0.0)
    d_gate, d_up = d * up * sigmoid * (1 + gate * (1 - sigmoid)), d * gate * sigmoid
    d_x = torch.cat([d_gate, d_up], dim=1)
    if c["clamp"] and c["inputs"]:
        d_x = torch.where(x.abs() <= c["clamp"], d_x, 0.0)
    d_x = d_x.to(s["x"].dtype)
    return torch.where(_used(s), d_x, 0) if s["num_valid"] is not None else d_x


# The library's calls: the problem, the output buffers and the workspace are made once per state, as a program
# keeps them.  Rows behind the last used one are left as they were.
def _own_sort(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        kind = {"bf16": mm.DTYPE_BF16, "f32": mm.DTYPE_F32, "e4m3": mm.DTYPE_E4M3}[c["rows"]]
        problem = mm.SortProblem.make(T, H, E, k, kind, recipe=c["recipe"],
                                      x_stride=s["x"].stride(0) if c["pad"] else 0)
        i32 = dict(dtype=torch.int32, device="cuda")
        rows, rows_sf = torch.zeros(T * k, H, dtype=s["x"].dtype, device="cuda"), None
        out = {"pair_pos": torch.zeros(T, k, **i32), "pool_src": torch.zeros(T * k, **i32),
               "expert_offset": torch.zeros(E + 1, **i32), "rows": rows.view(FP8) if c["rows"] == "e4m3" else rows}
        if s["x_sf"] is not None:
            rows_sf = torch.zeros(T * k, s["x_sf"].shape[1], dtype=s["x_sf"].dtype, device="cuda")
            out["rows_sf"] = rows_sf if c["recipe"] == 0 else rows_sf.view(torch.float8_e8m0fnu)
        workspace = torch.empty(mm.mega_moe_sort_workspace_size(problem), dtype=torch.uint8, device="cuda")
        s["call"] = (problem, rows, rows_sf, workspace, out)
    problem, rows, rows_sf, workspace, out = s["call"]
    mm.mega_moe_sort_tokens(problem, s["x"], s["topk_idx"], rows, out["pool_src"], out["pair_pos"],
                            out["expert_offset"], x_sf=s["x_sf"], rows_sf=rows_sf, workspace=workspace)
    return out


def _unsort_problem(mm, s, stride):
    c = s["case"]
    return mm.UnsortProblem.make(c["T"], c["H"], c["k"], mm.DTYPE_BF16 if c["rows"] == "bf16" else mm.DTYPE_F32,
                                 stride=stride)


def _own_unsort(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        y = _wide(c["T"], c["H"], s["rows"].dtype, c["pad"])
        s["call"] = (_unsort_problem(mm, s, y.stride(0) if c["pad"] else 0), y)
    problem, y = s["call"]
    mm.mega_moe_unsort_tokens(problem, s["rows"], s["pair_pos"], y, topk_w=s["topk_w"])
    return y


def _own_grad(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        s["call"] = (_unsort_problem(mm, s, s["dy"].stride(0) if c["pad"] else 0), torch.zeros_like(s["rows"]),
                     torch.zeros(c["T"], c["k"], device="cuda"))
    problem, d_rows, d_w = s["call"]
    mm.mega_moe_unsort_backward(problem, s["dy"], s["pair_pos"], rows=s["rows"], topk_w=s["topk_w"], d_rows=d_rows,
                                d_w=d_w)
    return {"d_rows": d_rows, "d_w": d_w}


def _own_product(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        y = _wide(c["M"], c["N"], torch.bfloat16, c["pad"])
        s["call"] = (mm.ProductProblem.make(c["M"], c["N"], c["K"], c["G"], x_stride=s["x"].stride(0) if c["pad"] else 0,
                                            y_stride=y.stride(0) if c["pad"] else 0), y)
    problem, y = s["call"]
    mm.mega_moe_block_product(problem, s["x"], s["x_sf"], s["w"], s["w_sf"], y, group_offset=s["group_offset"])
    return y


def _act_problem(mm, s):
    c = s["case"]
    return mm.ActProblem.make(c["M"], c["I"], mm.ACT_NONE if c.get("act") == "none" else mm.ACT_SWIGLU,
                              recipe=c.get("recipe", 0), x_dtype=mm.DTYPE_BF16 if c["x"] == "bf16" else mm.DTYPE_F32,
                              swiglu_clamp=c["clamp"], flags=mm.FLAG_CLAMP_INPUTS if c["inputs"] else 0,
                              x_stride=s["x"].stride(0) if c["pad"] else 0)


def _own_act(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        M, I = c["M"], c["I"]
        q = torch.zeros(M, I, dtype=torch.uint8, device="cuda")
        if c["recipe"] == 0:
            q_sf = values = torch.zeros(M, I // 128, device="cuda")
        else:
            q_sf = torch.zeros(M, I // 32, dtype=torch.uint8, device="cuda")
            values = q_sf.view(torch.float8_e8m0fnu)
        out = {"q": q.view(FP8), "q_sf": values}
        if c["out"]:
            out["out"] = torch.zeros(M, I, dtype=torch.bfloat16, device="cuda")
        s["call"] = (_act_problem(mm, s), q, q_sf, out)
    problem, q, q_sf, out = s["call"]
    mm.mega_moe_act_quant(problem, s["x"], q=q, q_sf=q_sf, out=out.get("out"), num_valid=s["num_valid"])
    return out


def _own_act_grad(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        s["call"] = (_act_problem(mm, s), _wide(s["x"].shape[0], s["x"].shape[1], s["x"].dtype, s["case"]["pad"]))
    problem, d_x = s["call"]
    mm.mega_moe_act_backward(problem, s["x"], s["d_out"], d_x, num_valid=s["num_valid"])
    return d_x


# ----------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"sort": _exact_sort, "unsort": _exact_unsort, "unsort_grad": _exact_grad, "product": _exact_product,
            "act": _exact_act, "act_grad": _exact_act_grad}[case["op"]](s)


def _exact_sort(s):
    """Sorting computes no number: the rows by one pass over the experts."""
    c = s["case"]
    T, k, E = c["T"], c["k"], c["E"]
    flat = s["topk_idx"].reshape(-1).cpu()
    lists = [[] for _ in range(E)]
    for pair, e in enumerate(flat.tolist()):
        if e >= 0:
            lists[e].append(pair)
    pairs = [p for one in lists for p in one]
    src, place, offset = torch.zeros(T * k, dtype=torch.int32), torch.full((T * k,), -1, dtype=torch.int32), [0]
    for one in lists:
        offset.append(offset[-1] + len(one))
    src[:len(pairs)] = torch.tensor(pairs, dtype=torch.int32)
    place[torch.tensor(pairs, dtype=torch.int64)] = torch.arange(len(pairs), dtype=torch.int32)
    token = torch.tensor(pairs, dtype=torch.int64).div(k, rounding_mode="floor").to(s["x"].device)

    def moved(x, as_type=None):
        out = torch.zeros(T * k, x.shape[1], dtype=x.dtype, device=x.device)
        out[:len(pairs)] = x.index_select(0, token)
        return (out.view(as_type) if as_type else out).to(torch.float64)

    out = {"pair_pos": place.view(T, k).to(s["x"].device), "pool_src": src.to(s["x"].device),
           "expert_offset": torch.tensor(offset, dtype=torch.int32, device=s["x"].device),
           "rows": moved(s["x"], FP8 if c["rows"] == "e4m3" else None)}
    if s["x_sf"] is not None:
        out["rows_sf"] = moved(s["x_sf"], None if c["recipe"] == 0 else torch.float8_e8m0fnu)
    return out


def _exact_unsort(s):
    c = s["case"]
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        at = s["pair_pos"][:, j].long()
        t = (at >= 0).nonzero()[:, 0]
        part = s["rows"].index_select(0, at[t]).to(torch.float64)
        if c["weights"]:
            part *= s["topk_w"][t, j].to(torch.float64)[:, None]
        y.index_add_(0, t, part)
    return y


def _exact_grad(s):
    c = s["case"]
    d_rows = torch.zeros(c["T"] * c["k"], c["H"], dtype=torch.float64, device="cuda")
    d_w = torch.zeros(c["T"], c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        at = s["pair_pos"][:, j].long()
        t = (at >= 0).nonzero()[:, 0]
        dy = s["dy"].index_select(0, t).to(torch.float64)
        d_w[t, j] = torch.linalg.vecdot(s["rows"].index_select(0, at[t]).to(torch.float64), dy)
        d_rows[at[t]] = dy * s["topk_w"][t, j].to(torch.float64)[:, None] if c["weights"] else dy
    return {"d_rows": d_rows, "d_w": d_w}


def _exact_product(s):
    c = s["case"]
    M, N, K, G = c["M"], c["N"], c["K"], c["G"]
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    ends = [0, M] if s["group_offset"] is None else s["group_offset"].tolist()
    for e in range(G):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        x = s["x"][lo:hi].contiguous().view(FP8).to(torch.float64).view(hi - lo, K // 128, 128)
        x = (x * s["x_sf"][lo:hi].to(torch.float64)[..., None]).view(hi - lo, K)
        for b in range(-(-N // 128)):
            w = s["w"][e, 128 * b:128 * b + 128].view(FP8).to(torch.float64)
            w = (w.view(-1, K // 128, 128) * s["w_sf"][e, b].to(torch.float64)[:, None]).view(-1, K)
            y[lo:hi, 128 * b:128 * b + 128] = x @ w.t()
    return y


def _exact_value(c, x):
    if c["act"] == "none":
        return x
    gate, up = x[:, :c["I"]], x[:, c["I"]:]
    if c["clamp"] and c["inputs"]:
        gate, up = gate.clip(-c["clamp"], c["clamp"]), up.clip(-c["clamp"], c["clamp"])
    v = torch.sigmoid(gate) * gate * up
    return v.clip(-c["clamp"], c["clamp"]) if c["clamp"] and not c["inputs"] else v


def _exact_act(s):
    """The 8-bit output stands as the scaled values before their rounding to 8 bits."""
    c = s["case"]
    M, I, n, g = c["M"], c["I"], c["M"] - c["behind"], 128 if c["recipe"] == 0 else 32
    q = torch.zeros(M, I, dtype=torch.float64, device="cuda")
    sf = torch.zeros(M, I // g, dtype=torch.float64, device="cuda")
    out = {"out": torch.zeros(M, I, dtype=torch.float64, device="cuda")} if c["out"] else {}
    if g == 32:
        sf += 2.0 ** -127                                          # code 0 behind the last row
    for lo in range(0, n, 8192):
        hi = min(n, lo + 8192)
        v = _exact_value(c, s["x"][lo:hi].to(torch.float64))
        blocks = v.view(hi - lo, I // g, g)
        largest = torch.maximum(blocks.amax(dim=2), -blocks.amin(dim=2)) / FP8_MAX
        if g == 32:
            # the smallest power of two that is at least `largest`; the logarithm's rounding is put right by comparing
            part = torch.exp2(torch.ceil(torch.log2(largest)))
            part = torch.where(part * 0.5 >= largest, part * 0.5, part)
            part = torch.where(part < largest, part * 2, part).clamp(2.0 ** -127, 2.0 ** 127)
        else:
            part = largest
        sf[lo:hi] = part
        q[lo:hi] = torch.nan_to_num(blocks / part[..., None], nan=0.0).view(hi - lo, I)
        if c["out"]:
            out["out"][lo:hi] = v
    return dict(out, q=q, q_sf=sf)


def _exact_act_grad(s):
    c = s["case"]
    n = c["M"] - c["behind"]
    d_x = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for lo in range(0, n, 8192):
        hi = min(n, lo + 8192)
        x = s["x"][lo:hi].to(torch.float64).requires_grad_()
        # differentiated by torch from the operator's definition
        v = _exact_value(dict(c, act="swiglu"), x)
        d_x[lo:hi] = torch.autograd.grad(v, x, s["d_out"][lo:hi].to(torch.float64))[0]
    return d_x
