"""The operators in front of the expert layer, as measured cases: the residual RMS norm with an 8-bit
output (`mega_moe_norm_quant`), the gate product (`mega_moe_gate_logits`) and the choice of experts
(`mega_moe_gate_topk`).  `run` computes them in elementary torch operations, or, with `own` set, through
the library's entry points.
"""
import math

import torch

own = False

FP8_MAX = 448.0
TINY = 1e-20           # added to the sum that renormalised weights are divided by


# ----------------------------------------------------------------------------- cases
def _norm(T, H, recipe, x="bf16", w="bf16", residual=True, normed=True, pad=0, **kw):
    return dict(kw, op="norm", T=T, H=H, recipe=recipe, x=x, w=w, residual=residual, normed=normed, pad=pad)


def _gate(T, H, E, w="bf16", pad=0, **kw):
    return dict(kw, op="gate", T=T, H=H, E=E, w=w, pad=pad)


def _topk(T, E, k, score="softmax", logits="f32", bias=False, groups=1, keep=1, best=1, renorm=True, scale=1.0,
          shared=0, offline=0, padded=0, pad=0, **kw):
    return dict(kw, op="topk", T=T, E=E, k=k, score=score, logits=logits, bias=bias, groups=groups, keep=keep,
                best=best, renorm=renorm, scale=scale, shared=shared, offline=offline, padded=padded, pad=pad)


def listed():
    return [
        # one new token of one sequence, per-32 scales: latency counts
        _norm(1, 7168, 2, name="norm one token"),
        # a decode batch in the float-scale recipe
        _norm(128, 7168, 0, name="norm decode"),
        # an odd batch, a float32 residual stream, rows cut out of a wider buffer, only the 8-bit output
        _norm(777, 3712, 0, x="f32", w="f32", normed=False, pad=64, name="norm ragged f32"),
        # a prefill batch with per-32 scales
        _norm(8192, 7168, 1, name="norm prefill"),
        # one new token against 256 experts' gate rows
        _gate(1, 7168, 256, name="gate one token"),
        # a decode batch, the gate kept in float32 as routers often are
        _gate(128, 7168, 256, w="f32", name="gate decode f32"),
        # a ragged mid-size batch with fewer experts
        _gate(1021, 4096, 128, name="gate mid"),
        # a prefill batch
        _gate(8192, 7168, 256, name="gate prefill"),
        # one new token: sigmoid scores, balance bias, 4 of 8 groups
        _topk(1, 256, 8, score="sigmoid", bias=True, groups=8, keep=4, best=2, scale=2.5, name="topk one token"),
        # a mid-size batch: softmax scores from bf16 logits, renormalised
        _topk(1024, 128, 8, logits="bf16", name="topk mid"),
        # a captured batch padded to 4096 rows, one shared expert, some experts switched off
        _topk(4096, 256, 8, renorm=False, shared=1, offline=5, padded=96, name="topk shared padded"),
        # a prefill batch: sigmoid scores, balance bias, 4 of 8 groups
        _topk(8192, 256, 8, score="sigmoid", bias=True, groups=8, keep=4, best=2, scale=2.5, name="topk prefill"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "gate", "topk"))
    if op == "norm":
        c = _norm(_log_int(rng, 1, 8192), 128 * _log_int(rng, 1, 56), rng.randrange(3), rng.choice(("bf16", "f32")),
                  rng.choice(("bf16", "f32")), rng.random() < 0.7, rng.random() < 0.7, rng.choice((0, 0, 8, 136)))
        most = work(listed()[3])["bytes"]
        while work(c)["bytes"] > most:
            c["T"] = c["T"] // 2 + 1
        return c
    if op == "gate":
        return _gate(_log_int(rng, 1, 8192), 128 * _log_int(rng, 2, 56), _log_int(rng, 4, 256),
                     rng.choice(("bf16", "f32")) if rng.random() < 0.7 else "bf16", rng.choice((0, 0, 8, 72)))
    T = _log_int(rng, 1, 8192)
    groups = rng.choice((1, 1, 2, 4, 8))
    E = groups * _log_int(rng, 2, 256 // groups)
    keep = rng.randint(1, groups)
    k = rng.randint(1, min(12, E // groups * keep))
    return _topk(T, E, k, rng.choice(("softmax", "sigmoid")), rng.choice(("f32", "bf16")), rng.random() < 0.5,
                 groups, keep, rng.choice((1, 2)), rng.random() < 0.6, rng.choice((1.0, 2.5)), rng.choice((0, 0, 1, 2)),
                 rng.choice((0, 0, min(3, E - 1))), rng.choice((0, 0, T // 5)), rng.choice((0, 0, 8)))


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        b = size[c["x"]] * (3 if c["residual"] else 1) + (2 if c["normed"] else 0) + 1
        sf = n // 128 * 4 if c["recipe"] == 0 else n // 32
        return {"bytes": n * b + sf + c["H"] * size[c["w"]], "flops": 8 * n}
    if c["op"] == "gate":
        return {"bytes": c["T"] * c["H"] * 2 + c["E"] * c["H"] * size[c["w"]] + c["T"] * c["E"] * 4,
                "flops": 2 * c["T"] * c["H"] * c["E"]}
    n = c["T"] * c["E"]
    return {"bytes": n * size[c["logits"]] + c["T"] * (c["k"] + c["shared"]) * 8 + (4 * c["E"] if c["bias"] else 0),
            "flops": 6 * n}


# ----------------------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(values, pad):
    """The values as rows of a buffer that is `pad` columns wider."""
    if not pad:
        return values.contiguous()
    wide = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device=values.device)
    wide[:, :values.shape[1]] = values
    return wide[:, :values.shape[1]]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        channel = torch.exp(0.5 * randn(H))          # some channels of a hidden state are far larger than others
        s["x"] = _rows((randn(T, H) * 0.3 * channel).to(_dtype(c["x"])), c["pad"])
        s["residual"] = (randn(T, H) * channel).to(_dtype(c["x"])) if c["residual"] else None
        s["weight"] = (1 + 0.2 * randn(H)).to(_dtype(c["w"]))
        s["eps"] = 1e-6
    elif c["op"] == "gate":
        s["x"] = _rows(randn(c["T"], c["H"]).to(torch.bfloat16), c["pad"])
        s["weight"] = (randn(c["E"], c["H"]) * (1.5 / math.sqrt(c["H"]))).to(_dtype(c["w"]))
    else:
        logits = randn(c["T"], c["E"]) * 1.5 + 0.5 * randn(c["E"])
        if c["offline"]:
            off = torch.randperm(c["E"], generator=g, device="cuda")[:c["offline"]]
            logits[:, off] = -math.inf
        s["logits"] = _rows(logits.to(_dtype(c["logits"])), c["pad"])
        s["bias"] = 0.1 * randn(c["E"]) if c["bias"] else None
        s["num_valid"] = (torch.tensor([c["T"] - c["padded"]], dtype=torch.int32, device="cuda")
                          if c["padded"] else None)
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return {"norm": _own_norm, "gate": _own_gate, "topk": _own_topk}[c["op"]](state)
    return {"norm": _plain_norm, "gate": _plain_gate, "topk": _plain_topk}[c["op"]](state)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    h = x + s["residual"].float() if c["residual"] else x
    rstd = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + s["eps"])
    v = h * rstd * s["weight"].float()
    out = {}
    if c["residual"]:
        out["residual_out"] = h.to(s["x"].dtype)
    if c["normed"]:
        out["normed"] = v.to(torch.bfloat16)
    T, H = v.shape
    if c["recipe"] == 0:
        grouped = v.view(T, H // 128, 128)
        sf = grouped.abs().amax(dim=2) / FP8_MAX
        out["q_sf"] = sf
        q = torch.where(sf[..., None] > 0, grouped / sf[..., None], 0.0)
    else:
        # a power-of-two scale jumps where amax / 448 passes a power of two: decided in 64 bits
        h64 = h.double()
        rstd64 = 1.0 / torch.sqrt((h64 * h64).mean(dim=1, keepdim=True) + s["eps"])
        amax = (h64 * s["weight"].double()).abs().view(T, H // 32, 32).amax(dim=2) * rstd64
        mantissa, exponent = torch.frexp(amax / FP8_MAX)
        exponent = exponent - (mantissa == 0.5).to(exponent.dtype)
        code = torch.where(amax > 0, (exponent + 127).clamp(0, 254), 0).to(torch.uint8)
        out["q_sf"] = code.view(torch.float8_e8m0fnu)
        q = v.view(T, H // 32, 32) * torch.exp2(127.0 - code.float())[..., None]
    out["q"] = q.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).view(T, H)
    return out


def _plain_gate(s):
    return s["x"].float() @ s["weight"].float().t()


def _plain_topk(s):
    c = s["case"]
    logits = s["logits"].double()          # the order of close scores is decided in 64 bits
    T, E = logits.shape
    on = logits > -math.inf
    if c["score"] == "sigmoid":
        score = torch.sigmoid(logits)
    else:
        e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    value = score + s["bias"].double() if c["bias"] else (score if c["best"] == 2 else logits)
    value = torch.where(on, value, -math.inf)
    if c["groups"] > 1:
        per = value.view(T, c["groups"], E // c["groups"])
        best = per.sort(dim=2, descending=True).values[..., :c["best"]]
        group = torch.where(best > -math.inf, best, 0.0).sum(dim=2)
        group = torch.where(best[..., 0] > -math.inf, group, -math.inf)
        kept = group.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        mask = torch.zeros(T, c["groups"], dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        value = torch.where(mask[..., None], per, -math.inf).view(T, E)
    order = value if c["bias"] else torch.where(value > -math.inf, logits, -math.inf)
    ranked = order.sort(dim=1, descending=True, stable=True)
    idx = ranked.indices[:, :c["k"]]
    found = ranked.values[:, :c["k"]] > -math.inf
    w = torch.where(found, score.gather(1, idx), 0.0)
    if c["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + TINY)
    w = w * c["scale"]
    idx = torch.where(found, idx, -1)
    if c["shared"]:
        ids = torch.arange(E, E + c["shared"], device=idx.device).expand(T, -1)
        idx, w = torch.cat([idx, ids], dim=1), torch.cat([w, torch.ones_like(ids, dtype=w.dtype)], dim=1)
    if c["padded"]:
        valid = torch.arange(T, device=idx.device)[:, None] < s["num_valid"]
        idx, w = torch.where(valid, idx, -1), torch.where(valid, w, 0.0)
    return {"topk_idx": idx.to(torch.int32), "topk_w": w.float()}


# The library's calls: the problem and the output buffers are made once per state, as a program keeps them.
def _own_norm(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        T, H, dev = c["T"], c["H"], s["x"].device
        kind = {"bf16": mm.DTYPE_BF16, "f32": mm.DTYPE_F32}
        problem = mm.NormProblem.make(T, H, c["recipe"], kind[c["x"]], kind[c["w"]], s["eps"],
                                      x_stride=s["x"].stride(0) if c["pad"] else 0)
        q = torch.empty(T, H, dtype=torch.uint8, device=dev)
        if c["recipe"] == 0:
            q_sf = sf_values = torch.empty(T, H // 128, dtype=torch.float32, device=dev)
        else:
            q_sf = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
            sf_values = q_sf.view(torch.float8_e8m0fnu)
        out = {"q": q.view(torch.float8_e4m3fn), "q_sf": sf_values}
        if c["residual"]:
            out["residual_out"] = torch.empty(T, H, dtype=s["x"].dtype, device=dev)
        if c["normed"]:
            out["normed"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        s["call"] = (problem, q, q_sf, out)
    problem, q, q_sf, out = s["call"]
    mm.mega_moe_norm_quant(problem, s["x"], s["weight"], residual=s["residual"],
                           residual_out=out.get("residual_out"), normed=out.get("normed"), q=q, q_sf=q_sf)
    return out


def _own_gate(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        kind = {"bf16": mm.DTYPE_BF16, "f32": mm.DTYPE_F32}
        problem = mm.GateProblem.make(c["T"], c["H"], c["E"], kind[c["w"]],
                                      x_stride=s["x"].stride(0) if c["pad"] else 0)
        s["call"] = (problem, torch.empty(c["T"], c["E"], dtype=torch.float32, device=s["x"].device))
    problem, logits = s["call"]
    mm.mega_moe_gate_logits(problem, s["x"], s["weight"], logits)
    return logits


def _own_topk(s):
    import dispatch_fp8_grouped_topk_amd as mm
    if "call" not in s:
        c = s["case"]
        dev = s["logits"].device
        problem = mm.TopkProblem.make(
            c["T"], c["E"], c["k"], score=mm.SCORE_SIGMOID if c["score"] == "sigmoid" else mm.SCORE_SOFTMAX,
            logits_dtype=mm.DTYPE_BF16 if c["logits"] == "bf16" else mm.DTYPE_F32, num_groups=c["groups"],
            topk_groups=c["keep"], group_top=c["best"], scale=c["scale"], num_shared=c["shared"], shared_weight=1.0,
            flags=mm.FLAG_TOPK_RENORM if c["renorm"] else 0,
            logits_stride=s["logits"].stride(0) if c["pad"] else 0)
        cols = c["k"] + c["shared"]
        s["call"] = (problem, {"topk_idx": torch.empty(c["T"], cols, dtype=torch.int32, device=dev),
                               "topk_w": torch.empty(c["T"], cols, dtype=torch.float32, device=dev)})
    problem, out = s["call"]
    mm.mega_moe_gate_topk(problem, s["logits"], out["topk_idx"], out["topk_w"], bias=s["bias"],
                          num_valid=s["num_valid"])
    return out


# ----------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "gate": _exact_gate, "topk": _exact_topk}[case["op"]](s)


def _exact_norm(s):
    """The 8-bit output stands as the scaled values before their rounding to 8 bits."""
    c = s["case"]
    h = s["x"].to(torch.float64)
    if s["residual"] is not None:
        h = h + s["residual"].to(torch.float64)
    out = {"residual_out": h} if c["residual"] else {}
    rms = torch.linalg.vector_norm(h, dim=1, keepdim=True).square().div(c["H"]).add(s["eps"]).sqrt()
    v = (h / rms).mul_(s["weight"].to(torch.float64))
    if c["normed"]:
        out["normed"] = v
    g = 128 if c["recipe"] == 0 else 32
    blocks = v.reshape(c["T"], c["H"] // g, g)
    largest = torch.maximum(blocks.amax(dim=2), -blocks.amin(dim=2)) / FP8_MAX
    if g == 128:
        sf = largest
    else:
        # the smallest power of two that is at least `largest`; the logarithm's rounding is put right by comparing
        sf = torch.exp2(torch.ceil(torch.log2(largest)))
        sf = torch.where(sf * 0.5 >= largest, sf * 0.5, sf)
        sf = torch.where(sf < largest, sf * 2, sf).clamp(2.0 ** -127, 2.0 ** 127)
    out["q_sf"] = sf
    out["q"] = torch.nan_to_num(blocks / sf[..., None], nan=0.0).reshape(c["T"], c["H"])
    return out


def _exact_gate(s):
    w = s["weight"].to(torch.float64).t().contiguous()
    return torch.cat([rows.to(torch.float64) @ w for rows in s["x"].split(2048)])


def _exact_topk(s):
    c = s["case"]
    l = s["logits"].to(torch.float64)
    T, E = l.shape
    dead = torch.isneginf(l)
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.exp(l - torch.logsumexp(l, dim=1, keepdim=True))
    v = p + s["bias"].to(torch.float64) if c["bias"] else l.clone()
    v[dead] = -math.inf
    ids = torch.arange(E, device=l.device)

    def best_of(values, where):      # the first of the largest values of each row, of those at `where`
        masked = values.masked_fill(~where, -math.inf)
        top = masked.amax(dim=1, keepdim=True)
        first = torch.where((masked == top) & where, torch.arange(values.shape[1], device=l.device), 1 << 30)
        return first.amin(dim=1), top[:, 0]

    allowed = ~dead
    if c["groups"] > 1:
        n = E // c["groups"]
        rank_by = v if c["bias"] or c["best"] == 1 else p.masked_fill(dead, -math.inf)
        total = torch.zeros(T, c["groups"], dtype=torch.float64, device=l.device)
        alive = torch.zeros(T, c["groups"], dtype=torch.bool, device=l.device)
        for j in range(c["groups"]):
            part, where = rank_by[:, j * n:(j + 1) * n], allowed[:, j * n:(j + 1) * n].clone()
            alive[:, j] = where.any(dim=1)
            for _ in range(c["best"]):
                at, top = best_of(part, where)
                some = where.any(dim=1)
                total[:, j] += torch.where(some, top, 0.0)
                where[some, at[some]] = False
        chosen = torch.zeros_like(alive)
        for _ in range(c["keep"]):
            at, _top = best_of(total, alive & ~chosen)
            some = (alive & ~chosen).any(dim=1)
            chosen[some, at[some]] = True
        allowed = allowed & chosen.repeat_interleave(n, dim=1)
    idx = torch.full((T, c["k"] + c["shared"]), -1, dtype=torch.int64, device=l.device)
    w = torch.zeros(T, c["k"] + c["shared"], dtype=torch.float64, device=l.device)
    left = allowed.clone()
    for j in range(c["k"]):
        some = left.any(dim=1)
        at, _top = best_of(v, left)
        idx[some, j] = ids[at[some]]
        w[some, j] = p[some, at[some]]
        left[some, at[some]] = False
    if c["renorm"]:
        w /= w.sum(dim=1, keepdim=True) + TINY
    w *= c["scale"]
    for j in range(c["shared"]):
        idx[:, c["k"] + j], w[:, c["k"] + j] = E + j, 1.0
    if c["padded"]:
        idx[T - c["padded"]:], w[T - c["padded"]:] = -1, 0.0
    return {"topk_idx": idx.to(torch.int32), "topk_w": w}
