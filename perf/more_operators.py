"""Measured cases of routing by groups of experts, the 8-bit expert operators and 8-bit activation checkpoints.

    route       top-k of the experts of the best groups, from logits; with `train` the gradient of the logits too
    quantize    rows to 8-bit integers under one scale a row, and back
    linear      product grouped by expert, 8-bit rows times 8-bit weights with a scale for each output channel
    experts     the SwiGLU expert FFN made of two such products
    checkpoint  pre-activations kept in 8 bits (a scale for 128 columns) and the SwiGLU backward pass from them

With `own` false every operator runs in elementary torch operations in 32 bits (the choice of experts in 64: it
decides between scores that are next to each other); with `own` true through the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
MASKED = -1e30                       # selection score of an expert whose logit is -inf
TINY = 2.0**-96                      # a row or block with no larger magnitude counts as zero
BLOCK = 128                          # columns under one scale of a checkpoint

# The largest listed case of each operator; draws stay below these.
MOST_LOGITS = 16384 * 256
MOST_VALUES = 131072 * 2048
MOST_LINEAR = 2.0 * 16384 * 14336 * 4096
MOST_FLOPS = 6.0 * 16384 * 4096 * 14336
MOST_WEIGHTS = 3 * 8 * 4096 * 14336
MOST_KEPT = 16384 * 14336


def listed():
    return [
        # four sequences decode one token each: 8 of 256 experts out of 4 of 8 groups; latency alone
        {"name": "route_token", "op": "route", "T": 4, "E": 256, "groups": 8, "top_groups": 4, "k": 8, "best": 2, "score": "sigmoid", "bias": True, "renorm": True, "scale": 2.5, "masked": 0.0, "train": False},
        # a prompt batch through the same router, some experts out of service
        {"name": "route_prompt", "op": "route", "T": 16384, "E": 256, "groups": 8, "top_groups": 4, "k": 8, "best": 2, "score": "sigmoid", "bias": True, "renorm": True, "scale": 2.5, "masked": 0.02, "train": False},
        # a training step of an odd number of tokens: softmax scores, groups of 20 experts, gradients of gates and balance loss
        {"name": "route_train", "op": "route", "T": 8191, "E": 160, "groups": 8, "top_groups": 3, "k": 6, "best": 1, "score": "softmax", "bias": False, "renorm": False, "scale": 16.0, "masked": 0.0, "train": True},
        # a ragged batch with an odd width: no row starts on a boundary
        {"name": "quantize_odd", "op": "quantize", "rows": 4099, "K": 999, "dtype": "fp16"},
        # the dispatched rows of 16384 tokens with 8 experts each
        {"name": "quantize_rows", "op": "quantize", "rows": 131072, "K": 2048, "dtype": "bf16"},
        # one decoded token: 8 of 128 experts get one row each
        {"name": "linear_token", "op": "linear", "G": 128, "rows": 8, "N": 1536, "K": 2048, "load": "even", "dtype": "bf16"},
        # sizes that fill no tile, in fp32 from end to end
        {"name": "linear_odd", "op": "linear", "G": 7, "rows": 1003, "N": 1001, "K": 1044, "load": "zipf", "dtype": "fp32"},
        # one matrix of 8 experts of inner size 14336 under a skewed load
        {"name": "linear_skewed", "op": "linear", "G": 8, "rows": 16384, "N": 14336, "K": 4096, "load": "zipf", "dtype": "bf16"},
        # a decode batch: 64 tokens spread over 128 experts, about 4 rows to an expert
        {"name": "experts_batch", "op": "experts", "E": 128, "k": 8, "T": 64, "h": 2048, "F": 768, "load": "even", "dtype": "bf16"},
        # a prompt batch through few large experts under a skewed load
        {"name": "experts_skewed", "op": "experts", "E": 8, "k": 2, "T": 8192, "h": 4096, "F": 14336, "load": "zipf", "dtype": "bf16"},
        # a small micro-batch with an inner size that fills no block
        {"name": "checkpoint_odd", "op": "checkpoint", "rows": 1003, "F": 1000},
        # the rows of 8192 tokens with 2 experts each, inner size 14336
        {"name": "checkpoint_rows", "op": "checkpoint", "rows": 16384, "F": 14336},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: mostly of whole 32s, as models have them, at times any number."""
    n = _log(rng, lo, hi)
    return max(lo, n // 32 * 32) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(("route", "quantize", "linear", "experts", "checkpoint"))
    case = {"op": op}
    if op == "route":
        groups = rng.choice((1, 2, 4, 4, 8, 8, 16))
        per = rng.choice((4, 8, 16, 32, 32, rng.randint(2, 64)))
        case.update(E=groups * per, groups=groups, top_groups=rng.randint(1, groups), best=rng.randint(1, 2),
                    score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.6, renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5, 16.0)), masked=rng.choice((0.0, 0.0, 0.05)), train=rng.random() < 0.5)
        case["k"] = rng.randint(1, min(16, case["top_groups"] * per))
        case["T"] = _log(rng, 1, min(16384, MOST_LOGITS // case["E"]))
        return case
    if op == "checkpoint":
        case["F"] = 8 * max(1, _width(rng, 64, 14336) // 8)
        case["rows"] = _log(rng, 1, min(131072, MOST_KEPT // case["F"]))
        return case
    case["dtype"] = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "quantize":
        case["K"] = _width(rng, 32, 14336)
        most = MOST_VALUES // (2 if case["dtype"] == "fp32" else 1)
        case["rows"] = _log(rng, 1, max(1, min(131072, most // case["K"])))
        return case
    case["load"] = rng.choice(("even", "zipf"))
    if op == "linear":
        case["G"] = _log(rng, 1, 128)
        case["K"] = _width(rng, 64, 12288)
        case["N"] = _width(rng, 32, max(32, min(14336, MOST_WEIGHTS // (case["G"] * case["K"]))))
        case["rows"] = _log(rng, 1, max(1, min(16384, int(MOST_LINEAR / (2.0 * case["N"] * case["K"])))))
        return case
    # 16-bit outputs: in the last bits of fp32 one would see which way an activation next to a tie was rounded
    # between the two products, and that follows the exponential's last bit
    case["dtype"] = "fp16" if case["dtype"] == "fp16" else "bf16"
    case["E"] = _log(rng, 1, 128)
    case["k"] = rng.randint(1, min(8, case["E"]))
    case["h"] = _width(rng, 64, 7168)
    case["F"] = _width(rng, 32, max(32, min(14336, MOST_WEIGHTS // (3 * case["E"] * case["h"]))))
    case["T"] = _log(rng, 1, max(1, min(16384, int(MOST_FLOPS / (6.0 * case["k"] * case["h"] * case["F"])))))
    return case


# ------------------------------------------------------------------------------------------------ inputs


def _shares(case, groups, gen):
    """Each group's share of the load: even, or falling with 1 / (rank + 1) in a shuffled order."""
    if case["load"] == "even":
        return np.full(groups, 1.0 / groups)
    p = 1.0 / np.arange(1, groups + 1)
    return gen.permutation(p / p.sum())


def _group_rows(case, seed):
    """Rows of each group of a `linear` case (host side)."""
    gen = np.random.default_rng(seed)
    if case["load"] == "even" and case["rows"] < case["G"]:
        n = np.zeros(case["G"], dtype=np.int64)
        n[gen.choice(case["G"], case["rows"], replace=False)] = 1
        return n
    return gen.multinomial(case["rows"], _shares(case, case["G"], gen))


def _routes(case, seed):
    """(rows of each expert, token of each row) of an `experts` case: k different experts to a token, rows in
    token order within an expert."""
    gen = np.random.default_rng(seed)
    p = np.log(_shares(case, case["E"], gen))
    noise = gen.gumbel(size=(case["T"], case["E"]))
    ids = np.argpartition(-(p + noise), case["k"] - 1, axis=1)[:, : case["k"]] if case["k"] < case["E"] else np.tile(np.arange(case["E"]), (case["T"], 1))
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    return np.bincount(flat, minlength=case["E"]), (order // case["k"]).astype(np.int32)


def _normal(shape, dtype, gen, scale=1.0):
    return torch.randn(shape, device=gen.device, dtype=torch.float32, generator=gen).mul_(scale).to(dtype)


def _activations(shape, dtype, gen):
    """Hidden states: normal, a few columns larger than the rest as trained models have them."""
    x = torch.randn(shape, device=gen.device, dtype=torch.float32, generator=gen)
    big = torch.rand(shape[-1], device=gen.device, generator=gen) < 0.01
    return x.mul_(torch.where(big, 8.0, 1.0)).to(dtype)


def _weight(groups, N, K, gen):
    """An 8-bit weight as a checkpoint holds it: codes [G, N, K] and a scale for each output channel [G, N]."""
    codes = torch.empty((groups, N, K), dtype=torch.int8, device=gen.device)
    scales = torch.empty((groups, N), dtype=torch.float32, device=gen.device)
    for g in range(groups):
        codes[g], scales[g] = quantize(_normal((N, K), torch.bfloat16, gen, 1.0 / math.sqrt(K)))
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if own:
        from top_routing_dispatch_moe_gb300 import moe
        s["moe"] = moe
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # router logits: normal about a level of each expert's own, as a trained router's are
        logits = _normal((T, E), torch.float32, gen, 1.5) + _normal((1, E), torch.float32, gen, 0.5)
        if case["masked"]:
            logits[:, torch.rand(E, device=dev, generator=gen) < case["masked"]] = -math.inf
        s["logits"] = logits
        s["bias"] = _normal((E,), torch.float32, gen, 0.05) if case["bias"] else None
        if case["train"]:
            s["d_gates"] = _normal((T, k), torch.float32, gen, 1.0 / math.sqrt(T))
        if own:
            s["ws"] = torch.empty(moe.moe_group_route_workspace_size(T, E), dtype=torch.uint8, device=dev)
        return s
    if op == "checkpoint":
        rows, F = case["rows"], case["F"]
        blocks = -(-F // BLOCK)
        gu = _normal((rows, blocks, 2, BLOCK), torch.bfloat16, gen)
        gu.permute(0, 2, 1, 3)[..., -1, F - (blocks - 1) * BLOCK:] = 0     # columns past F
        s["gu"] = gu.view(rows, -1)
        s["d_act"] = _normal((rows, F), torch.bfloat16, gen, 0.1)
        if own:
            s["codes"] = torch.empty(s["gu"].shape, dtype=torch.int8, device=dev)
            s["scales"] = torch.empty((rows, 2 * blocks), dtype=torch.float32, device=dev)
            s["d_gu"], s["act"] = torch.empty_like(s["gu"]), torch.empty_like(s["d_act"])
        return s
    dt = DTYPE[case["dtype"]]
    if op == "quantize":
        s["x"] = _activations((case["rows"], case["K"]), dt, gen)
        if own:
            s["codes"] = torch.empty((case["rows"], case["K"]), dtype=torch.int8, device=dev)
            s["scales"] = torch.empty((case["rows"],), dtype=torch.float32, device=dev)
            s["out"] = torch.empty_like(s["x"])
        return s
    if op == "linear":
        rows = _group_rows(case, seed)
        s["x"] = _activations((case["rows"], case["K"]), dt, gen)
        codes, s["scales"] = _weight(case["G"], case["N"], case["K"], gen)
        if own:
            s["packed"] = moe.moe_int8_pack_weight(codes)
            s["out"] = torch.empty((case["rows"], case["N"]), dtype=dt, device=dev)
            s["ws"] = torch.empty(moe.moe_int8_linear_workspace_size(case["G"], case["N"], case["K"], case["rows"]), dtype=torch.uint8, device=dev)
        else:
            s["codes"] = codes
    else:
        rows, src = _routes(case, seed)
        s["x"] = _activations((case["T"], case["h"]), dt, gen)
        s["src"] = torch.from_numpy(src).to(dev)
        w = [_weight(case["E"], n, k, gen) for n, k in ((case["F"], case["h"]), (case["F"], case["h"]), (case["h"], case["F"]))]
        s["scales"] = [v[1] for v in w]
        if own:
            s["packed"] = moe.moe_int8_pack_expert_weights(*(v[0] for v in w))
            s["out"] = torch.empty((len(src), case["h"]), dtype=dt, device=dev)
            s["ws"] = torch.empty(moe.moe_int8_expert_ffn_workspace_size(case["E"], case["h"], case["F"], len(src)), dtype=torch.uint8, device=dev)
        else:
            s["codes"] = [v[0] for v in w]
    bounds = np.concatenate([[0], np.cumsum(rows)])
    s["offsets"] = torch.from_numpy(bounds.astype(np.int32)).to(dev)
    s["bounds"] = [int(v) for v in bounds]
    return s


# ---------------------------------------------------------------------------------------------- plain form


def quantize(x):
    """Codes (int8) and scales of the rows of x [..., K]: scale = amax / 127, code = the whole number nearest to
    x * 127 / amax, ties to even (in 64 bits: 32 cannot tell which side of a border a value next to it is)."""
    amax = x.abs().amax(-1).float()
    live = amax >= TINY
    q = x.double() * 127 / torch.where(live, amax, math.inf).double().unsqueeze(-1)
    # (divided by a tensor: by a plain number torch multiplies with its rounded reciprocal)
    return torch.round(q).to(torch.int8), torch.where(live, amax / amax.new_full((1,), 127.0), 0.0)


def _choose(c, logits, bias):
    """The k experts of each token, by falling selection score, in 64 bits; ties go to the lowest index."""
    L = logits.double()
    T, E, G = L.shape[0], c["E"], c["groups"]
    masked = L == -math.inf
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-L))
    else:
        e = torch.exp(L - L.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    sel = torch.where(masked, MASKED, s if bias is None else s + bias.double())
    per = sel.view(T, G, E // G).sort(dim=2, descending=True).values[..., : min(c["best"], E // G)].sum(2)
    kept = per.sort(dim=1, descending=True, stable=True).indices[:, : c["top_groups"]]
    allowed = torch.zeros((T, G), dtype=torch.bool, device=L.device).scatter_(1, kept, True)
    allowed = allowed.repeat_interleave(E // G, 1)
    return torch.where(allowed, sel, -math.inf).sort(dim=1, descending=True, stable=True).indices[:, : c["k"]]


def _scores(c, logits):
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(s):
    c, L = s["case"], s["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    ids = _choose(c, L, s["bias"])
    p = _scores(c, L)
    chosen = p.gather(1, ids)
    S = chosen.sum(1, keepdim=True)
    gates = chosen * c["scale"]
    if c["renorm"]:
        gates = torch.where(S == 0, 0.0, gates / S)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    f = counts.float() / (k * T)
    total = p.sum(1, keepdim=True)
    q = p / total if c["score"] == "sigmoid" else p
    P = q.mean(0)
    alpha = 0.01
    out = {"ids": ids.int(), "gates": gates, "counts": counts.int(), "f": f, "P": P, "aux": (alpha * E * (f * P).sum()).view(1)}
    if c["train"]:
        # the gates' gradients and that of the balance loss (1), the choice held fixed
        dg = s["d_gates"]
        if c["renorm"]:
            ds = c["scale"] * (dg - (dg * chosen).sum(1, keepdim=True) / S) / S
        else:
            ds = c["scale"] * dg
        dp = torch.zeros_like(L).scatter_(1, ids, ds)
        a = (alpha * E / T) * f
        if c["score"] == "sigmoid":
            dp = dp + (a - (a * q).sum(1, keepdim=True)) / total
            out["d_logits"] = dp * p * (1 - p)
        else:
            dp = dp + a
            out["d_logits"] = p * (dp - (dp * p).sum(1, keepdim=True))
    return out


def _product(x, xs, codes, scales):
    """(x * xs) @ (codes * scales)^T for one group's rows: x and codes hold whole numbers, the scales come after the sum."""
    return (x @ codes.float().t()) * xs.unsqueeze(1) * scales


def _checkpoint(s):
    gu, d_act = s["gu"], s["d_act"].float()
    rows, F = d_act.shape
    codes, scales = quantize(gu.view(rows, -1, BLOCK))
    v = (codes.float() * scales.unsqueeze(-1)).view(rows, -1, 2, BLOCK)
    g, u = v[:, :, 0].flatten(1), v[:, :, 1].flatten(1)
    da = torch.zeros_like(g)
    da[:, :F] = d_act
    sg = 1 / (1 + torch.exp(-g))
    d_g, d_u = da * u * sg * (1 + g * (1 - sg)), da * g * sg
    d_gu = torch.stack((d_g.view(rows, -1, BLOCK), d_u.view(rows, -1, BLOCK)), 2).view(rows, -1)
    return {"act": (g * sg * u)[:, :F].to(gu.dtype), "d_gu": d_gu.to(gu.dtype)}


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        moe = s["moe"]
        if op == "route":
            r = moe.moe_group_route(s["logits"], s["bias"], c["k"], c["groups"], c["top_groups"], score=c["score"], best=c["best"], renorm=c["renorm"], scale=c["scale"], ws=s["ws"])
            out = {"ids": r["topk_ids"], "gates": r["gates"], "counts": r["counts"], "f": r["f"], "P": r["P"], "aux": r["aux"]}
            if c["train"]:
                out["d_logits"] = moe.moe_group_route_backward(s["logits"], r["topk_ids"], s["d_gates"], r["f"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
            return out
        if op == "checkpoint":
            moe.moe_checkpoint8_save(s["gu"], codes=s["codes"], scales=s["scales"])
            d_gu, act = moe.moe_checkpoint8_swiglu_backward(s["codes"], s["scales"], s["d_act"], d_gu=s["d_gu"], act=s["act"])
            return {"act": act, "d_gu": d_gu}
        if op == "quantize":
            moe.moe_int8_quantize(s["x"], codes=s["codes"], scales=s["scales"])
            return moe.moe_int8_dequantize(s["codes"], s["scales"], out=s["out"])
        if op == "linear":
            return moe.moe_int8_linear(s["x"], s["offsets"], s["packed"], s["scales"], out=s["out"], ws=s["ws"])
        return moe.moe_int8_expert_ffn(s["x"], s["offsets"], s["packed"], *s["scales"], src=s["src"], out=s["out"], ws=s["ws"])
    if op == "route":
        return _route(s)
    if op == "checkpoint":
        return _checkpoint(s)
    codes, scales = quantize(s["x"])
    if op == "quantize":
        return (codes.float() * scales.unsqueeze(1)).to(s["x"].dtype)
    rows = codes.float()
    if op == "linear":
        out = torch.empty((c["rows"], c["N"]), dtype=s["x"].dtype, device=rows.device)
    else:
        out = torch.empty((s["src"].numel(), c["h"]), dtype=s["x"].dtype, device=rows.device)
        rows, scales = rows[s["src"]], scales[s["src"]]
    # one group at a time: the groups' sizes differ, and their weights in 32 bits would fill the card together
    for g in [g for g in range(len(s["bounds"]) - 1) if s["bounds"][g] < s["bounds"][g + 1]]:
        lo, hi = s["bounds"][g], s["bounds"][g + 1]
        if op == "linear":
            out[lo:hi] = _product(rows[lo:hi], scales[lo:hi], s["codes"][g], s["scales"][g])
            continue
        gate, up = (_product(rows[lo:hi], scales[lo:hi], s["codes"][i][g], s["scales"][i][g]) for i in (0, 1))
        a, a_scales = quantize(gate / (1.0 + torch.exp(-gate)) * up)
        out[lo:hi] = _product(a.float(), a_scales, s["codes"][2][g], s["scales"][2][g])
    return out


# ------------------------------------------------------------------------------------------------- 64 bits


def _values(x, width):
    """x after the 8-bit format, by its definition: the nearest of the 255 multiples of the largest magnitude / 127 of each
    `width` columns."""
    v = x.double().reshape(*x.shape[:-1], -1, width)
    amax = v.abs().max(-1, keepdim=True).values
    return torch.where(amax >= TINY, torch.round(v * 127 / amax.clamp_min(TINY)) * (amax / 127), 0.0).reshape(x.shape)


def _exact_route(c, s):
    L = s["logits"].double()
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    p = torch.sigmoid(L) if c["score"] == "sigmoid" else torch.softmax(L, 1)
    sel = p + s["bias"].double() if s["bias"] is not None else p.clone()
    sel[L == -math.inf] = MASKED
    best = torch.topk(sel.view(T, G, -1), min(c["best"], E // G), dim=2).values.sum(2)
    # one expert after the other: the largest score among the groups left, the lowest index where several are equal
    index = torch.arange(G, device=L.device)
    taken = torch.zeros((T, G), dtype=torch.bool, device=L.device)
    for _ in range(c["top_groups"]):
        b = best.masked_fill(taken, -math.inf)
        g = torch.where(b == b.max(1, keepdim=True).values, index, G).min(1).values
        taken[torch.arange(T, device=L.device), g] = True
    left = sel.view(T, G, -1).masked_fill(~taken.unsqueeze(2), -math.inf).view(T, E)
    index, ids = torch.arange(E, device=L.device), []
    for _ in range(k):
        ids.append(torch.where(left == left.max(1, keepdim=True).values, index, E).min(1).values)
        left[torch.arange(T, device=L.device), ids[-1]] = -math.inf
    ids = torch.stack(ids, 1)
    counts = torch.zeros(E, dtype=torch.long, device=L.device).index_add_(0, ids.reshape(-1), torch.ones_like(ids.reshape(-1)))
    f = counts.double() / (k * T)
    x = L.clone().requires_grad_(True)
    with torch.enable_grad():
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
        w = p.gather(1, ids)
        gates = c["scale"] * (w / w.sum(1, keepdim=True).clamp_min(1e-300) if c["renorm"] else w)
        P = (p / p.sum(1, keepdim=True)).mean(0)
        aux = 0.01 * E * (f * P).sum()
        out = {"ids": None, "gates": gates.detach(), "counts": None, "f": f, "P": P.detach(), "aux": aux.detach().view(1)}
        if c["train"]:
            (out["d_logits"],) = torch.autograd.grad((gates * s["d_gates"].double()).sum() + aux, x)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, op = case, case["op"]
    if op == "route":
        return _exact_route(c, s)
    if op == "checkpoint":
        F = c["F"]
        v = _values(s["gu"], BLOCK).view(c["rows"], -1, 2, BLOCK)
        keep = [v[:, :, i].reshape(c["rows"], -1)[:, :F].clone().requires_grad_(True) for i in (0, 1)]
        with torch.enable_grad():
            act = torch.nn.functional.silu(keep[0]) * keep[1]
            grads = torch.autograd.grad(act, keep, s["d_act"].double())
        d_gu = torch.zeros((c["rows"], v.shape[1], 2, BLOCK), dtype=torch.float64, device=v.device)
        for i, d in enumerate(grads):
            d_gu[:, :, i] = torch.nn.functional.pad(d, (0, -F % BLOCK)).view(c["rows"], -1, BLOCK)
        return {"act": act.detach(), "d_gu": d_gu.view(c["rows"], -1)}
    x = _values(s["x"], s["x"].shape[1])
    if op == "quantize":
        return x
    parts = []
    for g, (lo, hi) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        if lo == hi:
            continue
        if op == "linear":
            parts.append(x[lo:hi] @ (s["codes"][g].double() * s["scales"][g].double().unsqueeze(1)).t())
            continue
        w = [s["codes"][i][g].double() * s["scales"][i][g].double().unsqueeze(1) for i in range(3)]
        a = x[s["src"][lo:hi].long()]
        a = torch.nn.functional.silu(a @ w[0].t()) * (a @ w[1].t())
        parts.append(_values(a, c["F"]) @ w[2].t())
    return torch.cat(parts)


# ---------------------------------------------------------------------------------------------------- work


def work(case):
    """Inputs read once, the weights of as many groups as the load reaches at most read once in 8 bits, outputs written once."""
    op = case["op"]
    if op == "route":
        n = case["T"] * case["E"]
        return {"bytes": 4.0 * n * (2 if case["train"] else 1) + (12.0 if case["train"] else 8.0) * case["T"] * case["k"], "flops": 0.0}
    if op == "checkpoint":
        # pre-activations read, codes written and read, the gradients of both halves and act written, d_act read
        kept = 2 * BLOCK * -(-case["F"] // BLOCK)
        return {"bytes": case["rows"] * ((2.0 + 1.0 + 1.0 + 2.0) * kept + 2 * 2.0 * case["F"]), "flops": 0.0}
    el = BYTES[case["dtype"]]
    if op == "quantize":
        return {"bytes": (2.0 * el + 2.0) * case["rows"] * case["K"], "flops": 0.0}
    if op == "linear":
        used = min(case["G"], case["rows"])
        return {"bytes": el * case["rows"] * (case["K"] + case["N"]) + 1.0 * used * case["N"] * case["K"], "flops": 2.0 * case["rows"] * case["N"] * case["K"]}
    rows = case["T"] * case["k"]
    used = min(case["E"], rows)
    return {"bytes": el * (case["T"] + rows) * case["h"] + 3.0 * used * case["h"] * case["F"], "flops": 6.0 * rows * case["h"] * case["F"]}
