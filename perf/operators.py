"""Measured cases of the 4-bit expert operators: block quantisation, the grouped product and the expert FFN.

Formats (`fmt`): "nv" holds 16 values under an e4m3 scale, "mx" 32 values under a power of two; the values are
e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the even column in the low half. With
`own` false every operator runs in elementary torch operations in 32 bits; with `own` true through the
framework's entry points.
"""
import math

import numpy as np
import torch

own = False

BLOCK = {"nv": 16, "mx": 32}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# The largest listed case of each operator; draws stay below these.
MOST_VALUES = 131072 * 2048          # quantised values
MOST_FLOPS = 6.0 * 16384 * 4096 * 14336
MOST_LINEAR = 2.0 * 16384 * 14336 * 4096
MOST_WEIGHTS = 3 * 8 * 4096 * 14336


def listed():
    return [
        # one token's eight copies on their way to eight experts (hidden size 7168): latency alone
        {"name": "quantize_token", "op": "quantize", "rows": 8, "K": 7168, "fmt": "nv", "dtype": "bf16", "scaled": False},
        # a ragged batch with an odd width: the last block of every row is partial and no row is aligned
        {"name": "quantize_odd", "op": "quantize", "rows": 4099, "K": 999, "fmt": "mx", "dtype": "fp16", "scaled": True},
        # one expert's fp32 master weight brought to 4 bits for serving
        {"name": "quantize_weight", "op": "quantize", "rows": 12288, "K": 4096, "fmt": "mx", "dtype": "fp32", "scaled": False},
        # the dispatched rows of 16384 tokens with 8 experts each
        {"name": "quantize_rows", "op": "quantize", "rows": 131072, "K": 2048, "fmt": "nv", "dtype": "bf16", "scaled": True},
        # one decoded token: 8 of 128 experts get one row each
        {"name": "linear_token", "op": "linear", "G": 128, "rows": 8, "N": 1536, "K": 2048, "load": "even", "fmt": "nv", "dtype": "bf16", "scaled": True},
        # sizes that fill no tile, in fp32 from end to end
        {"name": "linear_odd", "op": "linear", "G": 7, "rows": 1003, "N": 1001, "K": 1044, "load": "zipf", "fmt": "mx", "dtype": "fp32", "scaled": False},
        # the down product of 8 experts of inner size 12288 on 4096 tokens with 2 experts each
        {"name": "linear_down", "op": "linear", "G": 8, "rows": 8192, "N": 4096, "K": 12288, "load": "even", "fmt": "mx", "dtype": "bf16", "scaled": False},
        # one matrix of 8 experts of inner size 14336 under a skewed load
        {"name": "linear_skewed", "op": "linear", "G": 8, "rows": 16384, "N": 14336, "K": 4096, "load": "zipf", "fmt": "nv", "dtype": "bf16", "scaled": True},
        # one decoded token on a rank that holds 32 experts of a 256-expert layer: the weights' bytes and latency
        {"name": "experts_token", "op": "experts", "E": 32, "k": 8, "T": 1, "h": 7168, "F": 2048, "load": "even", "fmt": "nv", "dtype": "bf16", "scaled": True},
        # a decode batch: 64 tokens spread over 128 experts, about 4 rows to an expert
        {"name": "experts_batch", "op": "experts", "E": 128, "k": 8, "T": 64, "h": 2048, "F": 768, "load": "even", "fmt": "mx", "dtype": "bf16", "scaled": False},
        # a prompt batch through many small experts
        {"name": "experts_prompt", "op": "experts", "E": 128, "k": 8, "T": 16384, "h": 2048, "F": 768, "load": "even", "fmt": "nv", "dtype": "bf16", "scaled": True},
        # a prompt batch through few large experts under a skewed load
        {"name": "experts_skewed", "op": "experts", "E": 8, "k": 2, "T": 8192, "h": 4096, "F": 14336, "load": "zipf", "fmt": "nv", "dtype": "bf16", "scaled": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: mostly of whole 32s, as models have them, at times any number."""
    n = _log(rng, lo, hi)
    return max(lo, n // 32 * 32) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(("quantize", "linear", "experts"))
    case = {"op": op, "fmt": rng.choice(("nv", "mx")), "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32")), "scaled": rng.random() < 0.5}
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
    # 16-bit outputs: in the last bits of fp32 one would see which way a tied activation between the two products
    # was rounded, and that follows the order of the sums
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


def _weight(groups, N, K, fmt, scaled, gen):
    """A 4-bit weight as a checkpoint holds it: codes, block scales and the groups' fp32 multipliers (of the
    values, before they were quantised)."""
    codes, scales, mult = [], [], []
    for _ in range(groups):
        w = _normal((N, K), torch.bfloat16, gen, 1.0 / math.sqrt(K)).float()
        g = 448.0 * 6.0 / w.abs().max().clamp_min(1e-30) if scaled else None
        c, s = quantize(w, fmt, g)
        codes.append(c)
        scales.append(s)
        mult.append(g if scaled else torch.ones((), device=w.device))
    return torch.stack(codes), torch.stack(scales), torch.stack(mult)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    dt, fmt, op = DTYPE[case["dtype"]], case["fmt"], case["op"]
    # a calibrated multiplier of the activations (about 448 * 6 over their largest value), where the case has one
    mult = torch.full((1,), 58.35, device=dev) if case["scaled"] else None
    s = {"case": dict(case), "mult": mult}
    if op == "quantize":
        s["x"] = _activations((case["rows"], case["K"]), dt, gen)
        if own:
            from top_routing_dispatch_moe_gb300 import moe
            s["moe"] = moe
            s["codes"] = torch.empty((case["rows"], 16 * -(-case["K"] // 32)), dtype=torch.uint8, device=dev)
            s["scales"] = torch.empty((case["rows"], -(-case["K"] // BLOCK[fmt])), dtype=torch.uint8, device=dev)
            s["out"] = torch.empty_like(s["x"])
        return s
    inv = 1.0 / mult if mult is not None else torch.ones(1, device=dev)
    if op == "linear":
        rows = _group_rows(case, seed)
        s["x"] = _activations((case["rows"], case["K"]), dt, gen)
        codes, scales, wm = _weight(case["G"], case["N"], case["K"], fmt, case["scaled"], gen)
        s["alpha"] = (inv / wm) if case["scaled"] else None
        if own:
            from top_routing_dispatch_moe_gb300 import moe
            s["moe"] = moe
            s["packed"] = moe.moe_fp4_pack_weight(codes, scales, case["K"], fmt)
            s["out"] = torch.empty((case["rows"], case["N"]), dtype=dt, device=dev)
            s["ws"] = torch.empty(moe.moe_fp4_linear_workspace_size(case["G"], case["K"], case["rows"], fmt), dtype=torch.uint8, device=dev)
        else:
            s["weight"] = (codes, scales)
    else:
        rows, src = _routes(case, seed)
        s["x"] = _activations((case["T"], case["h"]), dt, gen)
        s["src"] = torch.from_numpy(src).to(dev)
        w = [_weight(case["E"], n, k, fmt, case["scaled"], gen) for n, k in ((case["F"], case["h"]), (case["F"], case["h"]), (case["h"], case["F"]))]
        act = torch.full((1,), 448.0 * 6.0 / 12.0, device=dev) if case["scaled"] else None
        s["act_mult"] = act
        s["alpha"] = [inv / w[0][2], inv / w[1][2], (1.0 / act) / w[2][2]] if case["scaled"] else [None] * 3
        if own:
            from top_routing_dispatch_moe_gb300 import moe
            s["moe"] = moe
            s["packed"] = moe.moe_fp4_pack_expert_weights(w[0][:2], w[1][:2], w[2][:2], case["h"], case["F"], fmt)
            s["out"] = torch.empty((len(src), case["h"]), dtype=dt, device=dev)
            s["ws"] = torch.empty(moe.moe_fp4_expert_ffn_workspace_size(case["E"], case["h"], case["F"], len(src), fmt), dtype=torch.uint8, device=dev)
        else:
            s["weight"] = [v[:2] for v in w]
    bounds = np.concatenate([[0], np.cumsum(rows)])
    s["offsets"] = torch.from_numpy(bounds.astype(np.int32)).to(dev)
    s["bounds"] = [int(v) for v in bounds]
    return s


# ---------------------------------------------------------------------------------------------- plain form


def quantize(x, fmt, mult=None):
    """Codes [rows, 16 * ceil(K / 32)] and scale bytes [rows, ceil(K / block)] of x [rows, K], in 32 bits."""
    rows, K = x.shape
    b, wide = BLOCK[fmt], -(-K // 32) * 32
    v = torch.zeros((rows, wide), dtype=torch.float32, device=x.device)
    v[:, :K] = x if mult is None else x.float() * mult
    v = v.view(rows, wide // b, b)
    most = v.abs().amax(-1)
    if fmt == "nv":
        # (divided by a tensor: by a plain number torch multiplies with its rounded reciprocal.) NaN stays NaN
        # through the clamp and the cast.
        s8 = (most / most.new_full((1,), 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale, byte = s8.float(), s8.view(torch.uint8)
    else:
        # the exponent field of a float is floor(log2) + 127; numbers below the normal range count as 0
        field = (most.view(torch.int32) >> 23) - 2
        byte = torch.where(most.isnan(), 255, field.clamp(0, 254)).to(torch.uint8)
        scale = torch.where(most.isnan(), torch.nan, torch.ldexp(torch.ones_like(most), byte.int() - 127))
    q = v / scale.unsqueeze(-1)
    m = q.abs()
    code = (m > 0.25).to(torch.uint8)
    code += m >= 0.75
    code += m > 1.25
    code += m >= 1.75
    code += m > 2.5
    code += m >= 3.5
    code += m > 5.0
    code = torch.where((scale == 0).unsqueeze(-1) | q.isnan(), 0, code)
    code |= v.signbit().to(torch.uint8) << 3
    code = torch.where(scale.isnan().unsqueeze(-1), 0, code).view(rows, wide // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), byte[:, : -(-K // b)].contiguous()


def dequantize(codes, scales, K, fmt):
    """The fp32 values [rows, K] that codes and scale bytes stand for."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).view(codes.shape[0], -1).int()][:, :K]
    if fmt == "nv":
        s = scales.view(torch.float8_e4m3fn).float()
    else:
        e = scales.int()
        s = torch.where(e == 255, torch.nan, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e - 127))
    return v * s.repeat_interleave(BLOCK[fmt], 1)[:, :K]


def _product(x, weight, alpha, g, K, fmt):
    """alpha[g] * x @ W[g]^T for one group's rows."""
    y = x @ dequantize(weight[0][g], weight[1][g], K, fmt).t()
    return y if alpha is None else y * alpha[g]


def _through(x, fmt, mult):
    """x after quantisation, as fp32 values (still times the multiplier)."""
    return dequantize(*quantize(x, fmt, mult), x.shape[1], fmt)


def run(s):
    c, fmt, dt = s["case"], s["case"]["fmt"], s["x"].dtype
    if own:
        moe = s["moe"]
        if c["op"] == "quantize":
            moe.moe_fp4_quantize(s["x"], fmt, gscale=s["mult"], codes=s["codes"], scales=s["scales"])
            return moe.moe_fp4_dequantize(s["codes"], s["scales"], c["K"], fmt, gscale=s["mult"], out=s["out"])
        if c["op"] == "linear":
            return moe.moe_fp4_linear(s["x"], s["offsets"], s["packed"], c["N"], fmt, alpha=s["alpha"], gscale=s["mult"], out=s["out"], ws=s["ws"])
        return moe.moe_fp4_expert_ffn(s["x"], s["offsets"], s["packed"], c["F"], fmt, src=s["src"], alpha_gate=s["alpha"][0], alpha_up=s["alpha"][1], alpha_down=s["alpha"][2],
                                      gscale=s["mult"], act_gscale=s["act_mult"], out=s["out"], ws=s["ws"])
    if c["op"] == "quantize":
        y = _through(s["x"], fmt, s["mult"])
        return (y if s["mult"] is None else y / s["mult"]).to(dt)
    x = _through(s["x"], fmt, s["mult"])
    if c["op"] == "linear":
        out = torch.empty((c["rows"], c["N"]), dtype=dt, device=x.device)
        K, rows = c["K"], x
    else:
        out = torch.empty((s["src"].numel(), c["h"]), dtype=dt, device=x.device)
        K, rows = c["h"], x[s["src"]]
    # one group at a time: the groups' sizes differ, and their weights in 32 bits would fill the card together
    for g in [g for g in range(len(s["bounds"]) - 1) if s["bounds"][g] < s["bounds"][g + 1]]:
        lo, hi = s["bounds"][g], s["bounds"][g + 1]
        if c["op"] == "linear":
            out[lo:hi] = _product(rows[lo:hi], s["weight"], s["alpha"], g, K, fmt)
            continue
        gate, up = (_product(rows[lo:hi], s["weight"][i], s["alpha"][i], g, K, fmt) for i in (0, 1))
        act = gate / (1.0 + torch.exp(-gate)) * up
        out[lo:hi] = _product(_through(act, fmt, s["act_mult"]), s["weight"][2], s["alpha"][2], g, c["F"], fmt)
    return out


# ------------------------------------------------------------------------------------------------- 64 bits


def _nearest(v, grid):
    """The index of the nearest of the rising `grid` to each v >= 0, a tie to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(v, mid)               # v <= mid[i]: an exact tie stays below
    tie = (i < len(mid)) & (v == mid[i.clamp(max=len(mid) - 1)]) & (i % 2 == 1)
    return i + tie.long()


def _rounded(x, fmt, mult):
    """Quantised and back by the formats' definition, in 64 bits: nearest values of the two grids."""
    rows, K = x.shape
    b = BLOCK[fmt]
    v = x.double() if mult is None else x.double() * mult.double()
    v = torch.nn.functional.pad(v, (0, -K % b)).view(rows, -1, b)
    most = v.abs().max(-1, keepdim=True).values
    if fmt == "nv":
        e = np.arange(127)                    # positive e4m3 bytes; 127 would be NaN
        grid = np.where(e < 8, e / 8.0 * 2.0**-6, (1 + e % 8 / 8.0) * 2.0 ** (e // 8 - 7.0))
        grid = torch.from_numpy(grid).to(v.device)
        s = grid[_nearest(most / 6, grid)]
    else:
        e = torch.frexp(most).exponent.double() - 1
        s = torch.exp2(torch.where(most > 0, e - 2, -127.0).clamp(-127, 127))
    m = (v / torch.where(s > 0, s, 1.0)).abs()
    grid = torch.tensor(VALUES, dtype=torch.float64, device=v.device)
    return (grid[_nearest(m, grid)] * s * torch.sign(v)).view(rows, -1)[:, :K]


def _weight64(weight, g, K, fmt):
    codes, scales = weight[0][g].long(), weight[1][g]
    v = torch.stack((codes % 16, codes // 16), -1).flatten(1)[:, :K]
    m, e = v % 2, v % 8 // 2
    mag = torch.where(e == 0, m / 2.0, (1 + m / 2.0) * torch.exp2(e.double() - 1)).double()
    byte = scales.long()
    s = torch.where(byte < 8, byte / 8.0 * 2.0**-6, (1 + byte % 8 / 8.0) * torch.exp2((byte // 8).double() - 7)) if fmt == "nv" else torch.exp2(byte.double() - 127)
    return mag * torch.where(v >= 8, -1.0, 1.0) * s.double().repeat_interleave(BLOCK[fmt], 1)[:, :K]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, fmt = case, case["fmt"]
    if c["op"] == "quantize":
        y = _rounded(s["x"], fmt, s["mult"])
        return y if s["mult"] is None else y / s["mult"].double()
    al = s["alpha"] if c["op"] == "experts" else [s["alpha"]]
    al = [None if a is None else a.double() for a in al]
    rows = [(lo, hi) for lo, hi in zip(s["bounds"][:-1], s["bounds"][1:])]
    x = _rounded(s["x"], fmt, s["mult"])
    parts = []
    for g, (lo, hi) in enumerate(rows):
        if lo == hi:
            continue

        def times(a, i, width):
            y = a @ _weight64(s["weight"] if c["op"] == "linear" else s["weight"][i], g, width, fmt).t()
            return y if al[i] is None else y * al[i][g]

        if c["op"] == "linear":
            parts.append(times(x[lo:hi], 0, c["K"]))
        else:
            a = x[s["src"][lo:hi].long()]
            a = torch.nn.functional.silu(times(a, 0, c["h"])) * times(a, 1, c["h"])
            parts.append(times(_rounded(a, fmt, s["act_mult"]), 2, c["F"]))
    return torch.cat(parts)


# ---------------------------------------------------------------------------------------------------- work


def work(case):
    """x read once, the weights of as many groups as the load reaches at most read once in 4 bits, y written once."""
    el = BYTES[case["dtype"]]
    if case["op"] == "quantize":
        return {"bytes": 2.0 * el * case["rows"] * case["K"], "flops": 0.0}
    per = 0.5 + 1.0 / BLOCK[case["fmt"]]
    if case["op"] == "linear":
        used = min(case["G"], case["rows"])
        return {"bytes": el * case["rows"] * (case["K"] + case["N"]) + per * used * case["N"] * case["K"], "flops": 2.0 * case["rows"] * case["N"] * case["K"]}
    rows = case["T"] * case["k"]
    used = min(case["E"], rows)
    return {"bytes": el * (case["T"] + rows) * case["h"] + 3 * per * used * case["h"] * case["F"], "flops": 6.0 * rows * case["h"] * case["F"]}
