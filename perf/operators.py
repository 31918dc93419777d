"""Cases for the expert products over unquantised and 8-bit weights.

Five operators that stand beside the packed-weight expert FFN.  Rows are in
expert order, expert e owning rows [offsets[e], offsets[e+1]) as the
permutation step writes them; rows behind offsets[E] stay as they were.

  mm     y[r]  = W[e] . x[r]              16-bit operands
  dx     dx[r] = W[e]^T . dy[r]           the gradient of the rows
  dw     dW[e] = sum_{r of e} dy[r] x[r]^T  the gradient of the weights
  quant  q[r, i] = e4m3(x[r, i] * (448 / a)), s = a / 448, where a is the
         largest |x| of the 128 inputs of i's block of row r
  fp8    y[r, o] = sum_g s_x[g, r] s_w[e, o/128, g] sum_{i of block g} q_x[r, i] q_w[e, o, i]
         with or without experts (one matrix for all rows)
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
WORKSPACE_BYTES = 40 << 20  # the library's workspace for grouped products, zeroed once
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -126          # the least scale: a block of zeros has it


# ------------------------------------------------------------------- cases
def _product(name, op, tokens, k, experts, n_in, n_out, dtype="bf16", out="bf16", skew=0.5, pad=0):
    return {"name": name, "op": op, "tokens": tokens, "k": k, "experts": experts, "n_in": n_in, "n_out": n_out,
            "dtype": dtype, "out": out, "skew": skew, "pad": pad}


def listed():
    return [
        # the gate projection of one decoded token over the layer's 256 experts: eight weight matrices are read
        _product("mm decode", "mm", 1, 8, 256, 4096, 2048),
        # the same projection for a prompt of 4096 tokens: every expert's weights, uneven row counts
        _product("mm prefill", "mm", 4096, 8, 256, 4096, 2048),
        # the down projection of the same prompt on a rank that owns few experts: long row ranges
        _product("mm slice", "mm", 4096, 8, 32, 2048, 4096, "fp16", "fp16"),
        # the rows' gradient for a short odd batch over a layer pruned to 161 experts
        _product("dx pruned", "dx", 37, 8, 161, 4096, 2048),
        # the rows' gradient of a large batch on a rank of few experts
        _product("dx slice", "dx", 4096, 8, 32, 4096, 2048),
        # the weights' gradient of the smallest layer: latency, and experts without rows
        _product("dw tiny", "dw", 4, 2, 8, 256, 128, "bf16", "fp32"),
        # the weights' gradient of a large batch on a rank of few experts
        _product("dw slice", "dw", 4096, 8, 32, 4096, 2048),
        # one token's activations to 8 bits: latency
        {"name": "quant token", "op": "quant", "rows": 1, "n_in": 4096, "dtype": "bf16"},
        # a prompt's permuted rows to 8 bits
        {"name": "quant prefill", "op": "quant", "rows": 32768, "n_in": 4096, "dtype": "bf16"},
        # the always-on shared expert's gate projection of one token: one 8-bit matrix
        _product("fp8 token", "fp8", 1, 1, 0, 4096, 2048, "e4m3"),
        # a decode batch of 32 tokens over 256 experts, most with one row or two
        _product("fp8 batch", "fp8", 32, 8, 256, 4096, 2048, "e4m3"),
        # a large batch on a rank of few experts, the rows padded behind the last expert's
        _product("fp8 slice", "fp8", 4096, 8, 32, 4096, 2048, "e4m3", "bf16", 0.5, 77),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, most):
    n = _log(rng, 64, most)
    step = rng.choice([128, 64, 16, 8, 1])  # whole blocks, vector widths, and odd widths
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(["mm", "dx", "dw", "quant", "fp8"])
    if op == "quant":
        n_in = _width(rng, 8192)
        return {"op": op, "rows": _log(rng, 1, min(32768, (1 << 27) // n_in)), "n_in": n_in,
                "dtype": rng.choice(["bf16", "fp16"])}
    n_in, n_out = _width(rng, 8192), _width(rng, 8192)
    experts = _log(rng, 1, 256)
    tokens = _log(rng, 1, 4096)
    k = rng.randint(1, min(8, experts))
    while tokens * k * n_in * n_out > 1 << 37 and tokens > 1:
        tokens = max(1, tokens * 2 // 3)
    while experts * n_in * n_out > 1 << 30 and experts > k:
        experts = max(k, experts * 2 // 3)
    c = _product("", op, tokens, k, experts, n_in, n_out, rng.choice(["bf16", "fp16"]), "bf16",
                 rng.choice([0.0, 0.5, 0.8]), rng.choice([0, 0, rng.randint(1, 130)]))
    if op == "fp8":
        c["dtype"] = "e4m3"
        c["out"] = rng.choice(["bf16", "fp16", "fp32"])
        if rng.random() < 0.4:  # one matrix for all rows
            c["experts"], c["k"], c["pad"] = 0, 1, 0
    else:
        c["out"] = rng.choice([c["dtype"], c["dtype"], "fp32"])
    del c["name"]
    return c


def _counts(case):
    """Rows of each expert: the case's alone, so that its work is too; the seed permutes the experts."""
    tokens, k, experts = case["tokens"], case["k"], case["experts"]
    if not experts:
        return np.array([tokens], np.int64)
    g = np.random.default_rng([tokens, k, experts, int(10 * case["skew"])])
    keys = case["skew"] * g.standard_normal(experts) + g.gumbel(size=(tokens, experts))
    picks = np.argpartition(-keys, k - 1, axis=1)[:, :k] if k < experts else np.tile(np.arange(experts), (tokens, 1))
    return np.bincount(picks.ravel(), minlength=experts)


def _groups(n):
    return (n + 127) // 128


def work(case):
    if case["op"] == "quant":
        rows, n = case["rows"], case["n_in"]
        return {"bytes": rows * (3 * n + 4 * _groups(n)), "flops": 3 * rows * n}
    counts = _counts(case)
    rows, active = int(counts.sum()), int((counts > 0).sum())
    n, o = case["n_in"], case["n_out"]
    size = 1 if case["dtype"] == "e4m3" else 2
    out = 4 if case["out"] == "fp32" else 2
    flops = 2 * rows * n * o
    table = 4 * (case["experts"] + 1)
    if case["op"] == "mm":
        return {"bytes": size * (active * n * o + rows * n) + out * rows * o + table, "flops": flops}
    if case["op"] == "dx":
        return {"bytes": size * (active * n * o + rows * o) + out * rows * n + table, "flops": flops}
    if case["op"] == "dw":
        return {"bytes": size * rows * (n + o) + out * len(counts) * n * o + table, "flops": flops}
    scales = 4 * (rows * _groups(n) + active * _groups(n) * _groups(o))
    return {"bytes": active * n * o + rows * n + scales + out * rows * o + table, "flops": flops}


# ------------------------------------------------------------------ inputs
def _normal(g, std, dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=DEVICE).normal_(0.0, std, generator=g)


def _scales(a):
    """What a block whose largest value is `a` is divided by, and what its codes are made with, each rounded once."""
    a = a.clamp(min=448 * TINY)
    top = torch.full_like(a, 448.0)
    return a / top, top / a


def _codes(v, scale):
    return (v * scale).to(torch.float8_e4m3fn)


def _fp8_rows(g, rows, n):
    """8-bit rows and their scales [groups, rows], as the quantisation step leaves them."""
    q = torch.empty(rows, n, dtype=torch.float8_e4m3fn, device=DEVICE)
    s = torch.empty(_groups(n), rows, dtype=torch.float32, device=DEVICE)
    for b in range(_groups(n)):
        x = _normal(g, 1.0, torch.float32, rows, min(128, n - 128 * b))
        s[b], inv = _scales(x.abs().amax(1))
        q[:, 128 * b:128 * b + 128] = _codes(x, inv[:, None])
    return q, s


def _fp8_weights(g, experts, n_out, n_in):
    """8-bit weights [E, out, in] with one scale for each 128 x 128 block."""
    q = torch.empty(experts, n_out, n_in, dtype=torch.float8_e4m3fn, device=DEVICE)
    s = torch.empty(experts, _groups(n_out), _groups(n_in), dtype=torch.float32, device=DEVICE)
    for b in range(_groups(n_out)):
        rows = min(128, n_out - 128 * b)
        w = torch.zeros(experts, rows, 128 * _groups(n_in), dtype=torch.float32, device=DEVICE)
        w[:, :, :n_in] = _normal(g, 0.02, torch.float32, experts, rows, n_in)
        w = w.view(experts, rows, _groups(n_in), 128)
        s[:, b], inv = _scales(w.abs().amax((1, 3)))
        q[:, 128 * b:128 * b + 128] = _codes(w, inv[:, None, :, None]).view(experts, rows, -1)[:, :, :n_in]
    return q, s


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    if case["op"] == "quant":
        rows, n = case["rows"], case["n_in"]
        x = _normal(g, 1.0, TYPES[case["dtype"]], rows, n)
        x.mul_(torch.empty(1, n, device=DEVICE).normal_(0.0, 1.0, generator=g).exp_().to(x.dtype))  # some wide channels
        return {"op": "quant", "x": x, "q": torch.empty(rows, n, dtype=torch.float8_e4m3fn, device=DEVICE),
                "s": torch.empty(_groups(n), rows, dtype=torch.float32, device=DEVICE)}
    counts = _counts(case)
    experts = len(counts)
    counts = counts[np.random.default_rng(seed).permutation(experts)]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    used, rows = int(offsets[-1]), int(offsets[-1]) + case["pad"]
    n, o, op = case["n_in"], case["n_out"], case["op"]
    s = {"op": op, "used": used, "most": int(counts.max()),
         "active": torch.from_numpy(np.flatnonzero(counts)).to(DEVICE),
         "offsets": torch.from_numpy(offsets).to(DEVICE) if case["experts"] else None,
         "bounds": torch.from_numpy(offsets.astype(np.int64)).to(DEVICE),
         "ws": torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device=DEVICE)}
    if op == "fp8":
        s["x"], s["sx"] = _fp8_rows(g, rows, n)
        s["w"], s["sw"] = _fp8_weights(g, experts, o, n)
        s["y"] = torch.zeros(rows, o, dtype=TYPES[case["out"]], device=DEVICE)
        return s
    dtype, out = TYPES[case["dtype"]], TYPES[case["out"]]
    if op != "dx":
        s["x"] = _normal(g, 1.0, dtype, rows, n)
    if op != "dw":
        s["w"] = _normal(g, 0.02, dtype, experts, o, n)
    if op != "mm":
        s["dy"] = _normal(g, 0.1, dtype, rows, o)
    s["y"] = torch.zeros({"mm": (rows, o), "dx": (rows, n), "dw": (experts, o, n)}[op], dtype=out, device=DEVICE)
    return s


# --------------------------------------------------------------- the passes
def _slots(s):
    """Each row's expert (its place among those with rows) and its place in that expert's range."""
    r = torch.arange(s["used"], device=DEVICE)
    e = torch.searchsorted(s["bounds"], r, right=True) - 1
    return torch.searchsorted(s["active"], e), r - s["bounds"][e]


def _by_expert(s, v, at):
    """[experts with rows, most rows, columns]: the rows of each expert, zeros behind them."""
    p = torch.zeros(len(s["active"]), s["most"], v.shape[1], dtype=torch.float32, device=DEVICE)
    p[at] = v[:s["used"]].float()
    return p


def _rows_out(s, products, at):
    y = torch.zeros(s["y"].shape, dtype=s["y"].dtype, device=DEVICE)
    y[:s["used"]] = products[at].to(y.dtype)
    return y


def _plain(s):
    op = s["op"]
    if op == "quant":
        x = s["x"].float()
        groups = s["s"].shape[0]
        wide = torch.zeros(x.shape[0], 128 * groups, dtype=torch.float32, device=DEVICE)
        wide[:, :x.shape[1]] = x
        wide = wide.view(x.shape[0], groups, 128)
        scales, inv = _scales(wide.abs().amax(2))
        q = _codes(wide, inv[:, :, None]).view(x.shape[0], -1)[:, :x.shape[1]].contiguous()
        return {"q": q, "s": scales.t().contiguous()}
    at = _slots(s)
    if op == "mm":
        return _rows_out(s, torch.bmm(_by_expert(s, s["x"], at), s["w"][s["active"]].float().transpose(1, 2)), at)
    if op == "dx":
        return _rows_out(s, torch.bmm(_by_expert(s, s["dy"], at), s["w"][s["active"]].float()), at)
    if op == "dw":
        dw = torch.zeros(s["y"].shape, dtype=s["y"].dtype, device=DEVICE)
        dw[s["active"]] = torch.bmm(_by_expert(s, s["dy"], at).transpose(1, 2), _by_expert(s, s["x"], at)).to(dw.dtype)
        return dw
    n, o = s["x"].shape[1], s["y"].shape[1]
    x = s["x"].float() * s["sx"].t().repeat_interleave(128, 1)[:, :n]
    sw = s["sw"][s["active"]].repeat_interleave(128, 1)[:, :o].repeat_interleave(128, 2)[:, :, :n]
    w = s["w"].view(torch.uint8)[s["active"]].view(torch.float8_e4m3fn).float() * sw
    return _rows_out(s, torch.bmm(_by_expert(s, x, at), w.transpose(1, 2)), at)


def _library(s):
    import bit_quantized_moe_route_b200 as moe
    op = s["op"]
    if op == "quant":
        moe.quant_fp8(s["x"], s["q"], s["s"])
        return {"q": s["q"], "s": s["s"]}
    if op == "mm":
        moe.grouped_mm(s["x"], s["w"], s["offsets"], s["y"], s["ws"])
    elif op == "dx":
        moe.grouped_mm_dx(s["dy"], s["w"], s["offsets"], s["y"], s["ws"])
    elif op == "dw":
        moe.grouped_mm_dw(s["dy"], s["x"], s["offsets"], s["y"], s["ws"])
    else:
        moe.grouped_mm_fp8(s["x"], s["sx"], s["w"], s["sw"], s["offsets"], s["y"], s["ws"])
    return s["y"]


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"].double()
        q = torch.empty_like(x)
        scales = torch.empty(s["s"].shape, dtype=torch.float64, device=DEVICE)
        for b in range(scales.shape[0]):
            x_b = x[:, 128 * b:128 * (b + 1)]
            scales[b] = (x_b.abs().max(1).values / 448).clamp(min=TINY)
            q[:, 128 * b:128 * (b + 1)] = x_b / scales[b][:, None]
        return {"q": q, "s": scales}
    bounds = s["bounds"].tolist()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEVICE)
    for e, (r0, r1) in enumerate(zip(bounds, bounds[1:])):
        if r0 == r1:
            continue
        if case["op"] == "mm":
            y[r0:r1] = s["x"][r0:r1].double() @ s["w"][e].double().t()
        elif case["op"] == "dx":
            y[r0:r1] = s["dy"][r0:r1].double() @ s["w"][e].double()
        elif case["op"] == "dw":
            y[e] = s["dy"][r0:r1].double().t() @ s["x"][r0:r1].double()
        else:
            for b in range(s["sx"].shape[0]):  # block by block, the products of the codes first
                part = s["x"][r0:r1, 128 * b:128 * (b + 1)].double() @ s["w"][e, :, 128 * b:128 * (b + 1)].double().t()
                scale = s["sw"][e, :, b].double().repeat_interleave(128)[:y.shape[1]]
                y[r0:r1] += part * s["sx"][b, r0:r1].double()[:, None] * scale
    return y
