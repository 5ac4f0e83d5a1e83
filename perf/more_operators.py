"""Workloads of a block's two halves around a low-precision linear layer: layer norm with its backward pass, and the
linear layer itself in microscaled 4-bit floating point (quantisation of its operands, products, gradients).

Each case is one pass through one operator. ``run`` computes it either in its plain form (elementary torch operations in
float32, rounded once where a result has a narrower type) or, with ``own`` set, through the framework's entry points.

Conventions shared by both forms:

Layer norm. s = x + residual, rounded to x's type, where there is a residual, else x; y = (s - mean) * rstd * weight + bias
over the last axis, rstd = 1 / sqrt(variance + eps). A "train" pass also takes the gradient with respect to x (which is the
residual's too), plus the gradient that reaches s directly where there is a residual, and those of weight and bias.

4-bit operands. Codes are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), blocks of consecutive entries along the axis that a
product contracts share a scale. Blocks of 32 have a power of two: the smallest that is at least max |x| / 6. Blocks of 16 have
an E4M3 number times one power of two for the tensor, the smallest for which no block's scale passes 448; a block's scale is
max |x| / 6, over that power, rounded to nearest, or upwards where rounding is stochastic. Codes are rounded to nearest even,
or stochastically with 16 bits of a counter hash of (seed, axis, entry). Where scales are rounded down, 6 is the largest code.
Quotients (max |x| / 6, and an entry by an E4M3 scale) are rounded to float32 before anything is decided by them.

``mode`` is what the pass does. "serve": activations are quantised and multiplied with weights that are kept in 4 bits.
"train": x, w and the output's gradient (this one stochastically) are quantised along both axes; output, gradient of x,
gradient of w. "values": both quantisations of a tensor, returned as the numbers that they stand for.
"""

import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
_TYPES = {"f32": F32, "bf16": BF16}
_SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-5


# ------------------------------------------------------------------------------------------- cases

def listed():
    norm = {"op": "norm", "residual": False, "bias": True, "pad": 0}
    fp4 = {"op": "fp4"}
    return [
        # one decoding step of 4 sequences through a 1600-wide model's norm, residual added: latency
        dict(norm, name="norm_token", rows=4, cols=1600, type="bf16", weight="bf16", residual=True, mode="forward"),
        # a prompt in float32, rows of odd length and no bias
        dict(norm, name="norm_prompt_odd_f32", rows=2051, cols=1217, type="f32", weight="f32", bias=False, mode="forward"),
        # a training step over 32768 tokens of a 1600-wide model, residual stream in bfloat16, gains in float32
        dict(norm, name="norm_train", rows=32768, cols=1600, type="bf16", weight="f32", residual=True, mode="train"),
        # the same in float32 for a 768-wide one, without residual
        dict(norm, name="norm_train_f32", rows=16384, cols=768, type="f32", weight="f32", mode="train"),
        # very wide rows of odd length inside a wider buffer
        dict(norm, name="norm_train_wide_odd", rows=3001, cols=12289, type="bf16", weight="bf16", pad=7, mode="train"),
        # one decoding step of 3 sequences through the up projection of a 1600-wide model: the weights are what is read
        dict(fp4, name="fp4_token", tokens=3, out=6400, cols=1600, type="bf16", block=32, result="bf16", mode="serve"),
        # 200 sequences at once through the attention projection, blocks of 16
        dict(fp4, name="fp4_batch", tokens=200, out=4800, cols=1600, type="bf16", block=16, result="bf16", mode="serve"),
        # a long prompt through a square layer, float32 logits
        dict(fp4, name="fp4_prompt_f32", tokens=8191, out=4096, cols=4096, type="bf16", block=16, result="f32", mode="serve"),
        # training step of the up projection, 16384 tokens
        dict(fp4, name="fp4_train", tokens=16384, out=6400, cols=1600, type="bf16", block=32, result="bf16", mode="train"),
        # the same with sizes that no tile divides, float32 activations and gradients
        dict(fp4, name="fp4_train_odd_f32", tokens=3001, out=1217, cols=777, type="f32", block=16, result="f32", mode="train"),
        # training step of a large square layer
        dict(fp4, name="fp4_train_wide", tokens=8192, out=8192, cols=8192, type="bf16", block=32, result="bf16", mode="train"),
        # a 50304 x 768 table in 4 bits, both ways, stochastic rounding
        dict(fp4, name="fp4_table_values", tokens=50304, out=1, cols=768, type="bf16", block=16, result="bf16", mode="values"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("bf16", "bf16", "f32"))
    if rng.random() < 0.45:
        cols = _log_uniform(rng, 16, 20_000)
        if rng.random() < 0.5:
            cols = cols // 8 * 8
        return {"op": "norm", "rows": _log_uniform(rng, 1, max(1, min(200_000, 70_000_000 // cols))), "cols": cols, "type": kind,
                "weight": rng.choice(("bf16", "f32")), "bias": rng.random() < 0.7, "residual": rng.random() < 0.5,
                "pad": rng.choice((0, 0, 1, 8)), "mode": rng.choice(("forward", "train"))}
    mode = rng.choice(("serve", "train", "train", "values"))
    few = mode == "serve" and rng.random() < 0.5
    tokens = _log_uniform(rng, 1, 64) if few else _log_uniform(rng, 65, 16384)
    out, cols = _log_uniform(rng, 33, 8192), _log_uniform(rng, 33, 8192)
    if rng.random() < 0.5:
        out, cols = max(64, out // 64 * 64), max(64, cols // 64 * 64)
    tokens = min(tokens, 8192 ** 3 // (out * cols))
    return {"op": "fp4", "tokens": tokens, "out": 1 if mode == "values" else out, "cols": cols, "type": kind,
            "block": rng.choice((16, 32)), "result": rng.choice(("bf16", "bf16", "f32")), "mode": mode}


# ------------------------------------------------------------------------------------------ inputs

def _prepare_norm(case, normal):
    rows, cols, kind, weights = case["rows"], case["cols"], _TYPES[case["type"]], _TYPES[case["weight"]]

    def rows_of(x):
        whole = torch.zeros((rows, cols + case["pad"]), dtype=kind, device="cuda")
        whole[:, :cols] = x
        return whole[:, :cols]

    # activations: a mean of their own in each column, a few columns far larger than the rest
    loud = torch.where(normal(cols) > 2.5, 8.0, 1.0)
    state = {"x": rows_of((normal(rows, cols) + 0.3 * normal(cols)) * loud), "weight": (1 + 0.2 * normal(cols)).to(weights),
             "bias": (0.1 * normal(cols)).to(weights) if case["bias"] else None,
             "residual": rows_of(normal(rows, cols)) if case["residual"] else None}
    if case["mode"] == "train":
        state["grad"] = rows_of(normal(rows, cols) / rows)
        state["grad_sum"] = rows_of(normal(rows, cols) / rows) if case["residual"] else None
    return state


def _prepare_fp4(case, normal, seed):
    tokens, out, cols, kind = case["tokens"], case["out"], case["cols"], _TYPES[case["type"]]
    state = {"x": (normal(tokens, cols) * torch.where(normal(cols) > 2.5, 8.0, 1.0)).to(kind), "seed": seed}
    if case["mode"] != "values":
        state["w"] = (normal(out, cols) / math.sqrt(cols)).to(kind)
    if case["mode"] == "train":
        state["grad"] = (normal(tokens, out) * (normal(tokens, 1) * 2 - 9).exp()).to(kind)
    if case["mode"] == "serve":  # what a program that serves keeps of its weights
        if own:
            from newton_schulz_08_gb300 import muon
            state["w"] = muon.fp4_quantize(state["w"], block=case["block"])
        else:
            state["w"] = _rounded(state["w"], case["block"])
    return state


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(1_000_003 * (int(seed) + 1))
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    with torch.no_grad():
        state = _prepare_norm(case, normal) if case["op"] == "norm" else _prepare_fp4(case, normal, int(seed))
    return state | {"case": case}


# ------------------------------------------------------------------------------------- plain forms

_M, _C0, _C1, _C2 = 0xFFFFFFFF, 0x9E3779B1, 0x6A09E667, 0xBB67AE85


def _mix(x):
    """Scrambles 32 bits (an int, or an int64 tensor of such)."""
    x = ((x ^ (x >> 16)) * _C1) & _M
    x = ((x ^ (x >> 15)) * _C2) & _M
    return x ^ (x >> 16)


def _random16(rows, cols, seed, axis):
    """16 random bits of each entry of a rows x cols operand: halves of a hash for two neighbours."""
    key = _mix(_mix((seed + _C0 * axis) & _M) ^ (seed >> 32 & _M))
    pairs = (cols + 1) // 2
    i = torch.arange(rows, device="cuda")[:, None] * pairs + torch.arange(pairs, device="cuda")
    h = _mix(((i & _M) * _C0 + key + (i >> 32) * _C1) & _M)
    return torch.stack((h & 0xFFFF, h >> 16), 2).view(rows, 2 * pairs)[:, :cols]


def _pow2(e):
    """2^e for whole numbers from -127 to 127 (2^-127 is subnormal)."""
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e.clamp_min(-126) + 127) << 23).view(F32)


def _least_power(a, mantissa, drop):
    """The exponent e with the smallest 2^e >= a / (1.mantissa * 2^drop), at least -127, of float32 a >= 0."""
    return ((a.contiguous().view(torch.int32) + (0x7FFFFF - mantissa)) >> 23).sub(127 + drop).clamp_min(-127).to(torch.int32)


def _rounded(x, block, seed=None, axis=1):
    """The values that x [rows, cols] has in 4 bits, blocks along the columns, in float32."""
    rows, cols = x.shape
    blocks = -(-cols // block)
    full = torch.zeros((rows, blocks * block), dtype=F32, device=x.device)
    full[:, :cols] = x
    a = full.view(rows, blocks, block).abs()
    largest = a.amax(2, keepdim=True)
    if block == 32:
        e = _least_power(largest, 0x400000, 2)          # 6 = 1.5 * 2^2
        scale = _pow2(e)
        y = a * _pow2(-e)
    else:
        k = _least_power(largest.max().view(1), 0x280000, 11)   # 6 * 448 = 1.3125 * 2^11
        up, down = _pow2(-k), _pow2(k)
        want = largest / torch.full_like(largest, 6) * up    # (a quotient by a plain number would be a product)
        s = want.to(torch.float8_e4m3fn)
        if seed is not None:  # upwards: nothing is cut off
            s = torch.where(s.to(F32) < want, (s.view(torch.uint8) + 1).view(torch.float8_e4m3fn).to(F32), s.to(F32))
        s = s.to(F32)
        y = torch.where(s > 0, (a * up / s).clamp_max(6), torch.zeros((), device=x.device))
        scale = s * down
    if seed is None:
        step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
        q = torch.round(y / step) * step
    else:  # in 64 bits: 32 would move entries next to a border over it
        r = torch.zeros((rows, blocks * block), dtype=torch.float64, device=x.device)
        r[:, :cols] = (_random16(rows, cols, seed, axis) + 0.5) / 65536
        step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).to(torch.float64)
        q = (torch.floor(y / step + r.view(rows, blocks, block)) * step).to(F32)
    return torch.copysign(q * scale, full.view(rows, blocks, block)).view(rows, -1)[:, :cols]


def _plain_fp4(s):
    case, block = s["case"], s["case"]["block"]
    result = _TYPES[case["result"]]
    if case["mode"] == "serve":
        return {"out": (_rounded(s["x"], block) @ s["w"].t()).to(result)}
    if case["mode"] == "values":
        return {"values": _rounded(s["x"], block, s["seed"], 1).to(BF16), "across": _rounded(s["x"].t(), block, s["seed"], 0).to(BF16)}
    g = _rounded(s["grad"], block, s["seed"], 1)
    out = _rounded(s["x"], block) @ _rounded(s["w"], block).t()
    grad_x = g @ _rounded(s["w"].t(), block, axis=0).t()
    g = _rounded(s["grad"].t(), block, s["seed"], 0)
    grad_w = g @ _rounded(s["x"].t(), block, axis=0).t()
    return {"out": out.to(result), "grad_x": grad_x.to(result), "grad_w": grad_w.to(result)}


def _plain_norm(s):
    x, kind = s["x"], s["x"].dtype
    out = {}
    if s["residual"] is not None:
        x = out["sum"] = (x.to(F32) + s["residual"].to(F32)).to(kind)
    x, w = x.to(F32), s["weight"].to(F32)
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    xhat = d * rstd
    y = xhat * w
    if s["bias"] is not None:
        y = y + s["bias"].to(F32)
    out |= {"y": y.to(kind), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["case"]["mode"] == "train":
        g = s["grad"].to(F32)
        gw = g * w
        grad_x = rstd * (gw - gw.mean(1, keepdim=True) - xhat * (gw * xhat).mean(1, keepdim=True))
        if s["grad_sum"] is not None:
            grad_x = grad_x + s["grad_sum"].to(F32)
        out |= {"grad_x": grad_x.to(kind), "grad_weight": (g * xhat).sum(0)}
        if s["bias"] is not None:
            out["grad_bias"] = g.sum(0)
    return out


# --------------------------------------------------------------------------------------- own forms

def _own_norm(s):
    from newton_schulz_08_gb300 import muon
    r = muon.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, residual=s["residual"])
    out = {"sum": r.sum} if s["residual"] is not None else {}
    out |= {"y": r.y, "mean": r.mean, "rstd": r.rstd}
    if s["case"]["mode"] == "train":
        x = s["x"] if r.sum is None else r.sum
        grad_x, grad_weight, grad_bias = muon.layer_norm_backward(s["grad"], x, r.mean, r.rstd, s["weight"], grad_sum=s["grad_sum"],
                                                                  bias=s["bias"] is not None)
        out |= {"grad_x": grad_x, "grad_weight": grad_weight}
        if s["bias"] is not None:
            out["grad_bias"] = grad_bias
    return out


def _own_fp4(s):
    from newton_schulz_08_gb300 import muon
    case, block = s["case"], s["case"]["block"]
    result = _TYPES[case["result"]]
    if case["mode"] == "serve":
        return {"out": muon.fp4_mm(muon.fp4_quantize(s["x"], block=block), s["w"], dtype=result)}
    if case["mode"] == "values":
        along, across = muon.fp4_quantize(s["x"], block=block, axis="both", seed=s["seed"])
        return {"values": muon.fp4_values(along), "across": muon.fp4_values(across)}
    x, x_t = muon.fp4_quantize(s["x"], block=block, axis="both")
    w, w_t = muon.fp4_quantize(s["w"], block=block, axis="both")
    out = muon.fp4_mm(x, w, dtype=result)
    g, g_t = muon.fp4_quantize(s["grad"], block=block, axis="both", seed=s["seed"])
    return {"out": out, "grad_x": muon.fp4_mm(g, w_t, dtype=result), "grad_w": muon.fp4_mm(g_t, x_t, dtype=result)}


def run(state):
    norm = state["case"]["op"] == "norm"
    with torch.no_grad():
        if own:
            return _own_norm(state) if norm else _own_fp4(state)
        return _plain_norm(state) if norm else _plain_fp4(state)


# ------------------------------------------------------------------------------------ work, 64 bits

def work(case):
    if case["op"] == "norm":
        n, s, w = case["rows"] * case["cols"], _SIZE[case["type"]], _SIZE[case["weight"]]
        extra = 1 if case["residual"] else 0
        size = n * s * (2 + 2 * extra) + 8 * case["rows"] + case["cols"] * w * (1 + case["bias"])
        if case["mode"] == "forward":
            return {"bytes": size, "flops": 8 * n}
        return {"bytes": size + n * s * (3 + extra) + 8 * case["rows"] + case["cols"] * (w + 4 * (1 + case["bias"])), "flops": 22 * n}
    m, n, k, s, r = case["tokens"], case["out"], case["cols"], _SIZE[case["type"]], _SIZE[case["result"]]
    held = 0.5 + 1 / case["block"]   # bytes of an entry in 4 bits
    if case["mode"] == "values":
        return {"bytes": m * k * (s + 4), "flops": 12 * m * k}
    if case["mode"] == "serve":
        return {"bytes": m * k * s + n * k * held + m * n * r, "flops": 2 * m * n * k}
    return {"bytes": (m * k + n * k + m * n) * (s + r), "flops": 6 * m * n * k}


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rounded(x, block, r=None):
    """x [rows, cols] in 4 bits, in float64: every grid number tried, ties to the one with an even code; r in (0, 1): stochastic."""
    rows, cols = x.shape
    pad = (-cols) % block
    z = torch.nn.functional.pad(x.to(torch.float64), (0, pad)).reshape(-1, block)
    top = z.abs().amax(1, keepdim=True)
    top = top / torch.full_like(top, 6)
    if block == 32:
        m, e = torch.frexp(top)
        scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), (e - (m == 0.5).to(torch.int32)).clamp_min(-127)), torch.ones_like(top))
    else:
        m, e = torch.frexp(z.abs().max() / torch.full_like(z[0, 0], 2688))
        k = e - (m == 0.5).to(torch.int32)
        want = torch.ldexp(top.to(F32).to(torch.float64), -k)
        step = torch.ldexp(torch.ones_like(top), (torch.frexp(want).exponent - 1).clamp_min(-6) - 3)
        units = want / step
        scale = torch.ldexp((torch.round(units) if r is None else torch.ceil(units)) * step, k)
    y = torch.where(scale > 0, z.abs() / scale, torch.zeros_like(z)).to(F32).to(torch.float64).clamp_max_(6)
    low, gap = torch.zeros_like(y), torch.full_like(y, 0.5)
    even = torch.ones_like(y, dtype=torch.bool)
    for code in range(1, 8):
        at = y >= _GRID[code]
        low = torch.where(at, _GRID[code], low)
        gap = torch.where(at, _GRID[min(code + 1, 7)] - _GRID[code], gap)
        even = torch.where(at, code % 2 == 0, even)
    part = torch.where(gap > 0, (y - low) / gap, torch.zeros_like(y))
    if r is None:
        up = (part > 0.5) | (part == 0.5) & ~even
    else:
        r = torch.nn.functional.pad(r, (0, pad)).reshape(-1, block)
        up = part + r >= 1
    q = torch.where(up, low + gap, low) * scale
    return torch.where(z < 0, -q, q).view(rows, -1)[:, :cols]


def _exact_fp4(case, s, w):
    block, f64 = case["block"], torch.float64
    chance = lambda rows, cols, axis: (_random16(rows, cols, s["seed"], axis).to(f64) + 0.5) / 65536  # noqa: E731
    x = s["x"]
    if case["mode"] == "values":
        return {"values": _exact_rounded(x, block, chance(*x.shape, 1)), "across": _exact_rounded(x.t(), block, chance(*x.t().shape, 0))}
    out = _exact_rounded(x, block) @ _exact_rounded(w, block).t()
    if case["mode"] == "serve":
        return {"out": out}
    g = s["grad"]
    grad_x = _exact_rounded(g, block, chance(*g.shape, 1)) @ _exact_rounded(w.t(), block).t()
    grad_w = _exact_rounded(g.t(), block, chance(*g.t().shape, 0)) @ _exact_rounded(x.t(), block).t()
    return {"out": out, "grad_x": grad_x, "grad_w": grad_w}


def _exact_norm(case, s):
    """Automatic differentiation of the definition in float64, some rows at a time."""
    f64, rows, train = torch.float64, case["rows"], case["mode"] == "train"
    w, out = s["weight"].to(f64).requires_grad_(train), {}
    b = None if s["bias"] is None else s["bias"].to(f64).requires_grad_(train)
    parts, sums = [], [0.0, 0.0]
    step = max(1, (1 << 25) // case["cols"])
    for a in range(0, rows, step):
        x = s["x"][a:a + step].to(f64)
        if s["residual"] is not None:  # the sum is kept in x's type
            x = (x + s["residual"][a:a + step].to(f64)).to(F32).to(s["x"].dtype).to(f64)
        x.requires_grad_(train)
        with torch.enable_grad():
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None] * w
            y = y if b is None else y + b
        got = {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach()}
        if s["residual"] is not None:
            got["sum"] = x.detach()
        if train:
            leaves = [x, w] + ([] if b is None else [b])
            grads = torch.autograd.grad(y, leaves, s["grad"][a:a + step].to(f64))
            got["grad_x"] = grads[0] if s["grad_sum"] is None else grads[0] + s["grad_sum"][a:a + step].to(f64)
            sums = [t + u for t, u in zip(sums, grads[1:])]
        parts.append(got)
    out = {k: torch.cat([p[k] for p in parts]) for k in (("sum",) if s["residual"] is not None else ()) + ("y", "mean", "rstd")}
    if train:
        out |= {"grad_x": torch.cat([p["grad_x"] for p in parts]), "grad_weight": sums[0]}
        if b is not None:
            out["grad_bias"] = sums[1]
    return out


def exact(case, seed):
    with torch.no_grad():
        s = prepare({**case, "mode": "train"} if case["op"] == "fp4" and case["mode"] == "serve" else case, seed)
        return _exact_norm(case, s) if case["op"] == "norm" else _exact_fp4(case, s, s.get("w"))
