"""Workloads of the operators at the two ends of a training step: the losses where gradients begin
(log probabilities of given tokens, balance loss of a router) and the AdamW step that consumes them.

Each case is one pass through one operator. ``run`` computes it either in its plain form (elementary
torch operations in float32, rounded once where a result has a narrower type) or, with ``own`` set,
through the framework's entry points.

Conventions shared by both forms:

AdamW. All tensors of a case are views into one flat bucket, each starting at a multiple of 256
elements (``odd`` shifts the whole bucket by one element, as a view into a larger buffer would).
8-bit moments: blocks of 256 consecutive elements of a tensor share a power-of-two scale; the first
moment's codes are E4M3, the second's E5M2. With E = max(floor(log2(max |x|)), -100) over the block the
scales are 2^(E-7) and 2^(E-14) (NaN where a value is not finite or 2^127 or more). Codes, and bfloat16 parameters, are rounded stochastically with 16 bits
each of a counter hash of (seed, step, tensor, element), so that moving averages whose change per step is
far below a code's spacing stay unbiased.

Token log probabilities. ``mode`` is what the pass does: "score" computes log probabilities, entropy and
alternatives; "loss" also the gradient of a loss whose weights are known beforehand; "policy" scores, forms
the gradient of a probability ratio from the result, and then runs the backward pass. A target below 0 marks a row that is left out: its outputs are 0 (ids -1) and its
gradient 0. Equal logits are ranked by the lower index. Entries of -inf have probability 0.

Balance loss. The tokens form ``groups`` sequences of equal length; the loss of a group is
E * sum_e f_e * P_e with f the share of the assignments and P the mean router probability over its unmasked
tokens, averaged over the groups that have any. The second value is the mean squared log-partition.
"""

import math

import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
_TYPES = {"f32": F32, "bf16": BF16}
_SIZE = {"f32": 4, "bf16": 2}
BLOCK = 256        # elements that share one scale of an 8-bit moment
FIRST_STEP = 10    # AdamW steps already taken when a pass begins
VOCAB = 50304      # padded vocabulary of the embedding bank
WIDTHS = (768, 1600)


# ------------------------------------------------------------------------------------------- cases

def listed():
    adamw = {"op": "adamw", "grad": "bf16", "odd": False, "cautious": False, "clip": False}
    logp = {"op": "logprobs", "scale": 1.0, "mask": 0, "ignored": 0.0, "pad": 0}
    bal = {"op": "balance", "masked": 0.0, "drop": 0.0}
    return [
        # gains and biases of a 48-layer model, 1600 wide: many tiny tensors, one launch's latency
        dict(adamw, name="adamw_gains_f32", sizes="1600*192,4800*48,6400*48", param="f32", state=32),
        # the embedding bank of four 50304 x 768 tables, moments in 32 bits
        dict(adamw, name="adamw_tables_f32", sizes="38633472*4", param="f32", state=32, cautious=True),
        # the same bank with moments in 8 bits
        dict(adamw, name="adamw_tables_8bit", sizes="38633472*4", param="f32", state=8, cautious=True),
        # bfloat16 weights of a 50257 x 1600 table, positions and gains, in a bucket at an odd offset, gradients clipped
        dict(adamw, name="adamw_bf16_odd_8bit", sizes="80411200,1638400,1600*97,50257", param="bf16", state=8, odd=True, clip=True),
        # scoring one decoding step of 8 sequences with 8 alternatives: latency
        dict(logp, name="logprobs_decode", rows=8, vocab=VOCAB, type="bf16", top=8, mode="score"),
        # evaluation of a 4096-token prompt over the unpadded vocabulary (rows of odd length), 5 alternatives
        dict(logp, name="logprobs_eval_odd", rows=4096, vocab=50257, type="bf16", top=5, mode="score"),
        # evaluation in float32 with padded columns masked, 20 alternatives, temperature 0.8
        dict(logp, name="logprobs_eval_f32", rows=6001, vocab=VOCAB, type="f32", top=20, scale=1.25, mask=47, mode="score"),
        # a training step's loss over 16384 tokens: forward and gradient, entropy bonus, some prompt tokens left out
        dict(logp, name="logprobs_loss", rows=16384, vocab=VOCAB, type="bf16", top=0, ignored=0.1, mask=47, mode="loss"),
        # a small policy update in float32 with a padded row pitch: forward, ratio, backward
        dict(logp, name="logprobs_policy_f32", rows=777, vocab=32001, type="f32", top=1, pad=3, ignored=0.3, mode="policy"),
        # router of a small mixture model on one micro-batch: latency
        dict(bal, name="balance_small", tokens=2048, experts=64, top=6, groups=1, type="bf16"),
        # router of a large batch: 256 experts, one loss per sequence, float32 scores
        dict(bal, name="balance_sequences_f32", tokens=131072, experts=256, top=8, groups=32, type="f32", drop=0.02),
        # an odd number of experts, padded sequences
        dict(bal, name="balance_masked_odd", tokens=65536, experts=161, top=4, groups=16, type="bf16", masked=0.2),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("adamw", "logprobs", "balance"))
    if op == "adamw":
        total, n, sizes = _log_uniform(rng, 2000, 120_000_000), rng.choice((1, 1, 3, 9, 40, 200)), []
        for _ in range(n):
            sizes.append(max(1, int(total * rng.uniform(0.2, 1.0) / n)))
        if rng.random() < 0.5:
            sizes[0] = max(1, sizes[0] // 768 * 768)
        sizes.append(rng.randrange(1, 3000))
        return {"op": op, "sizes": ",".join(map(str, sizes)), "param": rng.choice(("f32", "bf16")), "grad": rng.choice(("bf16", "f32")),
                "state": rng.choice((8, 32)), "odd": rng.random() < 0.3, "cautious": rng.random() < 0.5, "clip": rng.random() < 0.5}
    if op == "logprobs":
        vocab = _log_uniform(rng, 2, 160_000)
        return {"op": op, "rows": _log_uniform(rng, 1, max(1, min(65536, 400_000_000 // vocab))), "vocab": vocab,
                "type": rng.choice(("bf16", "f32")), "top": rng.choice((0, 1, min(5, vocab), min(20, vocab), min(32, vocab))),
                "mode": rng.choice(("score", "loss", "policy")), "scale": rng.choice((1.0, 1.0, 0.7, 1.25)), "mask": rng.randrange(0, max(1, vocab // 8)),
                "ignored": rng.choice((0.0, 0.2)), "pad": rng.choice((0, 0, 1, 8))}
    groups, experts = rng.choice((1, 1, 2, 8, 30, 64)), _log_uniform(rng, 2, 512)
    return {"op": op, "tokens": groups * _log_uniform(rng, 1, max(2, min(262144, 33_000_000 // experts) // groups)), "experts": experts,
            "top": rng.randrange(1, min(8, experts) + 1), "groups": groups, "type": rng.choice(("bf16", "f32")),
            "masked": rng.choice((0.0, 0.1, 0.5)), "drop": rng.choice((0.0, 0.05))}


def _sizes(case):
    got = []
    for part in case["sizes"].split(","):
        n, _, times = part.partition("*")
        got += [int(n)] * int(times or 1)
    return got


# ------------------------------------------------------------------------------------------ inputs

HYPER = {"beta1": 0.9, "beta2": 0.95, "eps": 1e-8}


def _rates(sizes):
    """Learning rate and weight decay of each tensor: tables decay, gains and biases (below 10,000 elements) do not."""
    return [3e-4 if n >= 10_000 else 6e-4 for n in sizes], [0.1 if n >= 10_000 else 0.0 for n in sizes]


def _prepare_adamw(case, gen, seed):
    sizes, dev = _sizes(case), "cuda"
    blocks = [-(-n // BLOCK) for n in sizes]
    first = np.concatenate([[0], np.cumsum(blocks)])
    total, shift = int(first[-1]) * BLOCK, int(case["odd"])
    tensor = torch.from_numpy(np.repeat(np.arange(len(sizes)), blocks)).to(dev)          # of each block
    number = torch.arange(total // BLOCK, device=dev) - torch.from_numpy(first[:-1]).to(dev)[tensor]  # within its tensor
    live = (number * BLOCK)[:, None] + torch.arange(BLOCK, device=dev) < torch.tensor(sizes, device=dev)[tensor][:, None]

    def bucket(kind, values):
        flat = torch.zeros(total + 16, dtype=kind, device=dev)[shift:shift + total]
        flat.copy_(values.view(-1))
        return flat

    draw_ = lambda std: torch.randn((total // BLOCK, BLOCK), generator=gen, device=dev).mul_(std) * live  # noqa: E731
    p, g = bucket(_TYPES[case["param"]], draw_(0.02)), bucket(_TYPES[case["grad"]], draw_(1e-3))
    state = {"p": p, "g": g}
    m, v = draw_(3e-4), draw_(1e-3).square_()
    if case["state"] == 32:
        state["m"], state["v"] = m.view(-1), v.view(-1)
    else:  # what earlier steps have left: codes and the blocks' scales
        for key, x, kind, shift_e in (("m", m, torch.float8_e4m3fn, 7), ("v", v, torch.float8_e5m2, 14)):
            s = _pow2(_exponent(x.abs().amax(1, keepdim=True)) - shift_e)
            state[key], state[key + "_scale"] = (x / s).to(kind).view(-1), s.view(-1)
    state |= {"case": case, "t": FIRST_STEP, "seed": seed, "sizes": sizes, "tensor": tensor, "number": number}
    state["clip"] = torch.tensor([0.37], device=dev) if case["clip"] else None
    if own:  # the optimizer object that a program keeps beside its parameters
        from newton_schulz_08_gb300 import muon
        cut = lambda x: [x[int(a) * BLOCK:int(a) * BLOCK + n] for a, n in zip(first, sizes)]  # noqa: E731
        part = lambda x: [x[int(a):int(a) + b] for a, b in zip(first, blocks)]  # noqa: E731
        if case["state"] == 32:
            states = list(zip(cut(state["m"]), cut(state["v"])))
        else:
            states = list(zip(cut(state["m"]), part(state["m_scale"]), cut(state["v"]), part(state["v_scale"])))
        lr, wd = _rates(sizes)
        state["opt"] = muon.AdamW(cut(p), grads=cut(g), states=states, lr=lr, weight_decay=wd, cautious=case["cautious"], seed=seed, step=FIRST_STEP, **HYPER)
    return state


def _prepare_logprobs(case, gen):
    rows, vocab, dev = case["rows"], case["vocab"], "cuda"
    kind, pitch = _TYPES[case["type"]], vocab + case["pad"]
    common = -torch.log(torch.randperm(vocab, generator=gen, device=dev).to(F32) + 2.0)   # how frequent each token is
    x = torch.empty((rows, pitch), dtype=kind, device=dev)
    step = max(1, (1 << 28) // pitch)
    for r in range(0, rows, step):
        part = x[r:r + step, :vocab]
        part.copy_(torch.randn(part.shape, generator=gen, device=dev).mul_(2.0).add_(common))
    x = x[:, :vocab]
    y = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
    if case["mask"]:  # columns beyond the real vocabulary
        x[:, vocab - case["mask"]:] = -math.inf
        y.remainder_(vocab - case["mask"])
    out = torch.rand(rows, generator=gen, device=dev) < case["ignored"]
    state = {"case": case, "x": x, "y": torch.where(out, torch.full_like(y, -100), y)}
    if case["mode"] != "score":
        state["gl"] = torch.randn(rows, generator=gen, device=dev) / rows   # advantages over the batch
        state["gh"] = torch.full((rows,), 0.01 / rows, device=dev)          # entropy bonus
    if case["mode"] == "policy":  # log probabilities under the policy that sampled the tokens
        at = x.gather(1, state["y"].clamp_min(0)[:, None]).to(F32)[:, 0] * case["scale"]
        step = max(1, (1 << 28) // vocab)
        lse = torch.cat([torch.logsumexp(x[r:r + step].to(F32) * case["scale"], 1) for r in range(0, rows, step)])
        state["old"] = at - lse + torch.randn(rows, generator=gen, device=dev) * 0.05
    return state


def _prepare_balance(case, gen):
    tokens, experts, dev = case["tokens"], case["experts"], "cuda"
    x = torch.randn((tokens, experts), generator=gen, device=dev).add_(torch.randn(experts, generator=gen, device=dev).mul_(0.5)).to(_TYPES[case["type"]])
    ids = torch.sort(x.to(F32), dim=1, descending=True, stable=True).indices[:, :case["top"]].contiguous()
    ids[torch.rand(ids.shape, generator=gen, device=dev) < case["drop"]] = -1    # assignments over an expert's capacity
    mask = torch.rand(tokens, generator=gen, device=dev) >= case["masked"] if case["masked"] else None
    return {"case": case, "x": x, "ids": ids, "mask": mask, "gb": torch.tensor([0.01], device=dev), "gz": torch.tensor([0.001], device=dev)}


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(1_000_003 * (int(seed) + 1))
    with torch.no_grad():
        if case["op"] == "adamw":
            return _prepare_adamw(case, gen, int(seed))
        return (_prepare_logprobs if case["op"] == "logprobs" else _prepare_balance)(case, gen)


# ------------------------------------------------------------------- random bits of the 8-bit state

_M, _C0, _C1, _C2 = 0xFFFFFFFF, 0x9E3779B1, 0x6A09E667, 0xBB67AE85


def _mix(x):
    """Scrambles 32 bits (an int, or an int64 tensor of such)."""
    x = ((x ^ (x >> 16)) * _C1) & _M
    x = ((x ^ (x >> 15)) * _C2) & _M
    return x ^ (x >> 16)


def _keys(seed, step, n):
    k = _mix(_mix((seed + _C0 * step) & _M) ^ (seed >> 32 & _M))
    return [_mix((k + _C0 * i) & _M) for i in range(n)]


def _bits(state):
    """32 random bits of every element of the bucket, as int64 [blocks, BLOCK]."""
    keys = torch.tensor(_keys(state["seed"], state["t"], len(state["sizes"])), device=state["p"].device)[state["tensor"]]
    i = (state["number"] * BLOCK)[:, None] + torch.arange(BLOCK, device=state["p"].device)
    return _mix(((i & _M) * _C0 + (keys + (i[:, 0] >> 32) * _C1)[:, None]) & _M)


# ------------------------------------------------------------------------------------- plain forms

def _exponent(a):
    """floor(log2(a)) of non-negative float32 values, at least -100."""
    return ((a.view(torch.int32) >> 23) - 127).clamp_min(-100)


def _pow2(e):
    """2^e for whole numbers from -126 to 127."""
    return ((e + 127) << 23).view(F32)


def _codes(x, r16, kind):
    """Block-wise 8-bit form of x [blocks, BLOCK] with 16 random bits per element: codes and scales."""
    top, drop, e_shift = (14, 20, 7) if kind == torch.float8_e4m3fn else (29, 21, 14)
    a = x.abs().amax(1, keepdim=True)
    e = _exponent(a).clamp_max(126)
    y = (x.abs() * _pow2(-e)) * 2.0 ** (top - 127)
    code = (y.view(torch.int32) + ((r16 << (drop - 16)) + (1 << (drop - 17))).to(torch.int32)) >> drop
    code = torch.where(x < 0, code + 128, code)
    s = torch.where(a < 2.0 ** 127, _pow2(e - e_shift), a * math.nan)
    return code.to(torch.uint8).view(kind), s


def _plain_adamw(s):
    case, blocks = s["case"], s["tensor"].numel()
    s["t"] += 1
    b1, b2, t = HYPER["beta1"], HYPER["beta2"], s["t"]
    bc1, r2 = 1 - b1 ** t, 1 / math.sqrt(1 - b2 ** t)
    lr, wd = (np.array(x) for x in _rates(s["sizes"]))
    per_block = lambda a: torch.from_numpy(a.astype(np.float32)).to(s["p"].device)[s["tensor"]][:, None]  # noqa: E731
    p, g = s["p"].view(blocks, BLOCK).to(F32), s["g"].view(blocks, BLOCK).to(F32)
    if s["clip"] is not None:
        g = g * s["clip"]
    small = case["state"] == 8
    m, v = (s[k].view(blocks, BLOCK).to(F32) * s[k + "_scale"][:, None] if small else s[k].view(blocks, BLOCK) for k in ("m", "v"))
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    u = m / (torch.sqrt(v) * r2 + HYPER["eps"])
    decay = p * per_block(lr * wd)
    if case["cautious"]:
        decay = torch.where((u > 0) & (p > 0) | (u < 0) & (p < 0), decay, torch.zeros_like(decay))
    p = p - (u * per_block(lr / bc1) + decay)
    bits = _bits(s) if small or case["param"] == "bf16" else None
    if case["param"] == "bf16":
        r = (bits * _C0 & _M) >> 16
        up = ((p.view(torch.int32).to(torch.int64) + r) >> 16 << 16).to(torch.int32).view(F32)
        p = torch.where(torch.isfinite(p), up, p)
    s["p"].view(blocks, BLOCK).copy_(p)  # what lies between two tensors is zero and stays so
    out = {"p": s["p"]}
    for key, x in (("m", m), ("v", v)):
        if small:
            code, scale = _codes(x, bits & 0xFFFF if key == "m" else bits >> 16, s[key].dtype)
            s[key].copy_(code.view(-1))
            s[key + "_scale"].copy_(scale.view(-1))
            out[key + "_scale"] = s[key + "_scale"]
        else:
            s[key].view(blocks, BLOCK).copy_(x)
        out[key] = s[key]
    return out


def _plain_logprobs(s):
    case, x, y = s["case"], s["x"], s["y"]
    kept = y >= 0
    z = x.to(F32) * case["scale"]
    m = z.amax(1, keepdim=True)
    d = z - torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    lse = m + log_total
    at = z.gather(1, y.clamp_min(0)[:, None])
    zero = torch.zeros((), device=x.device)
    d = torch.where(e > 0, d, zero)
    h = torch.where(total > 0, log_total - (e * d).sum(1, keepdim=True) / total, zero)
    out = {"logprobs": torch.where(kept, (at - lse)[:, 0], zero), "lse": torch.where(kept, lse[:, 0], zero), "entropy": torch.where(kept, h[:, 0], zero)}
    if case["top"]:  # value, then the lower index: one sortable whole number
        bits = (x.to(F32) + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
        order = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device=x.device))
        ids = 0xFFFFFFFF - (torch.topk(order, case["top"], dim=1).values & 0xFFFFFFFF)
        out["top_ids"] = torch.where(kept[:, None], ids, -torch.ones_like(ids))
        out["top_logprobs"] = torch.where(kept[:, None], z.gather(1, ids) - lse, zero)
    if case["mode"] != "score":
        p = torch.exp(z - lse)
        gl = s["gl"] if case["mode"] == "loss" else s["gl"] * torch.exp(out["logprobs"] - s["old"])
        gl, gh = torch.where(kept, gl, zero)[:, None], torch.where(kept, s["gh"], zero)[:, None]
        logp = torch.where(p > 0, z - lse, zero)
        grad = -p * (gl + gh * (logp + h))
        grad.scatter_add_(1, y.clamp_min(0)[:, None], gl)
        out["grad"] = (grad * case["scale"]).to(x.dtype)
    return out


def _plain_balance(s):
    case, x, ids, mask = s["case"], s["x"].to(F32), s["ids"], s["mask"]
    tokens, experts, groups = case["tokens"], case["experts"], case["groups"]
    z = x - x.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    p, lse = e / total, x.amax(1) + torch.log(total[:, 0])
    live = torch.ones(tokens, dtype=torch.bool, device=x.device) if mask is None else mask
    group = torch.arange(tokens, device=x.device) // (tokens // groups)
    slot = torch.where((ids >= 0) & (ids < experts) & live[:, None], group[:, None] * experts + ids, torch.full_like(ids, groups * experts))
    counts = torch.zeros(groups * experts + 1, dtype=torch.int32, device=x.device)
    counts = counts.index_add_(0, slot.view(-1), torch.ones(slot.numel(), dtype=torch.int32, device=x.device))[:-1].view(groups, experts)
    n = live.view(groups, -1).sum(1)
    f = counts / counts.sum(1, keepdim=True).clamp_min(1)
    mean = (p * live[:, None]).view(groups, -1, experts).sum(1) / n.clamp_min(1)[:, None]
    some, everyone = (n > 0).sum().clamp_min(1), n.sum().clamp_min(1)
    balance = experts * (f * mean).sum() / some
    z_loss = torch.where(live, lse * lse, torch.zeros_like(lse)).sum() / everyone
    a = (s["gb"] * experts / some / n.clamp_min(1))[:, None] * f
    a = a.repeat_interleave(tokens // groups, 0)
    grad = p * (a - (a * p).sum(1, keepdim=True) + (s["gz"] * 2 / everyone * lse)[:, None])
    return {"balance": balance, "z": z_loss, "counts": counts, "tokens": n.to(torch.int32), "mean": mean,
            "grad": torch.where(live[:, None], grad, torch.zeros_like(grad)).to(s["x"].dtype)}


# --------------------------------------------------------------------------------------- own forms

def _own_adamw(s):
    s["opt"].step(grad_scale=s["clip"])
    keys = ("p", "m", "v") if s["case"]["state"] == 32 else ("p", "m", "m_scale", "v", "v_scale")
    return {k: s[k] for k in keys}


def _own_logprobs(s):
    from newton_schulz_08_gb300 import muon
    case = s["case"]
    if case["mode"] == "loss":
        r = muon.token_logprobs_loss(s["x"], s["y"], s["gl"], s["gh"], top=case["top"], scale=case["scale"])
    else:
        r = muon.token_logprobs(s["x"], s["y"], top=case["top"], scale=case["scale"])
    out = {"logprobs": r.logprobs, "lse": r.lse, "entropy": r.entropy}
    if case["top"]:
        out |= {"top_ids": r.top_ids, "top_logprobs": r.top_logprobs}
    if case["mode"] == "loss":
        out["grad"] = r.grad
    elif case["mode"] == "policy":
        gl = s["gl"] * torch.exp(r.logprobs - s["old"])
        out["grad"] = muon.token_logprobs_backward(s["x"], s["y"], r.lse, gl, entropy=r.entropy, grad_entropy=s["gh"], scale=case["scale"])
    return out


def _own_balance(s):
    from newton_schulz_08_gb300 import muon
    r = muon.balance_loss(s["x"], s["ids"], mask=s["mask"], groups=s["case"]["groups"])
    grad = muon.balance_loss_backward(s["x"], r, s["gb"], s["gz"], mask=s["mask"])
    return {"balance": r.balance, "z": r.z, "counts": r.counts, "tokens": r.tokens, "mean": r.mean_probs, "grad": grad}


def run(state):
    op = state["case"]["op"]
    with torch.no_grad():
        if own:
            return {"adamw": _own_adamw, "logprobs": _own_logprobs, "balance": _own_balance}[op](state)
        return {"adamw": _plain_adamw, "logprobs": _plain_logprobs, "balance": _plain_balance}[op](state)


# ------------------------------------------------------------------------------------ work, 64 bits

def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["state"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (2 * _SIZE[case["param"]] + _SIZE[case["grad"]] + state), "flops": 16 * n}
    s = _SIZE[case["type"]]
    if case["op"] == "logprobs":
        kept, each = round(case["rows"] * (1 - case["ignored"])), case["vocab"] * s
        read, flops = kept * each, 6 * kept * case["vocab"]
        if case["mode"] != "score":  # the gradient written; a row that is held between its two uses is read once
            read, flops = read + case["rows"] * (each + 8), 2 * flops
        return {"bytes": read + case["rows"] * (20 + 12 * case["top"]), "flops": flops}
    kept = case["tokens"] * (1 - case["masked"])
    read = kept * (case["experts"] * s + 8 * case["top"]) + case["tokens"] * (case["experts"] * s + (1 if case["masked"] else 0))
    return {"bytes": read + 8 * case["groups"] * case["experts"], "flops": 12 * kept * case["experts"]}


def _spacing(x, least, mantissa):
    """Distance between neighbouring numbers of a narrow format around x > 0 (least: exponent of its smallest normal number)."""
    return torch.ldexp(torch.ones_like(x), (torch.frexp(x).exponent - 1).clamp_min(least) - mantissa)


def _exact_codes(x, r, mantissa, least, e_shift):
    """x [blocks, BLOCK] rounded stochastically (r in [0, 1)) to its block's 8-bit grid, in units of the scales, and those."""
    e = (torch.frexp(x.abs().amax(1, keepdim=True)).exponent - 1).clamp_min(-100)
    y = torch.ldexp(x, e_shift - e)
    grid = _spacing(y.abs(), least, mantissa)
    return torch.sign(y) * torch.floor(y.abs() / grid + r) * grid, torch.ldexp(torch.ones_like(x[:, :1]), e - e_shift)


def _exact_adamw(case, s):
    """Tensor by tensor in float64, the textbook formulas."""
    f64, t = torch.float64, FIRST_STEP + 1
    lr, wd = _rates(s["sizes"])
    out = {k: torch.zeros(s[k].shape, dtype=f64, device="cuda") for k in ("p", "m", "v")}
    if case["state"] == 8:
        out |= {k: s[k].to(f64) for k in ("m_scale", "v_scale")}
    at = 0
    for i, (n, key) in enumerate(zip(s["sizes"], _keys(s["seed"], t, len(s["sizes"])))):
        nb = -(-n // BLOCK)
        here, blk = slice(at * BLOCK, at * BLOCK + n), slice(at, at + nb)
        at += nb
        p, g, m, v = (s[k][here].to(f64) for k in ("p", "g", "m", "v"))
        if case["state"] == 8:
            m, v = (x * s[k][blk].to(f64).repeat_interleave(BLOCK)[:n] for x, k in ((m, "m_scale"), (v, "v_scale")))
        if s["clip"] is not None:
            g = g * s["clip"].to(f64)
        m = m.mul_(HYPER["beta1"]).add_(g, alpha=1 - HYPER["beta1"])
        v = v.mul_(HYPER["beta2"]).add_(g.square(), alpha=1 - HYPER["beta2"])
        u = (m / (1 - HYPER["beta1"] ** t)) / ((v / (1 - HYPER["beta2"] ** t)).sqrt() + HYPER["eps"])
        decay = wd[i] * p
        if case["cautious"]:
            decay = decay * (torch.sign(u) * torch.sign(p) > 0)
        p = p - lr[i] * (u + decay)
        h = _mix((torch.arange(n, device="cuda") * _C0 + key) & _M)
        if case["param"] == "bf16":
            grid = _spacing(p.abs(), -126, 7)
            p = torch.sign(p) * torch.floor(p.abs() / grid + ((h * _C0 & _M) >> 16) / 65536) * grid
        out["p"][here] = p
        if case["state"] == 32:
            out["m"][here], out["v"][here] = m, v
            continue
        full = lambda x: torch.nn.functional.pad(x, (0, nb * BLOCK - n)).view(nb, BLOCK)  # noqa: E731
        for k, x, r, form in (("m", m, h & 0xFFFF, (3, -6, 7)), ("v", v, h >> 16, (2, -14, 14))):
            value, scale = _exact_codes(full(x), (full(r.to(f64)) + 0.5) / 65536, *form)
            out[k][here], out[k + "_scale"][blk] = value.view(-1)[:n], scale[:, 0]
    return out


def _exact_logprobs(case, s):
    """Row blocks in float64: log-softmax from its definition, the gradient as a Jacobian product."""
    rows, f64 = case["rows"], torch.float64
    new = lambda *shape: torch.zeros(shape, dtype=f64, device="cuda")  # noqa: E731
    out = {"logprobs": new(rows), "lse": new(rows), "entropy": new(rows)}
    if case["top"]:
        out |= {"top_ids": None, "top_logprobs": new(rows, case["top"])}
    if case["mode"] != "score":
        out["grad"] = new(rows, case["vocab"])
    step = max(1, (1 << 26) // case["vocab"])
    for a in range(0, rows, step):
        b = min(rows, a + step)
        kept = (s["y"][a:b] >= 0).nonzero()[:, 0]
        z = s["x"][a:b][kept].to(f64) * case["scale"]
        y = s["y"][a:b][kept]
        lse = torch.logsumexp(z, 1)
        logp = z - lse[:, None]
        p = logp.exp()
        plogp = torch.where(p > 0, p * logp, torch.zeros_like(p))
        h = -plogp.sum(1)
        at = torch.arange(kept.numel(), device="cuda")
        rows_at = a + kept
        out["logprobs"][rows_at], out["lse"][rows_at], out["entropy"][rows_at] = logp[at, y], lse, h
        if case["top"]:
            out["top_logprobs"][rows_at] = logp.sort(1, descending=True).values[:, :case["top"]]
        if case["mode"] != "score":
            gl, gh = s["gl"][rows_at].to(f64), s["gh"][rows_at].to(f64)
            if case["mode"] == "policy":
                gl = gl * torch.exp(logp[at, y] - s["old"][rows_at].to(f64))
            up = torch.where(p > 0, -gh[:, None] * (logp + 1), torch.zeros_like(p)) * p   # through the probabilities
            grad = up - p * up.sum(1, keepdim=True) - gl[:, None] * p
            grad[at, y] += gl
            out["grad"][rows_at] = grad * case["scale"]
    return out


def _exact_balance(case, s):
    """One sequence at a time in float64, gradients by automatic differentiation of the loss."""
    groups, experts = case["groups"], case["experts"]
    x = s["x"].to(torch.float64).requires_grad_(True)
    ids = s["ids"].view(groups, -1, case["top"])
    live = torch.ones(case["tokens"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    live = live.view(groups, -1)
    losses, squares, means = [], [], []
    with torch.enable_grad():
        for k, rows in enumerate(x.view(groups, -1, experts)):
            kept = rows[live[k]]
            squares.append(torch.logsumexp(kept, 1).square().sum())
            mean = torch.softmax(kept, 1).sum(0) / max(1, kept.shape[0])
            means.append(mean)
            picked = ids[k][live[k]]
            picked = picked[(picked >= 0) & (picked < experts)]
            share = torch.bincount(picked, minlength=experts).to(torch.float64) / max(1, picked.numel())
            if kept.shape[0]:
                losses.append(experts * (share * mean).sum())
        balance = torch.stack(losses).mean() if losses else x.sum() * 0
        z = torch.stack(squares).sum() / max(1, int(live.sum()))
        (grad,) = torch.autograd.grad(balance * float(s["gb"]) + z * float(s["gz"]), x)
    return {"balance": balance.detach(), "z": z.detach(), "counts": None, "tokens": None, "mean": torch.stack(means).detach(), "grad": grad}


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        if case["op"] == "adamw":
            return _exact_adamw(case, s)
        return (_exact_logprobs if case["op"] == "logprobs" else _exact_balance)(case, s)
