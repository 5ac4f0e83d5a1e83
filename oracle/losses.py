"""Token log probabilities and the balance loss with their gradients, in
float64 from their definitions -- TEST INFRASTRUCTURE ONLY.

Log probabilities: z = scale x, lse = log sum exp z, logprob = z_target - lse,
entropy = -sum p log p; the alternatives are the largest x, equal ones by the
lower index.  Rows with a negative target are left out (zeros, ids -1); a
target past the vocabulary gives NaN.  A row of -inf only has lse = logprob =
-inf and entropy 0.

Balance loss: see balance_loss below.
"""

import numpy as np


def token_logprobs(x, targets, scale=1.0, top=0):
    """(logprobs, lse, entropy, top_logprobs, top_ids) of float64 rows."""
    x = np.asarray(x, np.float64)
    rows, vocab = x.shape
    lp, lse, h = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    tlp, ids = np.zeros((rows, top)), np.full((rows, top), -1, np.int64)
    for r in range(rows):
        t = int(targets[r])
        if t < 0:
            continue
        z = x[r] * scale
        nan = bool(np.isnan(z).any() or (z == np.inf).any())
        m = z.max() if not nan else np.nan
        if nan:
            lse[r] = h[r] = np.nan
        elif m == -np.inf:
            lse[r], h[r] = -np.inf, 0.0
        else:
            d = z - m
            e = np.exp(d)
            s = e.sum()
            lse[r] = m + np.log(s)
            h[r] = np.log(s) - (e[e > 0] * d[e > 0]).sum() / s
        # z_j - lse, with log s kept apart from a largest logit that may be the type's lowest value
        value = lambda j: -np.inf if lse[r] == -np.inf else (np.nan if nan else d[j] - np.log(s))  # noqa: E731
        lp[r] = np.nan if t >= vocab else value(t)
        rank = np.where(np.isnan(x[r]), -np.inf, x[r])
        ids[r] = np.argsort(-rank, kind="stable")[:top]
        tlp[r] = [value(j) for j in ids[r]]
    return lp, lse, h, tlp, ids


def token_logprobs_grad(x, targets, grad_logprobs, grad_entropy=None, scale=1.0):
    """d (sum gl logprob + ge entropy) / dx by the chain rule through log p:
    with c_k = d loss / d log p_k, dx_j = scale (c_j - p_j sum_k c_k)."""
    x = np.asarray(x, np.float64)
    rows, vocab = x.shape
    out = np.zeros((rows, vocab))
    for r in range(rows):
        t = int(targets[r])
        if t < 0:
            continue
        z = x[r] * scale
        if z.max() == -np.inf:
            continue
        d = z - z.max()
        logp = d - np.log(np.exp(d).sum())
        p = np.exp(logp)
        c = np.zeros(vocab)
        if grad_entropy is not None:
            live = p > 0
            c[live] = -grad_entropy[r] * p[live] * (logp[live] + 1)
        c[t] += grad_logprobs[r]
        out[r] = scale * (c - p * c.sum())
        if z[t] == -np.inf:
            out[r][t] = scale * grad_logprobs[r]
    return out


def _softmax(x):
    d = x - x.max(axis=1, keepdims=True)
    e = np.exp(d)
    s = e.sum(axis=1, keepdims=True)
    return e / s, (x.max(axis=1, keepdims=True) + np.log(s))[:, 0]


def balance_loss(x, ids, mask=None, groups=1):
    """dict of balance, z, counts, tokens, mean (float64).  Over the kept
    tokens of a group: f = counts / sum counts, P = mean softmax;
    balance = mean over the groups with tokens of E sum f P, z = mean over
    all kept tokens of lse^2."""
    x = np.asarray(x, np.float64)
    tokens, E = x.shape
    mask = np.ones(tokens, bool) if mask is None else np.asarray(mask, bool)
    counts, n, mean = np.zeros((groups, E), np.int64), np.zeros(groups, np.int64), np.zeros((groups, E))
    losses, squares = [], 0.0
    for g in range(groups):
        rows = np.arange(g * (tokens // groups), (g + 1) * (tokens // groups))
        rows = rows[mask[rows]]
        n[g] = rows.size
        if not rows.size:
            continue
        p, lse = _softmax(x[rows])
        squares += (lse ** 2).sum()
        mean[g] = p.mean(axis=0)
        k = np.asarray(ids)[rows].reshape(-1)
        counts[g] = np.bincount(k[(k >= 0) & (k < E)], minlength=E)
        losses.append(E * (counts[g] / max(1, counts[g].sum()) * mean[g]).sum())
    return {"balance": float(np.mean(losses)) if losses else 0.0, "z": squares / n.sum() if n.sum() else 0.0,
            "counts": counts, "tokens": n, "mean": mean}


def balance_loss_grad(x, ids, grad_balance, grad_z, mask=None, groups=1):
    """Gradient of grad_balance balance + grad_z z (the counts are constants)."""
    x = np.asarray(x, np.float64)
    tokens, E = x.shape
    mask = np.ones(tokens, bool) if mask is None else np.asarray(mask, bool)
    r = balance_loss(x, ids, mask, groups)
    some, kept = max(1, int((r["tokens"] > 0).sum())), max(1, int(r["tokens"].sum()))
    out = np.zeros((tokens, E))
    for t in np.nonzero(mask)[0]:
        g = t // (tokens // groups)
        p, lse = _softmax(x[t:t + 1])
        f = r["counts"][g] / max(1, r["counts"][g].sum())
        dp = grad_balance / some * E * f / r["tokens"][g]     # d loss / d p
        out[t] = p[0] * (dp - (dp * p[0]).sum()) + grad_z * 2 * lse[0] / kept * p[0]
    return out
