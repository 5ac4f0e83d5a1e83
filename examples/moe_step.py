"""A small mixture-of-experts language model trained with the library's parts
from end to end, on one GPU and synthetic tokens:

    tokens -> embedding, gain -> router -> top expert -> FP8 head -> loss

* the head is ``fp8_mm``; ``token_logprobs_loss`` turns its logits into their
  gradient in place, and ``fp8_mm_backward`` takes that from there;
* ``balance_loss`` keeps the router from sending every token to one expert;
* the experts' matrices take the Muon step, everything else (embedding and
  head with 8-bit moments, router and gain with 32-bit ones) AdamW.

Run it with ``python examples/moe_step.py [steps]``.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from newton_schulz_08_gb300 import muon  # noqa: E402

VOCAB, WIDTH, HIDDEN, EXPERTS, TOKENS = 512, 128, 256, 8, 2048


def scale_for(t, largest):
    """An FP8 scale that leaves 5 % above the largest magnitude of t."""
    return max(float(t.abs().max().float()) / largest * 1.05, 1e-12)


class Model:
    def __init__(self, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        normal = lambda *s, std: torch.randn(s, generator=g, device="cuda").mul_(std)  # noqa: E731
        self.embed, self.head = normal(VOCAB, WIDTH, std=1.0), normal(VOCAB, WIDTH, std=0.05)
        self.gain, self.router = torch.ones(WIDTH, device="cuda"), normal(EXPERTS, WIDTH, std=0.05)
        self.up = [normal(HIDDEN, WIDTH, std=0.05) for _ in range(EXPERTS)]
        self.down = [normal(WIDTH, HIDDEN, std=0.05) for _ in range(EXPERTS)]
        self.bank = self.up + self.down                                    # Muon
        self.others = [self.embed, self.head, self.gain, self.router]      # AdamW
        self.bufs = [torch.zeros_like(w) for w in self.bank]
        self.adamw = muon.AdamW(self.others, states=[muon.adamw_state(p, 8 if p.numel() >= 4096 else 32) for p in self.others],
                                lr=[1e-2, 1e-2, 1e-3, 1e-2], weight_decay=[0.01, 0.01, 0.0, 0.0], beta2=0.95, seed=seed)

    def hidden(self, tokens):
        """The head's input and the router's scores and choice (autograd)."""
        h = torch.nn.functional.embedding(tokens, self.embed) * self.gain
        scores = h @ self.router.t()
        gate, expert = torch.softmax(scores, 1).max(1)
        out = torch.zeros_like(h)
        for e in range(EXPERTS):
            rows = (expert == e).nonzero()[:, 0]
            out = out.index_add(0, rows, gate[rows, None] * (torch.relu(h[rows] @ self.up[e].t()).square() @ self.down[e].t()))
        return h + out, scores, expert[:, None]

    def step(self, tokens, targets, balance_weight=0.02, z_weight=1e-4):
        """One training step; returns (mean loss, entropy, balance loss, counts)."""
        every = self.others + self.bank
        for w in every:
            w.requires_grad_(True)
        h, scores, ids = self.hidden(tokens)
        # head and loss
        x, w = h.detach().bfloat16(), self.head.detach().bfloat16()
        x_s, w_s = scale_for(x, 448.0), scale_for(w, 448.0)
        logits, x_f8, w_f8 = muon.fp8_mm(x, w, x_s, w_s)
        kept = (targets >= 0).sum().clamp_min(1)
        r = muon.token_logprobs_loss(logits, targets, (-1.0 / kept).expand(len(targets)).contiguous(), out=logits)
        grad_s = scale_for(r.grad, 57344.0)
        grad_h, grad_head, _ = muon.fp8_mm_backward(r.grad, x_f8, w_f8, x_s, w_s, grad_s)
        # router
        b = muon.balance_loss(scores.detach(), ids)
        weight = lambda v: torch.full((1,), v, device="cuda")  # noqa: E731
        grad_scores = muon.balance_loss_backward(scores.detach(), b, weight(balance_weight), weight(z_weight))
        # through the model; an expert without tokens has no gradient
        rest = [self.embed, self.gain, self.router] + self.bank
        grads = torch.autograd.grad([h, scores], rest, [grad_h.float(), grad_scores], allow_unused=True)
        for w in every:
            w.requires_grad_(False)
        grads = [torch.zeros_like(w) if g is None else g.contiguous() for w, g in zip(rest, grads)]
        muon.muon_step(self.bank, grads[3:], self.bufs, lr=0.01)
        norm = torch.stack([g.norm() for g in grads[:3]]).norm()
        clip = (1.0 / norm.clamp_min(1.0)).reshape(1)
        self.adamw.step([grads[0], grad_head, grads[1], grads[2]], grad_scale=clip)
        return -(r.logprobs.sum() / kept), r.entropy.mean(), b.balance, b.counts


def batch(step):
    """Tokens of a fixed random successor table with 10 % noise; every 16th target is left out."""
    g = torch.Generator("cuda").manual_seed(12345)
    after = torch.randperm(VOCAB, generator=g, device="cuda")
    g = torch.Generator("cuda").manual_seed(step)
    tokens = torch.randint(0, VOCAB, (TOKENS,), generator=g, device="cuda")
    noise = torch.randint(0, VOCAB, (TOKENS,), generator=g, device="cuda")
    targets = torch.where(torch.rand(TOKENS, generator=g, device="cuda") < 0.1, noise, after[tokens])
    targets[::16] = -100
    return tokens, targets


def train(steps, report=None):
    """Trains a model; returns the loss, entropy, balance loss and counts of every step."""
    model, history = Model(), []
    for k in range(steps):
        history.append([x.detach().clone() for x in model.step(*batch(k))])
        if report and (k % 10 == 0 or k == steps - 1):
            loss, entropy, balance, counts = history[-1]
            report(f"step {k:4d}  loss {loss.item():.3f}  entropy {entropy.item():.3f}  "
                   f"balance {balance.item():.3f}  tokens per expert {counts[0].tolist()}")
    return history


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100, print)
