"""Trains a small language model on one GPU with the package's operators and
optimizer: FP16 weights, the embedding, layer norm, GELU and linear layers that keep
8-bit activations, the vocabulary's cross entropy without logits in memory, and
Fp8AdamW on the gradients, with a loss scale.

    python examples/train_lm.py [--steps 200] [--tokens 4096] [--vocab 5003]

The text is drawn from a fixed random table of likely successors, so that there
is something to learn: the loss falls from log(vocab) toward log(4).
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_optimizer_gb300 as bo  # noqa: E402
from bit_optimizer_gb300 import nn  # noqa: E402


class Model:
    """An embedding, residual feed-forward blocks over the current token, a
    final norm, and the embedding again as the output layer."""

    def __init__(self, vocab, dim, blocks, generator):
        def weight(*shape, std):
            w = torch.randn(*shape, device="cuda", generator=generator) * std
            return w.half().requires_grad_(True)

        def constant(n, value):
            return torch.full((n,), value, dtype=torch.float16, device="cuda",
                              requires_grad=True)
        self.wte = weight(vocab, dim, std=0.02)
        self.blocks = [dict(ln_w=constant(dim, 1.0), ln_b=constant(dim, 0.0),
                            fc_w=weight(4 * dim, dim, std=0.02), fc_b=constant(4 * dim, 0.0),
                            out_w=weight(dim, 4 * dim, std=0.02 / math.sqrt(2 * blocks)),
                            out_b=constant(dim, 0.0)) for _ in range(blocks)]
        self.lnf_w, self.lnf_b = constant(dim, 1.0), constant(dim, 0.0)

    def parameters(self):
        return [self.wte, *(p for b in self.blocks for p in b.values()), self.lnf_w, self.lnf_b]

    def loss(self, tokens, target):
        x = nn.embedding(tokens, self.wte)
        for b in self.blocks:
            h = nn.gelu(nn.linear(nn.layer_norm(x, b["ln_w"], b["ln_b"]), b["fc_w"], b["fc_b"]))
            x = x + nn.linear(h, b["out_w"], b["out_b"])
        return nn.linear_cross_entropy(nn.layer_norm(x, self.lnf_w, self.lnf_b), self.wte, target)


def train(steps=200, tokens=4096, vocab=5003, dim=256, blocks=2, seed=0, report=None):
    """Returns the loss of every step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    successors = torch.randint(0, vocab, (vocab, 4), device="cuda", generator=g)
    model = Model(vocab, dim, blocks, g)
    params = model.parameters()
    opt = bo.Fp8AdamW([p.data for p in params], lr=2e-3, weight_decay=0.01, scaled_v=True,
                      max_grad_norm=1.0)
    scale, losses = 2.0 ** 12, []
    for step in range(steps):
        now = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
        pick = torch.randint(0, 4, (tokens, 1), device="cuda", generator=g)
        target = successors[now].gather(1, pick)[:, 0]
        target[-tokens // 16:] = -100          # padding takes no part
        loss = model.loss(now, target)
        grads = torch.autograd.grad(loss * scale, params)
        if opt.step([d.contiguous() for d in grads], inv_loss_scale=1.0 / scale):
            scale /= 2                         # a skipped step: too large a scale
        losses.append(loss.item())
        if report and (step % report == 0 or step == steps - 1):
            print(f"step {step:4d}  loss {losses[-1]:.4f}  loss scale {scale:g}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=5003)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.vocab, report=20)
