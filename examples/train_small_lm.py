"""Trains a small language model with every operator of the package: blocks of
RMSNormLinear (the norm adds the residual and writes the FP8 operand), a
nonlinearity and a Float8BlockwiseLinear, a final RMSNorm, the vocabulary cross
entropy without logits, and AdamW with 8-bit states.

    python examples/train_small_lm.py [--steps 60] [--bits 8]

The text is synthetic: token t + 1 is a fixed function of token t, nine times
out of ten, so the loss falls from log(vocabulary) towards that rule's entropy.
Needs an MI355X."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import blockwise_scaled_fp8_amd as fp8  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, width, inner, device):
        super().__init__()
        self.up = fp8.RMSNormLinear(width, inner, device=device)
        self.down = fp8.Float8BlockwiseLinear(inner, width, device=device)

    def forward(self, x, residual):
        """x: the last block's output, not yet added to the residual stream."""
        y, residual = self.up(x, residual)
        return self.down(torch.nn.functional.silu(y)), residual


class SmallLM(torch.nn.Module):
    def __init__(self, vocab, width, inner, blocks, device):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(vocab, width, device=device).bfloat16())
        self.blocks = torch.nn.ModuleList(Block(width, inner, device) for _ in range(blocks))
        self.norm = fp8.RMSNorm(width, device=device)
        self.head = torch.nn.Parameter((torch.randn(vocab, width, device=device) / width ** 0.5).bfloat16())

    def loss(self, tokens, target):
        residual = self.embed[tokens]
        x = torch.zeros_like(residual)
        for block in self.blocks:
            x, residual = block(x, residual)
        h, _ = self.norm(x, residual)
        return fp8.linear_cross_entropy(h, self.head, target)


def batch(vocab, tokens, generator, device):
    """Tokens and their successors; the last one's is unknown (ignored)."""
    t = torch.randint(0, vocab, (tokens,), generator=generator, device=device)
    rule = (t * 7 + 3) % vocab
    noise = torch.randint(0, vocab, (tokens,), generator=generator, device=device)
    follow = torch.rand(tokens, generator=generator, device=device) < 0.9
    target = torch.where(follow, rule, noise)
    target[-1] = -100
    return t, target


def train(steps=60, bits=8, vocab=1000, width=256, inner=512, blocks=2, tokens=1024, lr=3e-3, say=print):
    device = torch.device("cuda", 0)
    torch.manual_seed(0)
    generator = torch.Generator(device=device)
    generator.manual_seed(1)
    model = SmallLM(vocab, width, inner, blocks, device)
    opt = fp8.AdamW(model.parameters(), lr=lr, weight_decay=0.01, state_bits=bits)
    losses = []
    for step in range(steps):
        loss = model.loss(*batch(vocab, tokens, generator, device))
        opt.zero_grad()
        loss.backward()
        # gradients clipped to norm 1 by the step itself
        norm = torch.stack([p.grad.float().norm() for p in model.parameters()]).norm()
        opt.step(grad_scale=(1.0 / norm.clamp(min=1.0)).reshape(1))
        losses.append(loss.item())
        if step % 10 == 0 or step == steps - 1:
            say(f"step {step}: loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--bits", type=int, default=8, choices=(8, 32))
    args = parser.parse_args()
    train(args.steps, args.bits)
