"""A small next-token model trained with the loss operators and the sharded step.

Four logical workers share one GPU. Two learn from hard targets (linear_xent, with
the first tokens of every row masked, as a prompt would be), two from a teacher's
top-K logits (linear_distill). Each worker's head gradient is written by the loss
straight into its flat gradient buffer; dhidden seeds the backward pass of the rest
of the model. One ZeroOptimizer step then averages the workers and updates.

    python examples/train_lm_head.py [--steps 60] [--precision bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from zero_sharded_optimizer_amd import losses  # noqa: E402
from zero_sharded_optimizer_amd.optimizer import ZeroOptimizer  # noqa: E402

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


class Body(torch.nn.Module):
    """What comes before the head: token embeddings, the token before, one hidden layer."""

    def __init__(self, vocab, dim):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, dim)
        self.mix = torch.nn.Linear(2 * dim, dim)
        self.out = torch.nn.Linear(dim, dim)

    def forward(self, tokens):
        x = self.embed(tokens)
        x = torch.cat([x, torch.roll(x, 1, dims=1)], dim=-1)
        return self.out(torch.nn.functional.gelu(self.mix(x)))


def train(steps=60, precision="bf16", vocab=2003, dim=128, length=64, batch=8, k=16, seed=0):
    """Runs the steps; returns the two losses, per live token, of the first and last."""
    gen = torch.Generator().manual_seed(seed)
    torch.manual_seed(seed)
    dtype = DTYPES[precision]
    body = Body(vocab, dim).to("cuda", dtype)
    head = torch.nn.Parameter((torch.randn(vocab, dim, generator=gen) / dim ** 0.5)
                              .to("cuda", dtype))
    params = list(body.parameters()) + [head]
    zo = ZeroOptimizer(params, n_workers=4, stage=2, precision=precision, lr=3e-3,
                       betas=(0.9, 0.99), weight_decay=0.01,
                       decay=[p.dim() >= 2 for p in params])
    scale = 1024.0 if precision == "fp16" else 1.0  # keeps fp16 gradients off their subnormals
    rule = torch.randperm(vocab, generator=gen)     # the language: each token has one successor
    history = []
    for _ in range(steps):
        zo.zero_grad()
        seen = {"xent": [], "distill": []}
        for w in range(4):
            text = torch.randint(0, vocab, (batch, length), generator=gen)
            target = rule[text]
            hidden = body(text.cuda())
            h = hidden.detach().reshape(-1, dim)
            grads = zo.worker_grads(w)
            if w % 2 == 0:
                target[:, :8] = -100                # the prompt is not learned from
                y = target.reshape(-1).cuda()
                live = int((target != -100).sum())
                loss, saved = losses.linear_xent(h, head.detach(), y, z_loss=1e-4)
                dh, _ = losses.linear_xent_grad(h, head.detach(), y, saved, scale / live,
                                                z_loss=1e-4, dweight=grads[-1])
            else:
                # a teacher that is sure of the successor and spreads the rest
                index = torch.randint(0, vocab, (batch * length, k), generator=gen)
                index[:, 0] = target.reshape(-1)
                logit = -torch.sort(torch.rand(batch * length, k, generator=gen) * 4, dim=1)[0]
                logit[:, 0] += 4.0
                index, logit, live = index.cuda(), logit.cuda(), batch * length
                loss, saved = losses.linear_distill(h, head.detach(), index, logit,
                                                    temperature=2.0)
                dh, _ = losses.linear_distill_grad(h, head.detach(), index, logit, saved,
                                                   scale / live, temperature=2.0,
                                                   dweight=grads[-1])
            seen["xent" if w % 2 == 0 else "distill"].append(float(loss.sum()) / live)
            body.zero_grad()
            hidden.backward(dh.view_as(hidden))
            for dst, p in zip(grads, body.parameters()):
                dst.copy_(p.grad)
            if scale != 1.0:
                zo.grads[w].mul_(1.0 / scale)
        zo.step(max_norm=1.0)
        history.append({name: sum(v) / len(v) for name, v in seen.items()})
    return history[0], history[-1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--precision", choices=sorted(DTYPES), default="bf16")
    a = ap.parse_args()
    first, last = train(a.steps, a.precision)
    for name in first:
        print(f"{name}: {first[name]:.3f} -> {last[name]:.3f} per token in {a.steps} steps")


if __name__ == "__main__":
    main()
