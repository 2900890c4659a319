"""A small pre-norm language model trained with the package's layers and its
clipped optimizer step: the layers, the gradient list and AdamW as they are
used together.

    python examples/residual_lm.py [--steps N] [--bf16]

The model predicts the next token of sequences that follow a fixed random
successor table: embeddings, dropout, and blocks of a residual step (add,
dropout, norm) and a two-layer perceptron.  Each optimizer step sums the
gradients of several microbatches, the norms' weight and bias gradients
among them, into the buffers of one GradList, whose global norm is clipped
inside the AdamW step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import global_l2_norm_amd as G  # noqa: E402


class Model:
    """Weights in binary32; activations in `dtype`."""

    def __init__(self, vocabulary=257, width=192, blocks=3, p=0.1, dtype=torch.float32, seed=0):
        g = torch.Generator().manual_seed(seed)
        new = lambda *shape, std: (torch.randn(*shape, generator=g) * std).cuda()  # noqa: E731
        self.embedding = new(vocabulary, width, std=0.02)
        self.norms = [(torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")) for _ in range(blocks + 1)]
        self.mlps = [(new(width, 4 * width, std=width ** -0.5), new(4 * width, width, std=(4 * width * blocks) ** -0.5))
                     for _ in range(blocks)]
        self.params = [self.embedding] + [t for pair in self.norms + self.mlps for t in pair]
        for t in self.params:
            t.requires_grad_()
            t.grad = torch.zeros_like(t)
        self.p, self.dtype, self.seed = p, dtype, seed

    def logits(self, tokens, step=None):
        """step: which dropout masks; None: none (evaluation)."""
        masks = None if step is None else G.DropoutMask(self.p, self.seed, step=step)
        at = lambda site: None if masks is None else masks.at(site=site)  # noqa: E731
        # every sublayer's output joins the stream in the next residual step,
        # the embeddings in the first
        x = self.embedding.to(self.dtype)[tokens.reshape(-1)]
        h = torch.zeros_like(x)
        for i, (up, down) in enumerate(self.mlps):
            h, y = G.residual_norm(x, h, *self.norms[i], mask=at(i))
            x = torch.nn.functional.gelu(y @ up.to(self.dtype)) @ down.to(self.dtype)
        _, y = G.residual_norm(x, h, *self.norms[-1], mask=at(len(self.mlps)))
        return y.float() @ self.embedding.t()


def batch(successor, sequences, length, generator):
    tokens = torch.empty(sequences, length + 1, dtype=torch.int64)
    tokens[:, 0] = torch.randint(0, len(successor), (sequences,), generator=generator)
    for t in range(length):
        tokens[:, t + 1] = successor[tokens[:, t]]
    return tokens.cuda()


def train(steps=60, microbatches=2, dtype=torch.float32, lr=3e-3, max_norm=1.0, seed=0, report=None):
    """The losses and gradient norms of the steps."""
    model = Model(dtype=dtype, seed=seed)
    grads = G.GradList([p.grad for p in model.params])
    weights = [p.detach() for p in model.params]
    opt = G.AdamWList(weights, grads.tensors, [torch.zeros_like(w) for w in weights],
                      [torch.zeros_like(w) for w in weights])
    generator = torch.Generator().manual_seed(seed + 1)
    successor = torch.randperm(model.embedding.shape[0], generator=generator)
    losses, norms = [], []
    for step in range(1, steps + 1):
        total = 0.0
        for p in model.params:
            p.grad.zero_()
        for micro in range(microbatches):
            tokens = batch(successor, 8, 32, generator)
            logits = model.logits(tokens[:, :-1], step * microbatches + micro)
            loss = torch.nn.functional.cross_entropy(logits, tokens[:, 1:].reshape(-1))
            loss.backward()
            total += loss.detach()
        grads.norm(1 / microbatches)
        opt.step(grads, lr=lr, step=step, max_norm=max_norm, avg_factor=1 / microbatches)
        losses.append(float(total) / microbatches)
        norms.append(grads.read()[1]["norm"])
        if report and (step == 1 or step % 10 == 0):
            report(f"step {step:4d}  loss {losses[-1]:.4f}  gradient norm {norms[-1]:.3f}")
    opt.close()
    grads.close()
    return losses, norms


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--bf16", action="store_true", help="activations in bfloat16")
    a = parser.parse_args()
    train(a.steps, dtype=torch.bfloat16 if a.bf16 else torch.float32, report=lambda s: print(s, flush=True))
