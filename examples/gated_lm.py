"""A small language model with RMS norms and gated perceptrons, trained on log
probabilities, whose blocks keep 8 bits of what their gradients need.

    python examples/gated_lm.py [--steps N] [--bf16] [--checkpoint] [--entropy W]

As examples/residual_lm.py, the model predicts the next token of sequences that
follow a fixed random successor table, and the gradients of the microbatches
are added up in the buffers of one GradList, whose global norm is clipped
inside the AdamW step.  The loss is the mean negative log probability of the
tokens that count (the first of each sequence does not), less W times their
mean entropy.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import global_l2_norm_amd as G  # noqa: E402

IGNORED = -100


class Model:
    """Weights in binary32; activations in `dtype`.  checkpoint: what the norms
    and the activations keep for their gradients is in 8 bits."""

    def __init__(self, vocabulary=257, width=192, inner=512, blocks=3, p=0.1, dtype=torch.float32, checkpoint=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        new = lambda *shape, std: (torch.randn(*shape, generator=g) * std).cuda()  # noqa: E731
        self.embedding = new(vocabulary, width, std=0.02)
        self.norms = [torch.ones(width, device="cuda") for _ in range(blocks + 1)]
        self.mlps = [(new(width, 2 * inner, std=width ** -0.5), new(inner, width, std=(inner * blocks) ** -0.5))
                     for _ in range(blocks)]
        self.params = [self.embedding] + self.norms + [t for pair in self.mlps for t in pair]
        for t in self.params:
            t.requires_grad_()
            t.grad = torch.zeros_like(t)
        self.inner, self.p, self.dtype, self.checkpoint, self.seed = inner, p, dtype, checkpoint, seed

    def logits(self, tokens, step=None):
        """step: which dropout masks; None: none (evaluation)."""
        masks = None if step is None else G.DropoutMask(self.p, self.seed, step=step)
        at = lambda site: None if masks is None else masks.at(site=site)  # noqa: E731
        x = self.embedding.to(self.dtype)[tokens.reshape(-1)]
        h = torch.zeros_like(x)
        for i, (into, down) in enumerate(self.mlps):
            h, y = G.residual_rms_norm(x, h, self.norms[i], mask=at(i), checkpoint=self.checkpoint)
            both = y @ into.to(self.dtype)
            z = G.activation(both[:, :self.inner], both[:, self.inner:], "silu", checkpoint=self.checkpoint)
            x = z @ down.to(self.dtype)
        _, y = G.residual_rms_norm(x, h, self.norms[-1], mask=at(len(self.mlps)), checkpoint=self.checkpoint)
        return y.float() @ self.embedding.t()

    def loss(self, tokens, targets, step=None, entropy=0.0):
        r = G.token_log_probs(self.logits(tokens, step), targets.reshape(-1), entropy=entropy != 0.0, ignore_index=IGNORED)
        count = (targets != IGNORED).sum()
        total = -r.logp.sum()  # rows that do not count are 0
        if entropy:
            total = total - entropy * r.entropy.sum()
        return total / count


def batch(successor, sequences, length, generator):
    """Tokens, and the targets that follow them."""
    tokens = torch.empty(sequences, length + 1, dtype=torch.int64)
    tokens[:, 0] = torch.randint(0, len(successor), (sequences,), generator=generator)
    for t in range(length):
        tokens[:, t + 1] = successor[tokens[:, t]]
    targets = tokens[:, 1:].clone()
    targets[:, 0] = IGNORED
    return tokens[:, :-1].cuda(), targets.cuda()


def train(steps=60, microbatches=2, dtype=torch.float32, checkpoint=False, entropy=0.0, lr=3e-3, max_norm=1.0, seed=0, report=None):
    """The losses and gradient norms of the steps."""
    model = Model(dtype=dtype, checkpoint=checkpoint, seed=seed)
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
            tokens, targets = batch(successor, 8, 32, generator)
            loss = model.loss(tokens, targets, step * microbatches + micro, entropy)
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
    parser.add_argument("--checkpoint", action="store_true", help="keep 8 bits for the gradients")
    parser.add_argument("--entropy", type=float, default=0.0, help="weight of the mean entropy")
    a = parser.parse_args()
    train(a.steps, dtype=torch.bfloat16 if a.bf16 else torch.float32, checkpoint=a.checkpoint, entropy=a.entropy,
          report=lambda s: print(s, flush=True))
