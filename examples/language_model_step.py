"""A language model's data-parallel training step on virtual ranks, every part of it through this package.

Each rank holds a replica of a small model that predicts the token after each
of its tokens: rows of a table by token, layer norm, and the same table as the
head.  One step:

1. forward: ``ar_embedding``, ``ar_layer_norm``, ``ar_cross_entropy``, each
   over every rank at once; no logits are stored, and with ``--packed`` the
   layer norm's input is kept in 8 bits (``ar_pack_activations``);
2. backward: ``ar_cross_entropy_backward`` writes the table's gradient as the
   head into each rank's flat gradient bucket, ``ar_layer_norm_backward`` (or
   ``ar_layer_norm_backward_packed``) its weights', and
   ``ar_embedding_backward`` adds the table's gradient as the embedding;
3. ``ar_reduce_scatter`` averages the buckets, ``ar_grad_norm`` and
   ``ar_adamw`` update each rank's chunk of the parameters, ``ar_all_gather``
   gives every rank all of them.

Usage: ``python examples/language_model_step.py [--ranks 4] [--steps 200] [--packed]``
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ring_allreduce_reduction_virtual_amd as ar  # noqa: E402

IGNORE = -100


class Replicas:
    """The ranks' parameters and gradients in flat buckets, and the sharded optimizer."""

    def __init__(self, ranks, vocab, width, packed=False, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ranks, self.vocab, self.width, self.packed = ranks, vocab, width, packed
        self.scale = math.sqrt(width)
        self.count = vocab * width + 2 * width                  # table, gamma, beta
        first = torch.cat([torch.randn(vocab * width, device="cuda", generator=gen) / self.scale,
                           torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")])
        self.params = [first.clone() for _ in range(ranks)]
        self.grads = [torch.empty(self.count, device="cuda") for _ in range(ranks)]
        spans = [ar.ar_chunk_range(r, self.count, ranks) for r in range(ranks)]
        self.shards = [first[b:e].clone() for b, e in spans]
        self.grad_shards = [torch.empty(e - b, device="cuda") for b, e in spans]
        self.states = [[torch.zeros(e - b, device="cuda") for b, e in spans] for _ in range(2)]
        self.update = ar.ar_adamw_init(self.shards, self.grad_shards, *self.states)
        self.norm = ar.ar_grad_norm_init(self.grad_shards)
        self.steps = 0

    def parts(self, flat):
        """(table, gamma, beta) of a flat buffer."""
        t, d = self.vocab * self.width, self.width
        return flat[:t].view(self.vocab, d), flat[t:t + d], flat[t + d:]

    def gradients(self, tokens, targets):
        """Every rank's gradients into its bucket, of the mean loss over its tokens; returns the losses per token."""
        tables, gammas, betas = zip(*(self.parts(p) for p in self.params))
        dtables, dgammas, dbetas = zip(*(self.parts(g) for g in self.grads))
        hs = ar.ar_embedding(tokens, tables, scale=self.scale)
        ys, means, rstds = ar.ar_layer_norm(hs, gammas, betas)
        if self.packed:
            kept = ar.ar_pack_activations(hs)
            backward = ar.ar_layer_norm_backward_packed
        else:
            kept, backward = hs, ar.ar_layer_norm_backward
        del hs
        losses, lses = ar.ar_cross_entropy(ys, tables, targets, ignore_index=IGNORE)
        dys, _ = ar.ar_cross_entropy_backward(None, ys, tables, targets, lses, dxs=ys, dweights=dtables,
                                              ignore_index=IGNORE, scale=1 / targets[0].numel())
        dhs, _, _ = backward(dys, kept, gammas, means, rstds, dxs=dys, dgammas=dgammas, dbetas=dbetas)
        ar.ar_embedding_backward(dhs, tokens, dtables=dtables, scale=self.scale, accumulate=True)
        return losses

    def step(self, tokens, targets, lr, weight_decay=0.01, max_norm=1.0):
        """One step on every rank's tokens; returns each rank's losses."""
        losses = self.gradients(tokens, targets)
        ar.ar_reduce_scatter(self.grads, self.grad_shards, op="avg")
        self.steps += 1
        self.update.start(step=self.steps, lr=lr, weight_decay=weight_decay, grad_norm=self.norm.start(),
                          max_norm=max_norm, skip_nonfinite=True)
        ar.ar_all_gather(self.shards, self.params)
        return losses


def batches(ranks, rows, vocab, seed=1):
    """Tokens of every rank and what follows each, batch after batch: a fixed successor nine times in ten, and no
    target for the last token of every 32."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    follows = torch.randperm(vocab, device="cuda", generator=gen)
    while True:
        tokens = [torch.randint(0, vocab, (rows,), device="cuda", generator=gen) for _ in range(ranks)]
        targets = []
        for t in tokens:
            noise = torch.rand(rows, device="cuda", generator=gen) < 0.1
            target = torch.where(noise, torch.randint(0, vocab, (rows,), device="cuda", generator=gen), follows[t])
            target[31::32] = IGNORE
            targets.append(target)
        yield tokens, targets


def train(ranks=4, steps=200, rows=512, vocab=1000, width=128, packed=False, lr=2e-2):
    """Train; returns the model and the mean loss of every step."""
    model = Replicas(ranks, vocab, width, packed)
    losses = []
    for k, (tokens, targets) in zip(range(steps), batches(ranks, rows, vocab)):
        losses.append(torch.stack(model.step(tokens, targets, lr * (1 - k / steps))).mean())
    return model, torch.stack(losses).tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--packed", action="store_true", help="the layer norm's input kept in 8 bits")
    a = p.parse_args()
    model, losses = train(a.ranks, a.steps, packed=a.packed)
    for k in sorted({0, a.steps // 4, a.steps // 2, a.steps - 1}):
        print(f"step {k + 1}: loss {losses[k]:.4f}")
    same = all(torch.equal(model.params[0], p) for p in model.params)
    print(f"{a.ranks} ranks hold {'the same' if same else 'DIFFERENT'} parameters")


if __name__ == "__main__":
    main()
