"""A data-parallel training step on virtual ranks, every part of it through this package.

Each rank holds a replica of a small model, layer norm followed by a linear
map, and its own tokens.  One step:

1. forward: ``ar_layer_norm`` of every rank's tokens in one launch, then the
   linear map;
2. backward: ``ar_layer_norm_backward`` writes each rank's part of the layer
   norm's weight gradient into that rank's flat gradient bucket, beside the
   linear map's;
3. ``ar_reduce_scatter`` averages the buckets: each rank owns one chunk of the
   gradient;
4. ``ar_grad_norm`` takes the norm over all chunks, which AdamW reads on the
   device to clip by: the host waits for nothing;
5. ``ar_adamw`` updates each rank's chunk of the parameters, its states in
   float32 or (``--packed``) in 8 bits; the optimizer's memory is split over
   the ranks;
6. ``ar_all_gather`` gives every rank all the new parameters.

Usage: ``python examples/data_parallel_step.py [--ranks 4] [--steps 200] [--packed]``
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ring_allreduce_reduction_virtual_amd as ar  # noqa: E402


class Replicas:
    """The ranks' parameters and gradients in flat buckets, and the sharded optimizer."""

    def __init__(self, ranks, width, out, packed=False, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ranks, self.width, self.out, self.packed = ranks, width, out, packed
        self.count = width * out + 2 * width                    # linear map, gamma, beta
        first = torch.cat([torch.randn(width * out, device="cuda", generator=gen) / width ** 0.5,
                           torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")])
        self.params = [first.clone() for _ in range(ranks)]
        self.grads = [torch.empty(self.count, device="cuda") for _ in range(ranks)]
        spans = [ar.ar_chunk_range(r, self.count, ranks) for r in range(ranks)]
        self.shards = [first[b:e].clone() for b, e in spans]
        self.grad_shards = [torch.empty(e - b, device="cuda") for b, e in spans]
        if packed:
            self.states = [[ar.PackedState.zeros(e - b, "cuda") for b, e in spans] for _ in range(2)]
            self.update = ar.ar_adamw_packed_init(self.shards, self.grad_shards, *self.states)
        else:
            self.states = [[torch.zeros(e - b, device="cuda") for b, e in spans] for _ in range(2)]
            self.update = ar.ar_adamw_init(self.shards, self.grad_shards, *self.states)
        self.norm = ar.ar_grad_norm_init(self.grad_shards)
        self.steps = 0

    def parts(self, flat):
        """(linear map, gamma, beta) of a flat buffer."""
        w, d = self.width * self.out, self.width
        return flat[:w].view(self.width, self.out), flat[w:w + d], flat[w + d:]

    def step(self, xs, targets, lr, weight_decay=0.01, max_norm=1.0):
        """One step on every rank's tokens; returns each rank's loss tensor."""
        weights, gammas, betas = zip(*(self.parts(p) for p in self.params))
        dweights, dgammas, dbetas = zip(*(self.parts(g) for g in self.grads))
        ys, means, rstds = ar.ar_layer_norm(xs, gammas, betas)
        losses, dys = [], []
        for y, w, dw, t in zip(ys, weights, dweights, targets):
            off = y @ w - t
            losses.append(off.square().mean())
            off.mul_(2 / off.numel())
            torch.mm(y.t(), off, out=dw)
            dys.append(off @ w.t())
        ar.ar_layer_norm_backward(dys, xs, gammas, means, rstds, dxs=dys, dgammas=dgammas, dbetas=dbetas)
        ar.ar_reduce_scatter(self.grads, self.grad_shards, op="avg")
        self.steps += 1
        config = {"seed": self.steps} if self.packed else {}
        self.update.start(step=self.steps, lr=lr, weight_decay=weight_decay, grad_norm=self.norm.start(),
                          max_norm=max_norm, skip_nonfinite=True, **config)
        ar.ar_all_gather(self.shards, self.params)
        return losses


def batches(ranks, rows, width, out, seed=1):
    """Tokens of every rank and a fixed teacher's answers to them, batch after batch."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher = torch.randn(width, out, device="cuda", generator=gen) / width ** 0.5
    scale = 1 + 0.5 * torch.randn(width, device="cuda", generator=gen)
    while True:
        xs = [3 * torch.randn(rows, width, device="cuda", generator=gen) + 1 for _ in range(ranks)]
        yield xs, [torch.nn.functional.layer_norm(x, (width,)) * scale @ teacher for x in xs]


def train(ranks=4, steps=200, rows=256, width=192, out=64, packed=False, lr=2e-2):
    """Train; returns the model and the mean loss of every step."""
    model = Replicas(ranks, width, out, packed)
    losses = []
    for k, (xs, targets) in zip(range(steps), batches(ranks, rows, width, out)):
        losses.append(torch.stack(model.step(xs, targets, lr * (1 - k / steps))).mean())
    return model, torch.stack(losses).tolist()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--packed", action="store_true", help="optimizer states in 8 bits")
    a = p.parse_args()
    model, losses = train(a.ranks, a.steps, packed=a.packed)
    for k in sorted({0, a.steps // 4, a.steps // 2, a.steps - 1}):
        print(f"step {k + 1}: loss {losses[k]:.6f}")
    same = all(torch.equal(model.params[0], p) for p in model.params)
    print(f"{a.ranks} ranks hold {'the same' if same else 'DIFFERENT'} parameters")


if __name__ == "__main__":
    main()
