"""The example training step: layer norm, its gradient, the reduction, the
norm and AdamW together, against the same model in float64 with torch's own
autograd, and to a small loss."""

import os
import sys

import pytest

from gpu_util import ROOT, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    require_gpu()
    path = os.path.join(ROOT, "examples")
    if path not in sys.path:
        sys.path.insert(0, path)
    import data_parallel_step

    return data_parallel_step


@pytest.mark.parametrize("ranks", [1, 3, 8])
def test_steps_follow_autograd_in_float64(example, ranks):
    """Six steps: every rank's replica is the same, and the mean loss follows the float64 model.

    The losses are means over thousands of terms of float32 products (1e-6
    relative); the parameters differ from the float64 ones by a few 1e-6 of an
    update (float32 moments) where the gradient is well away from 0, and by at
    most an update where it is not, on a few elements.  1e-3 relative covers
    six steps of both.
    """
    import torch

    rows, width, out, lr, steps = 64, 50, 20, 1e-2, 6
    model = example.Replicas(ranks, width, out)
    p = model.params[0].double().clone().requires_grad_(True)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    for t, (xs, targets) in zip(range(1, steps + 1), example.batches(ranks, rows, width, out)):
        got = torch.stack(model.step(xs, targets, lr)).mean().item()
        w, gamma, beta = model.parts(p)
        losses = [((torch.nn.functional.layer_norm(x.double(), (width,), gamma, beta) @ w - y.double()) ** 2).mean()
                  for x, y in zip(xs, targets)]
        want = torch.stack(losses).mean()
        assert abs(got / want.item() - 1) < 1e-3, t
        (g,) = torch.autograd.grad(want, p)
        with torch.no_grad():
            norm = g.norm()
            assert abs(model.norm.norm.item() / norm.item() - 1) < 1e-3
            g = g * min(1.0, 1.0 / (norm.item() + 1e-6))
            m = 0.9 * m + 0.1 * g
            v = 0.999 * v + 0.001 * g * g
            p -= lr * 0.01 * p + lr * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
        assert all(torch.equal(model.params[0], q) for q in model.params)
        assert torch.equal(torch.cat(model.shards), model.params[0])


@pytest.mark.parametrize("packed", [False, True])
def test_training_reaches_the_teacher(example, packed):
    import torch

    model, losses = example.train(ranks=4, steps=300, packed=packed)
    assert losses[-1] < 0.02 * losses[0]
    assert all(torch.equal(model.params[0], q) for q in model.params)
