"""The model's ends together, as a training step uses them: the example step's
gradients against float64, the whole chain in 16 bits and inside a graph, and
tensors whose offsets pass 32 bits."""

import math
import os
import sys

import pytest

from gpu_util import ROOT, require_gpu
from step_util import UNIT, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ar():
    require_gpu()
    import ring_allreduce_reduction_virtual_amd as ar

    return ar


@pytest.fixture(scope="module")
def example():
    require_gpu()
    path = os.path.join(ROOT, "examples")
    if path not in sys.path:
        sys.path.insert(0, path)
    import language_model_step

    return language_model_step


def reference(model, params, tokens, targets, ignore, packed_h=None):
    """(losses, flat gradient) of one rank in float64; `packed_h`: what layer norm's backward pass has for its input."""
    import torch

    table, gamma, beta = (p.double() for p in model.parts(params))
    h = table[tokens] * model.scale
    mean = h.mean(1, keepdim=True)
    rstd = ((h - mean) ** 2).mean(1, keepdim=True).add(1e-5).rsqrt()
    hat = (h - mean) * rstd
    y = hat * gamma + beta
    z = y @ table.t()
    lse = z.logsumexp(1)
    kept = targets != ignore
    losses = torch.where(kept, lse - z.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
    dz = torch.exp(z - lse[:, None])
    dz[kept, targets[kept]] -= 1
    dz *= kept[:, None] / tokens.numel()
    dy = dz @ table
    dtable = dz.t() @ y
    if packed_h is not None:
        hat = (packed_h.double() - mean) * rstd
    w = dy * gamma
    dh = rstd * (w - w.mean(1, keepdim=True) - hat * (w * hat).mean(1, keepdim=True))
    dtable.index_add_(0, tokens, dh * model.scale)
    return losses, torch.cat([dtable.reshape(-1), (dy * hat).sum(0), dy.sum(0)])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("ranks,rows,vocab,width", [(1, 64, 50, 20), (3, 200, 333, 66), (4, 512, 1000, 128)])
def test_gradients_follow_float64(example, ar, packed, ranks, rows, vocab, width):
    """Every rank's bucket, after some steps.

    Sums of up to 1,000 float32 terms of order of the result's largest (2^-24
    each: 6e-5), through three layers one after another: 2e-4 of the bucket's
    2-norm, and as much for its three parts one by one.
    """
    import torch

    model = example.Replicas(ranks, vocab, width, packed)
    for k, (tokens, targets) in zip(range(3), example.batches(ranks, rows, vocab)):
        before = [p.clone() for p in model.params]
        losses = model.step(tokens, targets, 1e-2)
        for r in range(ranks):
            h = None
            if packed:
                raw = ar.ar_embedding([tokens[r]], [model.parts(before[r])[0]], scale=model.scale)
                (h,) = ar.ar_unpack_activations(ar.ar_pack_activations(raw))
            want_losses, want = reference(model, before[r], tokens[r], targets[r], example.IGNORE, h)
            assert ((losses[r].double() - want_losses).abs() <= 1e-5 * (1 + want_losses.abs())).all()
            got = model.grads[r].double()
            for a, b in zip((got, *model.parts(got)), (want, *model.parts(want))):
                assert (a - b).norm() <= 2e-4 * b.norm(), (k, r, float((a - b).norm() / b.norm()))
        assert all(torch.equal(model.params[0], p) for p in model.params)
        assert torch.equal(torch.cat(model.shards), model.params[0])


@pytest.mark.parametrize("packed", [False, True])
def test_example_runs(example, packed):
    import torch

    model, losses = example.train(ranks=2, steps=5, rows=64, vocab=100, width=32, packed=packed)
    assert len(losses) == 5 and all(math.isfinite(x) for x in losses)
    assert all(torch.equal(model.params[0], p) for p in model.params)


def chain(ar, tokens, tables, gammas, targets, scale, grads):
    """Forward and backward over all ranks; everything that comes out."""
    hs = ar.ar_embedding(tokens, tables, scale=scale)
    ys, means, rstds = ar.ar_layer_norm(hs, gammas)
    packed = ar.ar_pack_activations(hs)
    losses, lses = ar.ar_cross_entropy(ys, tables, targets)
    dys, _ = ar.ar_cross_entropy_backward(None, ys, tables, targets, lses, dweights=grads, scale=1 / len(tokens[0]))
    dhs, dgammas, _ = ar.ar_layer_norm_backward_packed(dys, packed, gammas, means, rstds)
    ar.ar_embedding_backward(dhs, tokens, dtables=grads, scale=scale, accumulate=True)
    return losses + lses + dys + dhs + dgammas + list(grads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,width", [(48, 700, 96), (600, 3000, 200)])
def test_whole_chain_in_a_graph(ar, dtype, rows, vocab, width):
    """Replayed with new tokens and weights, it gives the eager chain's bits, and float64's within 16-bit roundings."""
    import torch

    dt, n, scale = torch_dtype(dtype), 2, 8.0
    tables = [torch.randn(vocab, width, device="cuda").mul_(0.1).to(dt) for _ in range(n)]
    gammas = [torch.ones(width, device="cuda", dtype=dt) for _ in range(n)]
    tokens = [torch.randint(0, vocab, (rows,), device="cuda") for _ in range(n)]
    targets = [torch.randint(0, vocab, (rows,), device="cuda") for _ in range(n)]
    grads = [torch.zeros(vocab, width, device="cuda", dtype=dt) for _ in range(n)]
    chain(ar, tokens, tables, gammas, targets, scale, grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = chain(ar, tokens, tables, gammas, targets, scale, grads)
    for _ in range(4):
        for t in tokens + targets:
            t.random_(0, vocab)
        for t in tables:
            t.normal_(0, 0.1)
        targets[1][::3] = -100
        graph.replay()
        torch.cuda.synchronize()
        mine = [torch.zeros_like(g) for g in grads]
        want = chain(ar, tokens, tables, gammas, targets, scale, mine)
        assert all(torch.equal(a, b) for a, b in zip(got, want))

    class Model:
        def parts(self, flat):
            t = vocab * width
            return flat[:t].view(vocab, width), flat[t:t + width], flat[t + width:]

    Model.scale = scale
    flat = torch.cat([tables[0].float().reshape(-1), torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")])
    losses, grad = reference(Model(), flat, tokens[0], targets[0], -100)
    # the hidden rows h and y are 16-bit: each logit is off by 2 UNIT of a sum of `width` terms' 2-norm (the roundings
    # are independent: no more than 4 of their root mean squares for all of them); the packed input, dz, dy, dh and the
    # table's gradient (twice) add their own roundings, 8 UNIT in 2-norm, and the 8-bit input half of 1/127 of a block's
    # largest, about 4 of its root mean square, through hat: 2%
    assert (got[0].double() - losses).abs().max() <= 40 * UNIT[dtype]
    dtable = Model().parts(grad)[0]
    away = (grads[0].double() - dtable).norm() / dtable.norm()
    assert away <= 0.02 + 16 * UNIT[dtype], float(away)


def test_offsets_past_32_bits(ar):
    """Tables, weights and activations of more than 2^32 bytes or elements, looked at where they end."""
    import torch

    vocab, width = 270_000, 16_384                              # 4.4e9 elements
    table = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    table[-1], table[-2] = 3.0, -2.0
    tokens = torch.tensor([vocab - 1, 5, vocab - 2, vocab - 1], device="cuda")
    (out,) = ar.ar_embedding([tokens], [table], scale=2.0)
    assert (out[0] == 6).all() and (out[1] == 0).all() and (out[2] == -4).all()
    ar.ar_embedding_backward([out], [tokens], dtables=[table])
    assert (table[-1] == 12).all() and (table[-2] == -4).all() and (table[:-2] == 0).all()
    del table
    rows = 270_000
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(width, device="cuda") % 128             # whole numbers: a block's scale holds them
    (packed,) = ar.ar_pack_activations([x])
    assert (packed.codes[-1, 1:] != 0).sum() == width - width // 128 and (packed.codes[:-1] == 0).all()
    (back,) = ar.ar_unpack_activations([packed], dtype=torch.bfloat16)
    assert torch.equal(back, x)
    del back, packed, x
    torch.cuda.empty_cache()
    vocab, width = 140_000, 16_384                              # a weight and its gradient of 4.6e9 bytes each
    w = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    w[-1, 0] = 10.0
    y = torch.zeros(3, width, dtype=torch.bfloat16, device="cuda")
    y[:, 0] = 1.0
    t = torch.tensor([vocab - 1, 0, -100], device="cuda")
    (loss,), (lse,) = ar.ar_cross_entropy([y], [w], [t])
    want = math.log(math.exp(10) + vocab - 1)
    # the sum of 140,000 ones and e^10 over tiles, and the logarithm: 1e-5 of 12
    assert abs(lse[0].item() - want) < 1e-4 and abs(loss[0].item() - (want - 10)) < 1e-4
    (dx,), (dw,) = ar.ar_cross_entropy_backward(None, [y], [w], [t], [lse])
    p = math.exp(10 - want)
    assert abs(dx[0, 0].item() / (10 * (p - 1)) - 1) < 3 * UNIT["bf16"]
    assert abs(dx[1, 0].item() / (10 * p) - 1) < 3 * UNIT["bf16"] and (dx[2] == 0).all() and (dx[:, 1:] == 0).all()
    assert abs(dw[-1, 0].item() / (2 * p - 1) - 1) < 8 * UNIT["bf16"] and (dw[:, 1:] == 0).all()
    assert abs(dw[1, 0].item() / (2 * math.exp(-want)) - 1) < 3 * UNIT["bf16"]


def test_many_tokens(ar):
    """A million places of a rank: the sort over many workgroups, and tokens of many chunks."""
    import torch

    rows, vocab = (1 << 20) + 5, 3000
    tokens = (torch.rand(rows, device="cuda") ** 3 * vocab).long()
    dy = torch.ones(rows, 5, device="cuda")
    (got,) = ar.ar_embedding_backward([dy], [tokens], vocab)
    want = torch.bincount(tokens, minlength=vocab)               # whole numbers below 2^24: exact in float32
    assert torch.equal(got, want.float()[:, None].expand(-1, 5))
