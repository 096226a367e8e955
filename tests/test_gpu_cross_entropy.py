"""The cross entropy of unstored logits on the GPU against the float64 oracle:
types, every shape's edge (rows, columns, vocabulary around tiles and pieces),
alignments and strides, ignored rows and what they hold, targets outside,
special values, streams, graphs, and the refusals."""

import math

import numpy as np
import pytest

from gpu_util import require_gpu
from oracle import model as oracle
from step_util import TINY, U32, UNIT, f64, rounded, torch_dtype

pytestmark = pytest.mark.gpu

IGNORE = -100
EXP = 4 * U32          # v_exp_f32 and v_log_f32: 1 unit in the last place, 2 U32; doubled


@pytest.fixture(scope="module")
def ar():
    require_gpu()
    import ring_allreduce_reduction_virtual_amd as ar

    return ar


def _torch():
    import torch

    return torch


def rows_of(rng, n, rows, cols, dtype, pad=0, scale=1.0, offset=0):
    """Tensors of rows `pad` elements apart, `offset` elements into their allocation."""
    torch = _torch()
    got = []
    for _ in range(n):
        values = torch.from_numpy((rng.standard_normal((rows, cols + pad)) * scale).astype(np.float32))
        flat = torch.full((rows * (cols + pad) + offset + 8,), math.nan, dtype=torch_dtype(dtype), device="cuda")
        part = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)
        part[:, :cols] = values[:, :cols].to("cuda")       # NaN everywhere else
        got.append(part[:, :cols])
    return got


def targets_of(rng, n, rows, vocab, index="i64", ignored=0.2):
    torch = _torch()
    got = []
    for _ in range(n):
        t = rng.integers(0, vocab, rows)
        t[rng.random(rows) < ignored] = IGNORE
        got.append(torch.tensor(t, dtype=torch.int64 if index == "i64" else torch.int32, device="cuda"))
    return got


def logit_error(x, w):
    """Bound on a float32 logit's error: cols products of exact factors, summed in float32 in some order.

    A sum of k terms in any order is off by at most (k - 1) U32 of the sum of
    magnitudes; float32 products add one rounding each.
    """
    return (x.shape[1] + 1) * U32 * (np.abs(x) @ np.abs(w).T)


def check_forward(ar, xs, weights, targets, **k):
    """lse: the logits' errors (weighted by p, at most their largest), and the exponentials' sum of V terms.

    Each term e^(z - top) has the difference's rounding times its argument
    (|z - top| U32, in base 2 another), the exponential's own, and as many
    additions as there are tiles and registers, below (V / 128 + 300); the
    logarithm's own error and two roundings of the result.
    """
    losses, lses = ar.ar_cross_entropy(xs, weights, targets, ignore_index=IGNORE, **k)
    for x, w, t, loss, lse in zip(xs, weights, targets, losses, lses):
        x, w, t = f64(x), f64(w), t.cpu().numpy()
        want_loss, want_lse = oracle.cross_entropy(x, w, t, IGNORE)
        z = x @ w.T
        off = logit_error(x, w)
        p = np.exp(z - want_lse[:, None])
        spread = np.abs(z - z.max(1, keepdims=True)) + off
        lse_off = ((p * (off + 4 * spread * U32)).sum(1) * 1.01 + EXP
                   + (w.shape[0] / 128 + 300) * U32 + 8 * U32 * (np.abs(want_lse) + np.abs(z).max(1) + 1))
        assert (np.abs(f64(lse) - want_lse) <= lse_off).all(), float((np.abs(f64(lse) - want_lse) / lse_off).max())
        kept = t != IGNORE
        loss_off = lse_off + np.array([off[i, v] if v >= 0 else 0 for i, v in enumerate(t)]) + 2 * U32 * np.abs(want_loss)
        assert (np.abs(f64(loss) - want_loss)[kept] <= loss_off[kept]).all()
        assert (f64(loss)[~kept] == 0).all()
    return losses, lses


def check_backward(ar, xs, weights, targets, lses, dlosses, dtype, scale=1.0, pad=0, offset=0, **k):
    """dz: p's relative error is that of its exponent (the logit's error, lse is given; the difference's roundings)
    and 4 roundings (g relative to the largest is a quotient), then the rounding to the type; dx and dweight: sums of
    at most k terms of float32 products, twice (pieces and splits are added up), the product with the largest g, one
    rounding."""
    torch = _torch()
    n, (rows, cols), vocab = len(xs), xs[0].shape, weights[0].shape[0]
    dxs = rows_of(np.random.default_rng(0), n, rows, cols, dtype, pad, offset=offset)
    dws = rows_of(np.random.default_rng(0), n, vocab, cols, dtype, pad, offset=offset)
    for t in dxs + dws:
        t.fill_(math.nan)
    got = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses, dxs, dws, ignore_index=IGNORE, scale=scale, **k)
    assert got[0] is dxs and got[1] is dws
    for r in range(n):
        x, w, t, lse = f64(xs[r]), f64(weights[r]), targets[r].cpu().numpy(), f64(lses[r])
        g = np.float64(np.float32(scale)) * (np.ones(rows) if dlosses is None else f64(dlosses[r]))
        want_dx, want_dw, dz = oracle.cross_entropy_backward(g, x, w, t, lse, IGNORE)
        live = (t != IGNORE) & (g != 0)
        x = np.where(live[:, None], x, 0)
        z = x @ w.T
        p = np.where(live[:, None], np.exp(z - lse[:, None]), 0)
        arg = np.abs(z - lse[:, None])
        p_off = p * 1.01 * (logit_error(x, w) + 3 * U32 * arg + 2 * U32 + EXP) + 2.0 ** -126
        # binary16's dz has 2^13 for the largest |g|: its subnormals' step relative to that
        floor = np.abs(g[live]).max(initial=0) * 2.0 ** -13 * TINY["f16"] if dtype == "f16" else TINY[dtype]
        dz_off = np.abs(g)[:, None] * (p_off + 3 * U32 * (p + 1)) + 4 * U32 * np.abs(dz)
        dz_off = np.where(live[:, None], dz_off + (0 if dtype == "f32" else UNIT[dtype] * (np.abs(dz) + dz_off) + floor), 0)
        for got, want, left, right, depth in ((dxs[r], want_dx, (np.abs(dz), dz_off), np.abs(w), vocab),
                                              (dws[r], want_dw, (np.abs(dz).T, dz_off.T), np.abs(x), rows)):
            off = left[1] @ right * 1.01 + (2 * (depth + 2) + 2) * U32 * ((left[0] + left[1]) @ right)
            away = np.abs(f64(got) - want)
            bad = away - off - rounded(np.abs(want) + off, dtype)
            assert (bad <= 0).all(), (got.shape, float(bad.max()), np.argwhere(~(bad <= 0))[:5])
        assert (f64(dxs[r])[~live] == 0).all()
    for t in dxs + dws:     # nothing beside the rows
        whole = torch.as_strided(t, (t.shape[0], cols + pad), (cols + pad, 1))
        assert pad == 0 or torch.isnan(whole[:, cols:]).all()
    return dxs, dws


def check(ar, rng, n, rows, cols, vocab, dtype, pad=0, offset=0, index="i64", ignored=0.2):
    xs = rows_of(rng, n, rows, cols, dtype, pad, 1.0, offset)
    weights = rows_of(rng, n, vocab, cols, dtype, pad, 1.5 / math.sqrt(max(cols, 1)), offset)
    targets = targets_of(rng, n, rows, vocab, index, ignored)
    _, lses = check_forward(ar, xs, weights, targets)
    dlosses = [t[:, 0].contiguous().abs() / rows for t in rows_of(rng, n, rows, 1, "f32")]
    check_backward(ar, xs, weights, targets, lses, dlosses, dtype, 1.5, pad, offset)
    return xs, weights, targets, lses, dlosses


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1, 2, 3, 7, 8, 9, 31, 32, 33, 63, 64, 65, 72, 127, 128, 129, 200, 257, 515])
def test_widths_and_types(ar, dtype, cols):
    """Columns around a step of the product and a chunk of 16 bytes, few rows."""
    check(ar, np.random.default_rng(cols), 2, 21, cols, 300, dtype, index="i32" if cols % 2 else "i64")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 520])
def test_row_counts(ar, dtype, rows):
    check(ar, np.random.default_rng(rows), 1, rows, 40, 270, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 5, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 5003])
@pytest.mark.parametrize("rows", [6, 140])
def test_vocabularies(ar, dtype, vocab, rows):
    check(ar, np.random.default_rng(vocab), 2, rows, 24, vocab, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,vocab", [(1, 4100, 700), (70, 1030, 600), (300, 1000, 800), (260, 264, 2500)])
def test_long_sums(ar, dtype, rows, cols, vocab):
    check(ar, np.random.default_rng(cols), 1, rows, cols, vocab, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (8, 0), (0, 8), (8, 3)])
@pytest.mark.parametrize("rows,cols", [(37, 64), (200, 40), (37, 61)])
def test_strides_and_alignments(ar, dtype, rows, cols, pad, offset):
    """Rows and starts off 16 bytes; NaN beside the rows reaches nothing."""
    check(ar, np.random.default_rng(pad + offset), 2, rows, cols, 333, dtype, pad, offset)


@pytest.mark.parametrize("rows,cols,vocab", [(50, 61, 40000), (64, 515, 9000), (32, 1003, 3000), (1, 2047, 500)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (2, 1)])
def test_few_float32_rows_anywhere(ar, rows, cols, vocab, pad, offset):
    """Few rows of float32 are read where they lie, in every tile that they get."""
    check(ar, np.random.default_rng(rows), 2, rows, cols, vocab, "f32", pad, offset)


@pytest.mark.parametrize("dtype,stride", [("f32", (1 << 21) + 1), ("f32", (1 << 21) + 4), ("bf16", (1 << 22) + 8)])
@pytest.mark.parametrize("rows", [5, 40, 70])
def test_rows_far_apart(ar, dtype, stride, rows):
    """Rows of the weight too far apart for 32-bit offsets: the same bits as from rows without gaps."""
    torch = _torch()
    rng = np.random.default_rng(rows)
    xs, weights = rows_of(rng, 1, rows, 64, dtype), rows_of(rng, 1, 70, 64, dtype)
    targets = targets_of(rng, 1, rows, 70)
    room = torch.full((69 * stride + 64,), math.nan, dtype=weights[0].dtype, device="cuda")
    far = [torch.as_strided(room, (70, 64), (stride, 1)).copy_(weights[0])]
    losses, lses = ar.ar_cross_entropy(xs, weights, targets)
    far_losses, far_lses = ar.ar_cross_entropy(xs, far, targets)
    assert torch.equal(losses[0], far_losses[0]) and torch.equal(lses[0], far_lses[0])
    dxs, dws = ar.ar_cross_entropy_backward(None, xs, weights, targets, lses)
    far_dxs, far_dws = ar.ar_cross_entropy_backward(None, xs, far, targets, lses)
    assert torch.equal(dxs[0], far_dxs[0]) and torch.equal(dws[0], far_dws[0])


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 8200, 33000), ("f32", 4100, 18000), ("bf16", 20, 140000)])
@pytest.mark.parametrize("offset", [0, 1])
def test_pieces_of_the_vocabulary(ar, dtype, rows, vocab, offset):
    """Several pieces, the last one short; the oracle on the GPU in float64.

    Columns are few, so that p's error is small against the type's rounding:
    the bounds are the whole results' 2-norms, relative: dz's rounding and the
    result's (each at most a unit UNIT of each term) for 16 bits, and for float32
    (a sum's terms up to `vocab`, its partial sums as large as the result at
    most) vocab U32.
    """
    torch = _torch()
    rng = np.random.default_rng(vocab)
    cols = 16
    (x,), (w,) = rows_of(rng, 1, rows, cols, dtype, 0, 1.0, offset), rows_of(rng, 1, vocab, cols, dtype, 0, 0.4, offset)
    (t,) = targets_of(rng, 1, rows, vocab)
    (loss,), (lse,) = ar.ar_cross_entropy([x], [w], [t])
    z = x.double() @ w.double().t()
    want = z.logsumexp(1)
    assert ((lse - want).abs() <= 1e-5 * (1 + want.abs())).all()
    kept = t != IGNORE
    at = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    assert ((loss - (want - at)).abs() <= 2e-5 * (1 + want.abs()))[kept].all() and (loss[~kept] == 0).all()
    g = torch.rand(rows, device="cuda") / rows
    (dx,), (dw,) = ar.ar_cross_entropy_backward([g], [x], [w], [t], [lse])
    dz = torch.exp(z.sub_(lse.double()[:, None]))
    dz[kept, t[kept]] -= 1
    dz *= (g.double() * kept)[:, None]
    for got, want in ((dx, dz @ w.double()), (dw, dz.t() @ x.double())):
        bound = 2 * UNIT[dtype] if dtype != "f32" else 1e-5
        assert torch.isfinite(got).all()
        assert (got.double() - want).norm() <= bound * want.norm(), float((got.double() - want).norm() / want.norm())
        # row by row as well, where a row is not all cancellation
        big = want.norm(dim=1) > 1e-3 * want.norm(dim=1).max()
        away = (got.double() - want).norm(dim=1) / want.norm(dim=1)
        assert (away[big] <= 4 * bound).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [40, 300])
def test_ignored_rows_reach_nothing(ar, dtype, rows):
    """NaN and infinities in ignored rows of x, in their lse and dloss; all rows ignored; weights of 0."""
    torch = _torch()
    rng = np.random.default_rng(9)
    xs, weights, targets, lses, dlosses = check(ar, rng, 1, rows, 48, 300, dtype, ignored=0.5)
    want = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses)
    dull = targets[0] == IGNORE
    xs[0][dull], lses[0][dull], dlosses[0][dull] = math.nan, math.inf, math.nan
    losses, _ = ar.ar_cross_entropy(xs, weights, targets)
    assert (losses[0][dull] == 0).all() and torch.isfinite(losses[0][~dull]).all()
    got = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    # the same rows left out by a weight of 0
    dlosses[0][dull] = 0.0
    some = [torch.where(dull, 3, targets[0])]
    got = ar.ar_cross_entropy_backward(dlosses, xs, weights, some, lses)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    nobody = [torch.full_like(targets[0], IGNORE)]
    (dx,), (dw,) = ar.ar_cross_entropy_backward(None, xs, weights, nobody, lses)
    assert (dx == 0).all() and (dw == 0).all()
    (loss,), _ = ar.ar_cross_entropy(xs, weights, nobody)
    assert (loss == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_targets_outside(ar, dtype):
    """Loss and row NaN, and dweight with it; another ignore_index, inside the vocabulary too."""
    torch = _torch()
    rng = np.random.default_rng(10)
    xs, weights = rows_of(rng, 1, 20, 16, dtype), rows_of(rng, 1, 90, 16, dtype)
    t = torch.arange(20, device="cuda")
    t[3], t[5], t[7] = 90, -1, 1 << 40
    (loss,), (lse,) = ar.ar_cross_entropy(xs, weights, [t])
    bad = torch.tensor([i in (3, 5, 7) for i in range(20)], device="cuda")
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all() and torch.isfinite(lse).all()
    (dx,), (dw,) = ar.ar_cross_entropy_backward(None, xs, weights, [t], [lse])
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[~bad]).all() and torch.isnan(dw).all()
    t[3], t[5], t[7] = 11, 11, 11
    (loss,), (lse,) = ar.ar_cross_entropy(xs, weights, [t], ignore_index=11)
    dull = t == 11
    assert (loss[dull] == 0).all() and (loss[~dull] > 0).all()
    (dx,), _ = ar.ar_cross_entropy_backward(None, xs, weights, [t], [lse], ignore_index=11)
    assert (dx[dull] == 0).all() and (dx[~dull] != 0).any(1).all()


@pytest.mark.parametrize("rows", [9, 140])
def test_special_values(ar, rows):
    """A NaN or infinite row of x spoils its own loss; equal logits, a logit far above the others, none of -inf."""
    torch = _torch()
    torch.manual_seed(0)
    x, w = torch.randn(rows, 32, device="cuda"), torch.randn(400, 32, device="cuda")
    x[1, 3], x[2, 3] = math.nan, math.inf
    x[4] = 0.0
    x[5] = 1e3 * w[7]
    t = torch.full((rows,), 7, device="cuda")
    (loss,), (lse,) = ar.ar_cross_entropy([x], [w], [t])
    assert torch.isnan(loss[1]) and not torch.isfinite(loss[2]) and torch.isfinite(loss[[0, 3, 4, 5, 6]]).all()
    # log 400, and e^-something tiny: the sum's and the logarithm's roundings
    assert abs(loss[4].item() - math.log(400)) < 1e-5
    assert abs(loss[5].item()) <= 1e-6 * abs(lse[5].item())
    low = torch.full((400, 32), 0.0, device="cuda")
    low[:, 0] = -math.inf
    low[13] = 1.0
    ones = torch.ones(rows, 32, device="cuda")
    (loss,), (lse,) = ar.ar_cross_entropy([ones], [low], [torch.full((rows,), 13, device="cuda")])
    assert (loss == 0).all() and (lse == 32).all()


def test_small_gradients_in_binary16(ar):
    """g of 1e-7, which binary16 would take for 0 or a subnormal: as exact as for g of 1, scaled."""
    torch = _torch()
    rng = np.random.default_rng(11)
    xs, weights = rows_of(rng, 1, 150, 64, "f16"), rows_of(rng, 1, 3000, 64, "f16", 0, 0.1)
    targets = targets_of(rng, 1, 150, 3000)
    _, lses = ar.ar_cross_entropy(xs, weights, targets)
    one = ar.ar_cross_entropy_backward(None, xs, weights, targets, lses)
    small = ar.ar_cross_entropy_backward(None, xs, weights, targets, lses, scale=2.0 ** -6)
    # a power of two changes nothing but the results' own exponents (and what becomes subnormal by it)
    for a, b in ((one[0][0], small[0][0]), (one[1][0], small[1][0])):
        assert ((a.float() * 2.0 ** -6 - b.float()).abs() <= TINY["f16"] * 1.01).all()
    tiny = [torch.full((150,), 1e-7, device="cuda")]
    dx, dw = ar.ar_cross_entropy_backward(tiny, xs, weights, targets, lses)
    assert (dx[0] != 0).any()


def test_one_gradient_alone_and_in_place(ar):
    torch = _torch()
    rng = np.random.default_rng(12)
    xs, weights, targets, lses, dlosses = check(ar, rng, 2, 150, 72, 500, "bf16")
    dxs, dws = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses)
    a, none = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses, weight_grads=False)
    assert none is None and all(torch.equal(p, q) for p, q in zip(a, dxs))
    none, b = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses, input_grads=False)
    assert none is None and all(torch.equal(p, q) for p, q in zip(b, dws))
    c, d = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses, dxs=xs)
    assert c is xs and all(torch.equal(p, q) for p, q in zip(xs + d, dxs + dws))


def test_ranks(ar):
    """One weight for all ranks, more ranks than one launch takes, each rank's results its own."""
    torch = _torch()
    rng = np.random.default_rng(13)
    n = 35
    xs, (w,) = rows_of(rng, n, 33, 24, "bf16"), rows_of(rng, 1, 200, 24, "bf16")
    targets = targets_of(rng, n, 33, 200)
    losses, lses = check_forward(ar, xs, [w] * n, targets)
    dxs, dws = ar.ar_cross_entropy_backward(None, xs, [w] * n, targets, lses)
    for r in (0, 31, 32, 34):
        (loss,), (lse,) = ar.ar_cross_entropy(xs[r:r + 1], [w], targets[r:r + 1])
        assert torch.equal(loss, losses[r]) and torch.equal(lse, lses[r])
        (dx,), (dw,) = ar.ar_cross_entropy_backward(None, xs[r:r + 1], [w], targets[r:r + 1], [lse])
        # one rank alone may be split another way: each within float32 sums' roundings and a rounding to bf16
        for a, b in ((dx, dxs[r]), (dw, dws[r])):
            assert (a.double() - b.double()).norm() <= 2 * UNIT["bf16"] * a.double().norm()


def test_no_rows_and_no_columns(ar):
    torch = _torch()
    e = lambda *s: [torch.empty(*s, device="cuda")]              # noqa: E731
    t = [torch.empty(0, dtype=torch.int64, device="cuda")]
    (loss,), (lse,) = ar.ar_cross_entropy(e(0, 8), e(300, 8), t)
    assert loss.shape == (0,) and lse.shape == (0,)
    mine = [torch.full((300, 8), math.nan, device="cuda")]
    ar.ar_cross_entropy_backward(None, e(0, 8), e(300, 8), t, e(0), dweights=mine)
    assert (mine[0] == 0).all()
    t = [torch.arange(5, device="cuda")]
    (loss,), (lse,) = ar.ar_cross_entropy(e(5, 0), e(300, 0), t)
    # log 300 with the logarithm's error and two roundings
    assert ((lse - math.log(300)).abs() <= 8 * U32 * 6).all() and torch.equal(loss, lse)
    dxs, dws = ar.ar_cross_entropy_backward(None, e(5, 0), e(300, 0), t, [lse])
    assert dxs[0].shape == (5, 0) and dws[0].shape == (300, 0)


@pytest.mark.parametrize("rows", [30, 700])
def test_same_bits_every_time(ar, rows):
    torch = _torch()
    rng = np.random.default_rng(14)
    xs, weights = rows_of(rng, 2, rows, 200, "bf16"), rows_of(rng, 2, 3000, 200, "bf16")
    targets = targets_of(rng, 2, rows, 3000)
    first = ar.ar_cross_entropy(xs, weights, targets)
    back = ar.ar_cross_entropy_backward(None, xs, weights, targets, first[1])
    for _ in range(4):
        again = ar.ar_cross_entropy(xs, weights, targets)
        assert all(torch.equal(a, b) for p, q in zip(first, again) for a, b in zip(p, q))
        again = ar.ar_cross_entropy_backward(None, xs, weights, targets, first[1])
        assert all(torch.equal(a, b) for p, q in zip(back, again) for a, b in zip(p, q))


def test_gradient_against_differences(ar):
    """Differences of the GPU's own losses, float32: h^2 / 6 times a third derivative of order one, and the losses'
    error (20 terms of 1e-6) over 2h: with h = 1e-2, 2e-5 + 1e-3; the bound is 1e-2."""
    torch = _torch()
    rng = np.random.default_rng(15)
    (x,), (w,) = rows_of(rng, 1, 20, 12, "f32"), rows_of(rng, 1, 30, 12, "f32")
    targets, h = targets_of(rng, 1, 20, 30), 1e-2
    _, lses = ar.ar_cross_entropy([x], [w], targets)
    (dx,), (dw,) = ar.ar_cross_entropy_backward(None, [x], [w], targets, lses)

    def loss(x, w):
        return float(ar.ar_cross_entropy([x], [w], targets)[0][0].double().sum())

    for at in [(0, 0), (7, 11), (19, 5)]:
        d = torch.zeros_like(x)
        d[at] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[at].item()) < 1e-2
    for at in [(0, 0), (17, 3), (29, 11)]:
        d = torch.zeros_like(w)
        d[at] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[at].item()) < 1e-2


@pytest.mark.parametrize("rows,cols", [(40, 64), (300, 61)])
def test_captured_into_a_graph_and_on_another_stream(ar, rows, cols):
    torch = _torch()
    xs = [torch.randn(rows, cols, device="cuda").bfloat16() for _ in range(2)]
    weights = [torch.randn(700, cols, device="cuda").bfloat16() for _ in range(2)]
    targets = [torch.randint(0, 700, (rows,), device="cuda") for _ in range(2)]

    def all_of(**k):
        losses, lses = ar.ar_cross_entropy(xs, weights, targets, **k)
        dxs, dws = ar.ar_cross_entropy_backward(losses, xs, weights, targets, lses, **k)
        return losses + lses + dxs + dws

    all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, all_of()))
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = all_of()
    for _ in range(4):
        for t in xs + weights:
            t.normal_()
        for t in targets:
            t.random_(0, 700)
        targets[0][:7] = IGNORE
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, all_of()))


def test_writes_are_counted(ar):
    torch = _torch()
    x, w, t = [torch.zeros(3, 8, device="cuda")], [torch.zeros(5, 8, device="cuda")], [torch.zeros(3, dtype=torch.int32, device="cuda")]
    outs = [torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda"), torch.zeros(3, 8, device="cuda"), torch.zeros(5, 8, device="cuda")]
    before = [o._version for o in outs]
    ar.ar_cross_entropy(x, w, t, outs[:1], outs[1:2])
    ar.ar_cross_entropy_backward(None, x, w, t, outs[1:2], outs[2:3], outs[3:])
    assert all(o._version > b for o, b in zip(outs, before))


def test_refusals(ar):
    torch = _torch()
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)              # noqa: E731
    x, w, t, s = [z(3, 8)], [z(5, 8)], [z(3, dtype=torch.int64)], [z(3)]
    f, b = ar.ar_cross_entropy, ar.ar_cross_entropy_backward
    for args in (([], [], []), ([z(3, 8, dtype=torch.float64)], w, t), (x, [z(5, 8, dtype=torch.bfloat16)], t),
                 (x, [z(5, 9)], t), (x, w, [z(4, dtype=torch.int64)]), (x, w, [z(3)]), (x, w * 2, t), (x, w, t * 2),
                 ([z(8, 3).t()], w, t), (x, [z(8, 5).t()], t), ([torch.zeros(3, 8)], w, t), (x, w, [t[0].cpu()]),
                 (x, w, [t[0].view(3, 1)])):
        with pytest.raises((ValueError, TypeError)):
            f(*args)
        with pytest.raises((ValueError, TypeError)):
            b(None, *args, s)
    with pytest.raises(ValueError, match="vocabulary of 0"):
        f(x, [z(0, 8)], t)
    with pytest.raises(ValueError):
        f(x, w, t, losses=[z(4)])
    with pytest.raises(TypeError):
        f(x, w, t, lses=[z(3, dtype=torch.float64)])
    with pytest.raises(ar.ArError, match="overlaps"):
        f(x, w, t, losses=s, lses=s)
    with pytest.raises(ar.ArError, match="workspace"):
        f(x, w, t, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        b([z(4)], x, w, t, s)
    with pytest.raises(ValueError):
        b(None, x, w, t, [z(2)])
    with pytest.raises(ValueError):
        b(None, x, w, t, s, dxs=[z(3, 9)])
    with pytest.raises(TypeError):
        b(None, x, w, t, s, dweights=[z(5, 8, dtype=torch.bfloat16)])
    with pytest.raises(ar.ArError, match="overlaps"):
        b(None, x, w, t, s, dweights=w)
    for scale in (math.nan, math.inf, 1e-60, 1e39):
        with pytest.raises(ar.ArError, match="scale"):
            b(None, x, w, t, s, scale=scale)
    need = ar.ar_cross_entropy_workspace_bytes(3, 5, 8, "f32", 1, True)
    with pytest.raises(ar.ArError, match="aligned"):
        b(None, x, w, t, s, workspace=torch.zeros(need + 32, dtype=torch.uint8, device="cuda")[4:need + 4])
    with pytest.raises(ar.ArError, match="workspace"):
        b(None, x, w, t, s, workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab", [(8, 300), (8, 5000), (200, 5000)])
def test_small_losses_of_large_logits(ar, dtype, rows, vocab):
    """Logits of up to 8,192 whose differences every type holds: the loss keeps what lse, a large number, rounds away.

    z = c (of the row) for the target and c - 12 for the others, exact in float32, so that the loss is
    log(1 + (V - 1) e^-12) for every c.  Its exponentials' sum is off by U32 for every addition to a sum that holds the
    target's 1 (32 of a lane, 4 across lanes and wavefronts, a tile in 16 and 16 joined: below V / 16 / 32 + 60) and as
    much for the small ones' own (relative: V / 128 + 300, EXP and the argument's rounding, 2 * 12 U32); the logarithm
    has EXP, and the last sum U32.
    """
    torch = _torch()
    c = torch.tensor([2.0 ** (k % 8 - 7) for k in range(rows)])          # 1/128 to 1
    x = torch.zeros(rows, 8)
    x[:, 0], x[:, 1] = c, 1.0
    w = torch.zeros(vocab, 8)
    w[:, 0], w[:, 1] = 8192.0, -12.0
    w[7, 1] = 0.0
    t = torch.full((rows,), 7, device="cuda")
    dt = torch_dtype(dtype)
    (loss,), (lse,) = ar.ar_cross_entropy([x.to("cuda", dt)], [w.to("cuda", dt)], [t])
    rest = (vocab - 1) * math.exp(-12)
    want = math.log1p(rest)
    off = (vocab / 512 + 60) * U32 + rest * ((vocab / 128 + 300 + 24) * U32 + EXP) + (EXP + U32) * want
    assert (np.abs(f64(loss) - want) <= off).all(), (f64(loss) - want, off)
    large = 8192 * f64(c) + want
    assert (np.abs(f64(lse) - large) <= off + 2 * U32 * large).all()


def test_most_rows(ar):
    """2^28 rows, the most: every grid at its largest.

    Two logits, 0 and k / 4 for k of 0 to 4 by the row: exact; the loss of a sum of two terms is off by the
    exponential's, the logarithm's and some 8 more roundings of numbers up to 2.
    """
    torch = _torch()
    rows = 1 << 28
    k = torch.arange(rows, dtype=torch.int32, device="cuda").remainder_(5)
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = k
    w = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    w[1, 0] = 0.25
    t = (k % 2).int()
    (loss,), (lse,) = ar.ar_cross_entropy([x], [w], [t])
    want = torch.log1p(torch.exp(torch.arange(5, dtype=torch.float64, device="cuda") / 4))
    for at in range(5):
        mine = k == at
        assert ((lse[mine] - want[at]).abs() <= 2 * (2 * EXP + 8 * U32)).all()
        assert ((loss[mine] - (want[at] - (at % 2) * at / 4)).abs() <= 2 * (2 * EXP + 8 * U32)).all()


def test_more_tiles_than_a_launch_counts(ar):
    """129 rows of float32 against 240,000,000 words: 18,750,000 tiles of 64 x 32, which take two launches.

    All logits are 0 but the last word's 20: the sums of ones are whole multiples of a tile's 64, below 2^24 of them, and
    exact; what the exponentials and the join of 16 sums add is below 30 U32 of the sum, the logarithm and the last sums
    10 U32 of 20.
    """
    torch = _torch()
    rows, vocab = 129, 240_000_000
    x = torch.zeros(rows, 4, device="cuda")
    x[:, 0] = torch.arange(rows, device="cuda") % 2
    w = torch.zeros(vocab, 4, device="cuda")
    w[-1, 0] = 20.0
    t = torch.full((rows,), vocab - 1, device="cuda")
    (loss,), (lse,) = ar.ar_cross_entropy([x], [w], [t])
    for odd in (0, 1):
        want = math.log(math.exp(20.0 * odd) + vocab - 1)
        off = 30 * U32 + 10 * U32 * 20
        assert (np.abs(f64(lse)[odd::2] - want) <= off).all() and (np.abs(f64(loss)[odd::2] - (want - 20 * odd)) <= off).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_rows_take_little_memory(ar, dtype):
    """16 rows against 131 to 262 MB of weight that lies on 16 bytes: no copy of it is made room for."""
    torch = _torch()
    rng = np.random.default_rng(16)
    xs, weights = rows_of(rng, 1, 16, 1024, dtype, 8), rows_of(rng, 1, 64000, 1024, dtype, 8)
    targets = targets_of(rng, 1, 16, 64000)
    losses, lses = ar.ar_cross_entropy(xs, weights, targets)
    dws = [torch.empty_like(weights[0])]
    most = {}
    for name, call in (("forward", lambda: ar.ar_cross_entropy(xs, weights, targets)),
                       ("backward", lambda: ar.ar_cross_entropy_backward(None, xs, weights, targets, lses, dweights=dws))):
        call()
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call()
        most[name] = torch.cuda.max_memory_allocated() - before
    logits = 16 * 64000 * 4
    # forward: 8 bytes per row and 64 words; backward: dz, 64 splits of dx's sums and the rest, which is x's size
    assert most["forward"] <= logits / 16 and most["backward"] <= 2 * logits + 64 * 16 * 1024 * 4
    # a workspace of the size for any operands serves as well
    for need in (ar.ar_cross_entropy_workspace_bytes, ar.ar_cross_entropy_aligned_workspace_bytes):
        ws = torch.empty(need(16, 64000, 1024, dtype, 1), dtype=torch.uint8, device="cuda")
        again = ar.ar_cross_entropy(xs, weights, targets, workspace=ws)
        assert torch.equal(again[0][0], losses[0]) and torch.equal(again[1][0], lses[0])


def random_case(n, rows, cols, vocab, dtype, seed):
    """check()'s inputs, made on the GPU: (xs, weights, targets, dlosses)."""
    torch = _torch()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch_dtype(dtype)
    xs = [torch.randn(rows, cols, device="cuda", generator=gen).to(dt) for _ in range(n)]
    weights = [(torch.randn(vocab, cols, device="cuda", generator=gen) * (1.5 / math.sqrt(cols))).to(dt) for _ in range(n)]
    targets = []
    for _ in range(n):
        t = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
        targets.append(torch.where(torch.rand(rows, device="cuda", generator=gen) < 0.2, IGNORE, t))
    return xs, weights, targets, [torch.rand(rows, device="cuda", generator=gen) / rows for _ in range(n)]


def check_large(ar, n, rows, cols, vocab, dtype):
    """Both passes against float64 on the GPU, row by row.

    lse and loss: check_forward()'s bound.  Gradients: the 2-norm of a row's error, relative to the row's.  What goes
    into it is independent from term to term and adds up as its root of squares: of 16-bit dz a rounding (UNIT at most)
    and one of the result; for float32 p's error, of some sqrt(cols) roundings of logits of a few units and 4 of
    arguments up to 16 (16 sqrt(cols) U32 hold both), and a sum's roundings, sqrt(depth) U32 of partial sums no larger
    than the result.  All rows together 2 times that, and a row (its largest of some thousand) 4 times: a step of the
    sum left out, 32 to 128 of its terms, is sqrt(32 / depth), 3% and more.
    """
    torch = _torch()
    xs, weights, targets, dlosses = random_case(n, rows, cols, vocab, dtype, rows + cols + vocab)
    losses, lses = ar.ar_cross_entropy(xs, weights, targets, ignore_index=IGNORE)
    dxs, dws = ar.ar_cross_entropy_backward(dlosses, xs, weights, targets, lses, ignore_index=IGNORE)
    for x, w, t, g, loss, lse, dx, dw in zip(xs, weights, targets, dlosses, losses, lses, dxs, dws):
        x, w, kept = x.double(), w.double(), t != IGNORE
        z = x @ w.t()
        want = z.logsumexp(1)
        spread = (z - z.amax(1, keepdim=True)).abs()
        off = (cols + 1) * U32 * (x.abs() @ w.abs().t())
        at = t.clamp(min=0)[:, None]
        lse_off = ((torch.exp(z - want[:, None]) * (off + 4 * (spread + off) * U32)).sum(1) * 1.01 + EXP
                   + (vocab / 128 + 300) * U32 + 8 * U32 * (want.abs() + z.abs().amax(1) + 1))
        assert ((lse - want).abs() <= lse_off).all()
        want_loss = want - z.gather(1, at)[:, 0]
        loss_off = lse_off + off.gather(1, at)[:, 0] + 2 * U32 * want_loss.abs()
        assert ((loss - want_loss).abs() <= loss_off)[kept].all() and (loss[~kept] == 0).all()
        del off, spread
        dz = torch.exp(z.sub_(lse.double()[:, None]))
        dz[kept, t[kept]] -= 1
        dz *= (g.double() * kept)[:, None]
        assert (dx[~kept] == 0).all()
        for got, want, depth, other in ((dx, dz @ w, vocab, w), (dw, dz.t() @ x, rows, x)):
            # below the normal numbers a rounding is no longer relative: the result's moves each of a row's `cols` elements
            # by at most TINY, their 2-norm by sqrt(cols) TINY (weights g near 0 make such rows of binary16); dz's moves each
            # of its elements by TINY times the largest |g| / 2^13 (binary16), and the row by that times the other
            # factor's 2-norm
            tiny = math.sqrt(cols) * TINY[dtype]
            if dtype == "f16":
                tiny = tiny + float(g[kept].max()) * 2.0 ** -13 * TINY["f16"] * float(other.norm())
            bound = 2 * UNIT[dtype] if dtype != "f32" else (math.sqrt(depth) + 16 * math.sqrt(cols)) * U32
            away, size = (got.double() - want).norm(dim=1), want.norm(dim=1)
            assert away.norm() <= 2 * bound * size.norm() + math.sqrt(len(got)) * tiny, float(away.norm() / size.norm() / bound)
            # a word that is no row's target has small terms only, whose rounding in a binary16 of 2^13 for the largest |g|
            # may be a subnormal's: what is far below the others counts with them
            size = size.clamp(min=1e-3 * float(size.max()))
            assert (away <= 4 * bound * size + tiny)[kept if got is dx else slice(None)].all(), float((away / size).max() / bound)


@pytest.mark.parametrize("n,rows,cols,vocab", [(3, 520, 100, 8200), (3, 2060, 100, 5000), (1, 3000, 100, 5000),
                                               (2, 150, 1500, 5000), (2, 2000, 390, 33000)])
def test_every_tile_in_float32(ar, n, rows, cols, vocab):
    """Sizes that the larger three tiles are picked for in each of the four products, all of several steps of the sum: the
    largest for the loss and dz in the third, for dweight in the fourth, for dx in the last."""
    check_large(ar, n, rows, cols, vocab, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,rows,cols,vocab", [(1, 260, 100, 8200), (3, 520, 130, 5000), (2, 150, 130, 16400),
                                               (2, 4100, 1000, 300), (1, 1500, 520, 33000), (1, 4096, 260, 16400)])
def test_every_tile_in_16_bits(ar, dtype, n, rows, cols, vocab):
    """The same: the largest for the loss and dz in the second and the last two, for dweight in the third and fifth, for dx
    in the fourth and last."""
    check_large(ar, n, rows, cols, vocab, dtype)


@pytest.mark.parametrize("large", ["weights", "rows"])
def test_small_gradients_keep_their_bits_in_binary16(ar, large):
    """g of 1e-7 against the float64 oracle, dx where the weights are large and dweight where x is, so that the results are
    normal binary16 numbers: the softmax's part of dz, 1e-7 of some 1/2,000 each, is below all of binary16 unless it is
    held relative to g.  Every third row has the target that its logits favour, so that its gradient is made of small
    terms only."""
    torch = _torch()
    rng = np.random.default_rng(17)
    up = 2000.0 if large == "weights" else 1 / 2000.0
    xs, weights = rows_of(rng, 1, 150, 64, "f16", 0, 1.2 / up), rows_of(rng, 1, 2000, 64, "f16", 0, 0.2 * up)
    targets = targets_of(rng, 1, 150, 2000)
    best = (xs[0].double() @ weights[0].double().t()).argmax(1)
    targets[0][::3] = best[::3]
    _, lses = check_forward(ar, xs, weights, targets)
    g = [torch.full((150,), 1e-7, device="cuda")]
    (dx,), (dw,) = check_backward(ar, xs, weights, targets, lses, g, "f16")
    x, w, t = f64(xs[0]), f64(weights[0]), targets[0].cpu().numpy()
    want_dx, want_dw, _ = oracle.cross_entropy_backward(f64(g[0]), x, w, t, f64(lses[0]), IGNORE)
    got, want = (f64(dx), want_dx) if large == "weights" else (f64(dw), want_dw)
    # a rounding of dz and one of the result, the subnormals' step for the result's small elements
    size = np.sqrt(np.maximum((want ** 2).sum(1), want.shape[1] * (2.0 ** 13 * TINY["f16"]) ** 2))
    assert (np.sqrt(((got - want) ** 2).sum(1)) <= 2 * UNIT["f16"] * size).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_copies_in_pieces(ar, dtype):
    """Rows that do not lie on 16 bytes, of a weight whose copy takes several pieces in both passes, the last one short."""
    check_large(ar, 1, 300, 1023, 160001, dtype)


def test_copied_forward_has_the_same_bits(ar):
    """The pieces of a copied weight leave every tile as it is: the bits of the same values on 16 bytes."""
    torch = _torch()
    (x,), (w,), (t,), _ = random_case(1, 300, 1016, 100000, "bf16", 18)
    flat = torch.empty(w.numel() + 1, dtype=w.dtype, device="cuda")
    off = flat[1:].view(w.shape)
    off.copy_(w)
    for a, b in zip(ar.ar_cross_entropy([x], [w], [t]), ar.ar_cross_entropy([x], [off], [t])):
        assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("odd", [0, 33])
def test_one_rank_of_many_off_16_bytes(ar, odd):
    """35 ranks, two launches: only the launch of the rank whose weight and x do not start on 16 bytes copies, and all
    have the same bits as without it."""
    torch = _torch()
    rng = np.random.default_rng(19)
    n = 35
    xs, weights = rows_of(rng, n, 33, 24, "bf16"), rows_of(rng, n, 700, 24, "bf16")
    targets = targets_of(rng, n, 33, 700)
    losses, lses = ar.ar_cross_entropy(xs, weights, targets)
    dxs, dws = ar.ar_cross_entropy_backward(None, xs, weights, targets, lses)
    for group in (xs, weights):
        flat = torch.empty(group[odd].numel() + 1, dtype=torch.bfloat16, device="cuda")
        group[odd] = flat[1:].view(group[odd].shape).copy_(group[odd])
    again = ar.ar_cross_entropy(xs, weights, targets)
    back = ar.ar_cross_entropy_backward(None, xs, weights, targets, lses)
    for a, b in zip((losses, lses, dxs, dws), again + back):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
