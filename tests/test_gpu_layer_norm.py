"""Layer norm's forward and backward pass on the GPU against the float64
oracle: types, widths around every row form, ranks, strides, special rows,
in place, streams, and the refusals."""

import math

import numpy as np
import pytest

from gpu_util import require_gpu
from oracle import step as oracle
from step_util import U32, f32, f64, rounded, torch_dtype

pytestmark = pytest.mark.gpu

COLS = [1, 2, 7, 8, 63, 127, 128, 129, 511, 512, 513, 1003, 1024, 1025, 2048, 2049, 4095, 4097, 8192, 8193, 16384,
        16391, 40001]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


@pytest.fixture(scope="module")
def ar():
    require_gpu()
    import ring_allreduce_reduction_virtual_amd as ar

    return ar


def _torch():
    import torch

    return torch


def additions(cols):
    """Longest chain of float32 additions of a row sum: at most 32 elements (or 1/1024 of a wide row) a
    thread, 6 exchanges, 16 wavefronts."""
    return 32 + cols / 1024 + 6 + 16


def make(rng, n, rows, cols, dtype, pad=0, scale=1.0, shift=0.0):
    torch = _torch()
    got = []
    for _ in range(n):
        wide = torch.from_numpy((rng.standard_normal((rows, cols + pad)) * scale + shift).astype(np.float32))
        got.append(wide.to("cuda").to(torch_dtype(dtype))[:, :cols])
    return got


def forward_bound(x, gamma, beta, mean, rstd, cols, dtype):
    """Bound on |y - y64|, and on the statistics, in half-ulp errors u.

    The mean is off by (k + 1) u mean|x| (k additions, one division); x - mean
    by u |x - mean| more; its square and the sum of squares by (k + 3) u plus
    twice the mean's error relative to the deviation, whose first order
    vanishes in the sum and whose square counts: rstd by (k + 3) / 2 + 3 u and
    half that square.  y's own products and sum add 4 u of each term.
    """
    k = additions(cols)
    x, h = np.abs(x), np.abs(x - mean[:, None]) * rstd[:, None]
    mean_off = (k + 1) * U32 * x.mean(1) + 2.0 ** -149
    rstd_off = ((k + 3) / 2 + 3) * U32 + 0.5 * (mean_off * rstd) ** 2
    g = 1.0 if gamma is None else np.abs(gamma)
    b = 0.0 if beta is None else np.abs(beta)
    y_off = g * (mean_off * rstd)[:, None] + g * h * (rstd_off[:, None] + 5 * U32) + 2 * U32 * b
    return y_off, mean_off, rstd_off * rstd


def check_forward(ar, xs, gammas, betas, dtype, eps=1e-5):
    ys, means, rstds = ar.ar_layer_norm(xs, gammas, betas, eps=eps)
    for r, x in enumerate(xs):
        g = None if gammas is None else f64(gammas[r])
        b = None if betas is None else f64(betas[r])
        y, mean, rstd = oracle.layer_norm(f64(x), g, b, eps)
        y_off, mean_off, rstd_off = forward_bound(f64(x), g, b, mean, rstd, x.shape[1], dtype)
        assert (np.abs(f64(means[r]) - mean) <= mean_off).all()
        assert (np.abs(f64(rstds[r]) - rstd) <= rstd_off).all()
        off = np.abs(f64(ys[r]) - y)
        assert (off <= y_off + rounded(np.abs(y) + y_off, dtype)).all(), (x.shape, float((off - y_off).max()))
    return ys, means, rstds


def check_backward(ar, dys, xs, gammas, means, rstds, dtype, wdtype):
    """Against float64 from the same statistics.

    With k additions a row: h has 2 u, w 1 u, sum(w)/cols (k + 2) u of mean|w|,
    sum(w h)/cols (k + 5) u of mean|w h|, and dx's products and differences
    3 u of each term.  A weight gradient's sum has at most one addition a
    row (and 20 in joining) over terms of 3 u.
    """
    dxs, dgs, dbs = ar.ar_layer_norm_backward(dys, xs, gammas, means, rstds)
    for r, x in enumerate(xs):
        g = None if gammas is None else f64(gammas[r])
        dy, x64, mean, rstd = f64(dys[r]), f64(x), f64(means[r]), f64(rstds[r])
        dx, dg, db = oracle.layer_norm_backward(dy, x64, g, mean, rstd)
        k = additions(x.shape[1])
        h = np.abs(x64 - mean[:, None]) * rstd[:, None]
        w = np.abs(dy if g is None else dy * g)
        off = rstd[:, None] * U32 * (5 * w + (k + 6) * w.mean(1, keepdims=True)
                                     + (k + 12) * h * (w * h).mean(1, keepdims=True))
        got = np.abs(f64(dxs[r]) - dx)
        assert (got <= off + rounded(np.abs(dx) + off, dtype)).all(), (x.shape, float((got - off).max()))
        rows = x.shape[0]
        for t, want, terms in ((dgs[r], dg, np.abs(dy) * h), (dbs[r], db, np.abs(dy))):
            off = (rows + 20 + 3) * U32 * terms.sum(0)
            got = np.abs(f64(t) - want)
            assert (got <= off + rounded(np.abs(want) + off, wdtype)).all(), (x.shape, float((got - off).max()))
    return dxs, dgs, dbs


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_widths_and_types(ar, dtype, wdtype, cols):
    rng = np.random.default_rng(cols)
    rows, n = (5, 2) if cols > 5000 else (37, 3)
    pad = cols % 3
    xs = make(rng, n, rows, cols, dtype, pad, 1.5, 0.4)
    gammas = [t[0].clone() for t in make(rng, n, 1, cols, wdtype, 0, 0.3, 1.0)]
    betas = [t[0].clone() for t in make(rng, n, 1, cols, wdtype, 0, 0.3)]
    _, means, rstds = check_forward(ar, xs, gammas, betas, dtype)
    dys = make(rng, n, rows, cols, dtype, pad + 1, 0.1)
    check_backward(ar, dys, xs, gammas, means, rstds, dtype, wdtype)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 63, 64, 65, 257, 2100])
@pytest.mark.parametrize("cols", [24, 300, 2500])
def test_row_counts(ar, rows, cols):
    """Below, at and above what one workgroup, and all of them together, take at a time."""
    rng = np.random.default_rng(rows)
    xs = make(rng, 1, rows, cols, "f32")
    gammas = [t[0].clone() for t in make(rng, 1, 1, cols, "f32")]
    _, means, rstds = check_forward(ar, xs, gammas, None, "f32")
    check_backward(ar, make(rng, 1, rows, cols, "f32"), xs, gammas, means, rstds, "f32", "f32")


@pytest.mark.parametrize("n", [1, 7, 31, 32, 33, 128])
def test_rank_counts(ar, n):
    """Across the ranks of one launch; each rank's own weights and rows."""
    rng = np.random.default_rng(n)
    xs = make(rng, n, 6, 100, "bf16")
    gammas = [t[0].clone() for t in make(rng, n, 1, 100, "bf16")]
    betas = [t[0].clone() for t in make(rng, n, 1, 100, "bf16")]
    _, means, rstds = check_forward(ar, xs, gammas, betas, "bf16")
    check_backward(ar, make(rng, n, 6, 100, "bf16"), xs, gammas, means, rstds, "bf16", "bf16")


def test_without_weights(ar):
    rng = np.random.default_rng(0)
    xs = make(rng, 2, 9, 200, "f32")
    _, means, rstds = check_forward(ar, xs, None, None, "f32")
    check_backward(ar, make(rng, 2, 9, 200, "f32"), xs, None, means, rstds, "f32", "f32")
    ys, none, also = ar.ar_layer_norm(xs, stats=False)
    assert none is None and also is None and len(ys) == 2
    dxs, dg, db = ar.ar_layer_norm_backward(xs, xs, None, means, rstds, weight_grads=False)
    assert dg is None and db is None and len(dxs) == 2


@pytest.mark.parametrize("cols", [100, 3000, 20000])
def test_one_weight_gradient_alone(ar, cols):
    torch = _torch()
    rng = np.random.default_rng(1)
    xs, dys = make(rng, 1, 11, cols, "f32"), make(rng, 1, 11, cols, "f32")
    _, means, rstds = ar.ar_layer_norm(xs)
    _, dg, db = ar.ar_layer_norm_backward(dys, xs, None, means, rstds)
    mine = [torch.full((cols,), math.nan, device="cuda")]
    _, got, none = ar.ar_layer_norm_backward(dys, xs, None, means, rstds, weight_grads=False, dgammas=mine)
    assert none is None and torch.equal(got[0], dg[0])
    _, none, got = ar.ar_layer_norm_backward(dys, xs, None, means, rstds, weight_grads=False, dbetas=mine)
    assert none is None and torch.equal(got[0], db[0])


@pytest.mark.parametrize("cols", [50, 700, 5000, 20000])
def test_in_place_and_interleaved(ar, cols):
    """y over x, dx over dy, and x and y as the two halves of one buffer's rows."""
    torch = _torch()
    rng = np.random.default_rng(cols)
    xs = make(rng, 2, 13, cols, "bf16", pad=3)
    dys = make(rng, 2, 13, cols, "bf16", pad=2)
    ys, means, rstds = ar.ar_layer_norm(xs)
    dxs, dg, db = ar.ar_layer_norm_backward(dys, xs, None, means, rstds)
    _, dg2, db2 = ar.ar_layer_norm_backward(dys, xs, None, means, rstds, dxs=dys)
    assert all(torch.equal(a, b) for a, b in zip(list(dys) + dg + db, list(dxs) + dg2 + db2))
    both = torch.full((13, 2 * cols + 1), 5.0, dtype=torch.bfloat16, device="cuda")
    both[:, :cols] = xs[0]
    ar.ar_layer_norm([both[:, :cols]], ys=[both[:, cols:2 * cols]])
    assert torch.equal(both[:, cols:2 * cols], ys[0]) and torch.equal(both[:, :cols], xs[0])
    assert (both[:, 2 * cols] == 5).all()
    ar.ar_layer_norm(xs, ys=xs)
    assert all(torch.equal(a, b) for a, b in zip(xs, ys))


@pytest.mark.parametrize("cols", [33, 600, 3000, 9000, 20000])
def test_special_rows(ar, cols):
    """A NaN or infinity spoils its own row only; equal rows normalise to beta; huge rows overflow nothing else."""
    torch = _torch()
    rng = np.random.default_rng(2)
    (x,) = make(rng, 1, 9, cols, "f32")
    x = x.contiguous()
    x[1, cols // 2] = math.nan
    x[3, 0] = math.inf
    x[5] = 0.25                            # its sums are exact: mean 0.25, deviation 0
    beta = torch.randn(cols, device="cuda")
    (y,), (mean,), (rstd,) = ar.ar_layer_norm([x], None, [beta])
    bad = [1, 3]
    good = [r for r in range(9) if r not in bad]
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).any() and torch.isfinite(y[good]).all()
    assert torch.equal(y[5], beta) and mean[5] == 0.25 and abs(rstd[5].item() * math.sqrt(1e-5) - 1) < 1e-6
    (clean,), _, _ = ar.ar_layer_norm([x[good].contiguous()], None, [beta])
    assert torch.equal(y[good], clean)
    (dy,) = make(rng, 1, 9, cols, "f32")
    (dx,), _, (db,) = ar.ar_layer_norm_backward([dy], [x], None, [mean], [rstd])
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[good]).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("cols", [10, 777, 9000, 17000])
def test_large_mean(ar, cols):
    """A mean a thousand deviations away: the sum of squares around it keeps the deviation."""
    rng = np.random.default_rng(3)
    xs = make(rng, 1, 8, cols, "f32", scale=1.0, shift=1000.0)
    check_forward(ar, xs, None, None, "f32")


def test_no_rows_and_no_columns(ar):
    torch = _torch()
    x = [torch.empty(0, 40, device="cuda")]
    w = [torch.ones(40, device="cuda")]
    ys, means, rstds = ar.ar_layer_norm(x, w, w)
    assert ys[0].shape == (0, 40) and means[0].numel() == 0
    mine = [[torch.full((40,), math.nan, device="cuda")] for _ in range(2)]
    ar.ar_layer_norm_backward(x, x, w, means, rstds, dgammas=mine[0], dbetas=mine[1])
    assert (mine[0][0] == 0).all() and (mine[1][0] == 0).all()
    x = [torch.empty(3, 0, device="cuda")]
    ys, means, rstds = ar.ar_layer_norm(x)
    assert ys[0].shape == (3, 0)


def test_gradient_against_differences(ar):
    """dx, dgamma and dbeta against differences of the GPU's own forward pass, float32.

    A central difference with step h has a cubic term of h^2 / 6 times a third
    derivative of order one and the forward pass's float32 error, some 30 u per
    term over sqrt(terms), divided by h: with h = 1e-2 and 96 terms, 2e-5 +
    2e-3; the bound is 1e-2 on derivatives of order one.
    """
    torch = _torch()
    rng = np.random.default_rng(6)
    rows, cols, h = 4, 24, 1e-2
    (x,) = make(rng, 1, rows, cols, "f32")
    (dy,) = make(rng, 1, rows, cols, "f32")
    gamma, beta = (torch.randn(cols, device="cuda") for _ in range(2))

    def loss(x, gamma, beta):
        y = ar.ar_layer_norm([x], [gamma], [beta])[0][0]
        return float((dy.double() * y.double()).sum())

    _, means, rstds = ar.ar_layer_norm([x], [gamma], [beta])
    (dx,), (dg,), (db,) = ar.ar_layer_norm_backward([dy], [x], [gamma], means, rstds)
    for at in [(0, 0), (1, 5), (2, 23), (3, 11)]:
        d = torch.zeros_like(x)
        d[at] = h
        slope = (loss(x + d, gamma, beta) - loss(x - d, gamma, beta)) / (2 * h)
        assert abs(slope - dx[at].item()) < 1e-2
    for c in (0, 7, 23):
        d = torch.zeros_like(gamma)
        d[c] = h
        assert abs((loss(x, gamma + d, beta) - loss(x, gamma - d, beta)) / (2 * h) - dg[c].item()) < 1e-2
        assert abs((loss(x, gamma, beta + d) - loss(x, gamma, beta - d)) / (2 * h) - db[c].item()) < 1e-2


@pytest.mark.parametrize("cols", [64, 1500, 6000, 12000, 30000])
def test_same_bits_every_time(ar, cols):
    torch = _torch()
    rng = np.random.default_rng(7)
    xs, dys = make(rng, 3, 200, cols, "bf16"), make(rng, 3, 200, cols, "bf16")
    _, means, rstds = ar.ar_layer_norm(xs)
    first = ar.ar_layer_norm_backward(dys, xs, None, means, rstds)
    for _ in range(4):
        again = ar.ar_layer_norm_backward(dys, xs, None, means, rstds)
        assert all(torch.equal(a, b) for p, q in zip(first, again) for a, b in zip(p, q))


def test_captured_into_a_graph(ar):
    torch = _torch()
    xs = [torch.randn(300, 1000, device="cuda") for _ in range(2)]
    dys = [torch.randn(300, 1000, device="cuda") for _ in range(2)]
    ar.ar_layer_norm_backward(dys, xs, None, *ar.ar_layer_norm(xs)[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ys, means, rstds = ar.ar_layer_norm(xs)
        dxs, dgs, dbs = ar.ar_layer_norm_backward(dys, xs, None, means, rstds)
    for _ in range(4):
        for t in xs + dys:
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = ar.ar_layer_norm(xs)
        back = ar.ar_layer_norm_backward(dys, xs, None, want[1], want[2])
        for got, w in zip((ys, means, rstds, dxs, dgs, dbs), (*want, *back)):
            assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_on_another_stream(ar):
    torch = _torch()
    stream = torch.cuda.Stream()
    xs = [torch.randn(2000, 1111, device="cuda")]
    stream.wait_stream(torch.cuda.current_stream())
    ys, means, rstds = ar.ar_layer_norm(xs, stream=stream)
    dxs, dgs, dbs = ar.ar_layer_norm_backward(xs, xs, None, means, rstds, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    want = ar.ar_layer_norm(xs)
    back = ar.ar_layer_norm_backward(xs, xs, None, want[1], want[2])
    for got, w in zip((ys, means, rstds, dxs, dgs, dbs), (*want, *back)):
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_refusals(ar):
    torch = _torch()
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)              # noqa: E731
    x, st = [z(3, 8)], [z(3)]
    with pytest.raises(ValueError):
        ar.ar_layer_norm([])
    with pytest.raises(ValueError):
        ar.ar_layer_norm([torch.zeros(3, 8)])
    with pytest.raises(ValueError):
        ar.ar_layer_norm([z(8)])
    with pytest.raises(TypeError):
        ar.ar_layer_norm([z(3, 8, dtype=torch.float64)])
    with pytest.raises(ValueError):
        ar.ar_layer_norm([z(3, 8), z(4, 8)])
    with pytest.raises(ValueError, match="contiguous rows"):
        ar.ar_layer_norm([z(8, 3).t()])
    with pytest.raises(ValueError, match="contiguous rows"):
        ar.ar_layer_norm([z(1, 8).expand(3, 8)])
    with pytest.raises(ValueError, match="stride"):
        ar.ar_layer_norm([z(3, 8), z(3, 9)[:, :8]])
    with pytest.raises(TypeError, match="weights"):
        ar.ar_layer_norm(x, [z(8, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        ar.ar_layer_norm(x, [z(9)])
    with pytest.raises(ValueError):
        ar.ar_layer_norm(x, [z(8), z(8)])
    with pytest.raises(ValueError):
        ar.ar_layer_norm([z(3, 8) for _ in range(129)])
    for eps in (-1.0, math.nan, math.inf):
        with pytest.raises(ar.ArError, match="eps"):
            ar.ar_layer_norm(x, eps=eps)
    buf = z(40)
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_layer_norm([buf[:24].view(3, 8)], ys=[buf[4:28].view(3, 8)])
    y = z(3, 8)
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_layer_norm([z(3, 8), z(3, 8)], ys=[y, y])
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_layer_norm_backward([z(3, 8)], x, None, st, st, dxs=x)
    with pytest.raises(ValueError):
        ar.ar_layer_norm_backward([z(3, 8)], x, None, [z(4)], st)
    with pytest.raises(ValueError):
        ar.ar_layer_norm_backward([z(3, 8)], x, None, st + st, st)
    with pytest.raises(ar.ArError, match="workspace"):
        ar.ar_layer_norm_backward([z(3, 8)], x, None, st, st, workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("cols", [31, 32, 33, 64, 65, 255, 256, 257, 767, 2047, 4096, 8191, 16383])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bounds_of_the_row_forms(ar, dtype, cols):
    """Widths at and beside the forms' bounds, with enough rows that every workgroup takes several."""
    torch = _torch()
    rng = np.random.default_rng(cols)
    rows, n = (1500, 2) if cols < 1024 else (40, 2)
    xs = make(rng, n, rows, cols, dtype, 1, 1.2, -0.3)
    gammas = [t[0].clone() for t in make(rng, n, 1, cols, dtype, 0, 0.3, 1.0)]
    _, means, rstds = check_forward(ar, xs, gammas, gammas, dtype)
    dys = make(rng, n, rows, cols, dtype, 3)
    dxs, _, _ = check_backward(ar, dys, xs, gammas, means, rstds, dtype, dtype)
    # nothing is written beside the rows
    wide = [torch.full((rows, cols + 9), 3.0, dtype=torch_dtype(dtype), device="cuda") for _ in range(n)]
    ar.ar_layer_norm_backward(dys, xs, gammas, means, rstds, dxs=[w[:, 4:cols + 4] for w in wide])
    for w, d in zip(wide, dxs):
        assert torch.equal(w[:, 4:cols + 4], d) and (w[:, :4] == 3).all() and (w[:, cols + 4:] == 3).all()


def test_made_outputs_are_tensors_of_their_own(ar):
    """The outputs a call makes share memory side by side, but are no views of one another."""
    torch = _torch()
    xs = [torch.randn(5, 33, device="cuda") for _ in range(3)]
    ys, means, rstds = ar.ar_layer_norm(xs)
    for group, shape in ((ys, (5, 33)), (means, (5,)), (rstds, (5,))):
        assert [tuple(t.shape) for t in group] == [shape] * 3
        assert all(t.is_contiguous() and not t._is_view() for t in group)
    kept = [t.clone() for t in (*ys, *means, *rstds)]
    ys[1].requires_grad_()
    with torch.no_grad():
        ys[1].fill_(7.0)
        means[2].fill_(8.0)
    for i, (a, b) in enumerate(zip((*ys, *means, *rstds), kept)):
        assert torch.equal(a, torch.full_like(b, 7.0 if i == 1 else 8.0) if i in (1, 5) else b)
    only = ys[2]
    del ys, means, rstds
    torch.empty(1 << 20, device="cuda").fill_(3.0)
    assert torch.equal(only, kept[2])


@pytest.mark.parametrize("cols", [9, 17, 1003, 4095])
def test_infinite_weight(ar, cols):
    """One infinite weight in the last columns: the formula's infinities, and NaN only where it has them."""
    torch = _torch()
    for at in (cols - 1, cols - 5):
        x = torch.randn(6, cols, device="cuda")
        dy = torch.randn(6, cols, device="cuda").abs() + 0.1
        g = torch.ones(cols, device="cuda")
        g[at] = math.inf
        _, m, s = ar.ar_layer_norm([x])
        dxs, _, _ = ar.ar_layer_norm_backward([dy], [x], [g], m, s)
        d, h = dy.double(), (x.double() - m[0].double()[:, None]) * s[0].double()[:, None]
        w = d * g.double()
        want = s[0].double()[:, None] * (w - w.mean(1, keepdim=True) - h * (w * h).mean(1, keepdim=True))
        got = dxs[0].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        inf = torch.isinf(want)
        assert inf.any() and torch.equal(got[inf], want[inf])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ranks,rows,cols", [(1, 70, 33000), (3, 11, 40001), (2, 300, 16385), (40, 3, 33001), (1, 5, 300007)])
def test_wide_rows_weight_gradients(ar, dtype, ranks, rows, cols):
    """Rows past the registers: every stretch of columns and every share of the rows reaches the sums."""
    from step_util import UNIT

    torch = _torch()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    xs = [torch.randn(rows, cols, device="cuda").to(dt) for _ in range(ranks)]
    dys = [torch.randn(rows, cols, device="cuda").to(dt) for _ in range(ranks)]
    _, m, s = ar.ar_layer_norm(xs)
    _, dg, db = ar.ar_layer_norm_backward(dys, xs, None, m, s)
    for r in range(ranks):
        d = dys[r].double()
        h = (xs[r].double() - m[r].double()[:, None]) * s[r].double()[:, None]
        for got, terms in ((dg[r], d * h), (db[r], d)):
            want, size = terms.sum(0), terms.abs().sum(0)
            # float32 sums of `rows` terms, each with three roundings, then the type's own
            bound = size * (rows + 5) * 2.0 ** -23 + want.abs() * UNIT[dtype] + 1e-30
            assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("cols", [72, 768, 1000, 1024, 1536, 5120, 6144, 12288])
def test_infinite_weight_in_rows_of_whole_vectors(ar, dtype, wdtype, cols):
    """The same where the row is a whole number of vectors, which leaves some of its threads without one."""
    torch = _torch()
    dt, wdt = torch_dtype(dtype), torch_dtype(wdtype)
    for at in (cols - 1, cols - 4, 0):
        x = torch.randn(6, cols, device="cuda").to(dt)
        dy = (torch.randn(6, cols, device="cuda").abs() + 0.1).to(dt)
        g = torch.ones(cols, device="cuda", dtype=wdt)
        g[at] = math.inf
        _, m, s = ar.ar_layer_norm([x])
        dxs, dgs, dbs = ar.ar_layer_norm_backward([dy], [x], [g], m, s)
        d, h = dy.double(), (x.double() - m[0].double()[:, None]) * s[0].double()[:, None]
        w = d * g.double()
        want = s[0].double()[:, None] * (w - w.mean(1, keepdim=True) - h * (w * h).mean(1, keepdim=True))
        got = dxs[0].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        inf = torch.isinf(want)
        assert inf.any() and torch.equal(got[inf], want[inf])
        assert torch.isfinite(dgs[0]).all() and torch.isfinite(dbs[0]).all()
