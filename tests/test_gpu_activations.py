"""Activations in 8 bits on the GPU: codes and scales against the oracle bit for
bit, their values, and layer norm's backward pass from them."""

import math

import numpy as np
import pytest

from gpu_util import require_gpu
from oracle import model as oracle
from oracle import step
from step_util import U32, f64, rounded, torch_dtype

pytestmark = pytest.mark.gpu

COLS = [1, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 511, 513, 1003, 1024, 2049, 4095, 4100, 8193, 16390,
        33001]
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


@pytest.fixture(scope="module")
def ar():
    require_gpu()
    import ring_allreduce_reduction_virtual_amd as ar

    return ar


def _torch():
    import torch

    return torch


def make(rng, n, rows, cols, dtype, pad=0, scale=1.0, shift=0.0):
    torch = _torch()
    got = []
    for _ in range(n):
        wide = torch.from_numpy((rng.standard_normal((rows, cols + pad)) * scale + shift).astype(np.float32))
        got.append(wide.to("cuda").to(torch_dtype(dtype))[:, :cols])
    return got


def same(got, want):
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", COLS)
def test_codes_and_values(ar, dtype, cols):
    torch = _torch()
    rng = np.random.default_rng(cols)
    rows, n = (3, 1) if cols > 3000 else (11, 3)
    sizes = np.exp2(rng.integers(-6, 7, cols)).astype(np.float32)
    xs = [x.mul_(torch.from_numpy(sizes).to("cuda")) for x in make(rng, n, rows, cols, dtype, cols % 5)]
    packed = ar.ar_pack_activations(xs)
    values = ar.ar_unpack_activations(packed)
    narrow = {t: ar.ar_unpack_activations(packed, dtype=t) for t in (torch.bfloat16, torch.float16)}
    for r, x in enumerate(xs):
        codes, scales = oracle.pack_activations(f64(x))
        assert np.array_equal(packed[r].codes.cpu().numpy(), codes)
        assert np.array_equal(packed[r].scales.cpu().numpy(), scales)
        want = oracle.unpack_activations(codes, scales)
        assert np.array_equal(f64(values[r]), want) and np.array_equal(f64(narrow[torch.bfloat16][r]), want)
        assert torch.equal(narrow[torch.float16][r], values[r].to(torch.float16))
        wide = [torch.full((rows, cols + 9), 3.0, device="cuda")]
        ar.ar_unpack_activations([packed[r]], [wide[0][:, 4:cols + 4]])
        assert np.array_equal(f64(wide[0][:, 4:cols + 4]), want)
        assert (wide[0][:, :4] == 3).all() and (wide[0][:, cols + 4:] == 3).all()


def test_special_values(ar):
    """NaN, infinities and what is too large mark their block alone; subnormals, zeros and ties."""
    torch = _torch()
    x = torch.zeros(6, 100, device="cuda")
    x[0, 5], x[0, 40], x[0, 99] = math.nan, math.inf, -math.inf
    x[1] = torch.linspace(-1, 1, 100, device="cuda") * 2.0 ** -126
    x[2, 0], x[2, 1:7] = 127.0, torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5], device="cuda")
    x[3, 0], x[3, 32], x[3, 64], x[3, 96] = 127 * 2.0 ** 121, 3.4e38, 2.0 ** -149, -127 / 64
    x[4] = -0.0
    x[5] = torch.randn(100, device="cuda") * 1e30
    (packed,) = ar.ar_pack_activations([x])
    codes, scales = oracle.pack_activations(f64(x))
    assert np.array_equal(packed.codes.cpu().numpy(), codes) and np.array_equal(packed.scales.cpu().numpy(), scales)
    assert scales[0].tolist().count(255) == 3 and scales[3].tolist() == [254, 255, 1, 127]
    (back,) = ar.ar_unpack_activations([packed])
    assert same(f64(back), oracle.unpack_activations(codes, scales))


def test_every_scale_and_code(ar):
    """All 256 scale bytes with all codes, -128 and scale 0 too, which packing never makes."""
    torch = _torch()
    codes = (torch.arange(256, device="cuda") - 128).to(torch.int8).repeat(256, 1)
    scales = torch.arange(256, device="cuda").to(torch.uint8)[:, None].repeat(1, 8)
    (got,) = ar.ar_unpack_activations([ar.PackedRows(codes, scales)])
    with np.errstate(over="ignore"):
        want = oracle.unpack_activations(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)
    assert same(got.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 63, 65, 300, 70001])
@pytest.mark.parametrize("cols", [3, 40, 300])
def test_row_counts(ar, rows, cols):
    torch = _torch()
    if rows > 1000 and cols > 3:
        return
    (x,) = make(np.random.default_rng(rows), 1, rows, cols, "f32")
    (packed,) = ar.ar_pack_activations([x])
    (back,) = ar.ar_unpack_activations([packed])
    blocks = torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)
    half = torch.exp2(packed.scales.double() - 134)[..., None]
    away = torch.nn.functional.pad(back - x, (0, -cols % 32)).view(rows, -1, 32)
    assert (away.abs().double() <= half).all() and (blocks.abs().amax(-1) <= 254 * half[..., 0]).all()


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm_backward(ar, dtype, wdtype, cols):
    """Against float64 from the values that the codes stand for (the counts of roundings are those of the
    backward pass from the input as it was: the codes' values are exact)."""
    torch = _torch()
    rng = np.random.default_rng(cols)
    rows, n = (5, 2) if cols > 5000 else (37, 3)
    xs = make(rng, n, rows, cols, dtype, cols % 3, 1.5, 0.4)
    gammas = [t[0].clone() for t in make(rng, n, 1, cols, wdtype, 0, 0.3, 1.0)]
    _, means, rstds = ar.ar_layer_norm(xs, gammas)
    packed = ar.ar_pack_activations(xs)
    dys = make(rng, n, rows, cols, dtype, 1 + cols % 3, 0.1)
    dxs, dgs, dbs = ar.ar_layer_norm_backward_packed(dys, packed, gammas, means, rstds)
    for r in range(n):
        x = oracle.unpack_activations(packed[r].codes.cpu().numpy(), packed[r].scales.cpu().numpy())
        dy, g, mean, rstd = f64(dys[r]), f64(gammas[r]), f64(means[r]), f64(rstds[r])
        dx, dg, db = step.layer_norm_backward(dy, x, g, mean, rstd)
        k = 32 + cols / 1024 + 6 + 16
        h = np.abs(x - mean[:, None]) * rstd[:, None]
        w = np.abs(dy * g)
        off = rstd[:, None] * U32 * (5 * w + (k + 6) * w.mean(1, keepdims=True)
                                     + (k + 12) * h * (w * h).mean(1, keepdims=True))
        assert (np.abs(f64(dxs[r]) - dx) <= off + rounded(np.abs(dx) + off, dtype)).all()
        for t, want, terms in ((dgs[r], dg, np.abs(dy) * h), (dbs[r], db, np.abs(dy))):
            off = (rows + 20 + 3) * U32 * terms.sum(0)
            assert (np.abs(f64(t) - want) <= off + rounded(np.abs(want) + off, wdtype)).all()
    # the same bits as from the unpacked values, where their type holds them: the arithmetic is the same
    if dtype != "f16":
        plain = ar.ar_layer_norm_backward(dys, ar.ar_unpack_activations(packed, dtype=torch_dtype(dtype)), gammas,
                                          means, rstds)
        assert all(torch.equal(a, b) for p, q in zip(plain, (dxs, dgs, dbs)) for a, b in zip(p, q))


@pytest.mark.parametrize("cols", [40, 700, 5000, 20000])
def test_layer_norm_backward_in_place_and_beside(ar, cols):
    torch = _torch()
    rng = np.random.default_rng(cols)
    xs, dys = make(rng, 2, 13, cols, "bf16"), make(rng, 2, 13, cols, "bf16", 2)
    _, means, rstds = ar.ar_layer_norm(xs)
    packed = ar.ar_pack_activations(xs)
    dxs, dgs, dbs = ar.ar_layer_norm_backward_packed(dys, packed, None, means, rstds)
    _, none, also = ar.ar_layer_norm_backward_packed(dys, packed, None, means, rstds, dxs=dys, weight_grads=False)
    assert none is None and also is None and all(torch.equal(a, b) for a, b in zip(dys, dxs))
    mine = [torch.full((cols,), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    dys = make(np.random.default_rng(cols), 4, 13, cols, "bf16", 0)[2:]
    want = ar.ar_layer_norm_backward_packed(dys, packed, None, means, rstds)
    ar.ar_layer_norm_backward_packed(dys, packed, None, means, rstds, weight_grads=False, dgammas=mine)
    assert all(torch.equal(a, b) for a, b in zip(mine, want[1]))


@pytest.mark.parametrize("cols", [50, 1000, 20000])
def test_a_block_of_nan_spoils_its_row(ar, cols):
    torch = _torch()
    x, dy = torch.randn(6, cols, device="cuda"), torch.randn(6, cols, device="cuda")
    _, (m,), (s,) = ar.ar_layer_norm([x])
    x[2, cols - 1] = math.inf
    packed = ar.ar_pack_activations([x])
    (dx,), (dg,), (db,) = ar.ar_layer_norm_backward_packed([dy], packed, None, [m], [s])
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[[0, 1, 3, 4, 5]]).all() and torch.isfinite(db).all()
    first = (cols - 1) // 32 * 32
    assert torch.isnan(dg[first:]).all() and torch.isfinite(dg[:first]).all()


def test_no_rows_and_no_columns(ar):
    torch = _torch()
    for shape in ((0, 40), (3, 0)):
        (p,) = ar.ar_pack_activations([torch.empty(*shape, device="cuda")])
        assert p.codes.shape == shape and ar.ar_unpack_activations([p])[0].shape == shape
    p = [ar.PackedRows.empty(0, 40, "cuda")]
    none = [torch.empty(0, device="cuda")]
    mine = [[torch.full((40,), math.nan, device="cuda")] for _ in range(2)]
    ar.ar_layer_norm_backward_packed([torch.empty(0, 40, device="cuda")], p, None, none, none, dgammas=mine[0],
                                     dbetas=mine[1])
    assert (mine[0][0] == 0).all() and (mine[1][0] == 0).all()


@pytest.mark.parametrize("n", [1, 33, 128])
def test_rank_counts(ar, n):
    rng = np.random.default_rng(n)
    xs = make(rng, n, 5, 70, "bf16")
    packed = ar.ar_pack_activations(xs)
    _, m, s = ar.ar_layer_norm(xs)
    whole = ar.ar_layer_norm_backward_packed(xs, packed, None, m, s)
    for r in (0, n // 2, n - 1):
        codes, scales = oracle.pack_activations(f64(xs[r]))
        assert np.array_equal(packed[r].codes.cpu().numpy(), codes)
        one = ar.ar_layer_norm_backward_packed(xs[r:r + 1], packed[r:r + 1], None, m[r:r + 1], s[r:r + 1])
        assert all(_torch().equal(a[r], b[0]) for a, b in zip(whole[:1], one[:1]))


def test_captured_into_a_graph_and_on_another_stream(ar):
    torch = _torch()
    xs, dys = ([torch.randn(300, 1000, device="cuda") for _ in range(2)] for _ in range(2))
    stats = ar.ar_layer_norm(xs)[1:]

    def all_of(**k):
        packed = ar.ar_pack_activations(xs, **k)
        back = ar.ar_unpack_activations(packed, **k)
        return [t for p in packed for t in p] + back + [
            t for g in ar.ar_layer_norm_backward_packed(dys, packed, None, *stats, **k) for t in g]

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
        for t in xs + dys:
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, all_of()))


def test_refusals(ar):
    torch = _torch()
    x = [torch.zeros(3, 40, device="cuda")]
    (p,) = ar.ar_pack_activations(x)
    st = [torch.zeros(3, device="cuda")]
    with pytest.raises(ValueError):
        ar.ar_pack_activations([])
    with pytest.raises(TypeError):
        ar.ar_pack_activations([torch.zeros(3, 40, dtype=torch.float64, device="cuda")])
    with pytest.raises(ValueError, match="contiguous rows"):
        ar.ar_pack_activations([torch.zeros(40, 3, device="cuda").t()])
    with pytest.raises(ValueError):
        ar.ar_pack_activations(x, [p, p])
    with pytest.raises(ValueError):
        ar.ar_pack_activations(x, [ar.PackedRows.empty(3, 41, "cuda")])
    with pytest.raises(ValueError, match="codes"):
        ar.ar_pack_activations(x, [ar.PackedRows(p.codes.view(40, 3), p.scales)])
    with pytest.raises(TypeError):
        ar.ar_pack_activations(x, [(p.codes.view(torch.uint8), p.scales)])
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_pack_activations(x * 2, [p, p])
    with pytest.raises(ValueError):
        ar.ar_unpack_activations([])
    with pytest.raises(ValueError):
        ar.ar_unpack_activations([x[0]])
    with pytest.raises(TypeError):
        ar.ar_unpack_activations([p], dtype=torch.float64)
    with pytest.raises(ValueError):
        ar.ar_unpack_activations([p], [torch.zeros(3, 41, device="cuda")])
    with pytest.raises(ValueError):
        ar.ar_unpack_activations([p] * 129)
    with pytest.raises(ValueError):
        ar.ar_layer_norm_backward_packed(x, [p, p], None, st, st)
    with pytest.raises(ValueError):
        ar.ar_layer_norm_backward_packed([torch.zeros(3, 39, device="cuda")], [p], None, st, st)
    with pytest.raises(ar.ArError, match="workspace"):
        ar.ar_layer_norm_backward_packed(x, [p], None, st, st,
                                         workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))
