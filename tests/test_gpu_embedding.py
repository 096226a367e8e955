"""The embedding and its gradient on the GPU against the float64 oracle: types,
widths around every row form, token counts around chunks and both sorts, skewed
tokens, padding, tokens outside, strides, streams, graphs, and the refusals."""

import math

import numpy as np
import pytest

from gpu_util import require_gpu
from oracle import model as oracle
from step_util import U32, f64, rounded, torch_dtype

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]
COLS = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 257, 512, 513, 1003, 1024, 2048, 2049, 4100, 9001]


@pytest.fixture(scope="module")
def ar():
    require_gpu()
    import ring_allreduce_reduction_virtual_amd as ar

    return ar


def _torch():
    import torch

    return torch


def rows_of(rng, n, rows, cols, dtype, pad=0, scale=1.0):
    torch = _torch()
    got = []
    for _ in range(n):
        wide = torch.from_numpy((rng.standard_normal((rows, cols + pad)) * scale).astype(np.float32))
        got.append(wide.to("cuda").to(torch_dtype(dtype))[:, :cols])
    return got


def tokens_of(values, index="i64"):
    torch = _torch()
    return [torch.tensor(np.asarray(v), dtype=torch.int64 if index == "i64" else torch.int32, device="cuda")
            for v in values]


def check_backward(ar, dys, tokens, vocab, dtype, wdtype, scale=1.0, padding=None, held=None, pad=0):
    """Each gradient within what its float32 sum and its one rounding allow.

    A token's sum has as many additions as it has rows (a chunk's sum starts at
    0), one for each partial sum, at most as many again, each off by half a unit
    of at most the sum of the terms' magnitudes; the scale's product, the scale
    itself and the sum with what was held add a rounding each.
    """
    torch = _torch()
    n, cols = len(dys), dys[0].shape[1]
    dt = torch_dtype(wdtype)
    wide = [torch.full((vocab, cols + pad), math.nan, dtype=dt, device="cuda") for _ in range(n)]
    outs = [w[:, :cols] for w in wide]
    if held is not None:
        for o, h in zip(outs, held):
            o.copy_(h)
    got = ar.ar_embedding_backward(dys, tokens, dtables=outs, scale=scale, padding_index=padding,
                                   accumulate=held is not None)
    assert got is outs
    for r in range(n):
        t = tokens[r].cpu().numpy()
        want, size, terms = oracle.embedding_backward(f64(dys[r]), t, vocab, scale, padding,
                                                      None if held is None else f64(held[r]))
        off = (2 * terms[:, None] + 3) * U32 * size
        bad = np.abs(f64(outs[r]) - want) - off - rounded(np.abs(want) + off, wdtype)
        assert (bad <= 0).all(), (r, float(bad.max()), np.argwhere(bad > 0)[:5])
        none = terms == 0
        assert (f64(outs[r])[none] == (0 if held is None else f64(held[r])[none])).all()
        assert pad == 0 or torch.isnan(wide[r][:, cols:]).all()
    return outs


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_widths_and_types(ar, dtype, wdtype, cols):
    torch = _torch()
    rng = np.random.default_rng(cols)
    n, rows, vocab = 2, 77, 50
    index = "i32" if cols % 2 else "i64"
    tokens = tokens_of([rng.integers(0, vocab, rows) for _ in range(n)], index)
    tables = rows_of(rng, n, vocab, cols, wdtype, cols % 3)
    wide = [torch.full((rows, cols + 5), 7.0, dtype=torch_dtype(dtype), device="cuda") for _ in range(n)]
    outs = [w[:, 2:cols + 2] for w in wide]
    ar.ar_embedding(tokens, tables, outs, scale=1.7)
    for o, t, w, x in zip(outs, tokens, tables, wide):
        # the float32 scale's product is off by at most 2^-24 of itself, then one rounding to the type; the
        # hardware's product that rounds to binary16 leaves the first out, so that a product within 2^-24 of
        # the middle between two of binary16's values may go either way
        want = oracle.embedding(t.cpu().numpy(), f64(w), float(np.float32(1.7)))
        off = 0 if dtype == "f32" else U32 * np.abs(want)
        assert (np.abs(f64(o) - want) <= off + rounded(np.abs(want) + off, dtype)).all()
        assert (x[:, :2] == 7).all() and (x[:, cols + 2:] == 7).all()
    check_backward(ar, rows_of(rng, n, rows, cols, dtype, cols % 4), tokens, vocab, dtype, wdtype, 1.7, pad=cols % 2)


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 64, 65, 1000, 4097, 8191, 8192, 8193, 12289, 40000])
@pytest.mark.parametrize("vocab", [1, 3, 511, 512, 70000])
def test_token_counts(ar, rows, vocab):
    """Around a chunk, a sort's tile, the largest sort in one workgroup, and one to three digits of token."""
    rng = np.random.default_rng(rows + vocab)
    tokens = tokens_of([rng.integers(0, vocab, rows) for _ in range(2)])
    check_backward(ar, rows_of(rng, 2, rows, 5, "f32"), tokens, vocab, "f32", "f32")


@pytest.mark.parametrize("vocab", [300000])
@pytest.mark.parametrize("rows", [500, 9000])
def test_three_passes(ar, rows, vocab):
    rng = np.random.default_rng(4)
    tokens = tokens_of([rng.integers(0, vocab, rows)])
    check_backward(ar, rows_of(rng, 1, rows, 3, "f32"), tokens, vocab, "f32", "f32")


@pytest.mark.parametrize("rows", [700, 20000])
@pytest.mark.parametrize("cols", [4, 100, 2100])
def test_skewed_tokens(ar, rows, cols):
    """One token for nearly all places, runs that end on a chunk's end, the first and the last token."""
    if rows * cols > 3e6:
        rows = 1500
    rng = np.random.default_rng(rows)
    vocab = 40
    few = np.where(rng.random(rows) < 0.95, 17, rng.integers(0, vocab, rows))
    runs = np.repeat(np.arange(-(-rows // 32)) % vocab, 32)[:rows]
    same = np.full(rows, vocab - 1)
    tokens = tokens_of([few, runs, same, np.zeros(rows, int)])
    check_backward(ar, rows_of(rng, 4, rows, cols, "f32"), tokens, vocab, "f32", "f32", scale=0.25)


@pytest.mark.parametrize("rows", [130, 9000])
def test_padding_and_tokens_outside(ar, rows):
    torch = _torch()
    rng = np.random.default_rng(3)
    vocab = 511                                              # vocab itself, the key of no part, needs a digit more
    values = rng.integers(-3, vocab + 3, rows)
    values[::7] = 5
    values[0], values[1] = 1 << 40, -(1 << 40)
    tokens = tokens_of([values])
    dys = rows_of(rng, 1, rows, 33, "bf16")
    dys[0][0] = math.nan                                     # a row outside spoils nothing
    check_backward(ar, dys, tokens, vocab, "bf16", "f32", padding=5)
    (table,) = rows_of(rng, 1, vocab, 33, "bf16")
    (out,) = ar.ar_embedding(tokens, [table])
    inside = (tokens[0] >= 0) & (tokens[0] < vocab)
    assert torch.isnan(out[~inside]).all() and torch.equal(out[inside], table[tokens[0][inside]])
    nobody = tokens_of([np.full(rows, -1)])
    check_backward(ar, dys, nobody, vocab, "bf16", "bf16")
    check_backward(ar, dys, tokens_of([np.full(rows, 5)]), vocab, "bf16", "bf16", padding=5)


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(90, 40), (9000, 17), (300, 2500)])
def test_accumulates(ar, dtype, wdtype, rows, cols):
    """Added to what is there; rows of other tokens are not touched, infinities and NaN among them."""
    torch = _torch()
    rng = np.random.default_rng(5)
    vocab = 100
    tokens = tokens_of([np.where(rng.random(rows) < 0.5, 7, rng.integers(0, 60, rows))])
    held = rows_of(rng, 1, vocab, cols, wdtype, 1)
    check_backward(ar, rows_of(rng, 1, rows, cols, dtype), tokens, vocab, dtype, wdtype, 2.0, held=held, pad=2)
    held[0][80], held[0][81] = math.inf, math.nan
    mine = held[0].clone()
    ar.ar_embedding_backward(rows_of(rng, 1, rows, cols, dtype), tokens, dtables=[mine], accumulate=True)
    assert torch.isinf(mine[80]).all() and torch.isnan(mine[81]).all()


def test_no_rows(ar):
    torch = _torch()
    none = tokens_of([[]])
    assert ar.ar_embedding(none, [torch.ones(4, 3, device="cuda")])[0].shape == (0, 3)
    dy = [torch.empty(0, 3, device="cuda")]
    mine = [torch.full((700, 3), math.nan, device="cuda")]
    ar.ar_embedding_backward(dy, none, dtables=mine)
    assert (mine[0] == 0).all()
    mine[0].fill_(2.0)
    ar.ar_embedding_backward(dy, none, dtables=mine, accumulate=True)
    assert (mine[0] == 2).all()
    assert ar.ar_embedding_backward(dy, none, 0)[0].shape == (0, 3)
    assert ar.ar_embedding_backward([torch.empty(2, 0, device="cuda")], tokens_of([[0, 1]]), 3)[0].shape == (3, 0)
    (out,) = ar.ar_embedding(tokens_of([[0, 1]]), [torch.empty(0, 3, device="cuda")])   # every token is outside
    assert torch.isnan(out).all()


@pytest.mark.parametrize("n", [1, 31, 33, 128])
def test_rank_counts(ar, n):
    rng = np.random.default_rng(n)
    tokens = tokens_of([rng.integers(0, 9, 40) for _ in range(n)])
    tables = rows_of(rng, n, 9, 20, "bf16")
    for o, t, w in zip(ar.ar_embedding(tokens, tables), tokens, tables):
        assert _torch().equal(o, w[t])
    check_backward(ar, rows_of(rng, n, 40, 20, "bf16"), tokens, 9, "bf16", "bf16")


def test_special_values(ar):
    """NaN and infinities reach their token's row only, and one table serves all ranks."""
    torch = _torch()
    dy = torch.ones(100, 70, device="cuda")
    dy[3, 5], dy[40, 6] = math.nan, math.inf
    tokens = torch.arange(100, device="cuda") % 10
    (g,) = ar.ar_embedding_backward([dy], [tokens], 10)
    want = torch.full((10, 70), 10.0, device="cuda")
    want[3, 5], want[0, 6] = math.nan, math.inf
    assert torch.equal(torch.isnan(g), torch.isnan(want)) and torch.equal(g.nan_to_num(1.0), want.nan_to_num(1.0))
    table = torch.randn(10, 70, device="cuda")
    a, b = ar.ar_embedding([tokens, tokens.flip(0)], [table, table])
    assert torch.equal(a, table[tokens]) and torch.equal(b, table[tokens.flip(0)])


@pytest.mark.parametrize("rows,cols", [(900, 100), (20000, 600)])
def test_same_bits_every_time(ar, rows, cols):
    torch = _torch()
    dy = torch.randn(rows, cols, device="cuda")
    tokens = (torch.rand(rows, device="cuda") ** 4 * 50).long()
    first = ar.ar_embedding_backward([dy], [tokens], 50)[0]
    for _ in range(4):
        assert torch.equal(ar.ar_embedding_backward([dy], [tokens], 50)[0], first)


def test_gradient_against_differences(ar):
    """The loss sum(dy * y) is linear in the table: a difference gives the gradient up to float32's rounding of y."""
    torch = _torch()
    rng = np.random.default_rng(6)
    tokens = tokens_of([rng.integers(0, 6, 30)])
    (table,), (dy,) = rows_of(rng, 1, 6, 8, "f32"), rows_of(rng, 1, 30, 8, "f32")
    (g,) = ar.ar_embedding_backward([dy], tokens, 6, scale=3.0)

    def loss(w):
        return float((dy.double() * ar.ar_embedding(tokens, [w], scale=3.0)[0].double()).sum())

    for at in [(0, 0), (3, 7), (5, 2)]:
        d = torch.zeros_like(table)
        d[at] = 0.5
        # each of 30 outputs of order 10 is off by 2^-24 of itself on either side: 30 * 10 * 2 * 2^-24 < 1e-4
        assert abs((loss(table + d) - loss(table - d)) - g[at].item()) < 1e-4


@pytest.mark.parametrize("rows", [400, 9000])
def test_captured_into_a_graph(ar, rows):
    torch = _torch()
    tokens = [torch.randint(0, 50, (rows,), device="cuda") for _ in range(2)]
    tables = [torch.randn(50, 70, device="cuda") for _ in range(2)]
    dys = [torch.randn(rows, 70, device="cuda") for _ in range(2)]
    ar.ar_embedding_backward(dys, tokens, 50)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = ar.ar_embedding(tokens, tables)
        grads = ar.ar_embedding_backward(dys, tokens, 50)
    for _ in range(4):
        for t in tokens:
            t.random_(0, 50)
        for t in tables + dys:
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = ar.ar_embedding(tokens, tables) + ar.ar_embedding_backward(dys, tokens, 50)
        assert all(torch.equal(a, b) for a, b in zip(outs + grads, want))


def test_on_another_stream(ar):
    torch = _torch()
    stream = torch.cuda.Stream()
    tokens = [torch.randint(0, 500, (20000,), device="cuda")]
    dys = [torch.randn(20000, 300, device="cuda")]
    stream.wait_stream(torch.cuda.current_stream())
    grads = ar.ar_embedding_backward(dys, tokens, 500, stream=stream)
    outs = ar.ar_embedding(tokens, grads, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    want = ar.ar_embedding_backward(dys, tokens, 500)
    assert torch.equal(grads[0], want[0]) and torch.equal(outs[0], want[0][tokens[0]])


def test_writes_are_counted(ar):
    torch = _torch()
    tokens = [torch.zeros(3, dtype=torch.int64, device="cuda")]
    out, grad = [torch.zeros(3, 4, device="cuda")], [torch.zeros(5, 4, device="cuda")]
    before = out[0]._version, grad[0]._version
    ar.ar_embedding(tokens, [torch.ones(5, 4, device="cuda")], out)
    ar.ar_embedding_backward(out, tokens, dtables=grad)
    assert out[0]._version > before[0] and grad[0]._version > before[1]


def test_refusals(ar):
    torch = _torch()
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)              # noqa: E731
    t = [torch.zeros(3, dtype=torch.int64, device="cuda")]
    w = [z(5, 8)]
    with pytest.raises(ValueError):
        ar.ar_embedding([], [])
    with pytest.raises(TypeError, match="tokens"):
        ar.ar_embedding([z(3)], w)
    with pytest.raises(ValueError, match="flat"):
        ar.ar_embedding([t[0].view(3, 1)], w)
    with pytest.raises(ValueError):
        ar.ar_embedding([t[0].cpu()], w)
    with pytest.raises(ValueError):
        ar.ar_embedding([torch.zeros(6, dtype=torch.int64, device="cuda")[::2]], w)
    with pytest.raises(ValueError):
        ar.ar_embedding(t * 2, w)
    with pytest.raises(ValueError, match="contiguous rows"):
        ar.ar_embedding(t, [z(8, 5).t()])
    with pytest.raises(TypeError):
        ar.ar_embedding(t, [z(5, 8, dtype=torch.bfloat16)], dtype=torch.float32)
    with pytest.raises(TypeError):
        ar.ar_embedding(t, w, dtype=torch.float64)
    with pytest.raises(ValueError):
        ar.ar_embedding(t, w, [z(4, 8)])
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_embedding(t, w, [w[0][:3]])
    for scale in (math.nan, math.inf, 1e-60, 1e39):
        with pytest.raises(ar.ArError, match="scale"):
            ar.ar_embedding(t, w, scale=scale)
    dy = [z(3, 8)]
    with pytest.raises(ValueError, match="vocab"):
        ar.ar_embedding_backward(dy, t)
    with pytest.raises(ValueError, match="rows, not"):
        ar.ar_embedding_backward(dy, t, 6, dtables=w)
    with pytest.raises(ValueError, match="accumulate"):
        ar.ar_embedding_backward(dy, t, 5, accumulate=True)
    with pytest.raises(ValueError, match="padding_index"):
        ar.ar_embedding_backward(dy, t, 5, padding_index=5)
    with pytest.raises(TypeError):
        ar.ar_embedding_backward(dy, t, 5, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ar.ar_embedding_backward(dy, [t[0][:2]], 5)
    with pytest.raises(ar.ArError, match="workspace"):
        ar.ar_embedding_backward(dy, t, 5, workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ar.ArError, match="overlaps"):
        ar.ar_embedding_backward(dy * 2, t * 2, dtables=w * 2)
    need = ar.ar_embedding_workspace_bytes(3, 5, 8, 1)
    odd = torch.zeros(need + 8, dtype=torch.uint8, device="cuda")[1:need + 1]
    with pytest.raises(ar.ArError, match="aligned"):
        ar.ar_embedding_backward(dy, t, 5, workspace=odd)


def test_most_tokens(ar):
    """2^31 - 1 places, the most: the sort's counts and every grid at their largest."""
    torch = _torch()
    rows, vocab = (1 << 31) - 1, 1024
    tokens = torch.arange(rows, dtype=torch.int32, device="cuda").remainder_(vocab)
    got = ar.ar_embedding_backward([torch.ones(rows, 1, device="cuda")], [tokens], vocab)[0]
    want = torch.full((vocab, 1), float(1 << 21), device="cuda")   # whole numbers below 2^24 throughout
    want[-1] -= 1
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [1 << 20, (1 << 22) + 8193 * 5 + 7])
def test_one_token_of_a_million_places(ar, rows):
    """All places of one token, with values whose partial sums are no whole numbers.

    The sums are of 32 places, 256 of those, 256 of those again and the rest: as many roundings one after another, of
    at most the whole sum (all terms are positive) each; the scale's product and the last sums add 4.  One chain of
    all of a million places' partial sums is off by thousands.
    """
    torch = _torch()
    values = torch.tensor([1 / (c + 3) for c in range(8)], device="cuda")
    dy = values.expand(rows, 8).contiguous()
    tokens = torch.full((rows,), 3, device="cuda")
    (got,) = ar.ar_embedding_backward([dy], [tokens], 5)
    want = values.double() * rows
    off = (32 + 256 + 256 + rows / 32 / 65536 + 4) * U32 * want
    assert ((got[3].double() - want).abs() <= off).all(), ((got[3].double() - want) / want / U32).tolist()
    assert (got[[0, 1, 2, 4]] == 0).all()


@pytest.mark.parametrize("n", [4, 5])
def test_bits_on_every_rank(ar, n):
    """4,096 places on each of 4 ranks, the most that are added in groups of 8, and of 5 (groups of 32): ranks with the
    same tokens and dy have the same bits, in every run; both groupings stay within the sum's roundings."""
    torch = _torch()
    rng = np.random.default_rng(7)
    tokens = tokens_of([(rng.random(4096) ** 3 * 60).astype(int)]) * n
    dys = rows_of(rng, 1, 4096, 40, "f32") * n
    outs = check_backward(ar, dys, tokens, 60, "f32", "f32", 1.5)
    again = ar.ar_embedding_backward(dys, tokens, 60, scale=1.5)
    assert all(torch.equal(o, outs[0]) for o in outs + again)
