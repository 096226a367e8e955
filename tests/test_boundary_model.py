"""The entry points of the model's ends without a GPU: every argument error is
reported before anything touches a device, empty work succeeds, workspaces
cover what the calls say they need, and the binding's constants are the
header's."""

import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000           # fake device addresses: only compared, never read
GAP = 1 << 36
INVALID = 1
F32, BF16, I32, F16 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from ring_allreduce_reduction_virtual_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return _lib.lib()


def ptrs(values):
    return None if values is None else (ctypes.c_void_p * max(len(values), 1))(*values)


def detail(lib):
    return lib.ar_get_last_error_detail().decode()


def buffers(start, n=2):
    return [BASE + (start + i) * GAP for i in range(n)]


WS = BASE + 90 * GAP
NONE = (1 << 64) - 1


def test_binding_matches_the_header():
    from ring_allreduce_reduction_virtual_amd import _lib as m

    text = open(os.path.join(ROOT, "include", "ar.h")).read()
    values = {k: int(v) for k, v in re.findall(r"\b(AR_[A-Z0-9_]+)\s*=\s*(\d+)", re.sub(r"/\*.*?\*/", "", text, flags=re.S))}
    assert {"i32": values["AR_INDEX_INT32"], "i64": values["AR_INDEX_INT64"]} == m.INDICES
    assert int(re.search(r"#define\s+AR_ACTIVATION_BLOCK\s+(\d+)", text).group(1)) == m.ACTIVATION_BLOCK


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def embed(lib, tokens=None, table=None, out=None, rows=10, vocab=20, cols=8, ts=8, os_=8, index=1, dt=F32, tdt=F32,
          scale=1.0, n=2, null=()):
    args = [buffers(0) if tokens is None else tokens, buffers(10) if table is None else table,
            buffers(20) if out is None else out]
    args = [None if k in null else ptrs(a) for k, a in enumerate(args)]
    return lib.ar_embedding(*args, rows, vocab, cols, ts, os_, index, dt, tdt, scale, n, None)


def test_embedding_errors(lib):
    assert embed(lib, dt=I32) == INVALID and "dtype" in detail(lib)
    assert embed(lib, dt=BF16, tdt=F16) == INVALID and embed(lib, dt=F32, tdt=BF16) == INVALID
    assert embed(lib, index=2) == INVALID and "index" in detail(lib)
    assert embed(lib, n=0) == INVALID and embed(lib, n=129) == INVALID and "nranks" in detail(lib)
    assert embed(lib, ts=7) == INVALID and "table_stride" in detail(lib)
    assert embed(lib, os_=7) == INVALID and "out_stride" in detail(lib)
    assert embed(lib, rows=1 << 31) == INVALID and embed(lib, vocab=1 << 31) == INVALID
    assert embed(lib, cols=1 << 23, ts=1 << 23, os_=1 << 23) == INVALID and "too large" in detail(lib)
    for scale in (math.nan, math.inf, -math.inf, 1e39, 1e-60):
        assert embed(lib, scale=scale) == INVALID and "scale" in detail(lib)
    for k in range(3):
        assert embed(lib, null=(k,)) == INVALID and "null" in detail(lib)
    assert embed(lib, tokens=[BASE, 0]) == INVALID and "tokens[1] is null" in detail(lib)
    assert embed(lib, tokens=[BASE + 4, BASE + GAP]) == INVALID and "aligned" in detail(lib)
    assert embed(lib, table=[BASE + 10 * GAP + 2, BASE + 11 * GAP]) == INVALID and "aligned" in detail(lib)
    assert embed(lib, out=buffers(10)) == INVALID and "overlaps" in detail(lib)
    assert embed(lib, out=[BASE + 20 * GAP] * 2) == INVALID and "overlaps" in detail(lib)
    assert embed(lib, rows=0) == 0 and embed(lib, cols=0, ts=0, os_=0) == 0


def embed_back(lib, dy=None, tokens=None, dtable=None, rows=10, vocab=20, cols=8, ds=8, ts=8, index=1, dt=F32, tdt=F32,
               scale=1.0, padding=-1, accumulate=0, n=2, ws=WS, have=None, null=()):
    args = [buffers(0) if dy is None else dy, buffers(10) if tokens is None else tokens,
            buffers(20) if dtable is None else dtable]
    args = [None if k in null else ptrs(a) for k, a in enumerate(args)]
    if have is None:
        have = lib.ar_embedding_workspace_bytes(rows, vocab, cols, n)
    return lib.ar_embedding_backward(*args, rows, vocab, cols, ds, ts, index, dt, tdt, scale, padding, accumulate, n, ws,
                                     have, None)


def test_embedding_backward_errors(lib):
    need = lib.ar_embedding_workspace_bytes(10, 20, 8, 2)
    assert 0 < need < 1 << 20
    assert embed_back(lib, have=need - 1) == INVALID and "workspace" in detail(lib)
    assert embed_back(lib, ws=None) == INVALID
    assert embed_back(lib, ws=WS + 2) == INVALID and "aligned" in detail(lib)
    assert embed_back(lib, ws=BASE) == INVALID and "overlaps" in detail(lib)
    assert embed_back(lib, dt=BF16, tdt=F16) == INVALID and embed_back(lib, dt=4) == INVALID
    assert embed_back(lib, ds=7) == INVALID and embed_back(lib, ts=7) == INVALID
    assert embed_back(lib, index=7) == INVALID and embed_back(lib, scale=math.nan) == INVALID
    for k in range(3):
        assert embed_back(lib, null=(k,)) == INVALID and "null" in detail(lib)
    assert embed_back(lib, dtable=buffers(0)) == INVALID and "overlaps" in detail(lib)
    assert embed_back(lib, dtable=[BASE + 20 * GAP] * 2) == INVALID and "overlaps" in detail(lib)
    assert embed_back(lib, vocab=0) == 0 and embed_back(lib, cols=0, ds=0, ts=0) == 0
    assert lib.ar_embedding_workspace_bytes(1 << 31, 5, 5, 1) == NONE
    assert lib.ar_embedding_workspace_bytes(5, 5, 5, 0) == NONE and lib.ar_embedding_workspace_bytes(5, 5, 5, 129) == NONE
    assert lib.ar_embedding_workspace_bytes(5, 5, 0, 1) == 0


@pytest.mark.parametrize("rows", [1, 8, 100, 8192, 8193, 100000])
@pytest.mark.parametrize("n", [1, 5, 128])
def test_embedding_workspace_holds_its_parts(lib, rows, n):
    """Keys and places twice, and two partial sums for every chunk of at most 32 places."""
    cols = 40
    least = n * (4 * rows + -(-rows // 32) * 2 * cols) * 4
    assert least <= lib.ar_embedding_workspace_bytes(rows, 1000, cols, n) <= 8 * least + n * 4 * 512 * (rows // 4096 + 1)


# --------------------------------------------------------------------------
# activations
# --------------------------------------------------------------------------

def test_pack_and_unpack_errors(lib):
    def pack(x=buffers(0), codes=buffers(10), scales=buffers(20), rows=5, cols=40, stride=40, dt=F32, n=2):
        return lib.ar_pack_activations(ptrs(x), ptrs(codes), ptrs(scales), rows, cols, stride, dt, n, None)

    def unpack(codes=buffers(10), scales=buffers(20), x=buffers(0), rows=5, cols=40, stride=40, dt=F32, n=2):
        return lib.ar_unpack_activations(ptrs(codes), ptrs(scales), ptrs(x), rows, cols, stride, dt, n, None)

    for call in (pack, unpack):
        assert call(dt=I32) == INVALID and "dtype" in detail(lib)
        assert call(n=0) == INVALID and call(n=129) == INVALID
        assert call(stride=39) == INVALID and "x_stride" in detail(lib)
        assert call(rows=1 << 41) == INVALID and call(cols=1 << 27, stride=1 << 27) == INVALID
        for name in ("x", "codes", "scales"):
            assert call(**{name: None}) == INVALID and "null" in detail(lib)
            assert call(**{name: [0, BASE]}) == INVALID and "is null" in detail(lib)
        assert call(x=[BASE + 2, BASE + GAP]) == INVALID and "aligned" in detail(lib)
        assert call(codes=buffers(0)) == INVALID and "overlaps" in detail(lib)
        assert call(rows=0) == 0 and call(cols=0, stride=0) == 0
    assert pack(scales=[BASE + 10 * GAP + 5 * 40 - 1, BASE + 21 * GAP]) == INVALID and "overlaps" in detail(lib)
    assert pack(codes=[BASE + 10 * GAP] * 2) == INVALID and unpack(x=[BASE] * 2) == INVALID


def test_layer_norm_backward_packed_errors(lib):
    need = lib.ar_layer_norm_workspace_bytes(5, 40, 2)

    def call(dy=buffers(0), codes=buffers(10), scales=buffers(20), gamma=None, mean=buffers(30), rstd=buffers(40),
             dx=buffers(50), dg=buffers(60), db=buffers(70), rows=5, cols=40, dys=40, dxs=40, dt=BF16, wdt=F32, n=2,
             ws=WS, have=need):
        return lib.ar_layer_norm_backward_packed(ptrs(dy), ptrs(codes), ptrs(scales), ptrs(gamma), ptrs(mean), ptrs(rstd),
                                                 ptrs(dx), ptrs(dg), ptrs(db), rows, cols, dys, dxs, dt, wdt, n, ws, have,
                                                 None)

    for name in ("dy", "codes", "scales", "mean", "rstd", "dx"):
        assert call(**{name: None}) == INVALID and "null" in detail(lib)
    assert call(dt=I32) == INVALID and call(dt=F32, wdt=BF16) == INVALID
    assert call(dys=39) == INVALID and call(dxs=39) == INVALID and call(n=0) == INVALID
    assert call(have=need - 1) == INVALID and "workspace" in detail(lib)
    assert call(dx=buffers(10)) == INVALID and "overlaps" in detail(lib)
    assert call(dg=[BASE + 20 * GAP, BASE + 61 * GAP]) == INVALID and "overlaps" in detail(lib)
    assert call(cols=0, dys=0, dxs=0) == 0 and call(rows=0, dg=None, db=None) == 0


# --------------------------------------------------------------------------
# cross entropy
# --------------------------------------------------------------------------

def cross(lib, x=buffers(0), w=buffers(10), t=buffers(20), loss=buffers(30), lse=buffers(40), rows=6, vocab=50, cols=16,
          xs=16, wst=16, index=1, ignore=-100, dt=BF16, n=2, ws=WS, have=None):
    if have is None:
        have = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 0)
    return lib.ar_cross_entropy(ptrs(x), ptrs(w), ptrs(t), ptrs(loss), ptrs(lse), rows, vocab, cols, xs, wst, index,
                                ignore, dt, n, ws, have, None)


def cross_back(lib, dl=buffers(60), x=buffers(0), w=buffers(10), t=buffers(20), lse=buffers(40), dx=buffers(70),
               dw=buffers(80), rows=6, vocab=50, cols=16, xs=16, wst=16, dxs=16, dws=16, index=1, ignore=-100, dt=BF16,
               scale=1.0, n=2, ws=WS, have=None):
    if have is None:
        have = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 1)
    return lib.ar_cross_entropy_backward(ptrs(dl), ptrs(x), ptrs(w), ptrs(t), ptrs(lse), ptrs(dx), ptrs(dw), rows, vocab,
                                         cols, xs, wst, dxs, dws, index, ignore, dt, scale, n, ws, have, None)


def test_cross_entropy_errors(lib):
    for call in (cross, cross_back):
        assert call(lib, dt=I32, have=1 << 40) == INVALID and "dtype" in detail(lib)
        assert call(lib, index=3) == INVALID and "index" in detail(lib)
        assert call(lib, n=0, have=1 << 40) == INVALID and call(lib, n=129, have=1 << 40) == INVALID
        assert call(lib, vocab=0, have=1 << 40) == INVALID and "vocabulary of 0" in detail(lib)
        assert call(lib, xs=15) == INVALID and "x_stride" in detail(lib)
        assert call(lib, wst=15) == INVALID and "weight_stride" in detail(lib)
        assert call(lib, rows=1 << 31, have=1 << 40) == INVALID and "too large" in detail(lib)
        assert call(lib, rows=1 << 30, vocab=1 << 22, have=1 << 60) == INVALID and "too large" in detail(lib)
        for name in ("x", "w", "t", "lse"):
            assert call(lib, **{name: None}) == INVALID and "null" in detail(lib)
            assert call(lib, **{name: [0, BASE + 5 * GAP]}) == INVALID and "is null" in detail(lib)
        assert call(lib, x=[BASE + 1, BASE + GAP]) == INVALID and "aligned" in detail(lib)
        assert call(lib, ws=WS + 8) == INVALID and "aligned" in detail(lib)
        assert call(lib, ws=None) == INVALID and call(lib, have=16) == INVALID and "workspace" in detail(lib)
        assert call(lib, ws=BASE) == INVALID and "overlaps" in detail(lib)
    assert cross(lib, loss=None) == INVALID and cross(lib, loss=buffers(40)) == INVALID and "overlaps" in detail(lib)
    assert cross(lib, rows=0) == 0
    for scale in (math.nan, math.inf, 1e39, 1e-60):
        assert cross_back(lib, scale=scale) == INVALID and "scale" in detail(lib)
    assert cross_back(lib, dxs=15) == INVALID and cross_back(lib, dws=15) == INVALID
    assert cross_back(lib, dw=buffers(10)) == INVALID and "overlaps" in detail(lib)
    assert cross_back(lib, dx=buffers(0), dxs=32) == INVALID and "overlaps" in detail(lib)
    assert cross_back(lib, dl=[BASE + 2, BASE + GAP]) == INVALID and "aligned" in detail(lib)
    # nothing wanted, or nothing to do
    assert cross_back(lib, dx=None, dw=None) == 0 and cross_back(lib, rows=0, dw=None) == 0
    assert cross_back(lib, cols=0, xs=0, wst=0, dxs=0, dws=0) == 0


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 1), (16, 8192, 1024), (129, 5003, 515), (8192, 65536, 4096),
                                             (4096, 131072, 8192), (131072, 50257, 768), (3, 1 << 22, 64)])
def test_cross_entropy_workspaces(lib, dt, rows, vocab, cols):
    """The backward pass never needs memory for the logits: a piece of them, at most half a GiB or 2,048
    columns, beside copies and float32 sums of x's size."""
    es = 4 if dt == F32 else 2
    for n in (1, 4, 33):
        ranks = min(n, 32)
        forward = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 0)
        back = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 1)
        piece = max(512 << 20, ranks * rows * 2048 * es)
        width = cols + 8
        # x's copy, a piece of the weight's (no wider than the vocabulary or dz's bound), and 64 splits of dx at most
        copies = ranks * (rows + min(vocab + 256, piece // (ranks * rows * es) + 256)) * width * es
        assert 0 < forward <= copies + ranks * rows * (vocab // 64 + 3) * 8 + 8192
        assert back <= piece + ranks * 256 * rows * es + copies + ranks * rows * (64 * width * 4 + 64) + 16384
    assert lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, I32, 1, 0) == NONE
    assert lib.ar_cross_entropy_workspace_bytes(rows, 0, cols, dt, 1, 1) == NONE


def test_cross_entropy_launches_fit(lib):
    """More rows than one launch's threads can be counted for are refused before anything is launched."""
    for backward in (0, 1):
        assert lib.ar_cross_entropy_workspace_bytes(1 << 28, 64, 8, BF16, 1, backward) not in (0, NONE)
        assert lib.ar_cross_entropy_workspace_bytes((1 << 28) + 1, 64, 8, BF16, 1, backward) == NONE
        assert lib.ar_cross_entropy_workspace_bytes(1 << 29, 64, 8, BF16, 1, backward) == NONE


def test_cross_entropy_sizes_that_always_fit(lib):
    """2^25 rows, 2^36 rows x columns and 2^36 vocabulary x columns of all ranks together, the largest that each
    shape has room for, in every tile's odd sizes: neither pass refuses any.  The forward pass's own limit is 2^28 rows,
    whatever the columns are (its launches are cut)."""
    import random

    rng = random.Random(0)
    cases = [(32, 1, 4_000_000, 513), (32, 129, 8_000_000, 4), (1, 129, 240_000_000, 4), (1, 1, (1 << 27) - 5, 513),
             (1, 1 << 25, 100, 2048), (32, 1 << 20, 1, 1), (1, 1 << 25, (1 << 31) - 1, 1), (128, 1, 513, 1 << 20)]
    edges = [1, 2, 31, 33, 64, 65, 129, 160, 161, 192, 193, 257, 320, 385, 513, 640, 769, 1025]
    for _ in range(4000):
        n = rng.choice((1, 2, 5, 31, 32, 33, 128))
        some = lambda most: min(most, rng.choice((rng.choice(edges), int(2 ** rng.uniform(0, 31)), most)))   # noqa: E731
        cols = some(min(1 << 20, (1 << 36) // n))
        rows = some(min((1 << 25) // n, (1 << 36) // (n * cols)))
        vocab = some(min((1 << 31) - 1, (1 << 36) // (n * cols)))
        cases.append((n, rows, vocab, cols))
    for n, rows, vocab, cols in cases:
        for dt in (F32, BF16, F16):
            for backward in (0, 1):
                got = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, backward)
                assert got != NONE, (n, rows, vocab, cols, dt, backward)
    for dt in (F32, BF16):
        for n, rows in ((1, 1 << 28), (32, 1 << 23)):
            assert lib.ar_cross_entropy_workspace_bytes(rows, (1 << 31) - 1, 16, dt, n, 0) != NONE


def needed(lib):
    """What the last error said that the call needs."""
    said = re.search(r"needs a workspace of (\d+) bytes", detail(lib))
    assert said, detail(lib)
    return int(said.group(1))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,vocab,cols", [(1, 1, 8), (16, 65536, 4096), (129, 5003, 520), (4096, 65536, 4096),
                                             (4096, 131072, 8192), (131072, 50257, 768), (3, 1 << 22, 64)])
@pytest.mark.parametrize("n", [1, 8, 33])
def test_cross_entropy_workspace_without_copies(lib, dt, rows, vocab, cols, n):
    """Operands on 16 bytes need room for no copy: forward for 8 bytes per row and 64 words (4 per row beside), backward
    for x's rows, dz's piece and dx's sums; and a call asks for just that."""
    es, ranks = 4 if dt == F32 else 2, min(n, 32)
    forward = lib.ar_cross_entropy_aligned_workspace_bytes(rows, vocab, cols, dt, n, 0)
    back = lib.ar_cross_entropy_aligned_workspace_bytes(rows, vocab, cols, dt, n, 1)
    assert 0 < forward <= ranks * rows * (-(-vocab // 64) * 8 + 4) + 512
    piece = max(512 << 20, ranks * rows * 2048 * es)
    dz = min(piece, ranks * rows * vocab * es) + ranks * rows * 256 * es
    splits = 64 if rows <= 256 else 8
    assert 0 < back <= dz + ranks * rows * (cols * es + splits * cols * 4 + 64) + 2048
    spans = [BASE + k * (GAP << 4) for k in range(8 * n)]                # 1 TiB apart
    ptr = lambda k: spans[k * n:(k + 1) * n]                             # noqa: E731
    ws = BASE - (GAP << 4)
    for x, w, aligned, aligned_back in ((0, 0, True, True), (es, 0, False, True), (0, es, False, False)):
        xs, wst = cols + (8 if x == 0 else 1), cols
        at = dict(x=[p + x for p in ptr(0)], w=[p + w for p in ptr(1)], t=ptr(2), lse=ptr(3), rows=rows, vocab=vocab,
                  cols=cols, xs=xs, wst=wst, dt=dt, n=n, ws=ws, have=15)
        assert cross(lib, loss=ptr(4), **at) == INVALID
        need = needed(lib)
        any_operands = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 0)
        assert forward <= any_operands and (need == forward if aligned else forward <= need <= any_operands)
        assert cross_back(lib, dl=ptr(5), dx=ptr(6), dw=ptr(7), dxs=cols, dws=cols, **at) == INVALID
        need = needed(lib)
        any_operands = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 1)
        assert back <= any_operands and (need == back if aligned_back else 0 < need <= any_operands)
    # rows that are no whole 16 bytes need copies wherever they lie
    assert (lib.ar_cross_entropy_aligned_workspace_bytes(rows, vocab, cols + 1, dt, n, 0)
            == lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols + 1, dt, n, 0))
    assert lib.ar_cross_entropy_aligned_workspace_bytes(rows, 0, cols, dt, n, 1) == NONE


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,rows,vocab,cols", [(1, 80, 131072, 4095), (8, 80, 131072, 8191), (32, 100, 131072, 8191),
                                               (2, 4096, 65536, 4095), (1, 4096, 1 << 22, 2047), (33, 70, 1 << 20, 1023)])
def test_cross_entropy_copies_are_bounded(lib, dt, n, rows, vocab, cols):
    """Of a weight that is copied a piece is held at a time: 128 MiB of all ranks (backward 256, or 2,048 rows of each),
    or what gives 256 compute units a tile of at most 256 rows; x is copied whole."""
    es, ranks = 4 if dt == F32 else 2, min(n, 32)
    row = -(-cols * es // 16) * 16
    turn = 256 * (256 + ranks) * row
    forward = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 0)
    back = lib.ar_cross_entropy_workspace_bytes(rows, vocab, cols, dt, n, 1)
    assert forward <= ranks * rows * (row + -(-vocab // 64) * 8 + 4) + max(128 << 20, turn) + ranks * 256 * row + 4096
    dz = min(max(512 << 20, ranks * rows * 2048 * es), ranks * rows * (vocab + 256) * es) + ranks * rows * 256 * es
    weight = max(256 << 20, turn, ranks * 2048 * row) + ranks * 256 * row
    assert back <= dz + weight + ranks * rows * (row + 64 * (cols + 4) * 4 + 64) + 4096
