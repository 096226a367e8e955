"""Python binding of the operators at a model's ends (include/ar.h): the embedding with its gradient, the
cross entropy of unstored logits with its gradients, and activations in 8 bits.

Argument marshalling only, in the manner of the training-step operators: one
tensor per virtual rank in each sequence, checks of device, type and shape,
one call into the library.  Autograd records none of these functions; what a
call writes into counts as changed in place.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib
from .binding import _on_device, _stream_handle, _ws
from .step import (_array, _dtype_of, _fast, _first, _FLOATS, _new_parts, _norm_backward, _pointers, _rank_list,
                   _row_pointers, _scratch, _second_half, _written)

_INDICES = {torch.int32: "i32", torch.int64: "i64"}


def _index_list(tensors, what):
    """The first of the ranks' tokens or targets, and the C name of their type."""
    t = _first(tensors, what)
    name = _INDICES.get(t.dtype)
    if name is None:
        raise TypeError(f"unsupported {what} dtype {t.dtype}; use int32 or int64")
    if t.dim() != 1:
        raise ValueError(f"{what} must be flat tensors, one per rank")
    if len(tensors) > _lib.MAX_RANKS:
        raise ValueError(f"nranks must be in [1, {_lib.MAX_RANKS}]")
    return t, _lib.INDICES[name]


def _per_rank(tensors, n, what):
    if len(tensors) != n:
        raise ValueError(f"need one of {what} per rank")


def _out_rows(outs, shape, n, dt, dev, index, what, stream):
    """One [rows, cols] output per rank, made if not given: the tensors, their addresses and row stride."""
    if outs is None:
        parts, ptrs = _new_parts((n, *shape), dt, dev, stream)
        return parts, ptrs, shape[1]
    return (outs, *_row_pointers(outs, n, dev, index, dt, *shape, what))


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------

def ar_embedding(tokens, tables, outs=None, scale: float = 1.0, dtype=None, stream=None):
    """Rows of every rank's table by its tokens, times `scale`; one [rows, cols] tensor per rank.

    `tokens` are flat int32 or int64 tensors, `tables` [vocab, cols].  The
    output's type is that of `outs`, else `dtype`, else the tables'; a float32
    table gives any, a 16-bit one its own.  A token outside [0, vocab) gives a
    row of NaN.
    """
    t0, index_type = _index_list(tokens, "tokens")
    w0 = _rank_list(tables, "tables")
    n, rows = len(tokens), t0.numel()
    dev, index = w0.device, w0.get_device()
    vocab, cols = w0.shape
    tp = _pointers(tokens, dev, index, t0.dtype, [rows] * n, "tokens")
    wp, table_stride = _row_pointers(tables, n, dev, index, w0.dtype, vocab, cols, "tables")
    table_type = _lib.DTYPES[_dtype_of(w0, "tables")]
    dt = outs[0].dtype if outs is not None and len(outs) and isinstance(outs[0], torch.Tensor) else dtype or w0.dtype
    if dt not in _FLOATS or (dt is not w0.dtype and w0.dtype is not torch.float32):
        raise TypeError(f"tables in {w0.dtype} give no rows in {dt}")
    given = outs
    outs, op, out_stride = _out_rows(outs, (rows, cols), n, dt, dev, index, "outs", stream)
    with _on_device(dev):
        rc = _lib.lib().ar_embedding(tp, wp, op, rows, vocab, cols, table_stride, out_stride, index_type,
                                     _lib.DTYPES[_FLOATS[dt]], table_type, scale, n, _stream_handle(stream, dev.index))
    _lib.check("ar_embedding", rc)
    _written(given)
    return outs


def ar_embedding_workspace_bytes(rows: int, vocab: int, cols: int, nranks: int) -> int:
    v = _lib.lib().ar_embedding_workspace_bytes(rows, vocab, cols, nranks)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("invalid arguments for ar_embedding_workspace_bytes")
    return v


def ar_embedding_backward(dys, tokens, vocab=None, dtables=None, scale: float = 1.0, padding_index=None,
                          accumulate: bool = False, dtype=None, workspace=None, stream=None):
    """The tables' gradients, one [vocab, cols] tensor per rank: `scale` times each token's sum of rows of `dys`.

    `vocab` is needed unless `dtables` are given, whose type then counts
    (`dtype`, else that of `dys`).  With ``accumulate=True`` the sums are added
    to what `dtables` hold, and rows of other tokens are left alone, as where
    the table is also the head's weight.  `padding_index` takes no part.
    """
    dy0 = _rank_list(dys, "dys")
    t0, index_type = _index_list(tokens, "tokens")
    n, dev, index = len(dys), dy0.device, dy0.get_device()
    rows, cols = dy0.shape
    dyp, dy_stride = _row_pointers(dys, n, dev, index, dy0.dtype, rows, cols, "dys")
    tp = _pointers(tokens, dev, index, t0.dtype, [rows] * n, "tokens")
    name = _dtype_of(dy0, "dys")
    if dtables is None:
        if vocab is None or accumulate:
            raise ValueError("pass dtables to accumulate into" if accumulate else "pass vocab or dtables")
        wdt = dtype or dy0.dtype
    else:
        w0 = _rank_list(dtables, "dtables")
        if vocab is not None and vocab != w0.shape[0]:
            raise ValueError(f"dtables have {w0.shape[0]} rows, not {vocab}")
        vocab, wdt = w0.shape[0], w0.dtype
    if wdt is not dy0.dtype and wdt is not torch.float32:
        raise TypeError("the tables' gradients have the type of dys or float32")
    if padding_index is not None and not 0 <= padding_index < vocab:
        raise ValueError(f"padding_index must be in [0, {vocab})")
    given = dtables
    with _on_device(dev):
        workspace = _scratch(ar_embedding_workspace_bytes(rows, vocab, cols, n), workspace, dev, stream)
        dtables, wp, dtable_stride = _out_rows(dtables, (vocab, cols), n, wdt, dev, index, "dtables", stream)
        sp, sb = _ws(workspace, dev)
        rc = _lib.lib().ar_embedding_backward(dyp, tp, wp, rows, vocab, cols, dy_stride, dtable_stride, index_type,
                                              _lib.DTYPES[name], _lib.DTYPES[_FLOATS[wdt]], scale,
                                              -1 if padding_index is None else padding_index, 1 if accumulate else 0,
                                              n, sp, sb, _stream_handle(stream, dev.index))
    _lib.check("ar_embedding_backward", rc)
    _written(given)
    return dtables


# --------------------------------------------------------------------------
# cross entropy
# --------------------------------------------------------------------------

def _cross_entropy_bytes(call, rows, vocab, cols, dtype, nranks, backward):
    v = getattr(_lib.lib(), call)(rows, vocab, cols, _lib.DTYPES[dtype], nranks, 1 if backward else 0)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError(f"invalid arguments for {call}: " + _lib.lib().ar_get_last_error_detail().decode())
    return v


def ar_cross_entropy_workspace_bytes(rows: int, vocab: int, cols: int, dtype: str, nranks: int,
                                     backward: bool = False) -> int:
    """Enough for any operands."""
    return _cross_entropy_bytes("ar_cross_entropy_workspace_bytes", rows, vocab, cols, dtype, nranks, backward)


def ar_cross_entropy_aligned_workspace_bytes(rows: int, vocab: int, cols: int, dtype: str, nranks: int,
                                             backward: bool = False) -> int:
    """What operands need whose rows lie on 16 bytes (include/ar.h), so that none is copied."""
    return _cross_entropy_bytes("ar_cross_entropy_aligned_workspace_bytes", rows, vocab, cols, dtype, nranks, backward)


def _cross_entropy_scratch(shape, name, n, backward, aligned, dev, stream):
    need = ar_cross_entropy_aligned_workspace_bytes if aligned else ar_cross_entropy_workspace_bytes
    return _scratch(need(*shape, name, n, backward), None, dev, stream)


def _aligned(addresses, n, stride, cols, es):
    """Whether the ranks' operands need no copy: rows on 16 bytes, of whole 16 bytes and at most 8 MiB apart."""
    if (stride * es | cols * es) & 15 or stride * es > 1 << 23:
        return False
    for a in addresses[:n]:
        if a and a & 15:
            return False
    return True


def _flat_floats(tensors, n, dev, index, rows, what):
    """Addresses of one float32 tensor of `rows` elements per rank."""
    _per_rank(tensors, n, what)
    return _pointers(tensors, dev, index, torch.float32, [rows] * n, what)


def _cross_inputs(xs, weights, targets):
    """What both passes read: (first x, dev, index, (rows, vocab, cols), addresses, strides, index type)."""
    x0 = _rank_list(xs, "xs")
    w0 = _rank_list(weights, "weights")
    t0, index_type = _index_list(targets, "targets")
    n, dev, index = len(xs), x0.device, x0.get_device()
    _dtype_of(x0, "xs")
    (rows, cols), vocab = x0.shape, w0.shape[0]
    xp, x_stride = _row_pointers(xs, n, dev, index, x0.dtype, rows, cols, "xs")
    wp, w_stride = _row_pointers(weights, n, dev, index, x0.dtype, vocab, cols, "weights")
    tp = _pointers(targets, dev, index, t0.dtype, [rows] * n, "targets")
    _per_rank(targets, n, "targets")
    return x0, n, dev, index, (rows, vocab, cols), (xp, wp, tp), (x_stride, w_stride), index_type


def ar_cross_entropy(xs, weights, targets, losses=None, lses=None, ignore_index: int = -100, workspace=None,
                     stream=None):
    """Softmax cross entropy of every rank's logits ``x @ weight.t()``, which are never stored.

    `xs` are [rows, cols], `weights` [vocab, cols] of the same type, `targets`
    flat int32 or int64 tensors.  Returns (losses, lses): each row's loss (0
    where the target is `ignore_index`, NaN where it is outside the
    vocabulary) and the logarithm of its sum of exponentials, which
    :func:`ar_cross_entropy_backward` takes; float32, one tensor per rank in
    each.
    """
    x0, n, dev, index, shape, inputs, strides, index_type = _cross_inputs(xs, weights, targets)
    rows = shape[0]
    name = _FLOATS[x0.dtype]
    given = (losses, lses)
    if losses is None and lses is None:
        both, lp = _new_parts((2 * n, rows), torch.float32, dev, stream)
        losses, lses, sp = both[:n], both[n:], _second_half(lp, n)
    else:
        made = [None, None] if all(g is not None for g in given) else _new_parts((n, rows), torch.float32, dev, stream)
        losses, lp = made if losses is None else (losses, _flat_floats(losses, n, dev, index, rows, "losses"))
        lses, sp = made if lses is None else (lses, _flat_floats(lses, n, dev, index, rows, "lses"))
    if workspace is None:
        es = x0.element_size()
        aligned = (_aligned(inputs[0], n, strides[0], shape[2], es) and _aligned(inputs[1], n, strides[1], shape[2], es))
        workspace = _cross_entropy_scratch(shape, name, n, False, aligned, dev, stream)
    with _on_device(dev):
        wp, wb = _ws(workspace, dev)
        rc = _lib.lib().ar_cross_entropy(*inputs, lp, sp, *shape, *strides, index_type, ignore_index,
                                         _lib.DTYPES[name], n, wp, wb, _stream_handle(stream, dev.index))
    _lib.check("ar_cross_entropy", rc)
    _written(*given)
    return losses, lses


def ar_cross_entropy_backward(dlosses, xs, weights, targets, lses, dxs=None, dweights=None, input_grads: bool = True,
                              weight_grads: bool = True, ignore_index: int = -100, scale: float = 1.0, workspace=None,
                              stream=None):
    """Gradients of :func:`ar_cross_entropy`; returns (dxs, dweights), one tensor per rank in each.

    Row i's loss counts `scale` times ``dlosses[r][i]`` (None: 1).  Tensors may
    be passed for the results (a rank's slice of its gradient bucket); with
    ``input_grads=False`` or ``weight_grads=False`` those not passed are not
    made.  In place: ``dxs=xs``.
    """
    x0, n, dev, index, shape, inputs, strides, index_type = _cross_inputs(xs, weights, targets)
    rows, vocab, cols = shape
    dt, name = x0.dtype, _FLOATS[x0.dtype]
    sp = _flat_floats(lses, n, dev, index, rows, "lses")
    dp = None if dlosses is None else _flat_floats(dlosses, n, dev, index, rows, "dlosses")
    given = (dxs, dweights)
    gx = gw = None
    x_stride = w_stride = cols
    if dxs is not None or input_grads:
        dxs, gx, x_stride = _out_rows(dxs, (rows, cols), n, dt, dev, index, "dxs", stream)
    if dweights is not None or weight_grads:
        dweights, gw, w_stride = _out_rows(dweights, (vocab, cols), n, dt, dev, index, "dweights", stream)
    if workspace is None:
        aligned = _aligned(inputs[1], n, strides[1], cols, x0.element_size())
        workspace = _cross_entropy_scratch(shape, name, n, True, aligned, dev, stream)
    with _on_device(dev):
        wp, wb = _ws(workspace, dev)
        rc = _lib.lib().ar_cross_entropy_backward(dp, *inputs, sp, gx, gw, *shape, *strides, x_stride, w_stride,
                                                  index_type, ignore_index, _lib.DTYPES[name], scale, n, wp, wb,
                                                  _stream_handle(stream, dev.index))
    _lib.check("ar_cross_entropy_backward", rc)
    _written(*given)
    return dxs, dweights


# --------------------------------------------------------------------------
# activations in 8 bits
# --------------------------------------------------------------------------

class PackedRows(NamedTuple):
    """One rank's activations in 8 bits: an int8 code per element [rows, cols], a scale byte per 32 of a row (uint8)."""

    codes: torch.Tensor
    scales: torch.Tensor

    @classmethod
    def empty(cls, rows: int, cols: int, device) -> "PackedRows":
        """Memory for `rows` x `cols` activations, to pack into."""
        return cls(torch.empty(rows, cols, dtype=torch.int8, device=device),
                   torch.empty(rows, -(-cols // _lib.ACTIVATION_BLOCK), dtype=torch.uint8, device=device))


def _packed_rows(packed, n, dev, index, rows, cols, what):
    """Addresses of the ranks' codes and scales."""
    _per_rank(packed, n, what)
    if not all(isinstance(p, (tuple, list)) and len(p) == 2 for p in packed):
        raise ValueError(f"{what} must be PackedRows pairs of codes and scales")
    blocks = -(-cols // _lib.ACTIVATION_BLOCK)
    got = []
    for k, (part, dt, width) in enumerate((("codes", torch.int8, cols), ("scales", torch.uint8, blocks))):
        tensors = [p[k] for p in packed]
        fast = _fast and _fast.rows(tensors, dt, index, rows, width)
        if fast is not None and fast[1] == width:
            got.append(_array(fast[0]))
            continue
        got.append(_pointers(tensors, dev, index, dt, [rows * width] * n, f"the {part} of {what}"))
        if any(t.shape != (rows, width) for t in tensors):
            raise ValueError(f"the {part} of {what} must be [{rows}, {width}] tensors")
    return got


def _first_packed(packed):
    """The codes of the first rank's packed rows."""
    p = packed[0] if len(packed) else None
    if not isinstance(p, (tuple, list)) or len(p) != 2:
        raise ValueError("packed must be a non-empty sequence of PackedRows")
    c = _first([p[0]], "the codes of packed")
    if c.dim() != 2:
        raise ValueError("the codes of packed must be [rows, cols] tensors, one per rank")
    if len(packed) > _lib.MAX_RANKS:
        raise ValueError(f"nranks must be in [1, {_lib.MAX_RANKS}]")
    return c


def ar_pack_activations(xs, outs=None, stream=None):
    """Every rank's [rows, cols] activations in 8 bits, one :class:`PackedRows` per rank (`outs`, made if not given)."""
    x0 = _rank_list(xs, "xs")
    n, dev, index = len(xs), x0.device, x0.get_device()
    name = _dtype_of(x0, "xs")
    rows, cols = x0.shape
    xp, x_stride = _row_pointers(xs, n, dev, index, x0.dtype, rows, cols, "xs")
    given = outs
    if outs is None:
        codes, cp = _new_parts((n, rows, cols), torch.int8, dev, stream)
        scales, sp = _new_parts((n, rows, -(-cols // _lib.ACTIVATION_BLOCK)), torch.uint8, dev, stream)
        outs = [PackedRows(c, s) for c, s in zip(codes, scales)]
    else:
        cp, sp = _packed_rows(outs, n, dev, index, rows, cols, "outs")
    with _on_device(dev):
        rc = _lib.lib().ar_pack_activations(xp, cp, sp, rows, cols, x_stride, _lib.DTYPES[name], n,
                                            _stream_handle(stream, dev.index))
    _lib.check("ar_pack_activations", rc)
    _written(given)
    return outs


def ar_unpack_activations(packed, outs=None, dtype=torch.float32, stream=None):
    """The values of packed activations, one [rows, cols] tensor per rank (`outs`, or made in `dtype`)."""
    c0 = _first_packed(packed)
    n, dev, index = len(packed), c0.device, c0.get_device()
    rows, cols = c0.shape
    cp, sp = _packed_rows(packed, n, dev, index, rows, cols, "packed")
    given = outs
    dt = dtype if outs is None else _rank_list(outs, "outs").dtype
    if dt not in _FLOATS:
        raise TypeError(f"unsupported outs dtype {dt}; use float32, bfloat16 or float16")
    outs, op, stride = _out_rows(outs, (rows, cols), n, dt, dev, index, "outs", stream)
    with _on_device(dev):
        rc = _lib.lib().ar_unpack_activations(cp, sp, op, rows, cols, stride, _lib.DTYPES[_FLOATS[dt]], n,
                                              _stream_handle(stream, dev.index))
    _lib.check("ar_unpack_activations", rc)
    _written(given)
    return outs


def ar_layer_norm_backward_packed(dys, packed, gammas, means, rstds, dxs=None, weight_grads: bool = True,
                                  dgammas=None, dbetas=None, workspace=None, stream=None):
    """:func:`ar_layer_norm_backward` with the forward pass's input kept by :func:`ar_pack_activations`.

    The statistics are the forward pass's own, of the input as it was.
    """
    dy0 = _rank_list(dys, "dys")
    _dtype_of(dy0, "dys")
    inputs = _packed_rows(packed, len(dys), dy0.device, dy0.get_device(), *dy0.shape, "packed")
    return _norm_backward("ar_layer_norm_backward_packed", inputs, (), dy0, len(dys), dys, gammas, means, rstds, dxs,
                          weight_grads, dgammas, dbetas, workspace, stream)
