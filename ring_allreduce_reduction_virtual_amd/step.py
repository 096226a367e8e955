"""Python binding of the training-step operators of include/ar.h, taking torch tensors.

Argument marshalling only, as in the collectives' binding: each function
checks the tensors (same CUDA device, contiguous where the operator needs it,
matching dtypes and sizes), collects their addresses and the stream handle,
and makes one call into the library.

The optimizer's functions take one sequence per role with one tensor per
entry: ``params``, ``grads``, ``exp_avgs``, ``exp_avg_sqs``.  ``out``, when
given, is ``(params, exp_avgs, exp_avg_sqs)`` to write beside the inputs;
without it the step updates them in place.  ``copies`` receives the new
float32 parameters rounded to its 16-bit type.  The layer norm functions take
one tensor per virtual rank, as the collectives do.

Tensors the functions make themselves come from torch's allocator, in the
memory of the stream that the work is enqueued on, as if the call were made
under ``torch.cuda.stream(stream)``.

Autograd records none of these functions: their outputs require no gradient.
What a call or a plan's start writes into counts as changed in place (the
tensor's version), so that a backward pass which still needs the old values
raises; the replays of a HIP graph count nothing.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib
from .binding import _on_device, _stream_handle, _ws

try:
    from . import _armarshal as _fast   # csrc/ar_marshal.cpp: the same checks in one native pass
except ImportError:
    _fast = None

_FLOATS = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


class PackedState(NamedTuple):
    """One tensor's state in 8 bits: a code per element, a scale byte per 256 elements (both uint8)."""

    codes: torch.Tensor
    scales: torch.Tensor

    @classmethod
    def zeros(cls, numel: int, device) -> "PackedState":
        """A state of zeros for a tensor of `numel` elements."""
        blocks = -(-int(numel) // _lib.STATE_BLOCK)
        return cls(torch.zeros(numel, dtype=torch.uint8, device=device),
                   torch.zeros(blocks, dtype=torch.uint8, device=device))


def _dtype_of(t, what):
    name = _FLOATS.get(t.dtype)
    if name is None:
        raise TypeError(f"unsupported {what} dtype {t.dtype}; use float32, bfloat16 or float16")
    return name


def _array(addresses: bytes):
    """A ctypes array of addresses packed as bytes."""
    n = len(addresses) // ctypes.sizeof(ctypes.c_void_p)
    return (ctypes.c_void_p * n).from_buffer_copy(addresses) if n else (ctypes.c_void_p * 1)()


def _pointers(tensors, dev, index, dtype, counts, what):
    """Addresses of contiguous tensors on `dev` of one dtype and the given element counts (a list; None: any)."""
    n = len(tensors)
    if counts is not None and len(counts) != n:
        raise ValueError(f"need one of {what} per tensor")
    fast = _fast and _fast.pointers(tensors, dtype, index, counts)
    if fast is not None:
        return _array(fast)
    for i, t in enumerate(tensors):
        _refuse(t, dev, index, dtype, None if counts is None else counts[i], what, i)
    return (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in tensors])


def _refuse(t, dev, index, dtype, count, what, i):
    """Raise what is wrong with a tensor, if anything is (a subclass of torch.Tensor may be as good)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{what} must be tensors on {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must have one dtype, {dtype}")
    if not t.is_contiguous() or t.is_neg():
        raise ValueError(f"{what} must be contiguous, and no negative views")
    if count is not None and t.numel() != count:
        raise ValueError(f"{what}[{i}] must hold {count} elements")


def _written(*groups):
    """Count a write into every tensor of the sequences (of tensors or packed states; None: none)."""
    for group in groups:
        if group is None or (_fast and _fast.written(group)):
            continue
        for item in group:
            for t in (item,) if isinstance(item, torch.Tensor) else item:
                if not t.is_inference():
                    torch.autograd.graph.increment_version(t)


def _counts(sizes):
    return (ctypes.c_size_t * max(len(sizes), 1))(*sizes)


def _first(tensors, what):
    t = tensors[0] if len(tensors) else None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a non-empty sequence of CUDA tensors")
    return t


def _empty(shape, dtype, dev, stream):
    """A new tensor for work on `stream` (None: the current one), from that stream's own memory: what the
    allocator hands out on another stream may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        raise ValueError("pass every output and the workspace when the stream is a raw handle")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _scratch(need, workspace, dev, stream):
    return _empty(need, torch.uint8, dev, stream) if need and workspace is None else workspace


def _scalar(t, dev, what):
    """Address of a one-element float32 tensor on `dev`."""
    if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype is not torch.float32 or t.numel() != 1:
        raise ValueError(f"{what} must be a float32 tensor of one element on {dev}")
    if t.is_neg():
        raise ValueError(f"{what} must be no negative view")
    return t.data_ptr()


def ar_update_workspace_bytes(kind: str, counts) -> int:
    """Workspace of ar_grad_norm and of the plans ("grad_norm", "adamw" or "adamw_packed")."""
    counts = list(counts)
    if any(c < 0 for c in counts):
        raise ValueError("invalid arguments for ar_update_workspace_bytes")
    v = _lib.lib().ar_update_workspace_bytes(_lib.UPDATES[kind], _counts(counts), len(counts))
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("invalid arguments for ar_update_workspace_bytes")
    return v


# --------------------------------------------------------------------------
# gradient norm
# --------------------------------------------------------------------------

def _norm_call(grads, norm, workspace, stream):
    g0 = _first(grads, "grads")
    dev = g0.device
    sizes = [g.numel() for g in grads]
    gp = _pointers(grads, dev, g0.get_device(), g0.dtype, None, "grads")
    dtype = _lib.DTYPES[_dtype_of(g0, "grads")]
    if norm is None:
        norm = _empty(1, torch.float32, dev, stream)
    workspace = _scratch(ar_update_workspace_bytes("grad_norm", sizes), workspace, dev, stream)
    wp, wb = _ws(workspace, dev)
    return dev, (gp, _counts(sizes), len(sizes), dtype, _scalar(norm, dev, "norm"), wp, wb), norm, workspace


def ar_grad_norm(grads, norm=None, workspace=None, stream=None):
    """The global 2-norm of all the gradients, in a float32 tensor of one element (`norm`, made if not given)."""
    given = norm
    dev, args, norm, workspace = _norm_call(grads, norm, workspace, stream)
    with _on_device(dev):
        rc = _lib.lib().ar_grad_norm(*args, _stream_handle(stream, dev.index))
    _lib.check("ar_grad_norm", rc)
    if given is not None:
        _written((given,))
    return norm


# --------------------------------------------------------------------------
# AdamW
# --------------------------------------------------------------------------

def _config(step, lr, betas, eps, weight_decay, max_norm, grad_scale, skip_nonfinite, seed):
    step, seed = int(step), int(seed)
    if not 1 <= step < 1 << 64:
        raise ValueError("step counts from 1")
    return _lib.AdamwConfig(lr, betas[0], betas[1], eps, weight_decay, max_norm, grad_scale, step,
                            seed & 0xFFFFFFFF, 1 if skip_nonfinite else 0)


def _packed_pointers(states, dev, index, counts, what):
    """Addresses of the states' codes and scales, for the given element counts."""
    fast = _fast and _fast.states(states, index, counts)
    if fast is not None:
        return _array(fast[0]), _array(fast[1])
    if not all(isinstance(s, (tuple, list)) and len(s) == 2 for s in states):
        raise ValueError(f"{what} must be PackedState pairs of codes and scales")
    return (_pointers([s[0] for s in states], dev, index, torch.uint8, counts, f"the codes of {what}"),
            _pointers([s[1] for s in states], dev, index, torch.uint8, [-(-c // _lib.STATE_BLOCK) for c in counts],
                      f"the scales of {what}"))


def _tensors(params, grads, exp_avgs, exp_avg_sqs, out, copies, packed):
    """ar_adamw_tensors_t of the sequences; also the tensors and arrays it points to."""
    p0 = _first(params, "params")
    dev, index = p0.device, p0.get_device()
    sizes = [p.numel() for p in params]
    g0 = _first(grads, "grads")
    keep, t = [], _lib.AdamwTensors()

    def put(name, tensors, dtype):
        tensors = list(tensors)
        arr = _pointers(tensors, dev, index, dtype, sizes, name)
        keep.append((tensors, arr))
        setattr(t, name, arr)

    def put_states(name, states, suffix=""):
        if not packed:
            put(f"{name}s{suffix}", states, torch.float32)
            return
        states = list(states)
        codes, scales = _packed_pointers(states, dev, index, sizes, name + "s")
        keep.append((states, codes, scales))
        setattr(t, f"{name}s{suffix}", codes)
        setattr(t, f"{name}_scales{suffix}", scales)

    t.ntensors = len(sizes)
    counts = _counts(sizes)
    keep.append(counts)
    t.counts = counts
    t.param_dtype = _lib.DTYPES[_dtype_of(p0, "params")]
    t.grad_dtype = _lib.DTYPES[_dtype_of(g0, "grads")]
    put("params", params, p0.dtype)
    put("grads", grads, g0.dtype)
    put_states("exp_avg", exp_avgs)
    put_states("exp_avg_sq", exp_avg_sqs)
    if out is not None:
        if len(out) != 3:
            raise ValueError("out must be (params, exp_avgs, exp_avg_sqs)")
        put("params_out", out[0], p0.dtype)
        put_states("exp_avg", out[1], "_out")
        put_states("exp_avg_sq", out[2], "_out")
    if copies is not None:
        c0 = _first(copies, "copies")
        if c0.dtype not in (torch.bfloat16, torch.float16) or p0.dtype is not torch.float32:
            raise TypeError("copies are bfloat16 or float16, of float32 parameters")
        t.copy_dtype = _lib.DTYPES[_FLOATS[c0.dtype]]
        put("copies", copies, c0.dtype)
    return dev, sizes, t, keep


def _adamw(packed, params, grads, exp_avgs, exp_avg_sqs, out, copies, config, grad_norm, stream):
    name = "ar_adamw_packed" if packed else "ar_adamw"
    dev, _, t, keep = _tensors(params, grads, exp_avgs, exp_avg_sqs, out, copies, packed)
    norm = None if grad_norm is None else _scalar(grad_norm, dev, "grad_norm")
    with _on_device(dev):
        rc = getattr(_lib.lib(), name)(ctypes.byref(t), ctypes.byref(config), norm, _stream_handle(stream, dev.index))
    _lib.check(name, rc)
    del keep
    new = (params, exp_avgs, exp_avg_sqs) if out is None else out
    _written(*new, copies)
    return new


def ar_adamw(params, grads, exp_avgs, exp_avg_sqs, out=None, copies=None, *, step, lr, betas=(0.9, 0.999), eps=1e-8,
             weight_decay=0.0, grad_norm=None, max_norm=0.0, grad_scale=1.0, skip_nonfinite=False, stream=None):
    """One AdamW step over all the tensors, states in float32; returns (params, exp_avgs, exp_avg_sqs) as written.

    `step` counts from 1.  `grad_norm` is the tensor :func:`ar_grad_norm`
    returns, of the gradients as they are; `max_norm` > 0 clips by it,
    `grad_scale` multiplies the gradients (the inverse of a loss scale), and
    `skip_nonfinite` leaves everything as it is when the norm is not finite.
    """
    config = _config(step, lr, betas, eps, weight_decay, max_norm, grad_scale, skip_nonfinite, 0)
    return _adamw(False, params, grads, exp_avgs, exp_avg_sqs, out, copies, config, grad_norm, stream)


def ar_adamw_packed(params, grads, exp_avgs, exp_avg_sqs, out=None, copies=None, *, step, lr, seed,
                    betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, grad_norm=None, max_norm=0.0, grad_scale=1.0,
                    skip_nonfinite=False, stream=None):
    """The same step with states in 8 bits: exp_avgs and exp_avg_sqs are :class:`PackedState` pairs.

    New states are rounded up or down at random, from `seed`: give every step
    its own (the step's number will do).
    """
    config = _config(step, lr, betas, eps, weight_decay, max_norm, grad_scale, skip_nonfinite, seed)
    return _adamw(True, params, grads, exp_avgs, exp_avg_sqs, out, copies, config, grad_norm, stream)


def ar_unpack_states(states, kind: str, outs=None, dtype=torch.float32, stream=None):
    """The values of packed states, one flat tensor each (`outs`, or made in `dtype`).

    `kind` says which of the two states they are: "exp_avg" or "exp_avg_sq".
    """
    codes = [s[0] for s in states]
    c0 = _first(codes, "states")
    dev, index = c0.device, c0.get_device()
    sizes = [c.numel() for c in codes]
    cp, sp = _packed_pointers(states, dev, index, sizes, "states")
    given = outs
    if outs is None:
        outs = [_empty(s, dtype, dev, stream) for s in sizes]
    o0 = _first(outs, "outs")
    op = _pointers(outs, dev, index, o0.dtype, sizes, "outs")
    with _on_device(dev):
        rc = _lib.lib().ar_unpack_states(cp, sp, op, _counts(sizes), len(sizes), _lib.STATES[kind],
                                         _lib.DTYPES[_dtype_of(o0, "outs")], _stream_handle(stream, dev.index))
    _lib.check("ar_unpack_states", rc)
    _written(given)
    return outs


# --------------------------------------------------------------------------
# persistent norms and steps
# --------------------------------------------------------------------------

class Update:
    """A persistent gradient norm or AdamW step from one of the ``*_init`` calls.

    Holds references to its tensors and its workspace; :meth:`start` enqueues
    it; it is freed by :meth:`close` or when collected.  As with the
    collectives' plans, close it after the work it enqueued has completed, or
    keep the tensors alive until then.
    """

    def __init__(self, kind, handle, device, keep, writes, norm=None):
        self.kind = kind
        self.device = device
        self.norm = norm
        self._handle = handle
        self._index = device.index
        self._keep = keep
        self._writes = writes

    @property
    def num_launches(self) -> int:
        return _lib.lib().ar_update_num_launches(self._handle)

    def start(self, stream=None, **config):
        """Enqueue it.  A norm takes the stream only and returns its `norm` tensor; a step takes the
        keyword arguments of :func:`ar_adamw` (or :func:`ar_adamw_packed`) after the tensors.

        Captured into a HIP graph, a step replays with the arguments it was
        captured with: `step`, `lr` and, with packed states, the random bits
        of `seed` stay the same at every replay, which a training loop must
        not have.
        """
        if self._handle is None:
            raise ValueError("update is closed")
        if self.kind == "grad_norm":
            if config:
                raise TypeError(f"a gradient norm takes no {sorted(config)}")
            rc = _lib.lib().ar_grad_norm_start(self._handle, _stream_handle(stream, self._index))
            _lib.check("ar_grad_norm_start", rc)
            _written(self._writes)
            return self.norm
        self._start_step(stream, **config)
        return None

    def _start_step(self, stream, *, step, lr, seed=None, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                    grad_norm=None, max_norm=0.0, grad_scale=1.0, skip_nonfinite=False):
        if (seed is None) == (self.kind == "adamw_packed"):
            raise TypeError("a packed step needs a seed, and a step with float32 states takes none")
        config = _config(step, lr, betas, eps, weight_decay, max_norm, grad_scale, skip_nonfinite, seed or 0)
        norm = None if grad_norm is None else _scalar(grad_norm, self.device, "grad_norm")
        rc = _lib.lib().ar_adamw_start(self._handle, ctypes.byref(config), norm, _stream_handle(stream, self._index))
        _lib.check("ar_adamw_start", rc)
        _written(self._writes)

    def close(self):
        if self._handle is not None:
            _lib.lib().ar_update_free(self._handle)
            self._handle = None
            self._keep = self._writes = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass


def ar_grad_norm_init(grads, norm=None, workspace=None) -> Update:
    """Persistent gradient norm; the plan's table is made on the current stream."""
    dev, args, norm, workspace = _norm_call(grads, norm, workspace, None)
    handle = ctypes.c_void_p()
    with _on_device(dev):
        rc = _lib.lib().ar_grad_norm_init(*args, _stream_handle(None, dev.index), ctypes.byref(handle))
    _lib.check("ar_grad_norm_init", rc)
    return Update("grad_norm", handle, dev, (list(grads), workspace), (norm,), norm)


def _adamw_init(kind, params, grads, exp_avgs, exp_avg_sqs, out, copies, workspace):
    dev, sizes, t, keep = _tensors(params, grads, exp_avgs, exp_avg_sqs, out, copies, kind == "adamw_packed")
    workspace = _scratch(ar_update_workspace_bytes(kind, sizes), workspace, dev, None)
    wp, wb = _ws(workspace, dev)
    handle = ctypes.c_void_p()
    with _on_device(dev):
        rc = getattr(_lib.lib(), f"ar_{kind}_init")(ctypes.byref(t), wp, wb, _stream_handle(None, dev.index),
                                                    ctypes.byref(handle))
    _lib.check(f"ar_{kind}_init", rc)
    new = (params, exp_avgs, exp_avg_sqs) if out is None else out
    writes = [t for group in (*new, copies or ()) for item in group
              for t in ((item,) if isinstance(item, torch.Tensor) else item)]
    return Update(kind, handle, dev, (keep, workspace), writes)


def ar_adamw_init(params, grads, exp_avgs, exp_avg_sqs, out=None, copies=None, workspace=None) -> Update:
    """Persistent AdamW step over these tensors; the plan's table is made on the current stream."""
    return _adamw_init("adamw", params, grads, exp_avgs, exp_avg_sqs, out, copies, workspace)


def ar_adamw_packed_init(params, grads, exp_avgs, exp_avg_sqs, out=None, copies=None, workspace=None) -> Update:
    """Persistent AdamW step with packed states; the plan's table is made on the current stream."""
    return _adamw_init("adamw_packed", params, grads, exp_avgs, exp_avg_sqs, out, copies, workspace)


def ar_grad_norm_start(update: Update, stream=None):
    """Enqueue a persistent gradient norm (same as ``update.start``)."""
    if update.kind != "grad_norm":
        raise ValueError("not a plan of ar_grad_norm_init")
    return update.start(stream)


def ar_adamw_start(update: Update, stream=None, **config):
    """Enqueue a persistent AdamW step (same as ``update.start``)."""
    if update.kind == "grad_norm":
        raise ValueError("not a plan of ar_adamw_init or ar_adamw_packed_init")
    return update.start(stream, **config)


def ar_update_num_launches(update: Update) -> int:
    """Kernel launches one start enqueues (same as ``update.num_launches``)."""
    return update.num_launches


def ar_update_free(update: Update):
    """Release a persistent norm or step (same as ``update.close``)."""
    update.close()


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------

def _row_pointers(tensors, n, dev, index, dtype, rows, cols, what):
    """Addresses and common row stride of one [rows, cols] tensor per rank, rows contiguous."""
    if len(tensors) != n:
        raise ValueError(f"need one of {what} per rank")
    fast = _fast and _fast.rows(tensors, dtype, index, rows, cols)
    if fast is not None:
        return _array(fast[0]), fast[1]
    stride = cols
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != index:
            raise ValueError(f"{what} must be tensors on {dev}")
        if t.dtype is not dtype:
            raise TypeError(f"{what} must have one dtype, {dtype}")
        if t.shape != (rows, cols):
            raise ValueError(f"{what} must be [{rows}, {cols}] tensors, one per rank")
        s = t.stride()
        if t.is_neg() or (cols > 1 and s[1] != 1) or (rows > 1 and s[0] < cols):
            raise ValueError(f"{what} must have contiguous rows that do not overlap")
        if rows > 1:
            if i > 0 and s[0] != stride:
                raise ValueError(f"{what} must have one row stride")
            stride = s[0]
    return (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]), stride


def _new_parts(shape, dtype, dev, stream):
    """shape[0] new tensors of one allocation, and their addresses (a list)."""
    fast = _fast.new_parts(shape, dtype, dev.index) if _fast and stream is None else None
    if fast is not None:
        return fast[0], _array(fast[1])
    parts = list(_empty(shape, dtype, dev, stream).unbind(0))
    return parts, (ctypes.c_void_p * max(len(parts), 1))(*[t.data_ptr() for t in parts])


def _second_half(ptrs, n):
    """Entries n to 2n of an address array, as an array of its own in the same memory."""
    return (ctypes.c_void_p * n).from_buffer(ptrs, n * ctypes.sizeof(ctypes.c_void_p))


def _rank_list(tensors, what):
    t = _first(tensors, what)
    if t.dim() != 2:
        raise ValueError(f"{what} must be [rows, cols] tensors, one per rank")
    if len(tensors) > _lib.MAX_RANKS:
        raise ValueError(f"nranks must be in [1, {_lib.MAX_RANKS}]")
    return t


def _weights(tensors, n, dev, index, dtype, cols, what):
    if len(tensors) != n:
        raise ValueError(f"need one of {what} per rank")
    return _pointers(tensors, dev, index, dtype, [cols] * n, what)


def _weight_dtype(dtype, *lists):
    """The weights' type: that of the first list given, else the activations'."""
    for w in lists:
        if w is not None and len(w):
            if w[0].dtype is not dtype and w[0].dtype is not torch.float32:
                raise TypeError("the weights have the activations' type or float32")
            return w[0].dtype
    return dtype


def ar_layer_norm(xs, gammas=None, betas=None, ys=None, eps: float = 1e-5, stats: bool = True, stream=None):
    """Layer norm of every rank's [rows, cols] activations over the last axis.

    Returns (ys, means, rstds), one tensor per rank in each; with
    ``stats=False`` the two statistics, which only the backward pass needs,
    are None.  Rows may lie further apart than their length, by the same
    stride on every rank.  Weights are one per rank, in the activations' type
    or float32; None means 1 (`gammas`) or 0 (`betas`).  In place: ``ys=xs``.
    Autograd does not see the call: the gradients are the caller's to take
    with :func:`ar_layer_norm_backward`.
    """
    x0 = _rank_list(xs, "xs")
    n, dev, index, dt = len(xs), x0.device, x0.get_device(), x0.dtype
    name = _dtype_of(x0, "xs")
    rows, cols = x0.shape
    xp, x_stride = _row_pointers(xs, n, dev, index, dt, rows, cols, "xs")
    wdt = _weight_dtype(dt, gammas, betas)
    gp = None if gammas is None else _weights(gammas, n, dev, index, wdt, cols, "gammas")
    bp = None if betas is None else _weights(betas, n, dev, index, wdt, cols, "betas")
    given = ys
    if ys is None:
        (ys, yp), y_stride = _new_parts((n, rows, cols), dt, dev, stream), cols
    else:
        yp, y_stride = _row_pointers(ys, n, dev, index, dt, rows, cols, "ys")
    means = rstds = mp = rp = None
    if stats:
        both, ptrs = _new_parts((2 * n, rows), torch.float32, dev, stream)
        means, rstds, mp, rp = both[:n], both[n:], ptrs, _second_half(ptrs, n)
    with _on_device(dev):
        rc = _lib.lib().ar_layer_norm(xp, gp, bp, yp, mp, rp, rows, cols, x_stride, y_stride, _lib.DTYPES[name],
                                      _lib.DTYPES[_FLOATS[wdt]], eps, n, _stream_handle(stream, dev.index))
    _lib.check("ar_layer_norm", rc)
    _written(given)
    return ys, means, rstds


def ar_layer_norm_workspace_bytes(rows: int, cols: int, nranks: int) -> int:
    v = _lib.lib().ar_layer_norm_workspace_bytes(rows, cols, nranks)
    if v == ctypes.c_size_t(-1).value:
        raise ValueError("invalid arguments for ar_layer_norm_workspace_bytes")
    return v


def ar_layer_norm_backward(dys, xs, gammas, means, rstds, dxs=None, weight_grads: bool = True, dgammas=None,
                           dbetas=None, workspace=None, stream=None):
    """Backward pass of :func:`ar_layer_norm`; returns (dxs, dgammas, dbetas), one tensor per rank in each.

    `dgammas` and `dbetas` are each rank's part of the weight gradients, for
    the AllReduce to sum over the ranks; tensors may be passed for them (a
    rank's slices of its gradient bucket), and with ``weight_grads=False``
    those not passed are not made.  In place: ``dxs=dys``.
    """
    x0 = _rank_list(xs, "xs")
    _dtype_of(x0, "xs")
    rows, cols = x0.shape
    xp, x_stride = _row_pointers(xs, len(xs), x0.device, x0.get_device(), x0.dtype, rows, cols, "xs")
    return _norm_backward("ar_layer_norm_backward", (xp,), (x_stride,), x0, len(xs), dys, gammas, means, rstds, dxs,
                          weight_grads, dgammas, dbetas, workspace, stream)


def _norm_backward(call, inputs, strides, x0, n, dys, gammas, means, rstds, dxs, weight_grads, dgammas, dbetas,
                   workspace, stream):
    """The backward pass `call` from the addresses `inputs` of x, its row stride in `strides` if it has one; `x0` is
    a tensor of dx's shape, type and device."""
    dev, index, dt = x0.device, x0.get_device(), x0.dtype
    rows, cols = x0.shape
    dyp, dy_stride = _row_pointers(dys, n, dev, index, dt, rows, cols, "dys")
    wdt = _weight_dtype(dt, gammas, dgammas, dbetas)
    gp = None if gammas is None else _weights(gammas, n, dev, index, wdt, cols, "gammas")
    if len(means) != n or len(rstds) != n:
        raise ValueError("need one of means and rstds per rank")
    given = (dxs, dgammas, dbetas)
    mp = _pointers(means, dev, index, torch.float32, [rows] * n, "means")
    rp = _pointers(rstds, dev, index, torch.float32, [rows] * n, "rstds")
    if dxs is None:
        (dxs, dxp), dx_stride = _new_parts((n, rows, cols), dt, dev, stream), cols
    else:
        dxp, dx_stride = _row_pointers(dxs, n, dev, index, dt, rows, cols, "dxs")
    if weight_grads and dgammas is None and dbetas is None:
        both, ptrs = _new_parts((2 * n, cols), wdt, dev, stream)
        dgammas, dbetas, gout, bout = both[:n], both[n:], ptrs, _second_half(ptrs, n)
    else:
        if weight_grads:
            made = list(_empty((n, cols), wdt, dev, stream).unbind(0))
            dgammas, dbetas = made if dgammas is None else dgammas, made if dbetas is None else dbetas
        gout = None if dgammas is None else _weights(dgammas, n, dev, index, wdt, cols, "dgammas")
        bout = None if dbetas is None else _weights(dbetas, n, dev, index, wdt, cols, "dbetas")
    with _on_device(dev):
        if gout is not None or bout is not None:
            workspace = _scratch(ar_layer_norm_workspace_bytes(rows, cols, n), workspace, dev, stream)
        wp, wb = _ws(workspace, dev)
        rc = getattr(_lib.lib(), call)(dyp, *inputs, gp, mp, rp, dxp, gout, bout, rows, cols, dy_stride, *strides,
                                       dx_stride, _lib.DTYPES[_FLOATS[dt]], _lib.DTYPES[_FLOATS[wdt]], n, wp, wb,
                                       _stream_handle(stream, dev.index))
    _lib.check(call, rc)
    _written(*given)
    return dxs, dgammas, dbetas
