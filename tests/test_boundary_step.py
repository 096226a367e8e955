"""The training-step entry points without a GPU: every argument error is
reported before anything touches a device, empty work succeeds, and the
binding's tables and structures are the header's."""

import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000           # fake device addresses: only compared, never read
GAP = 1 << 32
INVALID = 1


@pytest.fixture(scope="module")
def lib():
    from ring_allreduce_reduction_virtual_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return _lib.lib()


def _mod():
    from ring_allreduce_reduction_virtual_amd import _lib

    return _lib


def ptrs(values):
    return (ctypes.c_void_p * max(len(values), 1))(*values)


def sizes(values):
    return (ctypes.c_size_t * max(len(values), 1))(*values)


def detail(lib):
    return lib.ar_get_last_error_detail().decode()


def buffers(start, n):
    return [BASE + (start + i) * GAP for i in range(n)]


def tensors(n=2, counts=None, packed=False, **change):
    m = _mod()
    counts = [1000] * n if counts is None else counts
    t = m.AdamwTensors()
    keep = [sizes(counts)]
    t.ntensors, t.counts, t.param_dtype, t.grad_dtype, t.copy_dtype = n, keep[0], 0, 0, 1
    roles = ["params", "grads", "exp_avgs", "exp_avg_sqs"] + (["exp_avg_scales", "exp_avg_sq_scales"] if packed else [])
    for k, name in enumerate(roles):
        keep.append(ptrs(buffers(100 * k, n)))
        setattr(t, name, keep[-1])
    for name, value in change.items():
        if isinstance(value, list):
            keep.append(ptrs(value))
            value = keep[-1]
        setattr(t, name, value)
    t._keep = keep
    return t


def config(**change):
    c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_norm=0.0, grad_scale=1.0, step=1,
             seed=0, skip_nonfinite=0)
    c.update(change)
    return _mod().AdamwConfig(**c)


def test_binding_matches_the_header():
    m = _mod()
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ar.h")).read(), flags=re.S)
    values = {k: int(v) for k, v in re.findall(r"\b(AR_[A-Z0-9_]+)\s*=\s*(\d+)", text)}
    assert {k: values["AR_STATE_" + k.upper()] for k in m.STATES} == m.STATES
    assert {k: values["AR_UPDATE_" + k.upper()] for k in m.UPDATES} == m.UPDATES
    assert int(re.search(r"#define\s+AR_STATE_BLOCK\s+(\d+)", text).group(1)) == m.STATE_BLOCK
    for struct, name in ((m.AdamwConfig, "ar_adamw_config_t"), (m.AdamwTensors, "ar_adamw_tensors_t")):
        body = re.search(r"typedef struct \{([^}]*)\}\s*" + name, text).group(1)
        fields = re.findall(r"(\w+)\s*;", body)
        assert fields == [f[0] for f in struct._fields_]


def test_grad_norm_errors(lib):
    ws = BASE + 900 * GAP
    need = lib.ar_update_workspace_bytes(0, sizes([10, 10]), 2)
    norm = BASE + 901 * GAP

    def call(g=None, counts=(10, 10), n=2, dtype=0, norm=norm, ws=ws, have=need):
        return lib.ar_grad_norm(ptrs(buffers(0, 2) if g is None else g), sizes(list(counts)), n, dtype, norm, ws, have,
                                None)

    assert call(n=-1) == INVALID and "ntensors" in detail(lib)
    assert call(n=65537) == INVALID
    assert call(dtype=2) == INVALID and call(dtype=4) == INVALID and "dtype" in detail(lib)
    assert call(norm=None) == INVALID and "norm" in detail(lib)
    assert call(norm=norm + 2) == INVALID and "aligned" in detail(lib)
    assert call(g=[0, BASE]) == INVALID and "null" in detail(lib)
    assert call(g=[BASE + 2, BASE + GAP]) == INVALID and "aligned" in detail(lib)
    assert call(counts=(10, 1 << 50)) == INVALID and "too large" in detail(lib)
    assert call(have=need - 1) == INVALID and "workspace" in detail(lib)
    assert call(ws=None) == INVALID
    assert call(ws=ws + 4) == INVALID and "aligned" in detail(lib)
    assert call(norm=BASE + 4) == INVALID and "overlaps" in detail(lib)
    assert call(ws=BASE) == INVALID and "overlaps" in detail(lib)
    assert lib.ar_grad_norm(None, sizes([10]), 1, 0, norm, ws, need, None) == INVALID
    assert lib.ar_grad_norm(ptrs([BASE]), None, 1, 0, norm, ws, need, None) == INVALID


@pytest.mark.parametrize("packed", [False, True])
def test_adamw_errors(lib, packed):
    fn = lib.ar_adamw_packed if packed else lib.ar_adamw

    def call(t=None, c=None, norm=None, **change):
        t = tensors(packed=packed, **change) if t is None else t
        return fn(ctypes.byref(t), ctypes.byref(config() if c is None else c), norm, None)

    assert fn(None, ctypes.byref(config()), None, None) == INVALID
    assert fn(ctypes.byref(tensors(packed=packed)), None, None, None) == INVALID and "config" in detail(lib)
    assert call(ntensors=-1) == INVALID and call(ntensors=1 << 20) == INVALID
    for name in ("params", "grads", "exp_avgs", "exp_avg_sqs"):
        assert call(**{name: None}) == INVALID and "null" in detail(lib)
        assert call(**{name: [0, BASE + 50 * GAP]}) == INVALID and "null" in detail(lib)
    assert call(param_dtype=2) == INVALID and call(grad_dtype=7) == INVALID and "dtype" in detail(lib)
    assert call(copies=buffers(700, 2), copy_dtype=0) == INVALID and "copy" in detail(lib)
    assert call(copies=buffers(700, 2), param_dtype=1) == INVALID and "copies" in detail(lib)
    assert call(counts=[1000, 1 << 50]) == INVALID and "too large" in detail(lib)
    assert call(params=[BASE + 2, BASE + GAP]) == INVALID and "aligned" in detail(lib)
    # outputs overlap nothing but their own input, exactly
    assert call(grads=buffers(0, 2)) == INVALID and "overlaps" in detail(lib)
    assert call(exp_avg_sqs=buffers(200, 2)) == INVALID and "overlaps" in detail(lib)
    assert call(params_out=[BASE + 4, BASE + GAP]) == INVALID and "overlaps" in detail(lib)
    assert call(params_out=[BASE + GAP, BASE]) == INVALID and "overlaps" in detail(lib)
    assert call(copies=[BASE, BASE + 710 * GAP]) == INVALID and "overlaps" in detail(lib)
    assert call(norm=BASE + 8) == INVALID and "overlaps" in detail(lib)
    if packed:
        assert call(exp_avg_scales=None) == INVALID and "scales" in detail(lib)
        assert call(exp_avg_sq_scales=buffers(400, 2)) == INVALID and "overlaps" in detail(lib)
    else:
        assert call(exp_avg_scales=buffers(600, 2)) == INVALID and "scales" in detail(lib)
    for bad in (dict(lr=-1), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=math.nan), dict(eps=-1e-9), dict(eps=math.nan), dict(weight_decay=-0.1),
                dict(weight_decay=math.inf), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(grad_scale=0.0),
                dict(grad_scale=-1.0), dict(grad_scale=math.inf), dict(step=0), dict(max_norm=1.0),
                dict(skip_nonfinite=1)):
        assert call(c=config(**bad)) == INVALID, bad
    assert call(c=config(max_norm=1.0), norm=BASE + 801 * GAP + 2) == INVALID and "aligned" in detail(lib)


@pytest.mark.parametrize("packed", [False, True])
def test_empty_steps_succeed_without_a_device(lib, packed):
    fn = lib.ar_adamw_packed if packed else lib.ar_adamw
    init = lib.ar_adamw_packed_init if packed else lib.ar_adamw_init
    for t in (tensors(0, packed=packed), tensors(2, [0, 0], packed=packed),
              tensors(1, [0], packed=packed, params=[0], grads=[0])):
        assert fn(ctypes.byref(t), ctypes.byref(config()), None, None) == 0 and detail(lib) == ""
        handle = ctypes.c_void_p()
        assert init(ctypes.byref(t), None, 0, None, ctypes.byref(handle)) == 0
        assert lib.ar_update_num_launches(handle) == 0
        assert lib.ar_adamw_start(handle, ctypes.byref(config()), None, None) == 0
        assert lib.ar_adamw_start(handle, ctypes.byref(config(step=0)), None, None) == INVALID
        assert lib.ar_grad_norm_start(handle, None) == INVALID and "plan" in detail(lib)
        assert lib.ar_update_free(handle) == 0
    assert lib.ar_update_free(None) == 0 and lib.ar_update_num_launches(None) == -1
    assert lib.ar_adamw_start(None, ctypes.byref(config()), None, None) == INVALID
    assert lib.ar_grad_norm_start(None, None) == INVALID
    t = tensors(packed=packed)
    assert init(ctypes.byref(t), None, 0, None, None) == INVALID
    handle = ctypes.c_void_p(1)
    assert init(ctypes.byref(t), None, 0, None, ctypes.byref(handle)) == INVALID and not handle.value


def test_workspace_sizes(lib):
    f = lib.ar_update_workspace_bytes
    bad = ctypes.c_size_t(-1).value
    assert f(0, sizes([10]), -1) == bad and f(3, sizes([10]), 1) == bad and f(0, None, 1) == bad
    assert f(1, sizes([1 << 50]), 1) == bad
    assert f(1, sizes([]), 0) == 0 and f(2, sizes([0, 0]), 2) == 0
    for kind in (0, 1, 2):
        assert 0 < f(kind, sizes([10]), 1) < f(kind, sizes([10] * 400), 400)
    g = lib.ar_layer_norm_workspace_bytes
    assert g(10, 10, 0) == bad and g(10, 10, 129) == bad and g(1 << 60, 10, 1) == bad
    assert g(0, 10, 1) == 0 and g(1, 10, 1) == 80 and g(1000, 4096, 8) <= 512 * 2 * 4 * 4096


def test_unpack_errors(lib):
    def call(c=None, s=None, o=None, counts=(300,), n=1, state=0, dtype=0):
        return lib.ar_unpack_states(ptrs([BASE] if c is None else c), ptrs([BASE + GAP] if s is None else s),
                                    ptrs([BASE + 2 * GAP] if o is None else o), sizes(list(counts)), n, state, dtype,
                                    None)

    assert call(state=2) == INVALID and "state" in detail(lib)
    assert call(dtype=2) == INVALID and "dtype" in detail(lib)
    assert call(n=-1) == INVALID
    assert call(c=[0]) == INVALID and call(s=[0]) == INVALID and call(o=[0]) == INVALID
    assert call(o=[BASE + 100]) == INVALID and "overlaps" in detail(lib)
    assert call(o=[BASE + 2 * GAP + 2]) == INVALID and "aligned" in detail(lib)
    assert call(counts=(0,), c=[0], s=[0], o=[0]) == 0


def test_layer_norm_errors(lib):
    n, rows, cols = 2, 8, 100
    x, y, g, b = (ptrs(buffers(10 * k, n)) for k in range(4))
    mean, rstd = (ptrs(buffers(10 * k, n)) for k in (5, 6))

    def call(x=x, g=g, b=b, y=y, mean=mean, rstd=rstd, rows=rows, cols=cols, xs=100, ys=100, dtype=0, wdtype=0,
             eps=1e-5, n=n):
        return lib.ar_layer_norm(x, g, b, y, mean, rstd, rows, cols, xs, ys, dtype, wdtype, eps, n, None)

    assert call(x=None) == INVALID and call(y=None) == INVALID
    assert call(n=0) == INVALID and call(n=129) == INVALID and "nranks" in detail(lib)
    assert call(dtype=2) == INVALID and call(dtype=0, wdtype=1) == INVALID and call(dtype=1, wdtype=3) == INVALID
    assert call(xs=99) == INVALID and "x_stride" in detail(lib)
    assert call(ys=99) == INVALID and "y_stride" in detail(lib)
    assert call(xs=1 << 41) == INVALID and call(rows=1 << 41) == INVALID and call(cols=1 << 27, xs=1 << 27,
                                                                                ys=1 << 27) == INVALID
    for eps in (-1.0, math.nan, math.inf):
        assert call(eps=eps) == INVALID and "eps" in detail(lib)
    assert call(mean=None) == INVALID and "together" in detail(lib)
    assert call(g=ptrs([0, BASE])) == INVALID and "gamma" in detail(lib)
    assert call(y=ptrs([buffers(0, 1)[0] + 4, BASE + 77 * GAP])) == INVALID and "overlaps" in detail(lib)
    assert call(y=x, ys=101) == INVALID and "overlaps" in detail(lib)
    assert call(y=ptrs([BASE + 77 * GAP] * 2)) == INVALID and "overlaps" in detail(lib)
    assert call(mean=rstd) == INVALID and "overlaps" in detail(lib)
    assert call(mean=g) == INVALID and "overlaps" in detail(lib)
    # empty: no device is touched
    assert call(rows=0) == 0 and call(cols=0) == 0 and detail(lib) == ""


def test_layer_norm_backward_errors(lib):
    n, rows, cols = 2, 8, 100
    names = ("dy", "x", "gamma", "mean", "rstd", "dx", "dgamma", "dbeta")
    good = {k: ptrs(buffers(10 * i, n)) for i, k in enumerate(names)}
    need = lib.ar_layer_norm_workspace_bytes(rows, cols, n)

    def call(rows=rows, cols=cols, strides=(100, 100, 100), dtype=0, wdtype=0, n=n, ws=BASE + 500 * GAP, have=need,
             **change):
        a = dict(good, **change)
        return lib.ar_layer_norm_backward(*[a[k] for k in names], rows, cols, *strides, dtype, wdtype, n, ws, have,
                                          None)

    for name in ("dy", "x", "mean", "rstd", "dx"):
        assert call(**{name: None}) == INVALID and "null" in detail(lib), name
        assert call(**{name: ptrs([0, BASE + 600 * GAP])}) == INVALID and "null" in detail(lib), name
    for k in range(3):
        s = [100, 100, 100]
        s[k] = 50
        assert call(strides=s) == INVALID and "stride" in detail(lib)
    assert call(n=0) == INVALID and call(dtype=4) == INVALID and call(dtype=3, wdtype=1) == INVALID
    assert call(have=need - 1) == INVALID and call(ws=None) == INVALID and "workspace" in detail(lib)
    assert call(ws=BASE + 500 * GAP + 1) == INVALID and "aligned" in detail(lib)
    assert call(ws=BASE) == INVALID and "overlaps" in detail(lib)
    assert call(dx=good["x"]) == INVALID and "overlaps" in detail(lib)
    assert call(dgamma=good["dbeta"]) == INVALID and "overlaps" in detail(lib)
    assert call(dgamma=good["gamma"]) == INVALID and "overlaps" in detail(lib)
    assert call(dbeta=ptrs([0, BASE + 600 * GAP])) == INVALID
    assert call(cols=0, strides=(0, 0, 0)) == 0
    assert call(rows=0, dgamma=None, dbeta=None, ws=None, have=0) == 0


def test_native_marshalling_declines_what_it_does_not_know():
    """The native checks answer None, with no error left behind, for anything that is not theirs to take."""
    import torch

    m = pytest.importorskip("ring_allreduce_reduction_virtual_amd._armarshal")
    cpu, f32 = torch.zeros(4), torch.float32
    for bad in ([cpu], [None], [cpu, 3], 7, None):
        assert m.pointers(bad, f32, 0, None) is None
        assert m.rows(bad, f32, 0, 2, 2) is None
        assert m.states(bad, 0, [4]) is None
    assert m.pointers([], f32, 0, None) == b"" and m.states([], 0, []) == (b"", b"")
    assert m.pointers([], f32, 0, [1]) is None and m.pointers([], "float32", 0, None) is None
    assert m.pointers([], f32, 1 << 80, None) is None and m.pointers() is None
    assert m.states([(cpu, cpu)], 0, [4]) is None and m.states([(cpu,)], 0, [4]) is None
    assert m.new_parts([2, 3], f32, 0) is None and m.new_parts((), f32, 0) is None
    assert m.new_parts((2, "x"), f32, 0) is None and m.new_parts((2, -1), f32, 0) is None


@pytest.mark.parametrize("packed", [False, True])
def test_settings_that_float32_cannot_hold_are_refused(lib, packed):
    """A positive setting that would round to 0 would switch itself off, and an infinite scalar spoils parameters."""
    fn = lib.ar_adamw_packed if packed else lib.ar_adamw
    t = tensors(2, [0, 0], packed=packed)
    norm = BASE + 801 * GAP

    def call(**change):
        return fn(ctypes.byref(t), ctypes.byref(config(**change)), norm, None)

    for name in ("max_norm", "grad_scale", "eps"):
        for small in (1e-46, 5e-324):
            assert call(**{name: small}) == INVALID and name in detail(lib), (name, small)
        assert call(**{name: 1e-45}) == 0 and call(**{name: 3.4e38}) == 0, name
    assert call(eps=0.0, max_norm=0.0) == 0
    assert call(lr=3e38, beta1=0.99) == INVALID and "lr" in detail(lib)
    assert call(lr=3e38, beta1=0.0) == 0 and call(lr=3e38, beta1=0.99, step=10**6) == 0
    assert call(lr=1e30, weight_decay=1e30) == INVALID and "weight_decay" in detail(lib)
    assert call(lr=1e-46, weight_decay=1e-46) == 0
    handle = ctypes.c_void_p()
    init = lib.ar_adamw_packed_init if packed else lib.ar_adamw_init
    assert init(ctypes.byref(t), None, 0, None, ctypes.byref(handle)) == 0
    assert lib.ar_adamw_start(handle, ctypes.byref(config(max_norm=1e-46)), norm, None) == INVALID
    assert lib.ar_update_free(handle) == 0


def test_layer_norm_eps_that_float32_cannot_hold_is_refused(lib):
    x, y = ptrs([BASE]), ptrs([BASE + GAP])
    for eps, want in ((1e-46, INVALID), (5e-324, INVALID), (1e-45, 0), (0.0, 0)):
        assert lib.ar_layer_norm(x, None, None, y, None, None, 0, 8, 8, 8, 0, 0, eps, 1, None) == want, eps
        assert want == 0 or "eps" in detail(lib)


def test_read_only_buffers_of_one_span_are_each_checked(lib):
    """Rows with gaps and a whole buffer may start and end together: an output in the gaps overlaps the whole one."""
    names = ("dy", "x", "gamma", "mean", "rstd", "dx", "dgamma", "dbeta")
    good = {k: ptrs([BASE + 10 * i * GAP]) for i, k in enumerate(names)}
    x = good["x"][0]
    for a in ("mean", "rstd"):
        # two rows of one 2-byte element, 6 bytes apart: bytes 0-7 with x, and 2-9 with dx in x's gap
        args = dict(good, gamma=None, dgamma=None, dbeta=None, dx=ptrs([x + 2]), **{a: ptrs([x])})
        rc = lib.ar_layer_norm_backward(*[args[k] for k in names], 2, 1, 3, 3, 3, 1, 1, 1, None, 0, None)
        assert rc == INVALID and "overlaps" in detail(lib) and a in detail(lib)


def test_native_marshalling_counts_writes():
    """Tensors and pairs of them rise by one version each; tensors without a counter and other things are passed over."""
    import torch

    m = pytest.importorskip("ring_allreduce_reduction_virtual_amd._armarshal")
    a, b, c = (torch.zeros(4) for _ in range(3))
    assert m.written([a, (b, c), a[1:]]) is True and m.written(()) is True
    assert [t._version for t in (a, b, c)] == [2, 1, 1]
    with torch.inference_mode():
        d = torch.zeros(4)
        assert m.written([d, a]) is True
    assert m.written([d]) is True and a._version == 3
    for bad in (7, None, [3], [(a, 3)], [None]):
        assert m.written(bad) is None
    assert m.written() is None and m.written([a], [b]) is None
