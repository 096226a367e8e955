"""ctypes view of libar.so: the C ABI of include/ar.h, one Python call per C symbol.

Loading fails loudly when the library has not been built: there is no
fallback path.
"""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libar.so")

# values of the C enums in include/ar.h
AR_SUCCESS = 0
RESULT_NAMES = {0: "AR_SUCCESS", 1: "AR_ERR_INVALID_ARGUMENT", 2: "AR_ERR_UNSUPPORTED",
                3: "AR_ERR_HIP", 4: "AR_ERR_INTERNAL"}
DTYPES = {"f32": 0, "bf16": 1, "i32": 2, "f16": 3, "bf16acc32": 4}
OPS = {"sum": 0, "prod": 1, "min": 2, "max": 3, "avg": 4}
ALGOS = {"fused": 0, "ring": 1, "phases": 2, "auto": 3, "tree": 4, "tree_steps": 5, "recursive_doubling": 6,
         "halving_doubling": 7, "halving_doubling_steps": 8, "ring_persistent": 9, "ring_pipelined": 10,
         "staged": 11, "double_binary_tree": 12, "double_binary_tree_steps": 13}
# algorithms whose bracketing is a tree, not the ring's (AllReduce only)
TREE_ALGOS = ("tree", "tree_steps", "recursive_doubling", "halving_doubling", "halving_doubling_steps",
              "double_binary_tree", "double_binary_tree_steps")
COLLS = {"allreduce": 0, "reduce_scatter": 1, "all_gather": 2}
MAX_RANKS = 128

# every function include/ar.h declares
EXPORTS = (
    "ar_allreduce", "ar_reduce_scatter", "ar_all_gather",
    "ar_allreduce_ex", "ar_reduce_scatter_ex", "ar_all_gather_ex",
    "ar_workspace_bytes", "ar_chunk_range", "ar_get_error_string",
    "ar_get_last_error_detail", "ar_dtype_size",
    "ar_allreduce_init", "ar_reduce_scatter_init", "ar_all_gather_init",
    "ar_plan_start", "ar_plan_num_launches", "ar_plan_free", "ar_plan_limit_blocks",
    "ar_reduce_scatter_noalloc", "ar_plan_algo",
    "ar_grad_norm", "ar_grad_norm_init", "ar_grad_norm_start",
    "ar_adamw", "ar_adamw_init", "ar_adamw_packed", "ar_adamw_packed_init", "ar_adamw_start",
    "ar_unpack_states", "ar_update_workspace_bytes", "ar_update_num_launches", "ar_update_free",
    "ar_layer_norm", "ar_layer_norm_backward", "ar_layer_norm_workspace_bytes",
    "ar_embedding", "ar_embedding_backward", "ar_embedding_workspace_bytes",
    "ar_cross_entropy", "ar_cross_entropy_backward", "ar_cross_entropy_workspace_bytes",
    "ar_cross_entropy_aligned_workspace_bytes",
    "ar_pack_activations", "ar_unpack_activations", "ar_layer_norm_backward_packed",
)
# the training-step operators' enums and constants
STATES = {"exp_avg": 0, "exp_avg_sq": 1}
UPDATES = {"grad_norm": 0, "adamw": 1, "adamw_packed": 2}
STATE_BLOCK = 256
# the model's ends: types of tokens and targets, elements of a packed activations' block
INDICES = {"i32": 0, "i64": 1}
ACTIVATION_BLOCK = 32
# bytes of the fixed device array behind ar_reduce_scatter_noalloc
NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None

_vp = ctypes.c_void_p
_vpp = ctypes.POINTER(ctypes.c_void_p)
_sz = ctypes.c_size_t
_int = ctypes.c_int
_szp = ctypes.POINTER(ctypes.c_size_t)


class AdamwConfig(ctypes.Structure):
    """ar_adamw_config_t"""

    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("max_norm", ctypes.c_double),
                ("grad_scale", ctypes.c_double), ("step", ctypes.c_ulonglong), ("seed", ctypes.c_uint),
                ("skip_nonfinite", _int)]


class AdamwTensors(ctypes.Structure):
    """ar_adamw_tensors_t"""

    _fields_ = [("ntensors", _int), ("counts", _szp), ("param_dtype", _int), ("grad_dtype", _int),
                ("copy_dtype", _int)] + [(name, _vpp) for name in (
                    "params", "grads", "exp_avgs", "exp_avg_sqs", "exp_avg_scales", "exp_avg_sq_scales",
                    "params_out", "exp_avgs_out", "exp_avg_sqs_out", "exp_avg_scales_out", "exp_avg_sq_scales_out",
                    "copies")]


_tensors = ctypes.POINTER(AdamwTensors)
_config = ctypes.POINTER(AdamwConfig)


def _declare(lib):
    sig = {
        "ar_allreduce": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _vp]),
        "ar_reduce_scatter": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _vp]),
        "ar_all_gather": (_int, [_vpp, _vpp, _sz, _int, _int, _vp]),
        "ar_allreduce_ex": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _int, _vp, _sz, _vp]),
        "ar_reduce_scatter_ex": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _int, _vp, _sz, _vp]),
        "ar_all_gather_ex": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _vp, _sz, _vp]),
        "ar_workspace_bytes": (_sz, [_int, _int, _sz, _int, _int]),
        "ar_chunk_range": (_int, [_int, _sz, _int, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]),
        "ar_get_error_string": (ctypes.c_char_p, [_int]),
        "ar_get_last_error_detail": (ctypes.c_char_p, []),
        "ar_dtype_size": (_sz, [_int]),
        "ar_allreduce_init": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _int, _vp, _sz, _vpp]),
        "ar_reduce_scatter_init": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _int, _vp, _sz, _vpp]),
        "ar_all_gather_init": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _vp, _sz, _vpp]),
        "ar_plan_start": (_int, [_vp, _vp]),
        "ar_plan_num_launches": (_int, [_vp]),
        "ar_plan_algo": (_int, [_vp]),
        "ar_plan_free": (_int, [_vp]),
        "ar_plan_limit_blocks": (_int, [_vp, ctypes.c_uint]),
        "ar_reduce_scatter_noalloc": (_int, [_vpp, _vpp, _sz, _int, _int, _int, _int, _vp]),
        "ar_grad_norm": (_int, [_vpp, _szp, _int, _int, _vp, _vp, _sz, _vp]),
        "ar_grad_norm_init": (_int, [_vpp, _szp, _int, _int, _vp, _vp, _sz, _vp, _vpp]),
        "ar_grad_norm_start": (_int, [_vp, _vp]),
        "ar_adamw": (_int, [_tensors, _config, _vp, _vp]),
        "ar_adamw_packed": (_int, [_tensors, _config, _vp, _vp]),
        "ar_adamw_init": (_int, [_tensors, _vp, _sz, _vp, _vpp]),
        "ar_adamw_packed_init": (_int, [_tensors, _vp, _sz, _vp, _vpp]),
        "ar_adamw_start": (_int, [_vp, _config, _vp, _vp]),
        "ar_unpack_states": (_int, [_vpp, _vpp, _vpp, _szp, _int, _int, _int, _vp]),
        "ar_update_workspace_bytes": (_sz, [_int, _szp, _int]),
        "ar_update_num_launches": (_int, [_vp]),
        "ar_update_free": (_int, [_vp]),
        "ar_layer_norm": (_int, [_vpp, _vpp, _vpp, _vpp, _vpp, _vpp, _sz, _sz, _sz, _sz, _int, _int,
                                 ctypes.c_double, _int, _vp]),
        "ar_layer_norm_backward": (_int, [_vpp] * 8 + [_sz] * 5 + [_int, _int, _int, _vp, _sz, _vp]),
        "ar_layer_norm_workspace_bytes": (_sz, [_sz, _sz, _int]),
        "ar_embedding": (_int, [_vpp] * 3 + [_sz] * 5 + [_int] * 3 + [ctypes.c_double, _int, _vp]),
        "ar_embedding_backward": (_int, [_vpp] * 3 + [_sz] * 5 + [_int] * 3
                                  + [ctypes.c_double, ctypes.c_longlong, _int, _int, _vp, _sz, _vp]),
        "ar_embedding_workspace_bytes": (_sz, [_sz, _sz, _sz, _int]),
        "ar_cross_entropy": (_int, [_vpp] * 5 + [_sz] * 5 + [_int, ctypes.c_longlong, _int, _int, _vp, _sz, _vp]),
        "ar_cross_entropy_backward": (_int, [_vpp] * 7 + [_sz] * 7 + [_int, ctypes.c_longlong, _int, ctypes.c_double,
                                                                      _int, _vp, _sz, _vp]),
        "ar_cross_entropy_workspace_bytes": (_sz, [_sz, _sz, _sz, _int, _int, _int]),
        "ar_cross_entropy_aligned_workspace_bytes": (_sz, [_sz, _sz, _sz, _int, _int, _int]),
        "ar_pack_activations": (_int, [_vpp] * 3 + [_sz] * 3 + [_int, _int, _vp]),
        "ar_unpack_activations": (_int, [_vpp] * 3 + [_sz] * 3 + [_int, _int, _vp]),
        "ar_layer_norm_backward_packed": (_int, [_vpp] * 9 + [_sz] * 4 + [_int, _int, _int, _vp, _sz, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


def lib():
    """The loaded library; raises if libar.so is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is not built; build it with "
                "`python -m ring_allreduce_reduction_virtual_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        _declare(handle)
        _lib = handle
    return _lib


class ArError(RuntimeError):
    """A call into libar.so returned an error code."""

    def __init__(self, fn: str, code: int):
        L = lib()
        detail = L.ar_get_last_error_detail().decode()
        msg = L.ar_get_error_string(code).decode()
        super().__init__(f"{fn}: {RESULT_NAMES.get(code, code)} ({msg}){': ' + detail if detail else ''}")
        self.code = code
        self.detail = detail


def check(fn: str, code: int):
    if code != AR_SUCCESS:
        raise ArError(fn, code)


def ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(len(ptrs), 1))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr
