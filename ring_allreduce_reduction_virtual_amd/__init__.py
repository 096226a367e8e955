"""Ring AllReduce over N virtual ranks in one MI355X's HBM.

The computation lives in libar.so (HIP kernels for gfx950 behind the C ABI of
include/ar.h); this package is its Python binding, with the C functions'
names, taking torch tensors.  Importing the package does not load the
library; the first call does, and fails loudly if it is not built.
"""

from ._lib import ArError, lib  # noqa: F401
from .binding import (  # noqa: F401
    Plan,
    ar_all_gather,
    ar_all_gather_ex,
    ar_all_gather_init,
    ar_allreduce,
    ar_allreduce_ex,
    ar_allreduce_init,
    ar_chunk_range,
    ar_dtype_size,
    ar_get_error_string,
    ar_get_last_error_detail,
    ar_plan_algo,
    ar_plan_free,
    ar_plan_limit_blocks,
    ar_plan_num_launches,
    ar_plan_start,
    ar_reduce_scatter,
    ar_reduce_scatter_ex,
    ar_reduce_scatter_init,
    ar_reduce_scatter_noalloc,
    ar_workspace_bytes,
)
from .model import (  # noqa: F401
    PackedRows,
    ar_cross_entropy,
    ar_cross_entropy_aligned_workspace_bytes,
    ar_cross_entropy_backward,
    ar_cross_entropy_workspace_bytes,
    ar_embedding,
    ar_embedding_backward,
    ar_embedding_workspace_bytes,
    ar_layer_norm_backward_packed,
    ar_pack_activations,
    ar_unpack_activations,
)
from .step import (  # noqa: F401
    PackedState,
    Update,
    ar_adamw,
    ar_adamw_init,
    ar_adamw_packed,
    ar_adamw_packed_init,
    ar_adamw_start,
    ar_grad_norm,
    ar_grad_norm_init,
    ar_grad_norm_start,
    ar_layer_norm,
    ar_layer_norm_backward,
    ar_layer_norm_workspace_bytes,
    ar_unpack_states,
    ar_update_free,
    ar_update_num_launches,
    ar_update_workspace_bytes,
)

__all__ = [
    "ArError", "lib", "Plan",
    "ar_allreduce", "ar_allreduce_ex", "ar_reduce_scatter", "ar_reduce_scatter_ex",
    "ar_all_gather", "ar_all_gather_ex", "ar_workspace_bytes", "ar_chunk_range",
    "ar_get_error_string", "ar_get_last_error_detail", "ar_dtype_size",
    "ar_allreduce_init", "ar_reduce_scatter_init", "ar_all_gather_init", "ar_plan_start", "ar_plan_free",
    "ar_plan_limit_blocks", "ar_plan_num_launches", "ar_reduce_scatter_noalloc", "ar_plan_algo",
    "PackedState", "Update", "ar_grad_norm", "ar_grad_norm_init", "ar_grad_norm_start",
    "ar_adamw", "ar_adamw_init", "ar_adamw_packed", "ar_adamw_packed_init", "ar_adamw_start", "ar_unpack_states",
    "ar_update_workspace_bytes", "ar_update_num_launches", "ar_update_free",
    "ar_layer_norm", "ar_layer_norm_backward", "ar_layer_norm_workspace_bytes",
    "ar_embedding", "ar_embedding_backward", "ar_embedding_workspace_bytes",
    "ar_cross_entropy", "ar_cross_entropy_backward", "ar_cross_entropy_workspace_bytes",
    "ar_cross_entropy_aligned_workspace_bytes",
    "PackedRows", "ar_pack_activations", "ar_unpack_activations", "ar_layer_norm_backward_packed",
]
