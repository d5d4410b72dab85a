"""Bucketed gradient synchronisation for MI355X (gfx950).

The data-parallel reducer's hot path: parameters are assigned to buckets in
reverse definition order under a byte cap; each gradient hook marks its
variable ready; complete buckets are launched strictly in bucket-index order on
a side HIP stream, where hand-written CDNA4 kernels average the R replicas'
gradients in HBM and write the mean back to every replica; ``no_sync``
accumulates local steps before one synchronisation. Behind it, ``GradNorm`` and
``AdamW`` take the averaged gradients through the optimizer step: the global
norm with its clip coefficient, and AdamW over all tensors in one launch, with
32-bit or 8-bit states. Before it, ``layer_norm``, ``dropout`` and
``embedding`` with their backward passes make gradients where the reducer is
bound to them.

The native library (``lib/libddpb.so``, C ABI in ``include/ddpb.h``) does all
of the work; this package only marshals arguments. Importing the package does
not load the library; the first use does, and fails loudly if it was not built.
"""
from ._abi import (DdpbError, Lib, lib, F32, BF16, F16, MODE_FUSED, MODE_STAGED, STATIC_SCRATCH_BYTES,  # noqa: F401
                   BIND_DEVICE_TIMESTAMPS, BIND_TIME_LAUNCHES, BIND_ROCTX, BIND_OVERLAP, HIP_LIB, HOSTONLY_LIB, SYMBOLS,
                   NORM_SKIP_NONFINITE, STATE_F32, STATE_F8, STATE_BLOCK, ADAMW_MASTER,
                   OK, E_ARG, E_INDEX, E_DOUBLE_READY, E_INCOMPLETE, E_STATE, E_HIP, E_NOMEM)
from .layers import (Drop, Normed, NormGrads, dropout, dropout_backward, embedding, embedding_backward,  # noqa: F401
                     layer_norm, layer_norm_backward)
from .optim import AdamW, GradNorm  # noqa: F401
from .reducer import Reducer, StepTable  # noqa: F401


def _fwd(name):
    def f(*args, **kw):
        return getattr(lib(), name)(*args, **kw)
    f.__name__ = name
    f.__doc__ = f"Forwards to ddpb_{name} of the HIP library."
    return f


# Module-level functions with the C ABI's names (without the ddpb_ prefix). Those
# of layers.py, which have names of the ABI too, take tensors.
for _n in ["reducer_create", "destroy", "num_buckets", "get_locator", "get_bucket", "num_segments",
           "get_bucket_segments", "get_segment", "workspace_bytes", "bind", "ensure_prior_reduction_finished",
           "mark_ready", "mark_ready_many", "finalize", "set_sync", "no_sync_accumulate", "reset",
           "get_launch_log", "get_launch_times", "device_clock_hz", "last_error", "set_launch_blocks",
           "set_workgroups_per_cu",
           "view_storage_elems", "get_view_offset", "bind_bucket_views", "rebuild_buckets", "get_ready_order",
           "set_local_used", "set_sync_step", "bind_static",
           "norm_create", "norm_destroy", "norm_workspace_bytes", "norm_bind", "norm_compute",
           "adamw_create", "adamw_destroy", "adamw_workspace_bytes", "adamw_bind", "adamw_step",
           "adamw_set_step", "adamw_get_step", "check_writable", "begin_writes"]:
    globals()[_n] = _fwd(_n)
del _n
