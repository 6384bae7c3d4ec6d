"""GB300-native (sm_103a) ZeRO / FSDP sharded mixed-precision step over a
FlatParameter, with all N_d logical data-parallel ranks held in one GPU.

The compute lives in the CUDA library declared by ``include/zero_flat.h``;
``zero``, ``root_ops`` and ``layer_ops`` are its thin ctypes binding (same function names), ``buffers`` lays
out per-rank device buffers with PyTorch allocations, ``synthetic`` draws the
seeded synthetic workloads, and ``build`` compiles the library in-tree.
"""
from .zero import (ZERO_MAX_RANKS, zero1_accumulate, zero1_step, zero_param_layout,
                   zero_shard_numel, ZeroAdamW, ZeroError, ZeroLayout, load, zero_abi_version,
                   zero_adamw_shard_step, zero_all_gather, zero_device_status, zero_flat_layout,
                   zero_flatten, zero_last_error, zero_reduce_scatter,
                   zero_selftest_tile_wait_timeout, zero_selftest_wait_timeout,
                   zero_shard_segments, zero_step, zero_step_units, zero_step_units_clip,
                   zero_step_units_clip_noalloc, zero_clip_workspace_bytes, zero_unflatten,
                   zero_step_units_host, HostTables, ZERO_HOST_GRADS_FREE,
                   ZERO_HOST_SM_COPY)
from .root_ops import (ZERO_MAX_NORM_DIM, ZERO_MAX_TEACHER, zero_distill_loss,
                       zero_distill_loss_grad, zero_embedding, zero_embedding_grad,
                       zero_embedding_grad_workspace_bytes, zero_layer_norm, zero_layer_norm_grad,
                       zero_layer_norm_grad_workspace_bytes)
from .layer_ops import (ZERO_EIGHT_BLOCK, ZERO_MAX_HEAD_DIM, ZERO_MAX_HEAD_TOKENS,
                        ZERO_MAX_HEAD_VOCAB, zero_head_loss, zero_head_loss_grad,
                        zero_head_loss_grad_in_place_workspace_bytes,
                        zero_head_loss_grad_workspace_bytes,
                        zero_head_loss_in_place_workspace_bytes, zero_head_loss_workspace_bytes,
                        zero_pack_rows, zero_rms_norm, zero_rms_norm_grad,
                        zero_rms_norm_grad_workspace_bytes, zero_unpack_rows)

__all__ = [
    "ZERO_MAX_RANKS", "zero1_accumulate", "zero1_step", "zero_param_layout", "zero_shard_numel", "ZeroAdamW", "ZeroError", "ZeroLayout", "load", "zero_abi_version",
    "zero_adamw_shard_step", "zero_all_gather", "zero_device_status", "zero_flat_layout",
    "zero_flatten",
    "zero_last_error", "zero_reduce_scatter", "zero_selftest_tile_wait_timeout",
    "zero_selftest_wait_timeout",
    "zero_shard_segments", "zero_step", "zero_step_units", "zero_step_units_clip",
    "zero_clip_workspace_bytes", "zero_step_units_clip_noalloc",
    "zero_unflatten", "zero_step_units_host", "HostTables", "ZERO_HOST_GRADS_FREE", "ZERO_HOST_SM_COPY",
    "ZERO_MAX_NORM_DIM", "ZERO_MAX_TEACHER", "zero_distill_loss", "zero_distill_loss_grad",
    "zero_embedding", "zero_embedding_grad", "zero_embedding_grad_workspace_bytes",
    "zero_layer_norm", "zero_layer_norm_grad", "zero_layer_norm_grad_workspace_bytes",
    "ZERO_EIGHT_BLOCK", "zero_pack_rows", "zero_rms_norm", "zero_rms_norm_grad",
    "zero_rms_norm_grad_workspace_bytes", "zero_unpack_rows",
    "ZERO_MAX_HEAD_DIM", "ZERO_MAX_HEAD_TOKENS", "ZERO_MAX_HEAD_VOCAB", "zero_head_loss",
    "zero_head_loss_grad", "zero_head_loss_grad_in_place_workspace_bytes",
    "zero_head_loss_grad_workspace_bytes", "zero_head_loss_in_place_workspace_bytes",
    "zero_head_loss_workspace_bytes",
]
