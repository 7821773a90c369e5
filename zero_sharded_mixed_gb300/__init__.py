"""ZeRO stage-1/2/3 sharded mixed-precision step for GB300 (sm_103a).

The compute lives in ``libzero_gb300.so`` (hand-written CUDA kernels behind a
C ABI, declared in ``include/zero_gb300.h``); ``binding`` is a thin ctypes layer
with the same names.  The library is loaded on first use of a binding name, so
importing ``zero_sharded_mixed_gb300.inputs`` alone does not need a GPU or a
built library.  There is no CPU fallback: if the library is missing, every
binding call raises.
"""
from __future__ import annotations

_BINDING_NAMES = {
    "ZeroError", "ZeroLayout", "ZeroAdamW", "lib_path", "load",
    "zero_layout", "zero_reduce_scatter_adamw", "zero_gather_layer", "zero_accumulate", "zero_cast_bf16",
    "zero_reduce_scatter_adamw_clip", "zero_accumulate_adamw", "zero_grad_norm_workspace",
    "zero_grad_norm_sq", "zero_grad_norm_sq_static", "zero_quantize_int8", "zero_gather_layer_int8",
    "zero_reduce_scatter_adamw_int8", "zero_accumulate_int8", "zero_reduce_scatter_adamw_q8",
    "zero_reduce_scatter_adamw_int8_q8", "zero_schedule_fill", "zero_schedule_advance",
    "zero_status_check", "zero_strerror", "zero_memory_bytes", "zero_comm_bytes",
    "zero_bucket_range", "zero_shard_range", "zero_selftest_bounded_wait", "zero_lr_warmup_decay",
    "ZERO_OK", "ZERO_EINVAL", "ZERO_EALIGN", "ZERO_ERANGE", "ZERO_ECUDA", "ZERO_ETIMEOUT",
    "ZERO_EIO", "ZERO_ECORRUPT",
    "ZERO_BF16", "ZERO_F32", "ZERO_OUT_FULL", "ZERO_OUT_SHARD",
    "ZERO_ACC_LOCAL", "ZERO_ACC_REDUCE", "ZERO_MAX_SRC",
    "ZeroDropout", "ZeroRopePlan", "zero_linear", "zero_linear_grad_input", "zero_linear_grad_weight",
    "zero_dropout", "zero_dropout_grad", "zero_rope_plan", "zero_rope",
    "ZERO_ACT_NONE", "ZERO_ACT_RELU", "ZERO_ACT_GELU", "ZERO_ACT_GELU_TANH", "ZERO_ACT_SILU",
    "ZERO_ROPE_HALF", "ZERO_ROPE_INTERLEAVED", "ZERO_ROPE_NONE", "ZERO_ROPE_LINEAR", "ZERO_ROPE_NTK",
    "ZERO_ROPE_YARN", "ZERO_ROPE_MAX",
    "ZeroMuon", "zero_layer_norm", "zero_layer_norm_grad", "zero_layer_norm_grad_workspace",
    "zero_reduce_scatter_momentum", "zero_muon_update", "zero_orthogonalize", "zero_orthogonalize_workspace",
}


_ENGINE_NAMES = {"ZeroEngine", "Zero3Engine"}


_binding = None   # the module, looked up once; its names anew each time, so that a replaced one is seen


def __getattr__(name):
    if name in _BINDING_NAMES:
        global _binding
        if _binding is None:
            from . import binding
            _binding = binding
        return getattr(_binding, name)
    if name in _ENGINE_NAMES:
        from . import engine
        return getattr(engine, name)
    if name == "ZeroConfig":
        from .config import ZeroConfig
        return ZeroConfig
    raise AttributeError(name)
