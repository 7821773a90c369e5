"""Thin ctypes binding for libzero_gb300.so (names as in include/zero_gb300.h).

Argument marshalling only: torch tensors are checked (device, dtype,
contiguity, extent) and turned into pointers; every step of the computation
runs in the library's CUDA kernels.  There is no CPU fallback: if the library
is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libzero_gb300.so")

ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE, ZERO_ECUDA, ZERO_ETIMEOUT = 0, -1, -2, -3, -4, -5
ZERO_EIO, ZERO_ECORRUPT = -6, -7
ZERO_BF16, ZERO_F32 = 0, 1
ZERO_OUT_FULL, ZERO_OUT_SHARD = 0, 1
ZERO_ACC_LOCAL, ZERO_ACC_REDUCE = 0, 1
ZERO_MAX_SRC = 64
ZERO_ACT_NONE, ZERO_ACT_RELU, ZERO_ACT_GELU, ZERO_ACT_GELU_TANH, ZERO_ACT_SILU = 0, 1, 2, 3, 4
ZERO_ROPE_HALF, ZERO_ROPE_INTERLEAVED = 0, 1
ZERO_ROPE_NONE, ZERO_ROPE_LINEAR, ZERO_ROPE_NTK, ZERO_ROPE_YARN = 0, 1, 2, 3
ZERO_ROPE_MAX = 256


class ZeroError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        detail = ""
        if code == ZERO_ECUDA:
            detail = f" [{load().zero_last_cuda_error().decode()}]"
        super().__init__(f"{where}: {zero_strerror(code)} ({code}){detail}")


class ZeroLayout(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("padded_n", ctypes.c_int64), ("shard", ctypes.c_int64),
                ("align", ctypes.c_int64), ("bucket", ctypes.c_int64), ("n_buckets", ctypes.c_int64),
                ("n_dp", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "reserved"}

    def __repr__(self):
        return f"ZeroLayout({self.as_dict()})"


class ZeroCkptHeader(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("padded_n", ctypes.c_int64), ("shard", ctypes.c_int64),
                ("align", ctypes.c_int64), ("step", ctypes.c_int64), ("n_dp", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class ZeroAdamW(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("step", ctypes.c_int64),
                ("sched", ctypes.c_void_p)]

    @classmethod
    def make(cls, lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, sched=None):
        """sched: None, or a CUDA float32 tensor of 3 elements {lr, bc1, bc2}
        that the kernels read in place of lr and step.  The block keeps a
        reference to it, so the memory outlives every call made with the block."""
        ptr = None
        if sched is not None:
            ptr = _tensor(sched, "sched", torch.float32, 3)
        hp = cls(lr, beta1, beta2, eps, weight_decay, 0, step, ptr)
        hp._sched_tensor = sched
        return hp


class ZeroMuon(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale", ctypes.c_float), ("nesterov", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("sched", ctypes.c_void_p)]

    @classmethod
    def make(cls, lr=0.02, momentum=0.95, weight_decay=0.0, scale=1.0, nesterov=True, sched=None):
        """scale: what the orthogonalised matrix is multiplied with beside lr (for one
        of n rows and k columns 0.2 sqrt(max(n, k)) gives updates of AdamW's size).
        sched: None, or a CUDA float32 tensor whose first element the update reads in
        place of lr (a StepSchedule's sched); the block keeps a reference to it."""
        ptr = None if sched is None else _tensor(sched, "sched", torch.float32, 1)
        hp = cls(lr, momentum, weight_decay, scale, int(bool(nesterov)), 0, ptr)
        hp._sched_tensor = sched
        return hp


class ZeroDropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("site", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("step", ctypes.c_uint64),
                ("step_ptr", ctypes.c_void_p)]

    @classmethod
    def make(cls, p: float, seed: int = 0, site: int = 0, step: int = 0, step_ptr=None):
        """One place (site) and pass (step) of dropout with share p.  step_ptr:
        None, or a CUDA int64 tensor whose element the kernels add to step (a
        StepSchedule's step_index, so that each replay of a captured step drops
        other elements); the block keeps a reference to it."""
        if not (0 <= seed < 1 << 64 and 0 <= site < 1 << 32 and 0 <= step < 1 << 32):
            raise ValueError("seed must fit 64 bits, site and step 32, none negative")
        ptr = None if step_ptr is None else _tensor(step_ptr, "step_ptr", torch.int64, 1)
        drop = cls(p, seed, site, 0, step, ptr)
        drop._step_tensor = step_ptr
        return drop


class ZeroRopePlan(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turn", ctypes.c_uint64 * (ZERO_ROPE_MAX // 2))]


_lock = threading.Lock()
_lib = None


def load():
    """Load the library (raises if it has not been built)."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(lib_path):
            raise ImportError(
                f"{lib_path} is missing: build it with `python -m zero_sharded_mixed_gb300.build` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(lib_path)
        i32, i64, f32, p = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
        P = ctypes.POINTER
        lib.zero_layout.argtypes = [P(i64), i32, i32, i64, i64, P(i64), P(ZeroLayout)]
        lib.zero_bucket_range.argtypes = [P(ZeroLayout), i64, P(i64), P(i64)]
        lib.zero_shard_range.argtypes = [P(ZeroLayout), i32, P(i64), P(i64), P(i64)]
        lib.zero_reduce_scatter_adamw.argtypes = [
            P(ZeroLayout), P(p), i32, i32, i64, f32, i32, i32, i64, i64,
            p, p, p, p, i32, P(ZeroAdamW), p]
        lib.zero_reduce_scatter_adamw_clip.argtypes = [
            P(ZeroLayout), P(p), i32, i32, i64, f32, i32, i32, i64, i64,
            p, p, p, p, i32, P(ZeroAdamW), p, f32, p]
        lib.zero_accumulate_adamw.argtypes = [
            P(ZeroLayout), i32, P(p), i32, i64, P(p), i32, i64, f32, i32, i32, i64, i64,
            p, p, p, p, i32, P(ZeroAdamW), p]
        lib.zero_grad_norm_workspace.argtypes = [P(i64)]
        lib.zero_grad_norm_sq.argtypes = [P(ZeroLayout), P(p), i32, i32, i64, f32, i64, i64,
                                          p, i64, p, i32, p]
        lib.zero_grad_norm_sq_static.argtypes = [P(ZeroLayout), P(p), i32, i32, i64, f32, i64,
                                                 i64, p, i32, p]
        lib.zero_gather_layer.argtypes = [P(ZeroLayout), P(p), p, p]
        lib.zero_cast_bf16.argtypes = [p, p, i64, p]
        lib.zero_quantize_int8.argtypes = [P(ZeroLayout), p, p, p, i32, p]
        lib.zero_ckpt_write_shard.argtypes = [ctypes.c_char_p, P(ZeroCkptHeader), p, p, p, p]
        lib.zero_ckpt_read_header.argtypes = [ctypes.c_char_p, P(ZeroCkptHeader), P(i32)]
        lib.zero_ckpt_read_shard.argtypes = [ctypes.c_char_p, P(ZeroCkptHeader), p, p, p, p, i64]
        lib.zero_selftest_bounded_wait.argtypes = [i64, p]
        lib.zero_schedule_fill.argtypes = [P(ZeroAdamW), i64, i64, p, p]
        lib.zero_schedule_advance.argtypes = [p, i64, p, p, p]
        lib.zero_crc32.argtypes = [p, i64]
        lib.zero_ckpt_payload_crc.argtypes = [ctypes.c_char_p, P(ctypes.c_uint32)]
        lib.zero_crc32.restype = ctypes.c_uint32
        lib.zero_gather_layer_int8.argtypes = [P(ZeroLayout), P(p), P(p), i32, p, p]
        lib.zero_reduce_scatter_adamw_q8.argtypes = [
            P(ZeroLayout), P(p), i32, i32, i64, f32, i32, i32, i64, i64,
            p, p, p, p, p, i32, P(ZeroAdamW), p]
        lib.zero_reduce_scatter_adamw_int8_q8.argtypes = [
            P(ZeroLayout), P(p), P(p), i32, i32, f32, i32, i32, i64, i64,
            p, p, p, p, p, i32, P(ZeroAdamW), p]
        lib.zero_reduce_scatter_adamw_int8.argtypes = [
            P(ZeroLayout), P(p), P(p), i32, i32, f32, i32, i32, i64, i64,
            p, p, p, p, i32, P(ZeroAdamW), p]
        lib.zero_accumulate_int8.argtypes = [P(ZeroLayout), P(p), P(p), i32, i32, p, i64, i64, i64,
                                             i32, p]
        lib.zero_accumulate.argtypes = [P(ZeroLayout), i32, P(p), i32, i32, i64, p, i64, i64, i64,
                                        i32, p]
        D = P(ZeroDropout)
        lib.zero_linear.argtypes = [i64, i64, i64, p, i64, p, i64, p, i32, D, p, i64, p, i64, p, i32,
                                    i64, p]
        lib.zero_linear_grad_input.argtypes = [i64, i64, i64, p, i64, p, i64, i32, D, p, i64, p, i64, p,
                                               i32, i64, p]
        lib.zero_linear_grad_weight.argtypes = [i64, i64, i64, p, i64, p, i64, p, i64, p, i32, i64, p,
                                                p, p]
        lib.zero_dropout.argtypes = [i64, i64, p, i64, i32, D, p, i64, p, i64, p]
        lib.zero_dropout_grad.argtypes = [i64, i64, p, i64, i32, D, i32, p, i64, p, i32, i64, p, p, i32,
                                          p]
        lib.zero_rope_fill.argtypes = [i32, i32, ctypes.c_double, i32, ctypes.c_double, ctypes.c_double,
                                       P(ZeroRopePlan)]
        lib.zero_rope.argtypes = [P(ZeroRopePlan), i64, i64, i64, p, i64, i64, p, i64, i64, i32, p, i64,
                                  i32, p]
        lib.zero_layer_norm.argtypes = [i64, i64, p, i64, i32, p, i64, p, i64, p, p, f32, p, i32, i64, p, p, p]
        lib.zero_layer_norm_grad_workspace.argtypes = [i64, i64, P(i64)]
        lib.zero_layer_norm_grad.argtypes = [i64, i64, p, i64, i32, p, i64, p, p, p, p, i64, p, i32, i64,
                                             p, p, p, p, i32, p, i64, p]
        M = P(ZeroMuon)
        lib.zero_reduce_scatter_momentum.argtypes = [P(ZeroLayout), P(p), i32, i32, i64, f32, i32, i32, i64, i64,
                                                     p, p, i32, M, p]
        lib.zero_muon_update.argtypes = [P(ZeroLayout), p, i64, i32, i32, i64, i64, p, p, i32, M, p]
        lib.zero_orthogonalize_workspace.argtypes = [i64, i64, i64, P(i64)]
        lib.zero_orthogonalize.argtypes = [i64, i64, i64, p, i64, i64, i32, p, i64, i64, i32, P(f32), f32,
                                           p, i64, p]
        lib.zero_status_check.argtypes = [p]
        lib.zero_strerror.argtypes = [ctypes.c_int]
        lib.zero_strerror.restype = ctypes.c_char_p
        lib.zero_last_cuda_error.argtypes = []
        lib.zero_last_cuda_error.restype = ctypes.c_char_p
        lib.zero_memory_bytes.argtypes = [ctypes.c_double, i32, i32, ctypes.c_double,
                                          P(ctypes.c_double)]
        lib.zero_comm_bytes.argtypes = [ctypes.c_double, i32, i32, ctypes.c_double,
                                        ctypes.c_double, P(ctypes.c_double)]
        lib.zero_lr_warmup_decay.argtypes = [i64, ctypes.c_double, ctypes.c_double, i64, i64, P(f32)]
        for name in ("zero_layout", "zero_bucket_range", "zero_shard_range",
                     "zero_reduce_scatter_adamw", "zero_reduce_scatter_adamw_clip",
                     "zero_accumulate_adamw", "zero_grad_norm_workspace", "zero_grad_norm_sq",
                     "zero_grad_norm_sq_static", "zero_quantize_int8", "zero_gather_layer_int8",
                     "zero_ckpt_write_shard", "zero_ckpt_read_header", "zero_ckpt_read_shard",
                     "zero_ckpt_payload_crc",
                     "zero_selftest_bounded_wait", "zero_reduce_scatter_adamw_int8",
                     "zero_reduce_scatter_adamw_q8", "zero_reduce_scatter_adamw_int8_q8",
                     "zero_schedule_fill", "zero_schedule_advance",
                     "zero_accumulate_int8", "zero_gather_layer", "zero_accumulate",
                     "zero_status_check", "zero_memory_bytes", "zero_comm_bytes",
                     "zero_lr_warmup_decay", "zero_linear", "zero_linear_grad_input",
                     "zero_linear_grad_weight", "zero_dropout", "zero_dropout_grad",
                     "zero_rope_fill", "zero_rope", "zero_layer_norm", "zero_layer_norm_grad_workspace",
                     "zero_layer_norm_grad", "zero_reduce_scatter_momentum", "zero_muon_update",
                     "zero_orthogonalize_workspace", "zero_orthogonalize"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def zero_strerror(code: int) -> str:
    return load().zero_strerror(int(code)).decode()


def _check(rc: int, where: str):
    if rc != ZERO_OK:
        raise ZeroError(rc, where)


# --------------------------------------------------------------------------
# host-only calls
# --------------------------------------------------------------------------

def zero_layout(numels: Sequence[int], n_dp: int, align: int = 8,
                bucket_elems: int = 500_000_000, with_offsets: bool = False):
    arr = (ctypes.c_int64 * max(1, len(numels)))(*[int(x) for x in numels])
    offs = (ctypes.c_int64 * max(1, len(numels)))()
    L = ZeroLayout()
    _check(load().zero_layout(arr, len(numels), int(n_dp), int(align), int(bucket_elems), offs,
                              ctypes.byref(L)), "zero_layout")
    if with_offsets:
        return L, [offs[i] for i in range(len(numels))]
    return L


def zero_bucket_range(L: ZeroLayout, b: int):
    lo, hi = ctypes.c_int64(), ctypes.c_int64()
    _check(load().zero_bucket_range(ctypes.byref(L), int(b), ctypes.byref(lo), ctypes.byref(hi)),
           "zero_bucket_range")
    return lo.value, hi.value


def zero_shard_range(L: ZeroLayout, rank: int):
    lo, hi, valid = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(load().zero_shard_range(ctypes.byref(L), int(rank), ctypes.byref(lo), ctypes.byref(hi),
                                   ctypes.byref(valid)), "zero_shard_range")
    return lo.value, hi.value, valid.value


def zero_lr_warmup_decay(t: int, min_lr: float, max_lr: float, warmup_steps: int,
                         total_steps: int) -> float:
    """The learning rate of optimizer step t (>= 1) under WarmupDecayLR."""
    out = ctypes.c_float()
    _check(load().zero_lr_warmup_decay(int(t), float(min_lr), float(max_lr), int(warmup_steps),
                                       int(total_steps), ctypes.byref(out)), "zero_lr_warmup_decay")
    return out.value


def zero_memory_bytes(n, n_dp, stage, k_bytes=12.0) -> float:
    out = ctypes.c_double()
    _check(load().zero_memory_bytes(float(n), int(n_dp), int(stage), float(k_bytes),
                                    ctypes.byref(out)), "zero_memory_bytes")
    return out.value


def zero_comm_bytes(n, n_dp, stage, param_bytes=2.0, grad_bytes=2.0) -> float:
    out = ctypes.c_double()
    _check(load().zero_comm_bytes(float(n), int(n_dp), int(stage), float(param_bytes),
                                  float(grad_bytes), ctypes.byref(out)), "zero_comm_bytes")
    return out.value


# --------------------------------------------------------------------------
# device calls
# --------------------------------------------------------------------------

# The current stream's handle without a Stream object around it (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device_index = getattr(torch._C, "_cuda_getDevice", None)
_cuda_ready = torch.cuda.is_initialized


def _stream_ptr(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None and _device_index is not None and _cuda_ready():
            return _raw_stream(_device_index()) or None
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _tensor(t: torch.Tensor, name: str, dtype, min_numel: int, pinned_ok: bool = False) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        if not (pinned_ok and t.device.type == "cpu"):
            raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); there is no CPU path")
        if not t.is_pinned():
            raise ValueError(f"{name} is host memory but not pinned; the kernels read only "
                             "device memory or pinned host memory")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements, the call reads or writes {min_numel}")
    return t.data_ptr()


_SRC_DT = {ZERO_BF16: torch.bfloat16, ZERO_F32: torch.float32}


def _src_array(srcs, dtype, min_numel, pinned_ok=False):
    if len(srcs) == 0:
        raise ValueError("need at least one source")
    ptrs = [_tensor(s, f"src[{i}]", dtype, min_numel, pinned_ok) for i, s in enumerate(srcs)]
    return (ctypes.c_void_p * len(ptrs))(*ptrs), len(ptrs)


def zero_reduce_scatter_adamw(L: ZeroLayout, srcs, src_dtype: int, src_base: int, divisor: float,
                              rank_begin: int, rank_end: int, begin: int, end: int,
                              master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                              out: torch.Tensor, out_mode: int, hp: ZeroAdamW, stream=None):
    """Fused mean reduce-scatter + AdamW + bf16 cast + gather write over [begin, end).
    The sources may be pinned host tensors: the kernel then reads them over the
    host link."""
    if end <= begin:
        src_need = state_need = out_need = 0
    else:
        src_need = end - src_base
        state_need = end - rank_begin * L.shard
        out_need = end if out_mode == ZERO_OUT_FULL else state_need
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need, pinned_ok=True)
    rc = load().zero_reduce_scatter_adamw(
        ctypes.byref(L), arr, n, int(src_dtype), int(src_base), float(divisor),
        int(rank_begin), int(rank_end), int(begin), int(end),
        _tensor(master, "master", torch.float32, state_need),
        _tensor(m, "m", torch.float32, state_need),
        _tensor(v, "v", torch.float32, state_need),
        _tensor(out, "out", torch.bfloat16, out_need),
        int(out_mode), ctypes.byref(hp), _stream_ptr(stream))
    _check(rc, "zero_reduce_scatter_adamw")


def zero_reduce_scatter_adamw_clip(L: ZeroLayout, srcs, src_dtype: int, src_base: int,
                                   divisor: float, rank_begin: int, rank_end: int, begin: int,
                                   end: int, master: torch.Tensor, m: torch.Tensor,
                                   v: torch.Tensor, out: torch.Tensor, out_mode: int,
                                   hp: ZeroAdamW, norm_sq: torch.Tensor, max_norm: float,
                                   stream=None):
    """zero_reduce_scatter_adamw with the mean gradient scaled by
    min(1, max_norm / (sqrt(norm_sq) + 1e-6)); norm_sq is a 1-element fp64 CUDA tensor."""
    if end <= begin:
        src_need = state_need = out_need = 0
    else:
        src_need = end - src_base
        state_need = end - rank_begin * L.shard
        out_need = end if out_mode == ZERO_OUT_FULL else state_need
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need, pinned_ok=True)
    rc = load().zero_reduce_scatter_adamw_clip(
        ctypes.byref(L), arr, n, int(src_dtype), int(src_base), float(divisor),
        int(rank_begin), int(rank_end), int(begin), int(end),
        _tensor(master, "master", torch.float32, state_need),
        _tensor(m, "m", torch.float32, state_need),
        _tensor(v, "v", torch.float32, state_need),
        _tensor(out, "out", torch.bfloat16, out_need),
        int(out_mode), ctypes.byref(hp), _tensor(norm_sq, "norm_sq", torch.float64, 1),
        float(max_norm), _stream_ptr(stream))
    _check(rc, "zero_reduce_scatter_adamw_clip")


def zero_reduce_scatter_adamw_q8(L: ZeroLayout, srcs, src_dtype: int, src_base: int,
                                 divisor: float, rank_begin: int, rank_end: int, begin: int,
                                 end: int, master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                                 q_out: torch.Tensor, scales_out: torch.Tensor, block: int,
                                 hp: ZeroAdamW, stream=None):
    """The fused update with its result in the 8-bit block format (codes laid
    out like the state, one scale per 256 of them) instead of bf16."""
    if end <= begin:
        src_need = state_need = 0
    else:
        src_need = end - src_base
        state_need = end - rank_begin * L.shard
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need)
    rc = load().zero_reduce_scatter_adamw_q8(
        ctypes.byref(L), arr, n, int(src_dtype), int(src_base), float(divisor),
        int(rank_begin), int(rank_end), int(begin), int(end),
        _tensor(master, "master", torch.float32, state_need),
        _tensor(m, "m", torch.float32, state_need),
        _tensor(v, "v", torch.float32, state_need),
        _tensor(q_out, "q_out", torch.int8, state_need),
        _tensor(scales_out, "scales_out", torch.float32, -(-state_need // 256)),
        int(block), ctypes.byref(hp), _stream_ptr(stream))
    _check(rc, "zero_reduce_scatter_adamw_q8")


def zero_accumulate_adamw(L: ZeroLayout, mode: int, acc, acc_base: int, grads, grad_base: int,
                          divisor: float, rank_begin: int, rank_end: int, begin: int, end: int,
                          master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                          out: torch.Tensor, out_mode: int, hp: ZeroAdamW, stream=None):
    """The last micro-batch of an accumulation window fused with the update
    (LOCAL: sum_r (acc[r] + grads[r]); REDUCE: acc[0] + sum_r grads[r])."""
    if end <= begin:
        acc_need = grad_need = state_need = out_need = 0
    else:
        acc_need, grad_need = end - acc_base, end - grad_base
        state_need = end - rank_begin * L.shard
        out_need = end if out_mode == ZERO_OUT_FULL else state_need
    if len(acc) == 0 or len(grads) == 0:
        raise ValueError("need accumulators and gradients")
    acc_p = [_tensor(a, f"acc[{i}]", torch.float32, acc_need) for i, a in enumerate(acc)]
    g_p = [_tensor(g, f"grads[{i}]", torch.bfloat16, grad_need) for i, g in enumerate(grads)]
    rc = load().zero_accumulate_adamw(
        ctypes.byref(L), int(mode), (ctypes.c_void_p * len(acc_p))(*acc_p), len(acc_p), int(acc_base),
        (ctypes.c_void_p * len(g_p))(*g_p), len(g_p), int(grad_base), float(divisor),
        int(rank_begin), int(rank_end), int(begin), int(end),
        _tensor(master, "master", torch.float32, state_need),
        _tensor(m, "m", torch.float32, state_need),
        _tensor(v, "v", torch.float32, state_need),
        _tensor(out, "out", torch.bfloat16, out_need),
        int(out_mode), ctypes.byref(hp), _stream_ptr(stream))
    _check(rc, "zero_accumulate_adamw")


def zero_grad_norm_workspace() -> int:
    """Bytes of device workspace zero_grad_norm_sq needs on the current device."""
    out = ctypes.c_int64()
    _check(load().zero_grad_norm_workspace(ctypes.byref(out)), "zero_grad_norm_workspace")
    return out.value


def zero_grad_norm_sq(L: ZeroLayout, srcs, src_dtype: int, src_base: int, divisor: float,
                      begin: int, end: int, workspace: torch.Tensor, norm_sq: torch.Tensor,
                      accumulate: bool, stream=None):
    """norm_sq (1-element fp64 CUDA tensor) (+)= sum over [begin, end) of the
    squared mean gradient; workspace: a CUDA tensor of zero_grad_norm_workspace() bytes."""
    src_need = max(0, end - src_base) if end > begin else 0
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need)
    if workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().zero_grad_norm_sq(ctypes.byref(L), arr, n, int(src_dtype), int(src_base),
                                  float(divisor), int(begin), int(end), workspace.data_ptr(),
                                  int(ws_bytes), _tensor(norm_sq, "norm_sq", torch.float64, 1),
                                  int(bool(accumulate)), _stream_ptr(stream))
    _check(rc, "zero_grad_norm_sq")


def zero_grad_norm_sq_static(L: ZeroLayout, srcs, src_dtype: int, src_base: int, divisor: float,
                             begin: int, end: int, norm_sq: torch.Tensor, accumulate: bool,
                             stream=None):
    """zero_grad_norm_sq with its partial sums in the library's own device array:
    no workspace, nothing allocated.  Calls that overlap on the GPU race."""
    src_need = max(0, end - src_base) if end > begin else 0
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need)
    rc = load().zero_grad_norm_sq_static(ctypes.byref(L), arr, n, int(src_dtype), int(src_base),
                                         float(divisor), int(begin), int(end),
                                         _tensor(norm_sq, "norm_sq", torch.float64, 1),
                                         int(bool(accumulate)), _stream_ptr(stream))
    _check(rc, "zero_grad_norm_sq_static")


def zero_gather_layer(unit: ZeroLayout, shards, full_out: torch.Tensor, stream=None):
    """Concatenate unit.n_dp bf16 shards (unit.shard elements each) into full_out."""
    if len(shards) != unit.n_dp:
        raise ValueError(f"need {unit.n_dp} shards, got {len(shards)}")
    ptrs = [_tensor(s, f"shards[{i}]", torch.bfloat16, unit.shard) for i, s in enumerate(shards)]
    arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    rc = load().zero_gather_layer(ctypes.byref(unit), arr,
                                  _tensor(full_out, "full_out", torch.bfloat16, unit.padded_n),
                                  _stream_ptr(stream))
    _check(rc, "zero_gather_layer")


def zero_cast_bf16(src: torch.Tensor, dst: torch.Tensor, n: int = None, stream=None):
    """dst[:n] = bf16 of src[:n] (nearest, ties to even); n defaults to src.numel()."""
    n = src.numel() if n is None else int(n)
    rc = load().zero_cast_bf16(_tensor(src, "src", torch.float32, n), _tensor(dst, "dst", torch.bfloat16, n),
                               n, _stream_ptr(stream))
    _check(rc, "zero_cast_bf16")


def zero_accumulate(L: ZeroLayout, mode: int, srcs, src_dtype: int, src_base: int,
                    dst: torch.Tensor, dst_base: int, begin: int, end: int, first: bool,
                    stream=None):
    """dst[i - dst_base] (+)= src[0] (LOCAL) or sum_r src[r] (REDUCE) over [begin, end)."""
    src_need = max(0, end - src_base) if end > begin else 0
    dst_need = max(0, end - dst_base) if end > begin else 0
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need)
    rc = load().zero_accumulate(ctypes.byref(L), int(mode), arr, n, int(src_dtype), int(src_base),
                                _tensor(dst, "dst", torch.float32, dst_need), int(dst_base),
                                int(begin), int(end), int(bool(first)), _stream_ptr(stream))
    _check(rc, "zero_accumulate")


def zero_status_check(stream=None):
    _check(load().zero_status_check(_stream_ptr(stream)), "zero_status_check")


def zero_quantize_int8(unit: ZeroLayout, shards: torch.Tensor, q: torch.Tensor, scales: torch.Tensor,
                       block: int = 256, stream=None):
    """Quantize the unit's n_dp bf16 shards (back to back) to int8 + fp32 block scales."""
    nb = -(-unit.shard // block) if unit.shard else 0
    rc = load().zero_quantize_int8(
        ctypes.byref(unit), _tensor(shards, "shards", torch.bfloat16, unit.padded_n),
        _tensor(q, "q", torch.int8, unit.padded_n),
        _tensor(scales, "scales", torch.float32, nb * unit.n_dp), int(block), _stream_ptr(stream))
    _check(rc, "zero_quantize_int8")


def zero_gather_layer_int8(unit: ZeroLayout, q_shards, scale_shards, full_out: torch.Tensor,
                           block: int = 256, stream=None):
    """Rebuild the full bf16 unit from each rank's int8 shard and block scales."""
    if len(q_shards) != unit.n_dp or len(scale_shards) != unit.n_dp:
        raise ValueError(f"need {unit.n_dp} shards and scale arrays")
    nb = -(-unit.shard // block) if unit.shard else 0
    qp = [_tensor(x, f"q_shards[{i}]", torch.int8, unit.shard) for i, x in enumerate(q_shards)]
    sp = [_tensor(x, f"scale_shards[{i}]", torch.float32, nb) for i, x in enumerate(scale_shards)]
    rc = load().zero_gather_layer_int8(
        ctypes.byref(unit), (ctypes.c_void_p * max(1, len(qp)))(*qp),
        (ctypes.c_void_p * max(1, len(sp)))(*sp), int(block),
        _tensor(full_out, "full_out", torch.bfloat16, unit.padded_n), _stream_ptr(stream))
    _check(rc, "zero_gather_layer_int8")


def _qgrad_sources(L: ZeroLayout, q_src, scale_src, block: int, need: int):
    """Host arrays of the codes and scales of 8-bit gradient sources."""
    if len(q_src) == 0 or len(q_src) != len(scale_src):
        raise ValueError("need the same nonzero number of code and scale sources")
    nb = -(-L.shard // block) if L.shard else 0
    qp = [_tensor(x, f"q_src[{i}]", torch.int8, need) for i, x in enumerate(q_src)]
    sp = [_tensor(x, f"scale_src[{i}]", torch.float32, nb * L.n_dp if need else 0)
          for i, x in enumerate(scale_src)]
    n = len(qp)
    return (ctypes.c_void_p * n)(*qp), (ctypes.c_void_p * n)(*sp), n


def zero_reduce_scatter_adamw_int8(L: ZeroLayout, q_src, scale_src, block: int, divisor: float,
                                   rank_begin: int, rank_end: int, begin: int, end: int,
                                   master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                                   out: torch.Tensor, out_mode: int, hp: ZeroAdamW, stream=None):
    """The fused update over [begin, end) from 8-bit gradients: each rank's
    codes (padded_n int8) and block scales (n_dp * ceil(S / block) fp32)."""
    if end <= begin:
        src_need = state_need = out_need = 0
    else:
        src_need = end
        state_need = end - rank_begin * L.shard
        out_need = end if out_mode == ZERO_OUT_FULL else state_need
    qa, sa, n = _qgrad_sources(L, q_src, scale_src, block, src_need)
    rc = load().zero_reduce_scatter_adamw_int8(
        ctypes.byref(L), qa, sa, n, int(block), float(divisor), int(rank_begin), int(rank_end),
        int(begin), int(end),
        _tensor(master, "master", torch.float32, state_need),
        _tensor(m, "m", torch.float32, state_need),
        _tensor(v, "v", torch.float32, state_need),
        _tensor(out, "out", torch.bfloat16, out_need),
        int(out_mode), ctypes.byref(hp), _stream_ptr(stream))
    _check(rc, "zero_reduce_scatter_adamw_int8")


def zero_reduce_scatter_adamw_int8_q8(L: ZeroLayout, q_src, scale_src, block: int, divisor: float,
                                      rank_begin: int, rank_end: int, begin: int, end: int,
                                      master: torch.Tensor, m: torch.Tensor, v: torch.Tensor,
                                      q_out: torch.Tensor, scales_out: torch.Tensor, out_block: int,
                                      hp: ZeroAdamW, stream=None):
    """The update from 8-bit gradients with its result in the 8-bit block format."""
    if end <= begin:
        src_need = state_need = 0
    else:
        src_need = end
        state_need = end - rank_begin * L.shard
    qa, sa, n = _qgrad_sources(L, q_src, scale_src, block, src_need)
    rc = load().zero_reduce_scatter_adamw_int8_q8(
        ctypes.byref(L), qa, sa, n, int(block), float(divisor), int(rank_begin), int(rank_end),
        int(begin), int(end),
        _tensor(master, "master", torch.float32, state_need),
        _tensor(m, "m", torch.float32, state_need),
        _tensor(v, "v", torch.float32, state_need),
        _tensor(q_out, "q_out", torch.int8, state_need),
        _tensor(scales_out, "scales_out", torch.float32, -(-state_need // 256)),
        int(out_block), ctypes.byref(hp), _stream_ptr(stream))
    _check(rc, "zero_reduce_scatter_adamw_int8_q8")


def zero_accumulate_int8(L: ZeroLayout, q_src, scale_src, block: int, dst: torch.Tensor,
                         dst_base: int, begin: int, end: int, first: bool, stream=None):
    """dst[i - dst_base] (+)= sum over ranks of the dequantized 8-bit gradients."""
    src_need = end if end > begin else 0
    dst_need = max(0, end - dst_base) if end > begin else 0
    qa, sa, n = _qgrad_sources(L, q_src, scale_src, block, src_need)
    rc = load().zero_accumulate_int8(ctypes.byref(L), qa, sa, n, int(block),
                                     _tensor(dst, "dst", torch.float32, dst_need), int(dst_base),
                                     int(begin), int(end), int(bool(first)), _stream_ptr(stream))
    _check(rc, "zero_accumulate_int8")


def zero_schedule_fill(hp: ZeroAdamW, first_step: int, n_steps: int, lrs=None) -> torch.Tensor:
    """Host table [n_steps, 3] of {lr, bc1, bc2} for steps first_step..; lrs: a
    sequence of n_steps learning rates, or None for hp.lr."""
    table = torch.empty((int(n_steps), 3), dtype=torch.float32)
    lr_arr = None
    if lrs is not None:
        lr_t = torch.tensor([float(x) for x in lrs], dtype=torch.float32)
        if lr_t.numel() != n_steps:
            raise ValueError(f"need {n_steps} learning rates, got {lr_t.numel()}")
        lr_arr = lr_t
    rc = load().zero_schedule_fill(ctypes.byref(hp), int(first_step), int(n_steps),
                                   lr_arr.data_ptr() if lr_arr is not None else None, table.data_ptr())
    _check(rc, "zero_schedule_fill")
    return table


def zero_schedule_advance(table: torch.Tensor, step_index: torch.Tensor, sched: torch.Tensor,
                          stream=None):
    """On the device: sched = table[step_index]; step_index += 1."""
    rc = load().zero_schedule_advance(_tensor(table, "table", torch.float32, 3),
                                      table.numel() // 3,
                                      _tensor(step_index, "step_index", torch.int64, 1),
                                      _tensor(sched, "sched", torch.float32, 3), _stream_ptr(stream))
    _check(rc, "zero_schedule_advance")


def zero_selftest_bounded_wait(limit_cycles: int, stream=None):
    """Run the bounded-wait self test (see zero_gb300.h); follow with zero_status_check."""
    _check(load().zero_selftest_bounded_wait(int(limit_cycles), _stream_ptr(stream)),
           "zero_selftest_bounded_wait")


# --------------------------------------------------------------------------
# the dense operators of a unit
# --------------------------------------------------------------------------

_DT_CODE = {torch.bfloat16: ZERO_BF16, torch.float32: ZERO_F32}
_BF16_ONLY = {torch.bfloat16: ZERO_BF16}


def _matrix(t, name, rows, cols, dtypes):
    """Pointer, row stride and type code of a [rows, cols] matrix whose rows are
    contiguous; None gives a null pointer."""
    if t is None:
        return None, cols, ZERO_BF16
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = dtypes.get(t.dtype)
    if code is None or not t.is_cuda or t.shape != (rows, cols):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); there is no CPU path")
        if code is None:
            raise TypeError(f"{name} must be one of {list(dtypes)}, got {t.dtype}")
        raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
    ld, inner = t.stride()
    if rows <= 1 or cols == 0:
        ld = cols
    if (inner != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have rows of contiguous elements (strides {t.stride()})")
    return t.data_ptr(), ld, code


def _vector(t, name, n, code):
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        if t.numel() == n and t.is_cuda and t.dtype == _SRC_DT[code] and t.is_contiguous():
            return t.data_ptr()
        if t.numel() != n:
            raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return _tensor(t, name, _SRC_DT[code], n)


def _sizes(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape


def _same_type(name, code, t, other):
    if t is not None and _DT_CODE.get(t.dtype) != code:
        raise TypeError(f"{name} must have the type of {other}, got {t.dtype}")


def zero_linear(x, w, y, bias=None, act: int = ZERO_ACT_NONE, residual=None,
                drop: ZeroDropout | None = None, pre=None, stream=None):
    """y[m, n] = residual + D(act(x[m, k] w[n, k]^T + bias)); pre, if given,
    receives the value before the activation (bf16), for the gradient.  x, w, bias
    and pre are bf16; y and residual bf16 or fp32."""
    (m, k), n = _sizes(x, "x"), _sizes(w, "w")[0]
    xp, ldx, _ = _matrix(x, "x", m, k, _BF16_ONLY)
    wp, ldw, _ = _matrix(w, "w", n, k, _BF16_ONLY)
    yp, ldy, code = _matrix(y, "y", m, n, _DT_CODE)
    _same_type("residual", code, residual, "y")
    rp, ldr, _ = _matrix(residual, "residual", m, n, _DT_CODE)
    pp, ldp, _ = _matrix(pre, "pre", m, n, _BF16_ONLY)
    _check(load().zero_linear(m, n, k, xp, ldx, wp, ldw, _vector(bias, "bias", n, ZERO_BF16), act, drop,
                              rp, ldr, pp, ldp, yp, code, ldy, _stream_ptr(stream)), "zero_linear")


def zero_linear_grad_input(dz, w, dx, act: int = ZERO_ACT_NONE, pre=None,
                           drop: ZeroDropout | None = None, residual=None, stream=None):
    """dx[m, k] = residual + D'(dz[m, n] w[n, k]) act'(pre); act, pre and drop are
    those of the layer below (whose y was this layer's x), so that dx is its dz."""
    (m, n), k = _sizes(dz, "dz"), _sizes(w, "w")[1]
    zp, lddz, _ = _matrix(dz, "dz", m, n, _BF16_ONLY)
    wp, ldw, _ = _matrix(w, "w", n, k, _BF16_ONLY)
    xp, lddx, code = _matrix(dx, "dx", m, k, _DT_CODE)
    _same_type("residual", code, residual, "dx")
    rp, ldr, _ = _matrix(residual, "residual", m, k, _DT_CODE)
    pp, ldp, _ = _matrix(pre, "pre", m, k, _BF16_ONLY)
    _check(load().zero_linear_grad_input(m, n, k, zp, lddz, wp, ldw, act, drop, pp, ldp, rp, ldr, xp,
                                         code, lddx, _stream_ptr(stream)), "zero_linear_grad_input")


def zero_linear_grad_weight(dz, x, dw, db=None, acc=None, db_acc=None, stream=None):
    """dw[n, k] = acc + dz[m, n]^T x[m, k] and db[n] = db_acc + the column sums of
    dz.  dw, acc, db and db_acc have one type, bf16 or fp32; dw may be acc itself
    (and db db_acc): gradients are then accumulated in place."""
    (m, n), k = _sizes(dz, "dz"), _sizes(x, "x")[1]
    zp, lddz, _ = _matrix(dz, "dz", m, n, _BF16_ONLY)
    xp, ldx, _ = _matrix(x, "x", m, k, _BF16_ONLY)
    wp, lddw, code = _matrix(dw, "dw", n, k, _DT_CODE)
    _same_type("acc", code, acc, "dw")
    ap, ldacc, _ = _matrix(acc, "acc", n, k, _DT_CODE)
    _check(load().zero_linear_grad_weight(m, n, k, zp, lddz, xp, ldx, ap, ldacc, wp, code, lddw,
                                          _vector(db_acc, "db_acc", n, code),
                                          _vector(db, "db", n, code), _stream_ptr(stream)),
           "zero_linear_grad_weight")


def zero_dropout(x, y, drop: ZeroDropout | None, residual=None, stream=None):
    """y = residual + D(x), matrices of one type (bf16 or fp32)."""
    rows, cols = _sizes(x, "x")
    xp, ldx, code = _matrix(x, "x", rows, cols, _DT_CODE)
    _same_type("y", code, y, "x")
    _same_type("residual", code, residual, "x")
    yp, ldy, _ = _matrix(y, "y", rows, cols, _DT_CODE)
    rp, ldr, _ = _matrix(residual, "residual", rows, cols, _DT_CODE)
    _check(load().zero_dropout(rows, cols, xp, ldx, code, drop, rp, ldr, yp, ldy, _stream_ptr(stream)),
           "zero_dropout")


def zero_dropout_grad(dy, dx, drop: ZeroDropout | None = None, act: int = ZERO_ACT_NONE, pre=None,
                      db=None, db_acc=None, stream=None):
    """dx = D'(dy) act'(pre) and db = db_acc + the column sums of dx: with a
    linear's act, pre and drop, its dz and bias gradient.  dx may be dy itself."""
    rows, cols = _sizes(dy, "dy")
    dp, lddy, dcode = _matrix(dy, "dy", rows, cols, _DT_CODE)
    xp, lddx, xcode = _matrix(dx, "dx", rows, cols, _DT_CODE)
    pp, ldp, _ = _matrix(pre, "pre", rows, cols, _BF16_ONLY)
    bcode = ZERO_BF16
    if db is not None:
        bcode = _DT_CODE.get(getattr(db, "dtype", None), -1)
        if bcode < 0:
            raise TypeError("db must be a bfloat16 or float32 tensor")
    _check(load().zero_dropout_grad(rows, cols, dp, lddy, dcode, drop, act, pp, ldp, xp, xcode, lddx,
                                    _vector(db_acc, "db_acc", cols, bcode),
                                    _vector(db, "db", cols, bcode), bcode, _stream_ptr(stream)),
           "zero_dropout_grad")


def zero_rope_plan(rot: int, layout: int = ZERO_ROPE_HALF, base: float = 10000.0,
                   scaling: int = ZERO_ROPE_NONE, factor: float = 1.0,
                   context: float = 0.0) -> ZeroRopePlan:
    """The plan zero_rope turns by: the first `rot` elements of a head, pairs by
    `layout`, frequencies base^(-2i/rot) scaled for contexts `factor` times as long
    (YARN also needs the first context's length)."""
    plan = ZeroRopePlan()
    _check(load().zero_rope_fill(int(rot), int(layout), float(base), int(scaling), float(factor),
                                 float(context), ctypes.byref(plan)), "zero_rope_fill")
    return plan


def _heads(t, name, dtypes):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [tokens, heads, dim] tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); there is no CPU path")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {list(dtypes)}, got {t.dtype}")
    st, sh, inner = t.stride()
    if t.shape[2] > 1 and inner != 1:
        raise ValueError(f"{name} must have contiguous heads (strides {t.stride()})")
    return t.data_ptr(), st, sh


def zero_rope(plan: ZeroRopePlan, x, y, positions=None, pos0: int = 0, inverse: bool = False,
              stream=None):
    """Turns the pairs of x [tokens, heads, dim] into y (which may be x) by the
    int64 positions, or pos0 + token; inverse turns back, which is the gradient."""
    xp, xt, xh = _heads(x, "x", _DT_CODE)
    yp, yt, yh = _heads(y, "y", _DT_CODE)
    if x.shape != y.shape or x.dtype != y.dtype:
        raise ValueError("x and y must have one shape and type")
    tokens, heads, dim = x.shape
    if positions is not None and positions.numel() != tokens:
        raise ValueError(f"positions must have {tokens} elements, got {positions.numel()}")
    _check(load().zero_rope(plan, tokens, heads, dim, xp, xt, xh, yp, yt, yh, _DT_CODE[x.dtype],
                            None if positions is None else _tensor(positions, "positions", torch.int64, tokens),
                            pos0, bool(inverse), _stream_ptr(stream)), "zero_rope")


def _workspace(t, need: int):
    """Pointer and bytes of a workspace; None where none is given."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    size = t.numel() * t.element_size()
    if size < need:
        raise ValueError(f"workspace has {size} bytes, the call needs {need}")
    return t.data_ptr(), size


def zero_layer_norm(x, y, gamma=None, beta=None, eps: float = 1e-5, residual=None, sum=None, mean=None,
                    rstd=None, stream=None):
    """sum = x + residual (both or neither given) and y = (sum - mean) rstd gamma + beta
    over the rows of a matrix; mean and rstd (fp32, one a row), if given, receive the
    statistics for the gradient.  x, residual and sum are bf16 or fp32 alike, y the same
    or bf16, gamma and beta bf16.  sum may be x or residual itself, y may be x."""
    rows, cols = _sizes(x, "x")
    xp, ldx, code = _matrix(x, "x", rows, cols, _DT_CODE)
    yp, ldy, ycode = _matrix(y, "y", rows, cols, _DT_CODE)
    if ycode not in (code, ZERO_BF16):
        raise TypeError(f"y must be bfloat16 or have the type of x, got {y.dtype}")
    _same_type("residual", code, residual, "x")
    _same_type("sum", code, sum, "x")
    if (residual is None) != (sum is None):
        raise ValueError("residual and sum are given together")
    rp, ldr, _ = _matrix(residual, "residual", rows, cols, _DT_CODE)
    sp, lds, _ = _matrix(sum, "sum", rows, cols, _DT_CODE)
    _check(load().zero_layer_norm(rows, cols, xp, ldx, code, rp, ldr, sp, lds, _vector(gamma, "gamma", cols, ZERO_BF16),
                                  _vector(beta, "beta", cols, ZERO_BF16), eps, yp, ycode, ldy,
                                  _vector(mean, "mean", rows, ZERO_F32), _vector(rstd, "rstd", rows, ZERO_F32),
                                  _stream_ptr(stream)), "zero_layer_norm")


def zero_layer_norm_grad_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace zero_layer_norm_grad needs for dgamma or dbeta on the current device."""
    out = ctypes.c_int64()
    _check(load().zero_layer_norm_grad_workspace(rows, cols, ctypes.byref(out)), "zero_layer_norm_grad_workspace")
    return out.value


def zero_layer_norm_grad(dy, x, mean, rstd, dx, gamma=None, residual=None, dgamma=None, dbeta=None,
                         dgamma_acc=None, dbeta_acc=None, workspace=None, stream=None):
    """dx = residual + the gradient of zero_layer_norm by its input x (the sum, where it
    had a residual), dgamma = dgamma_acc + and dbeta = dbeta_acc + those by its weights.
    x, residual and dx (which may be residual, dy or x itself) are bf16 or fp32 alike,
    dy the same or bf16; dgamma, dbeta and what they are added to (which may be
    themselves) have one type.  workspace: a CUDA tensor of
    zero_layer_norm_grad_workspace(rows, cols) bytes, where dgamma or dbeta is given."""
    rows, cols = _sizes(x, "x")
    xp, ldx, code = _matrix(x, "x", rows, cols, _DT_CODE)
    dp, lddy, dcode = _matrix(dy, "dy", rows, cols, _DT_CODE)
    if dcode not in (code, ZERO_BF16):
        raise TypeError(f"dy must be bfloat16 or have the type of x, got {dy.dtype}")
    _same_type("residual", code, residual, "x")
    _same_type("dx", code, dx, "x")
    gp, lddx, _ = _matrix(dx, "dx", rows, cols, _DT_CODE)
    rp, ldr, _ = _matrix(residual, "residual", rows, cols, _DT_CODE)
    first = dgamma if dgamma is not None else dbeta
    wcode, wsp, ws = ZERO_BF16, None, 0
    if first is not None:
        wcode = _DT_CODE.get(getattr(first, "dtype", None), -1)
        if wcode < 0:
            raise TypeError("dgamma and dbeta must be bfloat16 or float32 tensors")
        need = zero_layer_norm_grad_workspace(rows, cols)
        if need and workspace is None:
            raise ValueError("dgamma and dbeta need a workspace")
        wsp, ws = _workspace(workspace, need)
    _check(load().zero_layer_norm_grad(rows, cols, dp, lddy, dcode, xp, ldx, _vector(mean, "mean", rows, ZERO_F32),
                                       _vector(rstd, "rstd", rows, ZERO_F32), _vector(gamma, "gamma", cols, ZERO_BF16),
                                       rp, ldr, gp, code, lddx, _vector(dgamma_acc, "dgamma_acc", cols, wcode),
                                       _vector(dgamma, "dgamma", cols, wcode), _vector(dbeta_acc, "dbeta_acc", cols, wcode),
                                       _vector(dbeta, "dbeta", cols, wcode), wcode, wsp, ws, _stream_ptr(stream)),
           "zero_layer_norm_grad")


# --------------------------------------------------------------------------
# a step by orthogonalised momentum
# --------------------------------------------------------------------------

def zero_reduce_scatter_momentum(L: ZeroLayout, srcs, src_dtype: int, src_base: int, divisor: float,
                                 rank_begin: int, rank_end: int, begin: int, end: int, m: torch.Tensor,
                                 u: torch.Tensor, out_mode: int, hp: ZeroMuon, stream=None):
    """Mean reduce-scatter into the momentum m (fp32) over [begin, end), and the bf16
    matrices u to orthogonalise, gathered (ZERO_OUT_FULL) or left with their owners."""
    if end <= begin:
        src_need = state_need = out_need = 0
    else:
        src_need = end - src_base
        state_need = end - rank_begin * L.shard
        out_need = end if out_mode == ZERO_OUT_FULL else state_need
    arr, n = _src_array(srcs, _SRC_DT.get(src_dtype, None), src_need, pinned_ok=True)
    _check(load().zero_reduce_scatter_momentum(L, arr, n, src_dtype, src_base, divisor, rank_begin, rank_end, begin, end,
                                               _tensor(m, "m", torch.float32, state_need),
                                               _tensor(u, "u", torch.bfloat16, out_need), out_mode, hp, _stream_ptr(stream)),
           "zero_reduce_scatter_momentum")


def zero_muon_update(L: ZeroLayout, update: torch.Tensor, update_base: int, rank_begin: int, rank_end: int,
                     begin: int, end: int, master: torch.Tensor, out: torch.Tensor, out_mode: int, hp: ZeroMuon,
                     stream=None):
    """w = w - lr weight_decay w - lr scale update over [begin, end) of the owners'
    master weights, and the bf16 cast with its gather write."""
    if end <= begin:
        up_need = state_need = out_need = 0
    else:
        up_need = end - update_base
        state_need = end - rank_begin * L.shard
        out_need = end if out_mode == ZERO_OUT_FULL else state_need
    _check(load().zero_muon_update(L, _tensor(update, "update", torch.bfloat16, up_need), update_base, rank_begin, rank_end,
                                   begin, end, _tensor(master, "master", torch.float32, state_need),
                                   _tensor(out, "out", torch.bfloat16, out_need), out_mode, hp, _stream_ptr(stream)),
           "zero_muon_update")


def zero_orthogonalize_workspace(batch: int, rows: int, cols: int) -> int:
    """Bytes of workspace zero_orthogonalize needs."""
    out = ctypes.c_int64()
    _check(load().zero_orthogonalize_workspace(batch, rows, cols, ctypes.byref(out)), "zero_orthogonalize_workspace")
    return out.value


def _matrices(t, name, dtypes):
    """Batch, rows, columns, pointer, matrix and row stride and type code of a matrix or
    a batch of them whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (2, 3):
        raise ValueError(f"{name} must be a matrix or a batch of them")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device}); there is no CPU path")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {list(dtypes)}, got {t.dtype}")
    if t.dim() == 2:
        t = t.unsqueeze(0)
    b, rows, cols = t.shape
    sb, ld, inner = t.stride()
    if rows <= 1 or cols == 0:
        ld = cols
    if (inner != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have rows of contiguous elements (strides {t.stride()})")
    return b, rows, cols, t.data_ptr(), (sb if b > 1 else 0), ld, dtypes[t.dtype]


_NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def zero_orthogonalize(x, y, steps: int = 5, coefficients=_NEWTON_SCHULZ, eps: float = 1e-7, workspace=None,
                       stream=None):
    """y (bf16) = the orthogonalised matrix, or batch of matrices, x (bf16 or fp32) by
    `steps` of the Newton-Schulz iteration with the quintic's coefficients; y may be x.
    workspace: a CUDA tensor of zero_orthogonalize_workspace(batch, rows, cols) bytes."""
    b, rows, cols, xp, xs, ldx, code = _matrices(x, "x", _DT_CODE)
    yb, yrows, ycols, yp, ys, ldy, _ = _matrices(y, "y", _BF16_ONLY)
    if (yb, yrows, ycols) != (b, rows, cols):
        raise ValueError(f"y must have the shape of x, {(b, rows, cols)}, got {(yb, yrows, ycols)}")
    coefficients = tuple(coefficients)
    if len(coefficients) != 3:
        raise ValueError("coefficients are three: of X, A X and A A X")
    need = zero_orthogonalize_workspace(b, rows, cols)
    if need and workspace is None:
        raise ValueError("zero_orthogonalize needs a workspace")
    wsp, ws = _workspace(workspace, need)
    _check(load().zero_orthogonalize(b, rows, cols, xp, xs, ldx, code, yp, ys, ldy, steps,
                                     (ctypes.c_float * 3)(*coefficients), eps, wsp, ws, _stream_ptr(stream)),
           "zero_orthogonalize")
