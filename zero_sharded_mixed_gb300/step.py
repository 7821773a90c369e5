"""Host-side orchestration of the C-ABI calls: the bucket loop of a ZeRO-1/2
step, the two gradient-accumulation orders, clipping by the global norm, the
ZeRO-3 per-unit gather / release / reduce-scatter / update sequence with a
two-slot ring of gathered buffers (and its prefetching variant), the ZeRO++
8-bit weight and gradient paths, steps fed from pinned host memory, and
per-step scalars in device memory for steps replayed from a CUDA graph, and the
step by orthogonalised momentum (Muon).  No arithmetic happens here; every element is touched only by the library's
kernels.

Buffer conventions (simulated ranks in one GPU):
* ``grads``: n_dp bf16 tensors, rank r's full local gradient of P elements.
* ``master``, ``m``, ``v``: fp32 tensors holding the owned shards of ranks
  ``rank_begin..rank_end-1`` back to back (all ranks: P elements).
* ``out``: the full flat bf16 weight buffer (P elements).
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import binding as zb


def bucket_ranges(L: zb.ZeroLayout, lo: int = 0, hi: int | None = None):
    """The non-empty intersections of [lo, hi) with the layout's buckets."""
    hi = L.padded_n if hi is None else hi
    out = []
    for b in range(L.n_buckets):
        b0, b1 = zb.zero_bucket_range(L, b)
        s, e = max(b0, lo), min(b1, hi)
        if s < e:
            out.append((s, e))
    return out


def zero12_step(L, grads, master, m, v, out, hp, rank_begin=0, rank_end=None, stream=None,
                grad_base=0, divisor=None):
    """One ZeRO-1/2 step for the owners rank_begin..rank_end-1, bucket by bucket
    ("ZeRO and FSDP": stage 2 reduce-scatters each bucket as it becomes ready;
    stage 1 once at the end -- the arithmetic is the same)."""
    rank_end = L.n_dp if rank_end is None else rank_end
    lo, hi = rank_begin * L.shard, rank_end * L.shard
    div = float(L.n_dp) if divisor is None else float(divisor)
    for s, e in bucket_ranges(L, lo, hi):
        zb.zero_reduce_scatter_adamw(L, grads, zb.ZERO_BF16, grad_base, div, rank_begin, rank_end,
                                     s, e, master, m, v, out, zb.ZERO_OUT_FULL, hp, stream)


def split_ranges(ranges, chunk_elems: int | None):
    """The ranges cut into pieces of at most chunk_elems elements (a multiple
    of 8, so every piece but a range's last keeps the 8-element grid); None
    keeps them whole.  The pieces change no number, only the granularity at
    which host copies and updates overlap."""
    if not chunk_elems:
        return list(ranges)
    if chunk_elems % 8:
        raise ValueError("chunk_elems must be a multiple of 8")
    return [(a, min(a + chunk_elems, e)) for s, e in ranges for a in range(s, e, chunk_elems)]


# --------------------------------------------------------------------------
# per-step scalars in device memory, and steps captured in CUDA graphs
# --------------------------------------------------------------------------

class StepSchedule:
    """lr and the bias corrections of steps first_step .. first_step+n_steps-1
    in device memory: advance() (a one-thread kernel on the stream) moves the
    current-step scalars to the next step, and hp() is the AdamW block whose
    kernels read them.  A step captured in a CUDA graph after advance() is
    then a new step at every replay; lrs gives a learning rate per step."""

    def __init__(self, lr, beta1, beta2, eps, weight_decay, n_steps: int, first_step: int = 1,
                 lrs=None, device="cuda"):
        base = zb.ZeroAdamW.make(lr, beta1, beta2, eps, weight_decay, first_step)
        self.table = zb.zero_schedule_fill(base, first_step, n_steps, lrs).to(device)
        self.index = torch.zeros(1, dtype=torch.int64, device=device)
        self.sched = torch.zeros(3, dtype=torch.float32, device=device)
        self._hp = zb.ZeroAdamW.make(lr, beta1, beta2, eps, weight_decay, first_step, sched=self.sched)

    def hp(self) -> zb.ZeroAdamW:
        return self._hp

    def advance(self, stream=None):
        zb.zero_schedule_advance(self.table, self.index, self.sched, stream)


class GraphStep:
    """A step captured once in a CUDA graph and replayed.  fn() must launch the
    whole step on the current stream with fixed buffers (the gradients of each
    step written into the same tensors) and read its per-step scalars from a
    StepSchedule that fn() advances first.  Capture runs one warm-up call on a
    side stream (which performs a step) before recording."""

    def __init__(self, fn, warmup: int = 1):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(warmup):
                fn()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            fn()

    def replay(self):
        self.graph.replay()


# --------------------------------------------------------------------------
# a step by orthogonalised momentum (Muon)
# --------------------------------------------------------------------------

def _runs(ranges):
    """Ranges in order, those that touch joined."""
    out = []
    for s, e in ranges:
        if s == e:
            continue
        if out and out[-1][1] == s:
            out[-1] = (out[-1][0], e)
        else:
            out.append((s, e))
    return out


def _batches(offsets, size: int, most: int):
    """(first, count, stride) of equal matrices at equal distances, at most `most` each."""
    out = []
    for o in offsets:
        if out:
            first, count, stride = out[-1]
            if count < most and (count == 1 or o == first + count * stride) and o - first >= size:
                out[-1] = (first, count + 1, o - first if count == 1 else stride)
                continue
        out.append((o, 1, size))
    return out


class MuonStep:
    """One step of the flat parameter vector in which the matrices (shapes of two
    dimensions) move by their orthogonalised momentum and everything else by
    AdamW.  The ranks' gradients are reduced into the owners' momentum m, whose
    bf16 form is gathered into `update`, orthogonalised there matrix by matrix
    (equal matrices at equal distances in one call), and moves the owners'
    master weights, which are cast and gathered.  A matrix of n rows and k
    columns moves by lr * 0.2 * sqrt(max(n, k)) times its orthogonal factor,
    which is about AdamW's size, so that one lr serves both (Liu et al., "Muon
    is scalable for LLM training", 2025).  `workspace_bytes` bounds what a call
    takes beside one matrix's need.  v of the matrices is not touched."""

    SCALE = 0.2
    MOST = 65535   # matrices that a call takes

    def __init__(self, L, offsets, shapes, device="cuda", workspace_bytes: int = 1 << 30):
        if len(shapes) != len(offsets):
            raise ValueError(f"need a shape for each of {len(offsets)} tensors, got {len(shapes)}")
        self.L = L
        shapes = [tuple(int(x) for x in s) for s in shapes]
        sizes = []
        for o, s in zip(offsets, shapes):
            n = 1
            for x in s:
                n *= x
            sizes.append(n)
            if o + n > L.n:
                raise ValueError(f"a tensor of shape {s} at {o} leaves the vector of {L.n} elements")
        spans = [(o, o + n) for o, n in zip(offsets, sizes)]
        self.matrices = [(o, s) for o, s, n in zip(offsets, shapes, sizes) if len(s) == 2 and n]
        matrix = {o for o, _ in self.matrices}
        self.matrix_runs = _runs([r for r in spans if r[0] in matrix and r[1] > r[0]])
        self.vector_runs = _runs([r for r in spans if r[0] not in matrix or r[0] == r[1]])
        self.update = torch.zeros(L.padded_n, dtype=torch.bfloat16, device=device)
        by_shape = {}
        for o, s in self.matrices:
            by_shape.setdefault(s, []).append(o)
        self.batches, need = [], 0
        for (n, k), at in by_shape.items():
            one = zb.zero_orthogonalize_workspace(1, n, k)
            for first, count, stride in _batches(at, n * k, min(self.MOST, max(1, workspace_bytes // one))):
                need = max(need, zb.zero_orthogonalize_workspace(count, n, k))
                self.batches.append(self.update.as_strided((count, n, k), (stride, k, 1), first))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)

    def run(self, srcs, src_dtype, divisor, master, m, v, out, adamw: zb.ZeroAdamW, lr: float, momentum: float,
            nesterov: bool = True, ns_steps: int = 5, stream=None):
        """srcs: every rank's bf16 gradients, or fp32 sums of them; divisor: what makes
        them a mean.  adamw.sched, if set, gives lr to the matrices as well."""
        L, sched = self.L, getattr(adamw, "_sched_tensor", None)
        for s, e in self.vector_runs:
            zb.zero_reduce_scatter_adamw(L, srcs, src_dtype, 0, divisor, 0, L.n_dp, s, e, master, m, v, out,
                                         zb.ZERO_OUT_FULL, adamw, stream)
        hp = zb.ZeroMuon.make(lr, momentum, adamw.weight_decay, 1.0, nesterov, sched)
        for s, e in self.matrix_runs:
            zb.zero_reduce_scatter_momentum(L, srcs, src_dtype, 0, divisor, 0, L.n_dp, s, e, m, self.update,
                                            zb.ZERO_OUT_FULL, hp, stream)
        for x in self.batches:
            zb.zero_orthogonalize(x, x, steps=ns_steps, workspace=self.workspace, stream=stream)
        for o, (n, k) in self.matrices:
            hp = zb.ZeroMuon.make(lr, momentum, adamw.weight_decay, self.SCALE * max(n, k) ** 0.5, nesterov, sched)
            zb.zero_muon_update(L, self.update, 0, 0, L.n_dp, o, o + n * k, master, out, zb.ZERO_OUT_FULL, hp, stream)


# --------------------------------------------------------------------------
# gradient accumulation ("ZeRO and FSDP", paragraph on accumulation)
# --------------------------------------------------------------------------

def zero1_accumulate_micro(L, grads, acc, first: bool, stream=None):
    """Stage 1: every rank adds its full local micro-batch gradient into its own
    full fp32 buffer acc[r]; nothing is communicated."""
    for r in range(L.n_dp):
        zb.zero_accumulate(L, zb.ZERO_ACC_LOCAL, [grads[r]], zb.ZERO_BF16, 0, acc[r], 0,
                           0, L.padded_n, first, stream)


def zero1_finish(L, acc, n_micro, master, m, v, out, hp, stream=None):
    """Stage 1 after K micro-batches: one reduce-scatter (mean over n_dp*K) of
    the fp32 buffers fused with the update, bucket by bucket."""
    for s, e in bucket_ranges(L):
        zb.zero_reduce_scatter_adamw(L, acc, zb.ZERO_F32, 0, float(L.n_dp * n_micro), 0, L.n_dp,
                                     s, e, master, m, v, out, zb.ZERO_OUT_FULL, hp, stream)


def zero2_accumulate_micro(L, grads, A, first: bool, stream=None):
    """Stage 2: after every micro-batch, each bucket is reduce-scattered into the
    owners' fp32 shard buffer A (all owners back to back, P elements)."""
    for s, e in bucket_ranges(L):
        zb.zero_accumulate(L, zb.ZERO_ACC_REDUCE, grads, zb.ZERO_BF16, 0, A, 0, s, e, first,
                           stream)


def zero2_finish(L, A, n_micro, master, m, v, out, hp, stream=None):
    for s, e in bucket_ranges(L):
        zb.zero_reduce_scatter_adamw(L, [A], zb.ZERO_F32, 0, float(L.n_dp * n_micro), 0, L.n_dp,
                                     s, e, master, m, v, out, zb.ZERO_OUT_FULL, hp, stream)


def zero1_finish_fused(L, acc, last_grads, n_micro, master, m, v, out, hp, stream=None):
    """Stage 1, last micro-batch fused with the update: each rank's final
    accumulator acc[r] + g_r is formed in registers, never written back."""
    for s, e in bucket_ranges(L):
        zb.zero_accumulate_adamw(L, zb.ZERO_ACC_LOCAL, acc, 0, last_grads, 0,
                                 float(L.n_dp * n_micro), 0, L.n_dp, s, e, master, m, v, out,
                                 zb.ZERO_OUT_FULL, hp, stream)


def zero2_finish_fused(L, A, last_grads, n_micro, master, m, v, out, hp, stream=None):
    """Stage 2, last micro-batch fused with the update: A + sum over ranks of
    the last micro-batch's gradients, formed in registers."""
    for s, e in bucket_ranges(L):
        zb.zero_accumulate_adamw(L, zb.ZERO_ACC_REDUCE, [A], 0, last_grads, 0,
                                 float(L.n_dp * n_micro), 0, L.n_dp, s, e, master, m, v, out,
                                 zb.ZERO_OUT_FULL, hp, stream)


# --------------------------------------------------------------------------
# clipping by the global gradient norm ("DeepSpeed ZeRO", "The configuration
# file": gradient_clipping)
# --------------------------------------------------------------------------

class NormBuffers:
    """Device workspace and the fp64 squared-norm scalar of a clipped step."""

    def __init__(self, device=None):
        nbytes = zb.zero_grad_norm_workspace()
        self.workspace = torch.empty(nbytes // 8, dtype=torch.float64, device=device)
        self.norm_sq = torch.zeros(1, dtype=torch.float64, device=device)


def zero12_step_clipped(L, grads, master, m, v, out, hp, max_norm, bufs: NormBuffers,
                        rank_begin=0, rank_end=None, stream=None, grad_base=0):
    """A ZeRO-1/2 step with the mean gradient clipped to max_norm: first the
    squared norm over every owned bucket (kept on the device), then the clipped
    fused update of every bucket."""
    rank_end = L.n_dp if rank_end is None else rank_end
    ranges = bucket_ranges(L, rank_begin * L.shard, rank_end * L.shard)
    div = float(L.n_dp)
    for j, (s, e) in enumerate(ranges):
        zb.zero_grad_norm_sq(L, grads, zb.ZERO_BF16, grad_base, div, s, e, bufs.workspace,
                             bufs.norm_sq, j > 0, stream)
    for s, e in ranges:
        zb.zero_reduce_scatter_adamw_clip(L, grads, zb.ZERO_BF16, grad_base, div, rank_begin,
                                          rank_end, s, e, master, m, v, out, zb.ZERO_OUT_FULL,
                                          hp, bufs.norm_sq, max_norm, stream)


# --------------------------------------------------------------------------
# ZeRO-3 ("DeepSpeed ZeRO", "Stage 3 step by step"; "ZeRO and FSDP", "FSDP,
# ZeRO-3 inside PyTorch": per-unit flat buffers, at most two gathered at once)
# --------------------------------------------------------------------------

@dataclass
class GatherRing:
    """Two gathered-unit buffers reused in turn.  ``acquire`` hands out a slot
    for a unit; ``release`` returns it.  ``peak`` counts the most units that
    were ever resident at once."""
    capacity: int
    device: str = "cuda"
    slots: int = 2
    buffers: list = field(default_factory=list)
    owner: list = field(default_factory=list)
    peak: int = 0

    def __post_init__(self):
        self.buffers = [torch.empty(self.capacity, dtype=torch.bfloat16, device=self.device)
                        for _ in range(self.slots)]
        self.owner = [None] * self.slots

    def acquire(self, unit_id, numel: int) -> torch.Tensor:
        if numel > self.capacity:
            raise ValueError(f"unit of {numel} elements exceeds the ring's {self.capacity}")
        for i, o in enumerate(self.owner):
            if o is None:
                self.owner[i] = unit_id
                self.peak = max(self.peak, sum(x is not None for x in self.owner))
                return self.buffers[i][:numel]
        raise RuntimeError("both gathered-unit slots are in use: release one first")

    def release(self, unit_id):
        for i, o in enumerate(self.owner):
            if o == unit_id:
                self.owner[i] = None
                return
        raise KeyError(unit_id)

    @property
    def resident(self) -> int:
        return sum(x is not None for x in self.owner)


@dataclass
class Zero3Unit:
    """One unit's sharded state: n_dp bf16 shards (one [n_dp, S] tensor whose row
    o is rank o's shard) and the owners' fp32 master / m / v (P elements)."""
    layout: zb.ZeroLayout
    shards: torch.Tensor
    master: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor

    def shard_list(self):
        return [self.shards[o] for o in range(self.layout.n_dp)]


def zero3_gather(unit: Zero3Unit, ring: GatherRing, unit_id, stream=None) -> torch.Tensor:
    buf = ring.acquire(unit_id, unit.layout.padded_n)
    zb.zero_gather_layer(unit.layout, unit.shard_list(), buf, stream)
    return buf


def zero3_layer_reduce_scatter(unit: Zero3Unit, layer_grads, A: torch.Tensor, first: bool = True,
                               stream=None):
    """Each owner receives the sum over ranks of its slice of the unit's
    gradient, in fp32 (the mean's division is applied by the update)."""
    L = unit.layout
    zb.zero_accumulate(L, zb.ZERO_ACC_REDUCE, layer_grads, zb.ZERO_BF16, 0, A, 0, 0, L.padded_n,
                       first, stream)


def zero3_update(unit: Zero3Unit, A: torch.Tensor, hp, n_micro: int = 1, stream=None):
    """Every owner updates its shard and writes bf16 into its own shard only
    (no final all-gather at stage 3)."""
    L = unit.layout
    zb.zero_reduce_scatter_adamw(L, [A], zb.ZERO_F32, 0, float(L.n_dp * n_micro), 0, L.n_dp,
                                 0, L.padded_n, unit.master, unit.m, unit.v,
                                 unit.shards.view(-1), zb.ZERO_OUT_SHARD, hp, stream)


def zero3_clipped_updates(units, grads_fp32, hp, max_norm: float, bufs: "NormBuffers",
                          n_micro: int = 1, stream=None):
    """Stage 3 with clipping by the global gradient norm: the norm covers every
    unit's reduced gradient, so the updates wait for the whole backward.
    grads_fp32[i] is unit i's fp32 owned-shard sums (zero3_layer_reduce_scatter);
    the squared norm of the mean gradient accumulates over the units on the
    device, then every unit updates with the clipped gradient."""
    for j, (u, A) in enumerate(zip(units, grads_fp32)):
        L = u.layout
        zb.zero_grad_norm_sq(L, [A], zb.ZERO_F32, 0, float(L.n_dp * n_micro), 0, L.padded_n,
                             bufs.workspace, bufs.norm_sq, j > 0, stream)
    for u, A in zip(units, grads_fp32):
        L = u.layout
        zb.zero_reduce_scatter_adamw_clip(L, [A], zb.ZERO_F32, 0, float(L.n_dp * n_micro), 0, L.n_dp,
                                          0, L.padded_n, u.master, u.m, u.v, u.shards.view(-1),
                                          zb.ZERO_OUT_SHARD, hp, bufs.norm_sq, max_norm, stream)


def zero3_reduce_scatter_update(unit: Zero3Unit, layer_grads, hp, stream=None):
    """The layer reduce-scatter and the update of the unit's owned shards in one
    pass, with bf16 into each rank's own shard.  Valid when the step has one
    micro-batch and no global-norm clipping: each element's update then needs
    only its own gradient, so a unit can be updated as soon as its gradient is
    reduced (the units still to run backward keep their weights).  The sum
    starts from +0 and is divided once, as in zero3_layer_reduce_scatter
    followed by zero3_update, so the result is bit-identical to that pair;
    it skips the fp32 buffer's write and re-read (8 bytes per element)."""
    L = unit.layout
    zb.zero_reduce_scatter_adamw(L, layer_grads, zb.ZERO_BF16, 0, float(L.n_dp), 0, L.n_dp,
                                 0, L.padded_n, unit.master, unit.m, unit.v,
                                 unit.shards.view(-1), zb.ZERO_OUT_SHARD, hp, stream)


# --------------------------------------------------------------------------
# host-resident gradients: copies overlapped with the per-bucket update
# --------------------------------------------------------------------------

class HostPipeline:
    """A ZeRO-1/2 step whose gradients arrive in pinned host memory and whose
    bf16 result goes back to pinned host memory.  Bucket b's host-to-device
    copies run on one stream, its fused update on the caller's stream once they
    have landed, and its device-to-host copy on a third stream, so the copies of
    one bucket overlap the update of the previous one ("ZeRO and FSDP", stage
    2: each bucket is reduce-scattered as soon as it is ready).  With
    defer_out the result copies start only once every gradient copy has
    landed: on hosts where the two directions of the link slow each other
    down, the gradients then have the link to themselves."""

    def __init__(self, L, device=None, chunk_elems: int | None = None, defer_out: bool = False):
        self.L = L
        self.defer_out = defer_out
        self.ranges = split_ranges(bucket_ranges(L), chunk_elems)
        self.h2d = torch.cuda.Stream(device=device)
        self.d2h = torch.cuda.Stream(device=device)
        self.ev_in = [torch.cuda.Event() for _ in self.ranges]
        self.ev_done = [torch.cuda.Event() for _ in self.ranges]
        self.ev_out = torch.cuda.Event()

    def step(self, host_grads, dev_grads, master, m, v, out, host_out, hp):
        L = self.L
        comp = torch.cuda.current_stream()
        self.h2d.wait_stream(comp)       # the device gradient buffer is free to overwrite
        with torch.cuda.stream(self.h2d):
            for j, (s, e) in enumerate(self.ranges):
                for r in range(L.n_dp):
                    dev_grads[r, s:e].copy_(host_grads[r, s:e], non_blocking=True)
                self.ev_in[j].record(self.h2d)
        rows = [dev_grads[r] for r in range(L.n_dp)]
        for j, (s, e) in enumerate(self.ranges):
            comp.wait_event(self.ev_in[j])
            zb.zero_reduce_scatter_adamw(L, rows, zb.ZERO_BF16, 0, float(L.n_dp), 0, L.n_dp, s, e,
                                         master, m, v, out, zb.ZERO_OUT_FULL, hp, comp)
            self.ev_done[j].record(comp)
        with torch.cuda.stream(self.d2h):
            if self.defer_out and self.ranges:
                self.d2h.wait_event(self.ev_in[-1])
            for j, (s, e) in enumerate(self.ranges):
                self.d2h.wait_event(self.ev_done[j])
                host_out[s:e].copy_(out[s:e], non_blocking=True)
            self.ev_out.record(self.d2h)
        comp.wait_event(self.ev_out)     # the step ends when the result is on the host


class HostDirect:
    """A ZeRO-1/2 step whose gradients stay in pinned host memory: the fused
    kernel reads the n_dp gradient rows over the host link itself (on
    Grace-Blackwell the NVLink-C2C), bucket by bucket, with no staging copy;
    each bucket's bf16 result is copied back to pinned host memory on a second
    stream while the next bucket updates."""

    def __init__(self, L, device=None):
        self.L = L
        self.ranges = bucket_ranges(L)
        self.d2h = torch.cuda.Stream(device=device)
        self.ev_done = [torch.cuda.Event() for _ in self.ranges]
        self.ev_out = torch.cuda.Event()

    def step(self, host_grads, master, m, v, out, host_out, hp):
        L = self.L
        comp = torch.cuda.current_stream()
        rows = [host_grads[r] for r in range(L.n_dp)]
        for j, (s, e) in enumerate(self.ranges):
            zb.zero_reduce_scatter_adamw(L, rows, zb.ZERO_BF16, 0, float(L.n_dp), 0, L.n_dp, s, e,
                                         master, m, v, out, zb.ZERO_OUT_FULL, hp, comp)
            self.ev_done[j].record(comp)
        with torch.cuda.stream(self.d2h):
            for j, (s, e) in enumerate(self.ranges):
                self.d2h.wait_event(self.ev_done[j])
                host_out[s:e].copy_(out[s:e], non_blocking=True)
            self.ev_out.record(self.d2h)
        comp.wait_event(self.ev_out)     # the step ends when the result is on the host


# --------------------------------------------------------------------------
# ZeRO-3 with 8-bit weight gathers ("ZeRO Optimizer, in depth", "Offload and
# ZeRO++": zero_quantized_weights)
# --------------------------------------------------------------------------

class Int8Shards:
    """A unit's quantized shards: int8 [n_dp, S] and fp32 block scales
    [n_dp, ceil(S / block)], what each rank would send in the all-gather."""

    def __init__(self, layout, block: int = 256, device="cuda"):
        self.layout = layout
        self.block = block
        self.nb = -(-layout.shard // block) if layout.shard else 0
        self.q = torch.empty((layout.n_dp, layout.shard), dtype=torch.int8, device=device)
        self.scales = torch.empty((layout.n_dp, max(self.nb, 1)), dtype=torch.float32, device=device)

    def wire_bytes(self) -> int:
        return self.q.numel() + self.layout.n_dp * self.nb * 4


def zero3_quantize(unit: Zero3Unit, qs: Int8Shards, stream=None):
    """Each owner quantizes its bf16 shard (after its update) for the next gathers."""
    zb.zero_quantize_int8(unit.layout, unit.shards.view(-1), qs.q.view(-1), qs.scales.view(-1),
                          qs.block, stream)


def zero3_update_q8(unit: Zero3Unit, A: torch.Tensor, qs: Int8Shards, hp, n_micro: int = 1,
                    stream=None):
    """zero3_update followed by zero3_quantize in one pass: the owners' update
    writes their shards straight in the 8-bit format (block 256; the unit laid
    out with align 256).  The bf16 shards are not written."""
    L = unit.layout
    zb.zero_reduce_scatter_adamw_q8(L, [A], zb.ZERO_F32, 0, float(L.n_dp * n_micro), 0, L.n_dp,
                                    0, L.padded_n, unit.master, unit.m, unit.v, qs.q.view(-1),
                                    qs.scales.view(-1), qs.block, hp, stream)


def zero3_reduce_scatter_update_q8(unit: Zero3Unit, layer_grads, qs: Int8Shards, hp, stream=None):
    """zero3_reduce_scatter_update with the 8-bit output of zero3_update_q8:
    the unit's gradient reduce-scatter, update and quantization in one pass
    (one micro-batch, no clipping)."""
    L = unit.layout
    zb.zero_reduce_scatter_adamw_q8(L, layer_grads, zb.ZERO_BF16, 0, float(L.n_dp), 0, L.n_dp,
                                    0, L.padded_n, unit.master, unit.m, unit.v, qs.q.view(-1),
                                    qs.scales.view(-1), qs.block, hp, stream)


def zero3_gather_int8(unit: Zero3Unit, qs: Int8Shards, ring: GatherRing, unit_id,
                      stream=None) -> torch.Tensor:
    buf = ring.acquire(unit_id, unit.layout.padded_n)
    n = unit.layout.n_dp
    zb.zero_gather_layer_int8(unit.layout, [qs.q[o] for o in range(n)],
                              [qs.scales[o] for o in range(n)], buf, qs.block, stream)
    return buf


# --------------------------------------------------------------------------
# 8-bit gradient reduce-scatter ("ZeRO Optimizer, in depth", "Offload and
# ZeRO++": zero_quantized_gradients; "ZeRO and FSDP", "Fewer bytes on the
# wire": gradients quantized during the reduce-scatter)
# --------------------------------------------------------------------------

def side_streams(n: int, device=None) -> list:
    """Side streams for n simulated ranks' independent launches (at most 8)."""
    return [torch.cuda.Stream(device=device) for _ in range(max(1, min(n, 8)))]


def quantize_ranks(L, grads, q, scales, block: int, side=None, stream=None):
    """Every simulated rank quantizes its bf16 gradient grads[r] into q[r] and
    scales[r] (zero_quantize_int8 over layout L).  With side streams the ranks
    quantize at the same time, as ranks on their own GPUs would: each rank's
    launch runs on a side stream forked from the caller's stream and joined
    back into it before returning -- bit-identical to one after another, and
    measured 7.04 against 6.78 TB/s on a Llama-7B block unit at n_dp = 8, where
    each rank's launch is short."""
    n = len(grads)
    if not side or n == 1 or isinstance(stream, int):
        for r in range(n):
            zb.zero_quantize_int8(L, grads[r], q[r], scales[r], block, stream)
        return
    cur = stream if stream is not None else torch.cuda.current_stream()
    for s in side:
        s.wait_stream(cur)
    for r in range(n):
        zb.zero_quantize_int8(L, grads[r], q[r], scales[r], block, side[r % len(side)])
    for s in side:
        cur.wait_stream(s)


class Int8Grads:
    """Every simulated rank's quantized gradient: codes [n_src, P] int8 and
    block scales [n_src, n_dp * ceil(S / block)] fp32.  Row r is what rank r
    sends in the reduce-scatter: its slice o (codes [o*S, (o+1)*S), scales
    [o*nb, (o+1)*nb)) to owner o."""

    def __init__(self, layout, n_src: int | None = None, block: int = 256, device="cuda"):
        self.layout = layout
        self.block = block
        self.n_src = layout.n_dp if n_src is None else n_src
        self.nb = -(-layout.shard // block) if layout.shard else 0
        self.q = torch.empty((self.n_src, layout.padded_n), dtype=torch.int8, device=device)
        self.scales = torch.empty((self.n_src, max(layout.n_dp * self.nb, 1)), dtype=torch.float32,
                                  device=device)

    def quantize(self, grads, stream=None, concurrent: bool = True):
        """Each rank quantizes its bf16 gradient (P elements), slice by slice;
        with concurrent, all ranks at once (quantize_ranks)."""
        if concurrent and getattr(self, "_side", None) is None:
            self._side = side_streams(self.n_src, self.q.device)
        quantize_ranks(self.layout, grads, [self.q[r] for r in range(self.n_src)],
                       [self.scales[r] for r in range(self.n_src)], self.block,
                       self._side if concurrent else None, stream)

    def sources(self):
        return [self.q[r] for r in range(self.n_src)], [self.scales[r] for r in range(self.n_src)]

    def wire_bytes(self) -> int:
        """Bytes one rank sends: its slices for the n_dp - 1 other owners."""
        L = self.layout
        return (L.n_dp - 1) * (L.shard + self.nb * 4)


def zero12_step_int8(L, qg: Int8Grads, master, m, v, out, hp, rank_begin=0, rank_end=None,
                     stream=None):
    """A ZeRO-1/2 step from 8-bit gradients, bucket by bucket: every owner
    dequantizes the ranks' slices, takes the fp32 mean and updates."""
    rank_end = L.n_dp if rank_end is None else rank_end
    qs, ss = qg.sources()
    for s, e in bucket_ranges(L, rank_begin * L.shard, rank_end * L.shard):
        zb.zero_reduce_scatter_adamw_int8(L, qs, ss, qg.block, float(L.n_dp), rank_begin, rank_end,
                                          s, e, master, m, v, out, zb.ZERO_OUT_FULL, hp, stream)


def zero3_layer_reduce_scatter_int8(unit: Zero3Unit, qg: Int8Grads, A: torch.Tensor,
                                    first: bool = True, stream=None):
    """The stage-3 layer reduce-scatter from 8-bit unit gradients: each owner
    receives the fp32 sum over ranks of its dequantized slice."""
    L = unit.layout
    qs, ss = qg.sources()
    zb.zero_accumulate_int8(L, qs, ss, qg.block, A, 0, 0, L.padded_n, first, stream)


def zero3_reduce_scatter_update_int8_q8(unit: Zero3Unit, qg: Int8Grads, qs: Int8Shards, hp,
                                        stream=None):
    """Both ZeRO++ 8-bit paths in one pass per unit (one micro-batch, no
    clipping): the owners dequantize the ranks' 8-bit gradient slices, update,
    and write their shards straight in the 8-bit format (block 256)."""
    L = unit.layout
    q_src, s_src = qg.sources()
    zb.zero_reduce_scatter_adamw_int8_q8(L, q_src, s_src, qg.block, float(L.n_dp), 0, L.n_dp, 0,
                                         L.padded_n, unit.master, unit.m, unit.v, qs.q.view(-1),
                                         qs.scales.view(-1), qs.block, hp, stream)


# --------------------------------------------------------------------------
# ZeRO-3 prefetch ("DeepSpeed ZeRO", "Stage 3 step by step": prefetching so
# that the gather for the next layer overlaps with the compute of the current
# one; "ZeRO and FSDP", "FSDP, ZeRO-3 inside PyTorch": with prefetching the
# next unit is being gathered while the current one computes, so up to two
# units are resident)
# --------------------------------------------------------------------------

class Zero3Prefetcher:
    """Gathers units one ahead on a side stream into a two-slot GatherRing.

    prefetch(i) first makes the side stream wait for everything already queued
    on the caller's stream -- in particular the release of the slot's previous
    unit and the last update of unit i's shards -- then enqueues the gather
    and records an event; get(i) makes the caller's stream wait for that event.
    """

    def __init__(self, units, ring: GatherRing, int8=None, device=None):
        self.units = units
        self.ring = ring
        self.int8 = int8
        self.side = torch.cuda.Stream(device=device)
        self.pending = {}

    def prefetch(self, i, tag):
        main = torch.cuda.current_stream()
        issued = torch.cuda.Event()
        issued.record(main)
        self.side.wait_event(issued)
        with torch.cuda.stream(self.side):
            if self.int8 is not None:
                buf = zero3_gather_int8(self.units[i], self.int8[i], self.ring, (tag, i), self.side)
            else:
                buf = zero3_gather(self.units[i], self.ring, (tag, i), self.side)
            ready = torch.cuda.Event()
            ready.record(self.side)
        self.pending[(tag, i)] = (buf, ready)

    def get(self, i, tag) -> torch.Tensor:
        buf, ready = self.pending.pop((tag, i))
        torch.cuda.current_stream().wait_event(ready)
        return buf

    def release(self, i, tag):
        self.ring.release((tag, i))


def zero3_step_prefetched(pf: Zero3Prefetcher, unit_grads, A: torch.Tensor, hp, compute=None):
    """One stage-3 step over all units with gathers one unit ahead: forward in
    order, backward in reverse (gather, compute, reduce-scatter the unit's
    gradient, update its owned shards).  unit_grads(i) returns unit i's n_dp
    bf16 gradient buffers; compute(i, gathered, phase) stands in for the
    layer's work and may be None."""
    units = pf.units
    n = len(units)
    if n == 0:
        return
    pf.prefetch(0, "fwd")
    for i in range(n):
        buf = pf.get(i, "fwd")
        if i + 1 < n:
            pf.prefetch(i + 1, "fwd")
        if compute is not None:
            compute(i, buf, "fwd")
        pf.release(i, "fwd")
    pf.prefetch(n - 1, "bwd")
    for i in reversed(range(n)):
        buf = pf.get(i, "bwd")
        if i > 0:
            pf.prefetch(i - 1, "bwd")
        if compute is not None:
            compute(i, buf, "bwd")
        P = units[i].layout.padded_n
        zero3_layer_reduce_scatter(units[i], unit_grads(i), A[:P])
        pf.release(i, "bwd")
        zero3_update(units[i], A[:P], hp)
        if pf.int8 is not None:
            zero3_quantize(units[i], pf.int8[i])
