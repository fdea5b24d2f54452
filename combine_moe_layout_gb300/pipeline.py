"""Steps through the C ABI, with torch for device memory.

``MoeStep`` owns the device buffers of one problem size and runs
layout -> dispatch -> experts -> combine on a stream. The experts are the
synthetic ones of the workloads: identity for bf16 steps (combine reads the
receive buffer itself) and ``moe_expert_stub`` for fp8 steps.

``LocalMoe`` is an MoE layer of one device that is no part of an EP group: router,
token sort, expert stage and the way back, the gradients of all but the experts,
and a projection shared by all requests with each request's low-rank adapter.
"""
from __future__ import annotations

import math
from contextlib import nullcontext
from dataclasses import dataclass

import numpy as np
import torch

from . import _binding as B


@dataclass
class DeviceInputs:
    topk_idx: torch.Tensor      # [R][T][k] int32
    topk_weights: torch.Tensor  # [R][T][k] float32
    x: torch.Tensor             # [R][T][H] uint8 (fp8 codes) or bfloat16
    x_scales: torch.Tensor | None


def to_pinned_host(inputs) -> DeviceInputs:
    """The generated inputs in pinned host memory, for kernels that read them
    directly over the CPU-GPU link (bf16 bits are reinterpreted, not converted)."""
    def t(a):
        return torch.from_numpy(np.ascontiguousarray(a)).pin_memory()

    x = t(inputs.x)
    if x.dtype == torch.uint16:
        x = x.view(torch.bfloat16)
    return DeviceInputs(t(inputs.topk_idx), t(inputs.topk_weights), x,
                        None if inputs.x_scales is None else t(inputs.x_scales))


def to_device(inputs, device, pin: bool = False) -> DeviceInputs:
    """Copy generated numpy inputs to the device (bf16 bits are reinterpreted, not converted)."""
    def t(a):
        ht = torch.from_numpy(np.ascontiguousarray(a))
        if pin:
            ht = ht.pin_memory()
        return ht.to(device, non_blocking=pin)

    x = t(inputs.x)
    if x.dtype == torch.uint16:
        x = x.view(torch.bfloat16)
    elif x.dtype != torch.uint8:
        raise ValueError("x must hold uint16 bf16 bits or uint8 e4m3 codes")
    return DeviceInputs(t(inputs.topk_idx), t(inputs.topk_weights), x,
                        None if inputs.x_scales is None else t(inputs.x_scales))


class MoeStep:
    def __init__(self, workload, device="cuda", num_sms: int = 0, buffers: B.MoeBuffers | None = None):
        self.w = workload
        self.desc = B.MoeDesc.of(workload, num_sms)
        self.fp8 = workload.dtype != "bf16"  # slots hold e4m3 rows + scales
        self.device = torch.device(device)
        self.buf = buffers if buffers is not None else B.allocate_buffers(self.desc, self.device)
        self.slots = workload.num_experts * workload.num_ranks * workload.max_m
        if self.buf.expert_out is not None:
            self.y = self.buf.expert_out
        else:  # identity experts: combine reads the dispatched rows themselves
            self.y = self.buf.recv_x.view(torch.bfloat16).view(self.slots, workload.hidden)

    def reset(self, stream=None):
        B.moe_reset(self.desc, self.buf.flags, self.buf.err, stream)

    def layout(self, d: DeviceInputs, stream=None):
        b = self.buf
        B.moe_layout(self.desc, d.topk_idx, b.counts, b.flags, b.tok_slot, b.err, stream)

    def dispatch(self, d: DeviceInputs, stream=None):
        b = self.buf
        B.moe_dispatch(self.desc, d.x, d.x_scales, b.tok_slot, b.flags, b.recv_x, b.recv_scales, b.recv_meta, b.err,
                       stream)

    def layout_dispatch(self, d: DeviceInputs, stream=None):
        b = self.buf
        B.moe_layout_dispatch(self.desc, d.topk_idx, d.x, d.x_scales, b.counts, b.flags, b.tok_slot, b.recv_x,
                              b.recv_scales, b.recv_meta, b.err, stream)

    def experts(self, stream=None):
        if self.fp8:
            b = self.buf
            B.moe_expert_stub(self.desc, b.recv_x, b.recv_scales, b.counts, b.expert_out, b.err, stream)

    def combine(self, d: DeviceInputs, stream=None, out=None):
        """out: the step's output buffer (default: the device buffer; may be pinned host memory)."""
        b = self.buf
        B.moe_combine(self.desc, self.y, d.topk_weights, b.tok_slot, b.flags, b.out if out is None else out, b.err,
                      stream)

    def run(self, d: DeviceInputs, stream=None, fused: bool = False):
        if fused:
            self.layout_dispatch(d, stream)
        else:
            self.layout(d, stream)
            self.dispatch(d, stream)
        self.experts(stream)
        self.combine(d, stream)

    def recv(self, packed: B.PackedBuffers, stream=None):
        """The receive hook: wait for the counts, pack the filled slots expert-major."""
        b = self.buf
        B.moe_dispatch_recv(self.desc, b.counts, b.flags, b.recv_x, b.recv_scales, b.recv_meta, b.tok_slot,
                            packed.region_offsets, packed.packed_x, packed.packed_scales, packed.packed_meta,
                            packed.tok_packed, b.err, stream)

    def combine_packed(self, d: DeviceInputs, packed_y: torch.Tensor, packed: B.PackedBuffers, stream=None,
                       out=None):
        b = self.buf
        B.moe_combine_packed(self.desc, packed_y, packed.tok_packed, d.topk_weights, b.flags,
                             b.out if out is None else out, b.err, stream)

    def expert_mlp(self, weights, packed: B.PackedBuffers, h: torch.Tensor, packed_y: torch.Tensor, stream=None):
        """The expert stage on the packed rows: linear 1 with SwiGLU into h [R*T*k][I],
        then linear 2 into packed_y [R*T*k][H] (what combine_packed reads)."""
        b = self.buf
        B.moe_expert_gate_up(self.desc, weights.inter, packed.region_offsets, packed.packed_x, weights.w_gate,
                             weights.w_up, h, b.err, stream)
        B.moe_expert_down(self.desc, weights.inter, packed.region_offsets, h, weights.w_down, packed_y, b.err, stream)

    def expert_mlp_fp8(self, weights, packed: B.PackedBuffers, h: torch.Tensor, h_scales: torch.Tensor,
                       packed_y: torch.Tensor, stream=None):
        """The fp8 expert stage on e4m3 packed rows: linear 1 with SwiGLU into h
        (e4m3 [R*T*k][I]) and h_scales ([R*T*k][I/128]), then linear 2 into
        packed_y [R*T*k][H] bf16."""
        b = self.buf
        B.moe_expert_gate_up_fp8(self.desc, weights.inter, packed.region_offsets, packed.packed_x,
                                 packed.packed_scales, weights.w_gate, weights.w_gate_scales, weights.w_up,
                                 weights.w_up_scales, h, h_scales, b.err, stream)
        B.moe_expert_down_fp8(self.desc, weights.inter, packed.region_offsets, h, h_scales, weights.w_down,
                              weights.w_down_scales, packed_y, b.err, stream)

    def error(self, stream=None) -> int:
        return B.moe_get_error(self.buf.err, stream)


def _expect(name: str, t, dtype, *shape):
    """A tensor argument of LocalMoe: its type and sizes, before a kernel reads by them. Leading sizes may be joined or
    split (rows of [batch][sequence][hidden] are as good as [tokens][hidden]); with a size of None, any, they are as
    listed."""
    good = isinstance(t, torch.Tensor) and t.dtype == dtype
    if good and None in shape:
        good = t.dim() == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape))
    elif good:
        good = t.dim() > 0 and t.numel() == math.prod(shape) and (len(shape) == 1 or t.shape[-1] == shape[-1])
    if not good:
        what = f"{t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else repr(t)
        sizes = ", ".join("any" if n is None else str(n) for n in shape)
        raise ValueError(f"LocalMoe: {name} is {what}, not {dtype} ({sizes})")


class LocalMoe:
    """An MoE layer of one device.

    forward: logits -> moe_gate -> moe_sort -> expert stage -> moe_unsort. backward takes the gradient of the
    output back through moe_unsort_grad, the caller's expert gradient, moe_sort_grad and moe_gate_grad. shared runs
    the projection beside the experts with the adapters of the batch's requests. The buffers of forward and backward
    are allocated once.

    Each method runs on ``stream`` (None: the current one) whole, what it does with torch and expert_grad included.
    The layer may have been made on another stream: the first call on a stream waits for that one's work up to then.
    Methods called on different streams share the layer's buffers, and ordering them is the caller's part.

    tokens x hidden bf16 rows, num_experts experts of width inter (a multiple of 128 when the expert stage runs)."""

    def __init__(self, tokens: int, hidden: int, num_experts: int, topk: int, opts: B.MoeGateOpts, device="cuda",
                 inter: int = 0):
        self.desc = B.MoeDesc(1, tokens, hidden, num_experts, topk, max(tokens, 1), B.MOE_BF16, 0)
        self.opts, self.inter = opts, inter
        n, dev = tokens * topk, torch.device(device)

        def rows(count, width):
            return torch.empty((count, width), dtype=torch.bfloat16, device=dev)

        def ints(*shape):
            return torch.empty(shape, dtype=torch.int32, device=dev)

        self.topk_idx, self.tok_packed = ints(tokens, topk), ints(tokens, topk)
        self.region_offsets = ints(num_experts + 1)
        self.topk_weights = torch.empty((tokens, topk), device=dev)
        self.packed_x, self.packed_y, self.out = rows(n, hidden), rows(n, hidden), rows(tokens, hidden)
        self.h = rows(n, inter) if inter else None
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.grad_y = self.grad_x = self.grad_weights = self.grad_logits = None  # allocated by the first backward
        self.u = None  # the last shared's scratch, its first part
        self.device = self.err.device
        self._streams = {}  # the streams that have used the buffers, by their handles
        if dev.type == "cuda":
            made_on = torch.cuda.current_stream(self.device)
            # (an event of a capture says nothing outside of it)
            self._made = None if torch.cuda.is_current_stream_capturing() else made_on.record_event()
            self._streams[made_on.cuda_stream] = made_on

    def _on(self, stream):
        """The context that a method runs in: ``stream`` is the current one there, and the layer's buffers may be used
        on it. Handles are compared, since building a Stream object takes longer than a small kernel's launch."""
        if self.device.type != "cuda":
            return nullcontext()  # the binding refuses it
        handle = torch._C._cuda_getCurrentRawStream(self.device.index) if stream is None else stream.cuda_stream
        if handle not in self._streams:
            s = torch.cuda.current_stream(self.device) if stream is None else stream
            with torch.cuda.stream(s):
                # (a capture begins with nothing pending, and a captured stream may not wait for an event before it)
                if self._made is not None and not torch.cuda.is_current_stream_capturing():
                    s.wait_event(self._made)
            self._streams[handle] = s
            self._keep_for([s])
        return nullcontext() if stream is None else torch.cuda.stream(stream)

    def _keep_for(self, streams):
        """The layer's buffers are given out again, after the layer, only when these streams have passed them."""
        for t in vars(self).values():
            if isinstance(t, torch.Tensor):
                for s in streams:
                    t.record_stream(s)

    def _expect_logits(self, logits):
        _expect("logits", logits, torch.bfloat16 if self.opts.logits_bf16 else torch.float32, self.desc.tokens_per_rank,
                self.desc.num_experts)

    def route(self, logits, bias=None, stream=None):
        self._expect_logits(logits)
        if bias is not None:
            _expect("bias", bias, torch.float32, self.desc.num_experts)
        with self._on(stream):
            B.moe_gate(self.desc, self.opts, logits, bias, self.topk_idx, self.topk_weights, self.err)

    def sort(self, x, stream=None):
        _expect("x", x, torch.bfloat16, *self.out.shape)
        with self._on(stream):
            B.moe_sort(self.desc, self.topk_idx, x, None, self.region_offsets, self.packed_x, None, self.tok_packed,
                       self.err)

    def experts(self, weights, stream=None):
        """The expert stage on the sorted rows (weights: workloads.ExpertWeights)."""
        E, H, I = self.desc.num_experts, self.desc.hidden, self.inter
        if not I:
            raise ValueError("LocalMoe: a layer made with inter = 0 has no expert stage")
        _expect("w_gate", weights.w_gate, torch.bfloat16, E, I, H)
        _expect("w_up", weights.w_up, torch.bfloat16, E, I, H)
        _expect("w_down", weights.w_down, torch.bfloat16, E, H, I)
        with self._on(stream):
            B.moe_expert_gate_up(self.desc, self.inter, self.region_offsets, self.packed_x, weights.w_gate,
                                 weights.w_up, self.h, self.err)
            B.moe_expert_down(self.desc, self.inter, self.region_offsets, self.h, weights.w_down, self.packed_y,
                              self.err)

    def unsort(self, stream=None):
        with self._on(stream):
            B.moe_unsort(self.desc, self.packed_y, self.tok_packed, self.topk_weights, self.out, self.err)
        return self.out

    def forward(self, x, logits, weights, bias=None, stream=None):
        """x [tokens][hidden], logits [tokens][num_experts] -> the routed experts' output [tokens][hidden], a buffer of
        the layer that the next forward writes again."""
        self.route(logits, bias, stream)
        self.sort(x, stream)
        self.experts(weights, stream)
        return self.unsort(stream)

    def backward(self, grad_out, logits, expert_grad, stream=None):
        """The gradients of x and of the logits, in buffers of the layer that the next backward writes again.
        expert_grad(packed_x, region_offsets, grad_y) is the caller's gradient of the experts: from the gradient of
        packed_y to that of packed_x, row by row, both bf16 [tokens * topk][hidden]. It is called with ``stream`` as
        the current one. Rows at or above region_offsets' last entry belong to no choice: packed_x and grad_y hold
        nothing of this batch there."""
        _expect("grad_out", grad_out, torch.bfloat16, *self.out.shape)
        self._expect_logits(logits)
        with self._on(stream):
            if self.grad_y is None:
                self.grad_y, self.grad_x = torch.zeros_like(self.packed_y), torch.empty_like(self.out)
                self.grad_weights = torch.empty_like(self.topk_weights)
                self.grad_logits = torch.empty_like(logits)
                self._keep_for(self._streams.values())
            B.moe_unsort_grad(self.desc, self.packed_y, self.tok_packed, self.topk_weights, grad_out, self.grad_y,
                              self.grad_weights, self.err)
            grad_packed = expert_grad(self.packed_x, self.region_offsets, self.grad_y)
            _expect("expert_grad's result", grad_packed, torch.bfloat16, *self.packed_x.shape)
            B.moe_sort_grad(self.desc, grad_packed, self.tok_packed, self.grad_x, self.err)
            B.moe_gate_grad(self.desc, self.opts, logits, self.topk_idx, self.grad_weights, self.grad_logits, self.err)
        return self.grad_x, self.grad_logits

    def shared(self, x, w, lora_a=None, lora_b=None, scales=None, adapter=None, stream=None, u_parts=2):
        """x w^T [tokens][out] with each token's adapter beside it (moe_lora_linear), or, without lora_a, alone: x
        [tokens][in] and w [out][in] bf16, lora_a [A][rank][in] and lora_b [A][out][rank] bf16, scales [A] float32 or
        None, adapter [tokens] int32. The result is the caller's own: it and the scratch u are new in each call, so
        that two projections, on one stream or on two, share nothing. u_parts: u = x lora_a^T as two bf16 parts, or as
        one, which takes up to a tenth less time and leaves 2^-9 of u."""
        bf16 = torch.bfloat16
        if u_parts not in (1, 2):
            raise ValueError(f"LocalMoe: u_parts is {u_parts!r}, not 1 or 2")
        _expect("x", x, bf16, None, None)
        (T, K), A, rank = x.shape, 0, 0
        _expect("w", w, bf16, None, K)
        N = w.shape[0]
        if lora_a is not None:
            _expect("lora_a", lora_a, bf16, None, None, K)
            A, rank, _ = lora_a.shape
            _expect("lora_b", lora_b, bf16, A, N, rank)
            _expect("adapter", adapter, torch.int32, T)
            if scales is not None:
                _expect("scales", scales, torch.float32, A)
        else:
            for name, t in (("lora_b", lora_b), ("scales", scales), ("adapter", adapter)):
                if t is not None:
                    raise ValueError(f"LocalMoe: {name} is given without lora_a")
        with self._on(stream):
            u = torch.empty((u_parts, T, rank), dtype=bf16, device=x.device) if A else None
            self.u = u[0] if A else None
            out = torch.empty((T, N), dtype=bf16, device=x.device)
            B.moe_lora_linear(B.MoeLoraDesc(T, K, N, rank, A, 0, u_parts), x, w, lora_a, lora_b, scales, adapter, u, out,
                              self.err)
        return out

    def error(self, stream=None) -> int:
        with self._on(stream):
            return B.moe_get_error(self.err)
