"""Steps through the C ABI, with torch for device memory.

``MoeStep`` owns the device buffers of one problem size and runs
layout -> dispatch -> experts -> combine on a stream. The experts are the
synthetic ones of the workloads: identity for bf16 steps (combine reads the
receive buffer itself) and ``moe_expert_stub`` for fp8 steps.

``LocalMoe`` is an MoE layer of one device that is no part of an EP group: router,
token sort, expert stage and the way back with their gradients, from what the
forward keeps in bf16 or in 8 bits; and what stands beside them: a projection shared
by all requests with each request's low-rank adapter, a dense feed-forward block (a
shared expert), and the norms before and after a block with its gate and residual.
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


SAVE = {None: B.MOE_SAVE_NONE, "bf16": B.MOE_SAVE_BF16, "fp8": B.MOE_SAVE_FP8}


@dataclass
class KeptFfn:
    """What a feed-forward block's forward keeps of its two projections for its gradients: bf16 rows, or e4m3 rows
    (uint8 codes) with a float scale for each 128 columns."""
    desc: B.MoeFfnDesc
    gate: torch.Tensor
    up: torch.Tensor
    gate_scales: torch.Tensor | None
    up_scales: torch.Tensor | None


@dataclass
class NormGrads:
    """Gradients of LocalMoe.norm; None for what it did not have."""
    x: torch.Tensor
    o: torch.Tensor | None
    w_pre: torch.Tensor
    w_post: torch.Tensor | None
    gate: torch.Tensor | None


def _keep(desc: B.MoeFfnDesc, device) -> KeptFfn:
    n, I, fp8 = desc.rows, desc.inter, desc.save == B.MOE_SAVE_FP8

    def rows():
        return torch.empty((n, I), dtype=torch.uint8 if fp8 else torch.bfloat16, device=device)

    def scales():
        return torch.empty((n, I // 128), dtype=torch.float32, device=device) if fp8 else None

    return KeptFfn(desc, rows(), rows(), scales(), scales())


class LocalMoe:
    """An MoE layer of one device.

    forward: logits -> moe_gate -> moe_sort -> expert stage -> moe_unsort. backward takes the gradient of the
    output back through moe_unsort_grad, the experts' gradient (moe_ffn_grad, from what a forward with ``save`` kept, or
    the caller's own), moe_sort_grad and moe_gate_grad. shared runs the projection beside the experts with the adapters
    of the batch's requests, dense a feed-forward block of all tokens, norm the norms around a block; their results are
    new tensors. The buffers of forward and backward are allocated once, those of a ``save`` by the first forward with
    it, and stay: a captured graph may be replayed after a forward that kept another format.

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
        self.kept = None  # what the last forward with ``save`` kept, for backward
        self._kept_by = {}  # by ``save``: a graph captured with one format writes to its buffers after a call with another
        self._kept_now = False  # it was kept of the batch that the layer's buffers hold
        self.grad_gate = self.grad_up = self.grad_packed_x = None
        self.grad_w_gate = self.grad_w_up = self.grad_w_down = None  # by the first backward with the experts' weights
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
        kept = (t for k in self._kept_by.values() for t in vars(k).values())
        for t in (*vars(self).values(), *kept):
            if isinstance(t, torch.Tensor):
                for s in streams:
                    t.record_stream(s)

    def _expect_logits(self, logits):
        _expect("logits", logits, torch.bfloat16 if self.opts.logits_bf16 else torch.float32, self.desc.tokens_per_rank,
                self.desc.num_experts)

    def _expect_routing(self, logits, bias):
        self._expect_logits(logits)
        if bias is not None:
            _expect("bias", bias, torch.float32, self.desc.num_experts)

    def route(self, logits, bias=None, stream=None):
        self._expect_routing(logits, bias)
        with self._on(stream):
            self._route(logits, bias)

    def _route(self, logits, bias):
        self._kept_now = False  # what was kept belongs to the choices before these
        B.moe_gate(self.desc, self.opts, logits, bias, self.topk_idx, self.topk_weights, self.err)

    def sort(self, x, stream=None):
        _expect("x", x, torch.bfloat16, *self.out.shape)
        with self._on(stream):
            self._sort(x)

    def _sort(self, x):
        self._kept_now = False
        B.moe_sort(self.desc, self.topk_idx, x, None, self.region_offsets, self.packed_x, None, self.tok_packed, self.err)

    def _expect_experts(self, weights, save):
        E, H, I = self.desc.num_experts, self.desc.hidden, self.inter
        if not I:
            raise ValueError("LocalMoe: a layer made with inter = 0 has no expert stage")
        _expect("w_gate", weights.w_gate, torch.bfloat16, E, I, H)
        _expect("w_up", weights.w_up, torch.bfloat16, E, I, H)
        _expect("w_down", weights.w_down, torch.bfloat16, E, H, I)
        if save not in SAVE:
            raise ValueError(f"LocalMoe: save is {save!r}, not None, 'bf16' or 'fp8'")

    def experts(self, weights, stream=None, save=None):
        """The expert stage on the sorted rows (weights: workloads.ExpertWeights). save: "bf16" or "fp8" keeps what
        backward needs of it (kept), until the next route, sort or experts."""
        self._expect_experts(weights, save)
        with self._on(stream):
            self._experts(weights, save)

    def _experts(self, weights, save):
        self._kept_now = False
        if save is not None:
            if save not in self._kept_by:
                n, H = self.packed_x.shape
                desc = B.MoeFfnDesc(n, H, self.inter, self.desc.num_experts, 1, B.MOE_ACT_SILU, SAVE[save], 0)
                self._kept_by[save] = _keep(desc, self.device)
                self._keep_for(self._streams.values())
            self.kept = k = self._kept_by[save]
            B.moe_ffn(k.desc, self.region_offsets, self.packed_x, weights.w_gate, weights.w_up, weights.w_down, self.h,
                      self.packed_y, k.gate, k.gate_scales, k.up, k.up_scales, self.err)
            self._kept_now = True
            return
        B.moe_expert_gate_up(self.desc, self.inter, self.region_offsets, self.packed_x, weights.w_gate, weights.w_up,
                             self.h, self.err)
        B.moe_expert_down(self.desc, self.inter, self.region_offsets, self.h, weights.w_down, self.packed_y, self.err)

    def unsort(self, stream=None):
        with self._on(stream):
            B.moe_unsort(self.desc, self.packed_y, self.tok_packed, self.topk_weights, self.out, self.err)
        return self.out

    def forward(self, x, logits, weights, bias=None, stream=None, save=None):
        """x [tokens][hidden], logits [tokens][num_experts] -> the routed experts' output [tokens][hidden], a buffer of
        the layer that the next forward writes again. save as in experts. What it refuses it refuses before its first
        launch, with the last batch as it was."""
        self._expect_routing(logits, bias)
        _expect("x", x, torch.bfloat16, *self.out.shape)
        self._expect_experts(weights, save)
        with self._on(stream):
            self._route(logits, bias)
            self._sort(x)
            self._experts(weights, save)
            return self.unsort()

    def backward(self, grad_out, logits, expert_grad, stream=None):
        """The gradients of x and of the logits, in buffers of the layer that the next backward writes again.
        expert_grad: the experts' weights, after a forward with ``save``, which leaves the weights' gradients in
        grad_w_gate, grad_w_up and grad_w_down, buffers of the layer too. Or a function of the caller's (whatever can be
        called, a module that holds weights among them), expert_grad(packed_x, region_offsets, grad_y): from the
        gradient of packed_y to that of packed_x, row by row, both bf16 [tokens * topk][hidden]. It is called with
        ``stream`` as the current one. Rows at or above region_offsets' last entry belong to no choice: packed_x and
        grad_y hold nothing of this batch there."""
        _expect("grad_out", grad_out, torch.bfloat16, *self.out.shape)
        self._expect_logits(logits)
        own = hasattr(expert_grad, "w_gate") and not callable(expert_grad)
        if own:
            self._expect_experts(expert_grad, None)
            if not self._kept_now:
                raise ValueError("LocalMoe: backward with the experts' weights follows a forward with save")
        with self._on(stream):
            if self.grad_y is None:
                self.grad_y, self.grad_x = torch.zeros_like(self.packed_y), torch.empty_like(self.out)
                self.grad_weights = torch.empty_like(self.topk_weights)
                self.grad_logits = torch.empty_like(logits)
                self._keep_for(self._streams.values())
            if own and self.grad_packed_x is None:
                self.grad_packed_x = torch.empty_like(self.packed_x)
                self.grad_gate, self.grad_up = torch.empty_like(self.h), torch.empty_like(self.h)
                self.grad_w_gate, self.grad_w_up, self.grad_w_down = (
                    torch.empty(t.shape, dtype=t.dtype, device=self.device)
                    for t in (expert_grad.w_gate, expert_grad.w_up, expert_grad.w_down))
                self._keep_for(self._streams.values())
            B.moe_unsort_grad(self.desc, self.packed_y, self.tok_packed, self.topk_weights, grad_out, self.grad_y,
                              self.grad_weights, self.err)
            if own:
                k, w = self.kept, expert_grad
                B.moe_ffn_grad(k.desc, self.region_offsets, self.packed_x, k.gate, k.gate_scales, k.up, k.up_scales,
                               w.w_gate, w.w_up, w.w_down, self.grad_y, self.h, self.grad_gate, self.grad_up,
                               self.grad_packed_x, self.grad_w_gate, self.grad_w_up, self.grad_w_down, self.err)
                grad_packed = self.grad_packed_x
            else:
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
        one, which takes up to a tenth less time and leaves up to 2^-8 of u."""
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

    def dense(self, x, w_gate, w_up, w_down, act=B.MOE_ACT_SILU, save=None, stream=None):
        """A feed-forward block of all tokens, act(x w_gate^T) * (x w_up^T) w_down^T (a shared expert): x [rows][in],
        w_gate and w_up [inter][in], w_down [in][inter] bf16. The result y [rows][in], a new tensor, and what dense_grad
        needs of it: None without save ("bf16" or "fp8")."""
        bf16 = torch.bfloat16
        if save not in SAVE:
            raise ValueError(f"LocalMoe: save is {save!r}, not None, 'bf16' or 'fp8'")
        _expect("x", x, bf16, None, None)
        _expect("w_gate", w_gate, bf16, None, x.shape[1])
        I = w_gate.shape[0]
        _expect("w_up", w_up, bf16, I, x.shape[1])
        _expect("w_down", w_down, bf16, x.shape[1], I)
        desc = B.MoeFfnDesc(*x.shape, I, 1, 1, act, SAVE[save], 0)
        with self._on(stream):
            h, y = torch.empty((x.shape[0], I), dtype=bf16, device=x.device), torch.empty_like(x)
            k = _keep(desc, x.device) if save is not None else None
            B.moe_ffn(desc, None, x, w_gate, w_up, w_down, h, y, *((k.gate, k.gate_scales, k.up, k.up_scales) if k else
                                                                   (None,) * 4), self.err)
        return y, k

    def dense_grad(self, kept: KeptFfn, x, w_gate, w_up, w_down, grad_y, stream=None):
        """Gradients of dense with respect to x, w_gate, w_up and w_down (new tensors), from what it kept."""
        n, H, I = kept.desc.rows, kept.desc.hidden, kept.desc.inter
        bf16 = torch.bfloat16
        for name, t, shape in (("x", x, (n, H)), ("w_gate", w_gate, (I, H)), ("w_up", w_up, (I, H)),
                               ("w_down", w_down, (H, I)), ("grad_y", grad_y, (n, H))):
            _expect(name, t, bf16, *shape)
        with self._on(stream):
            scratch = [torch.empty((n, I), dtype=bf16, device=x.device) for _ in range(3)]
            grads = [torch.empty_like(t) for t in (x, w_gate, w_up, w_down)]
            B.moe_ffn_grad(kept.desc, None, x, kept.gate, kept.gate_scales, kept.up, kept.up_scales, w_gate, w_up, w_down,
                           grad_y, *scratch, *grads, self.err)
        return tuple(grads)

    @staticmethod
    def _norm_desc(x, w_pre, o, w_post, gate, by, eps, alpha):
        _expect("x", x, x.dtype if isinstance(x, torch.Tensor) and x.dtype == torch.float32 else torch.bfloat16, None, None)
        T, H = x.shape
        _expect("w_pre", w_pre, torch.float32, H)
        if by not in ("row", "channel"):
            raise ValueError(f"LocalMoe: by is {by!r}, not 'row' or 'channel'")
        if o is not None:
            _expect("o", o, torch.bfloat16, T, H)
        elif w_post is not None or gate is not None:
            raise ValueError("LocalMoe: w_post or gate is given without o")
        if w_post is not None:
            _expect("w_post", w_post, torch.float32, H)
        kind = B.MOE_GATE_NONE
        if gate is not None:
            _expect("gate", gate, torch.float32, T if by == "row" else H)
            kind = B.MOE_GATE_ROW if by == "row" else B.MOE_GATE_CHANNEL
        return B.MoeNormDesc(T, H, int(x.dtype == torch.float32), kind, eps, alpha)

    def norm(self, x, w_pre, o=None, w_post=None, gate=None, by="channel", eps=1e-6, alpha=1.0, stream=None):
        """The stream with a block's output o added, r = x + alpha gate (o / rms(o) w_post), and n = r / rms(r) w_pre,
        the next block's input (new tensors). x [rows][width] bf16 or float32, o bf16 or None (r is x then); w_post or
        None: o as it is; gate: float32, a value for each row or channel (by), or None."""
        desc = self._norm_desc(x, w_pre, o, w_post, gate, by, eps, alpha)
        with self._on(stream):
            r = torch.empty_like(x) if o is not None else None
            n = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
            B.moe_norm(desc, x, o, w_post, gate, w_pre, r, n, self.err)
        return (r if o is not None else x), n

    def norm_grad(self, r, grad_n, w_pre, grad_r=None, o=None, w_post=None, gate=None, by="channel", eps=1e-6, alpha=1.0,
                  stream=None) -> NormGrads:
        """Gradients of norm (new tensors) from the stream r that it returned and the gradients of both its results;
        grad_r None: r was not used beside n."""
        desc = self._norm_desc(r, w_pre, o, w_post, gate, by, eps, alpha)
        _expect("grad_n", grad_n, torch.bfloat16, *r.shape)
        if grad_r is not None:
            _expect("grad_r", grad_r, r.dtype, *r.shape)
        with self._on(stream):
            g = NormGrads(torch.empty_like(r), torch.empty_like(o) if o is not None else None, torch.empty_like(w_pre),
                          torch.empty_like(w_post) if w_post is not None else None,
                          torch.empty_like(gate) if gate is not None else None)
            work = torch.empty(max(1, B.moe_norm_workspace(desc)), dtype=torch.uint8, device=r.device)
            B.moe_norm_grad(desc, r, o, w_post, gate, w_pre, grad_r, grad_n, g.x, g.o, g.w_post, g.gate, g.w_pre, work,
                            self.err)
        return g

    def error(self, stream=None) -> int:
        with self._on(stream):
            return B.moe_get_error(self.err)
