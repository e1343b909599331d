"""Autograd wrappers and the activation-checkpoint handle recorder.

Gate, dispatch and combine on a layout handle, and the operators around
them: layer norm, dense products with their epilogue, the balance loss
(``block.py`` strings all of them together).

DeepSpeed #8213 "Add an opt-in DeepEP transport for the AutoEP expert
all-to-all", description: the backward of a combine is a dispatch and the
backward of a dispatch is a combine, both replayed against the handle the
forward layout produced; review thread: the routing weights are an autograd
input of the combine, so their gradient reaches the router.

Automodel #3684 "perf(moe): reuse the DeepEP dispatch layout on
activation-checkpoint recompute", "How": one recorder per checkpointed call;
the forward logs each dispatch's handle and routing metadata in call order,
the recompute consumes them in the same order, the dispatched activation is
not retained, and a replay that outruns its log falls back to a full layout
build rather than replaying a mismatched one.  Replay is only valid when the
routing is pinned across recompute; the recorder checks the expert ids it is
given against the logged ones (on the device) when asked to.

All arithmetic runs in the CUDA library (``binding``); this module only
wires tensors and handles together.  The library's gradients carry no graph:
a second derivative is refused (``first_order``), not taken as zero.
"""
from __future__ import annotations

import functools
from collections import deque

import torch

from . import binding as B


_words: dict[int, torch.Tensor] = {}  # a device's status word, the same for its whole life


def _status(t: torch.Tensor) -> torch.Tensor | None:
    """The status word of t's device (a host tensor goes to the library, which rejects it)."""
    if not t.is_cuda:
        return None
    word = _words.get(t.get_device())
    if word is None:
        if torch.cuda.is_current_stream_capturing():
            return None  # it would belong to the graph; a run before the capture makes it
        word = torch.zeros(1, dtype=torch.int32, device=t.device)
        torch.cuda.current_stream(t.device).synchronize()  # it is written from any stream
        word = _words.setdefault(t.get_device(), word)  # another thread may have been first
    return word


def status(device: torch.device | int | None = None) -> int:
    """Synchronise, read and clear what the kernels behind these wrappers reported on a device since the last call:
    MOE_DEV_* bits, 0 when all went well.  A set MOE_DEV_TIMEOUT means that a product's outputs are not all there.
    (A layout handle has a status of its own, ``Handle.status``.)"""
    index = torch.device("cuda", device).index if isinstance(device, int) else \
        torch.device(device).index if device is not None else None
    word = _words.get(torch.cuda.current_device() if index is None else index)
    if word is None:
        return 0
    torch.cuda.synchronize(word.device)
    bits = int(word.item())
    if bits:
        word.zero_()
        torch.cuda.synchronize(word.device)
    return bits


class _NoSecondDerivative(torch.autograd.Function):
    """The first argument, tied to the tensors that it depends on by a node that raises."""

    @staticmethod
    def forward(ctx, value: torch.Tensor, *sources):
        return value.view_as(value)

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError("the MoE library's gradients cannot be differentiated again")


def first_order(backward):
    """For a ``backward`` whose results carry no graph.  Under ``create_graph=True`` they are tied to the incoming
    gradients and the saved inputs, so that a derivative that would go through them raises.  (torch's
    ``once_differentiable`` ties them to nothing: ``torch.autograd.grad`` then never reaches its error.)"""

    @functools.wraps(backward)
    def call(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        sources = [t for t in (*grads, *ctx.saved_tensors) if t is not None and t.requires_grad]
        if not sources:
            return out
        tied = tuple(t if t is None else _NoSecondDerivative.apply(t, *sources)
                     for t in (out if isinstance(out, tuple) else (out,)))
        return tied if isinstance(out, tuple) else tied[0]

    return call


def _rows(t: torch.Tensor | None) -> torch.Tensor | None:
    """A contiguous tensor on 16 bytes, as the library wants its pointers: autograd hands out views (of a
    concatenation's gradient, say), and so do users (one expert's bias out of a packed one), that may start anywhere."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _strided(t: torch.Tensor | None, multiple: int = 1) -> torch.Tensor | None:
    """The same for calls that take rows apart from one another: a copy only where the rows are not contiguous, overlap
    (a broadcast), or start off the boundary (the first on 16 bytes, the others `multiple` elements apart)."""
    if t is None or (t.dim() == 2 and t.data_ptr() % 16 == 0 and (t.stride(1) == 1 or t.shape[1] == 1) and
                     (t.shape[0] == 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % multiple == 0))):
        return t
    return _rows(t)


class MoETopkGateFn(torch.autograd.Function):
    """(idx, gate) = topk_gate(logits); dlogits = topk_gate_bwd(dgate).  The
    expert ids are not differentiable; the gates' gradient reaches the router."""

    @staticmethod
    def forward(ctx, logits: torch.Tensor, k: int, renorm: int):
        logits = _rows(logits)
        idx, gate = B.moe_topk_gate(logits, k, renorm, device_status=_status(logits))
        ctx.renorm = int(renorm)
        ctx.e = logits.shape[1]
        ctx.save_for_backward(None if renorm else logits, idx, gate)
        ctx.mark_non_differentiable(idx)
        return idx, gate

    @staticmethod
    @first_order
    def backward(ctx, didx, dgate: torch.Tensor):
        logits, idx, gate = ctx.saved_tensors
        dl = B.moe_topk_gate_bwd(logits, idx, gate, _rows(dgate), ctx.e, ctx.renorm)
        return dl, None, None


def topk_gate(logits: torch.Tensor, k: int, renorm: int = 1):
    # copies are made before the node, so that what it saves is its own input
    return MoETopkGateFn.apply(_rows(logits), k, renorm)


class MoEDispatchFn(torch.autograd.Function):
    """X = dispatch(x) on a layout handle; dx = dispatch_bwd(dX) on the same handle."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, handle: B.Handle):
        ctx.handle = handle
        return B.moe_dispatch(handle, _rows(x))

    @staticmethod
    @first_order
    def backward(ctx, dX: torch.Tensor):
        return B.moe_dispatch_bwd(ctx.handle, _rows(dX)), None


class MoECombineFn(torch.autograd.Function):
    """out = combine(y, gate); (dY, dgate) = combine_bwd(dout, gate, y)."""

    @staticmethod
    def forward(ctx, y: torch.Tensor, gate: torch.Tensor, handle: B.Handle):
        y, gate = _rows(y), _rows(gate)
        ctx.handle = handle
        ctx.save_for_backward(y, gate)
        return B.moe_combine(handle, y, gate)

    @staticmethod
    @first_order
    def backward(ctx, dout: torch.Tensor):
        y, gate = ctx.saved_tensors
        dY, dgate = B.moe_combine_bwd(ctx.handle, _rows(dout), gate, y)
        return dY, dgate, None


def dispatch(x: torch.Tensor, handle: B.Handle) -> torch.Tensor:
    return MoEDispatchFn.apply(_rows(x), handle)


def combine(y: torch.Tensor, gate: torch.Tensor, handle: B.Handle) -> torch.Tensor:
    return MoECombineFn.apply(_rows(y), _rows(gate), handle)


class LayerNormFn(torch.autograd.Function):
    """y = layernorm(x) weight + bias; the weight gradients are summed in fp32 and rounded once to their type."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight, bias, eps: float):
        y, mean, rstd = B.moe_layernorm(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @first_order
    def backward(ctx, dy: torch.Tensor):
        x, weight, mean, rstd = ctx.saved_tensors
        _, need_w, need_b, _ = ctx.needs_input_grad
        dx, dw, db = B.moe_layernorm_bwd(_rows(dy), x, weight, mean, rstd, need_dweight=need_w, need_dbias=need_b)
        return dx, dw if dw is None else dw.to(weight.dtype), db if db is None else db.to(ctx.bias_dtype), None


def layernorm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
              eps: float = 1e-5) -> torch.Tensor:
    """Layer norm of [s, m] rows."""
    return LayerNormFn.apply(_strided(x), _rows(weight), _rows(bias), eps)


class LinearFn(torch.autograd.Function):
    """y = act(x W^T + bias) + residual; z is kept (bf16) where the activation's slope needs it.  grad: whether a
    gradient can be asked for at all (needs_input_grad stays true for parameters under no_grad)."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, W: torch.Tensor, bias, residual, act: str, out_dtype, grad: bool):
        save_z = grad and act != "none" and any(ctx.needs_input_grad[:3])
        out = B.moe_linear(x, W, bias, act, residual, out_dtype=out_dtype, save_z=save_z, device_status=_status(x))
        y, z = out if save_z else (out, None)
        ctx.save_for_backward(x, W, z)
        ctx.act = act
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.residual_dtype = None if residual is None else residual.dtype
        return y

    @staticmethod
    @first_order
    def products(ctx, dy: torch.Tensor):
        x, W, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        if not any(need[:3]):
            return None, None, None
        dx, dW, db = B.moe_linear_bwd(_rows(dy), x, W, z, ctx.act, need[0], need[1], need[2], device_status=_status(x))
        return dx, dW, db if db is None else db.to(ctx.bias_dtype)

    @staticmethod
    def backward(ctx, dy: torch.Tensor):
        # the residual's gradient is dy itself, which may be differentiated
        dres = dy.to(ctx.residual_dtype) if ctx.needs_input_grad[3] else None
        return (*LinearFn.products(ctx, dy), dres, None, None, None)


def linear(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
           residual: torch.Tensor | None = None, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """y [s, N] = act(x W^T + bias) + residual, bf16 (or fp32) out."""
    return LinearFn.apply(_strided(x, 8), _strided(W, 8), _rows(bias), _strided(residual), act, out_dtype,
                          torch.is_grad_enabled())


class BalanceLossFn(torch.autograd.Function):
    """loss [2] (balance, z) of the router's logits, with the counts held fixed in the gradient."""

    @staticmethod
    def forward(ctx, logits: torch.Tensor, topk_idx: torch.Tensor, valid, seq_offsets):
        r = B.moe_balance_loss(logits, topk_idx, valid, seq_offsets, device_status=_status(logits))
        ctx.save_for_backward(logits, r.lse, r.coef, r.norm, valid, seq_offsets)
        ctx.mark_non_differentiable(r.counts, r.mean_prob)
        return r.loss, r.counts, r.mean_prob

    @staticmethod
    @first_order
    def backward(ctx, dloss: torch.Tensor, dcounts, dmean_prob):
        logits, lse, coef, norm, valid, seq_offsets = ctx.saved_tensors
        d = B.moe_balance_loss_bwd(logits, lse, coef, norm, dloss.contiguous(), valid, seq_offsets)
        return d, None, None, None


def balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, valid: torch.Tensor | None = None,
                 seq_offsets: torch.Tensor | None = None):
    """(loss f32 [2]: the balance loss and the z loss, counts i32 [num_seqs, e], mean_prob f32 [num_seqs, e])."""
    return BalanceLossFn.apply(_rows(logits), _rows(topk_idx), _rows(valid), _rows(seq_offsets))


class HandleRecorder:
    """Per-checkpointed-call log of layout handles.

    ``layout(topk_idx, ...)`` builds a fresh layout while recording (the
    forward) and appends it to the log; once ``replay()`` is entered (the
    recompute) it returns the logged handles in call order without
    launching the layout kernel.  A replay past the end of the log builds a
    fresh layout (``fallbacks`` counts those).  ``build`` is the layout
    constructor, injectable so the bookkeeping can be tested without a GPU.
    """

    def __init__(self, build=None, verify: bool = False):
        self._build = build or _build_layout
        self._log: deque = deque()
        self._replaying = False
        self.verify = verify
        self.recorded = 0
        self.replayed = 0
        self.fallbacks = 0

    def replay(self):
        """Switch to replay mode (the recompute of the checkpointed call)."""
        self._replaying = True
        return self

    def record(self):
        self._replaying = False
        self._log.clear()
        return self

    def __len__(self):
        return len(self._log)

    def layout(self, topk_idx: torch.Tensor, e: int, capacity: int = 0, num_virtual_ranks: int = 0,
               priority: str = "token", pad_multiple: int = 1, send_slots: bool = False):
        """The layout of ``topk_idx`` (options as ``moe_dispatch_layout_ex``):
        built and logged while recording, the logged handle while replaying."""
        opts = {}
        if priority != "token" or pad_multiple != 1 or send_slots:
            opts = dict(priority=priority, pad_multiple=int(pad_multiple), send_slots=bool(send_slots))
        key = (tuple(topk_idx.shape), int(e), int(capacity), int(num_virtual_ranks), tuple(sorted(opts.items())))
        if not self._replaying:
            h = self._build(topk_idx, e, capacity, num_virtual_ranks, **opts)
            # routing metadata: the expert ids; the dispatched activation is not kept
            self._log.append((key, h, topk_idx.detach() if self.verify else None))
            self.recorded += 1
            return h
        if self._log:
            k0, h, logged_idx = self._log.popleft()
            if k0 == key and (logged_idx is None or torch.equal(logged_idx, topk_idx)):
                self.replayed += 1
                return h
        # outran the log, or the call does not match what was logged: build afresh
        self.fallbacks += 1
        return self._build(topk_idx, e, capacity, num_virtual_ranks, **opts)


def _build_layout(topk_idx, e, capacity, num_virtual_ranks, priority="token", pad_multiple=1, send_slots=False):
    """Plain layouts through moe_dispatch_layout, variants through _ex."""
    if priority == "token" and pad_multiple == 1 and not send_slots:
        return B.moe_dispatch_layout(topk_idx, e, capacity, num_virtual_ranks)
    return B.moe_dispatch_layout_ex(topk_idx, e, capacity, num_virtual_ranks, priority, pad_multiple, send_slots)
