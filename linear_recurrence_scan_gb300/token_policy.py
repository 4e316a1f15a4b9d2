"""A recurrent token policy's other operators for PyTorch tensors: the gated
recurrence (one state a channel), the gated feed-forward block's projections,
and the loss that distils a teacher's top logits into the policy.

They follow the state-space layer's functions (``state_space.py``): arguments
are checked, outputs allocated with torch, one librlscan call is made on the
current CUDA stream of the tensors' device, without synchronising; there is no
CPU path.  What has gradients has them once, in reverse mode; the
``*_backward`` functions are the same gradients as plain calls; dual tensors
are refused.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from . import _native
from .api import _stream_handle
from .state_space import (_ARRAY3, _TYPES, _act, _at, _changed, _check, _dense, _flags, _lead, _load_fast, _on,
                          _refuse_tangents, _scratch, _wants_grad)

__all__ = [
    "gated_scan", "gated_scan_backward", "gated_scan_step", "GatedScanGrads",
    "gated_projection", "gated_projection_backward", "GatedProjectionGrads",
    "distill_loss", "distill_loss_backward", "distill_loss_and_grad",
]

GATED_CHECKPOINT = 32   # tokens between two checkpoints of the gated scan (RLSCAN_GATED_SCAN_CHECKPOINT)

_GATED_ARGS = struct.Struct("=17q")
_GATED_GRADS = struct.Struct("=5q")
_PROJECTION_ARGS = struct.Struct("=10q")
_ACTIVATIONS = {"silu": 0, "gelu": 1}
_DISTILL_ARGS = struct.Struct("=13qd")

MAX_TEACHER_TOKENS = 256   # RLSCAN_DISTILL_MOST


_fast = None


def _load():
    """The native call layer (csrc_sequence/fastcall.c), or one that leaves all to Python."""
    global _fast
    if _fast is None:
        fast = _load_fast()
        lib = _native.lib()
        fast.setup_token_policy(torch, GatedScanGrads, GatedProjectionGrads, *(
            ctypes.cast(getattr(lib, "rlscan_" + name), ctypes.c_void_p).value for name in (
                "gated_scan", "gated_scan_backward_workspace_bytes", "gated_scan_backward", "gated_scan_step",
                "gated_projection_workspace_bytes", "gated_projection", "gated_projection_backward_workspace_bytes",
                "gated_projection_backward", "distill_loss", "distill_loss_and_grad")))
        _fast = fast
    return _fast


# ---------------------------------------------------------------------------
# gated scan

class GatedScanGrads(NamedTuple):
    """Gradients of gated_scan's inputs."""
    x: torch.Tensor
    gate: torch.Tensor
    input_gate: torch.Tensor
    log_decay: torch.Tensor
    initial_state: torch.Tensor


def _gated_args(step, x, gate, input_gate, log_decay, initial_state, resets, lengths):
    """Checks; (device, (N, T, channels), the packed arguments, the tensors they point at)."""
    dev = _lead("x", x, 2 if step else 3)
    dtype, shape = x.dtype, x.shape
    N, T, width = (shape[0], 1, shape[1]) if step else shape
    xp, xr, xt, x = _act("x", x, shape, dtype, dev)
    gp, gr, gt, gate = _act("gate", gate, shape, dtype, dev)
    ip, ir, it, input_gate = _act("input_gate", input_gate, shape, dtype, dev)
    if log_decay is None:
        raise TypeError("log_decay must be a torch.Tensor")
    log_decay = _dense("log_decay", log_decay, (width,), torch.float32, dev)
    initial_state = _dense("initial_state", initial_state, (N, width), torch.float32, dev)
    resets = _flags(resets, (N, T), dev)
    lengths = _dense("lengths", lengths, (N,), torch.int32, dev)
    packed = _GATED_ARGS.pack(N, T, width, _TYPES[dtype], xp, xr, xt, gp, gr, gt, ip, ir, it, log_decay.data_ptr(),
                              _at(initial_state), _at(resets), _at(lengths))
    return dev, (N, T, width), packed, (x, gate, input_gate, log_decay, initial_state, resets, lengths)


def _gated_forward(want_checkpoints, *args):
    dev, (N, T, width), packed, kept = _gated_args(False, *args)
    x = kept[0]
    f32 = dict(dtype=torch.float32, device=x.device)
    y = torch.empty((N, T, width), dtype=x.dtype, device=x.device)
    final = torch.empty((N, width), **f32)
    marks = torch.empty((N, -(-T // GATED_CHECKPOINT), width), **f32) if want_checkpoints else None
    with _on(dev):
        _native.check(_native.lib().rlscan_gated_scan(packed, y.data_ptr(), final.data_ptr(), _at(marks),
                                                      _stream_handle(x.device)), "rlscan_gated_scan")
    return y, final, marks


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, input_gate, log_decay, initial_state, resets, lengths):
        y, final, marks = _gated_forward(True, x, gate, input_gate, log_decay, initial_state, resets, lengths)
        ctx.started = initial_state is not None
        ctx.save_for_backward(x, gate, input_gate, log_decay, resets, lengths, marks)
        ctx.mark_non_differentiable(marks)
        ctx.set_materialize_grads(False)
        return y, final, marks

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_final, _):
        x, gate, input_gate, log_decay, resets, lengths, marks = ctx.saved_tensors
        if grad_y is None:
            if grad_final is None:
                return (None,) * 7
            grad_y = torch.zeros_like(x)
        g = gated_scan_backward(grad_y, x, gate, input_gate, log_decay, marks, resets, lengths, grad_final)
        return g.x, g.gate, g.input_gate, g.log_decay, g.initial_state if ctx.started else None, None, None


def gated_scan(x, gate, input_gate, log_decay, initial_state=None, resets=None, lengths=None,
               return_checkpoints=False):
    """The gated linear recurrence over prompts, for every channel

        r_t = sigmoid(gate_t),  i_t = sigmoid(input_gate_t),  a_t = exp(log_decay r_t)
        y_t = h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,    h_{-1} = initial_state

    x, gate and input_gate [N,T,channels] are float32 or bfloat16 (one type,
    any strides over rows and tokens); log_decay [channels], below 0, and
    initial_state [N,channels] float32.  ``resets`` and ``lengths`` as in
    selective_scan (at a reset h_{t-1} counts 0, the input keeps its root).
    Returns (y, final_state): y like x, the states [N,channels] float32 after
    each row's last token.  With ``return_checkpoints`` a third value, what
    gated_scan_backward needs: the states before every 32nd token (these
    carry no gradient)."""
    args = (x, gate, input_gate, log_decay, initial_state, resets, lengths)
    out = (_fast or _load()).gated_scan(*args, return_checkpoints)
    if out is not None:
        return out
    _refuse_tangents(*args[:5])
    out = _GatedScan.apply(*args) if _wants_grad(*args[:5]) else _gated_forward(return_checkpoints, *args)
    return out if return_checkpoints else out[:2]


def gated_scan_backward(grad_y, x, gate, input_gate, log_decay, checkpoints, resets=None, lengths=None,
                        grad_final_state=None):
    """Gradients of gated_scan: ``grad_y`` like x, ``checkpoints`` from the
    forward call on the same inputs, ``grad_final_state`` [N,channels] float32
    or None.  Returns GatedScanGrads."""
    g = (_fast or _load()).gated_scan_backward(grad_y, x, gate, input_gate, log_decay, checkpoints, resets, lengths,
                                               grad_final_state)
    if g is not None:
        return g
    _refuse_tangents(grad_y, x, gate, input_gate, log_decay, checkpoints, grad_final_state)
    dev, (N, T, width), packed, kept = _gated_args(False, x, gate, input_gate, log_decay, None, resets, lengths)
    x = kept[0]
    gp, gr, gt, grad_y = _act("grad_y", grad_y, x.shape, x.dtype, dev)
    if checkpoints is None:
        raise ValueError("checkpoints is required (gated_scan(..., return_checkpoints=True))")
    marks = _dense("checkpoints", checkpoints, (N, -(-T // GATED_CHECKPOINT), width), torch.float32, dev)
    gfinal = _dense("grad_final_state", grad_final_state, (N, width), torch.float32, dev)
    acts, f32 = dict(dtype=x.dtype, device=x.device), dict(dtype=torch.float32, device=x.device)
    g = GatedScanGrads(x=torch.empty((N, T, width), **acts), gate=torch.empty((N, T, width), **acts),
                       input_gate=torch.empty((N, T, width), **acts), log_decay=torch.empty((width,), **f32),
                       initial_state=torch.empty((N, width), **f32))
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_gated_scan_backward_workspace_bytes(packed), x.device)
        _native.check(lib.rlscan_gated_scan_backward(
            packed, _ARRAY3.pack(gp, gr, gt), _at(gfinal), marks.data_ptr(),
            _GATED_GRADS.pack(g.x.data_ptr(), g.gate.data_ptr(), g.input_gate.data_ptr(), g.log_decay.data_ptr(),
                              g.initial_state.data_ptr()),
            _at(ws), 0 if ws is None else ws.numel(), _stream_handle(x.device)), "rlscan_gated_scan_backward")
    return g


def gated_scan_step(state, x, gate, input_gate, log_decay, slots=None):
    """One token of each of N sequences: x, gate, input_gate [N,channels];
    ``state`` [P,channels] float32 (dense) is updated in place, with ``slots``
    as in selective_scan_step.  Returns y [N,channels].  Not differentiable."""
    y = (_fast or _load()).gated_scan_step(state, x, gate, input_gate, log_decay, slots)
    if y is not None:
        return y
    _refuse_tangents(state, x, gate, input_gate, log_decay)
    dev, (N, _, width), packed, kept = _gated_args(True, x, gate, input_gate, log_decay, None, None, None)
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be a [slots, channels] tensor")
    P = state.shape[0]
    _check("state", state, (P, width), torch.float32, dev)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous: it is updated in place")
    slots = _dense("slots", slots, (N,), torch.int32, dev)
    if slots is None and P < N:
        raise ValueError(f"state holds {P} slots for {N} sequences")
    x = kept[0]
    y = torch.empty((N, width), dtype=x.dtype, device=x.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_gated_scan_step(packed, state.data_ptr(), P, _at(slots), y.data_ptr(),
                                                           _stream_handle(x.device)), "rlscan_gated_scan_step")
    _changed(state)
    return y


# ---------------------------------------------------------------------------
# gated feed-forward block

class GatedProjectionGrads(NamedTuple):
    """Gradients of gated_projection's inputs."""
    x: torch.Tensor
    gate_weight: torch.Tensor
    up_weight: torch.Tensor


def _matrix(name, t, shape, device):
    """(tensor, address, row stride) of a bfloat16 [..., columns] array as rows."""
    _check(name, t, shape, torch.bfloat16, device)
    if len(shape) != 2:
        t = t.reshape(t.numel() // max(shape[-1], 1), shape[-1])
    if t.stride(1) != 1 and t.shape[1] > 1:
        t = t.contiguous()
    return t, t.data_ptr(), t.stride(0)


def _projection_args(x, gate_weight, up_weight, activation):
    """Checks; (device, the packed arguments, (x, both weights) as rows)."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be a [..., values] tensor of at least 2 dimensions")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or 'gelu', got {activation!r}")
    dev = _lead("x", x, x.dim())
    D = x.shape[-1]
    if not isinstance(gate_weight, torch.Tensor) or gate_weight.dim() != 2:
        raise ValueError("gate_weight must be a [features, values] tensor")
    F = gate_weight.shape[0]
    if D == 0:
        raise ValueError("x must have values")
    x, xp, xs = _matrix("x", x, x.shape, dev)
    gate_weight, gp, gs = _matrix("gate_weight", gate_weight, (F, D), dev)
    up_weight, up, us = _matrix("up_weight", up_weight, (F, D), dev)
    packed = _PROJECTION_ARGS.pack(x.shape[0], D, F, _ACTIVATIONS[activation], xp, xs, gp, gs, up, us)
    return dev, packed, (x, gate_weight, up_weight)


def _projection_forward(x, gate_weight, up_weight, activation):
    dev, packed, (rows, gate, up) = _projection_args(x, gate_weight, up_weight, activation)
    h = torch.empty((*x.shape[:-1], gate.shape[0]), dtype=x.dtype, device=x.device)
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_gated_projection_workspace_bytes(packed), x.device)
        _native.check(lib.rlscan_gated_projection(packed, h.data_ptr(), _at(ws), 0 if ws is None else ws.numel(),
                                                  _stream_handle(x.device)), "rlscan_gated_projection")
    return h


class _GatedProjection(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate_weight, up_weight, activation):
        ctx.activation = activation
        ctx.save_for_backward(x, gate_weight, up_weight)
        ctx.set_materialize_grads(False)
        return _projection_forward(x, gate_weight, up_weight, activation)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_h):
        if grad_h is None:
            return None, None, None, None
        x, gate_weight, up_weight = ctx.saved_tensors
        g = _projection_backward(grad_h, x, gate_weight, up_weight, ctx.activation, ctx.needs_input_grad[0],
                                 ctx.needs_input_grad[1] or ctx.needs_input_grad[2])
        return (*g, None)


def gated_projection(x, gate_weight, up_weight, activation="silu"):
    """The gated feed-forward block's projections, activation and product:

        z = x gate_weight^T,  u = x up_weight^T,  h = act(z) * u

    x [..., D] and both weights [F, D] are bfloat16 (rows of any stride:
    halves of one [2F, D] weight are taken as they are); the sums, z and u are
    float32, h [..., F] is rounded once.  ``activation`` is "silu" or "gelu"
    (z times the normal distribution up to z).  float32 is refused: the tensor
    cores would round its factors to 11 bits."""
    h = (_fast or _load()).gated_projection(x, gate_weight, up_weight, activation)
    if h is not None:
        return h
    _refuse_tangents(x, gate_weight, up_weight)
    if _wants_grad(x, gate_weight, up_weight):
        return _GatedProjection.apply(x, gate_weight, up_weight, activation)
    return _projection_forward(x, gate_weight, up_weight, activation)


def _projection_backward(grad_h, x, gate_weight, up_weight, activation, want_x, want_weights):
    shape = x.shape
    dev, packed, (rows, gate, up) = _projection_args(x, gate_weight, up_weight, activation)
    grad_h, ghp, ghs = _matrix("grad_h", grad_h, (*shape[:-1], gate.shape[0]), dev)

    def like(size, wanted):
        return torch.empty(size, dtype=x.dtype, device=x.device) if wanted else None

    g = GatedProjectionGrads(like(shape, want_x), like(gate.shape, want_weights), like(gate.shape, want_weights))
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_gated_projection_backward_workspace_bytes(packed), x.device)
        _native.check(lib.rlscan_gated_projection_backward(
            packed, ghp, ghs, _at(g.x), _at(g.gate_weight), _at(g.up_weight), _at(ws),
            0 if ws is None else ws.numel(), _stream_handle(x.device)), "rlscan_gated_projection_backward")
    return g


def gated_projection_backward(grad_h, x, gate_weight, up_weight, activation="silu"):
    """Gradients of gated_projection: ``grad_h`` [..., F] bfloat16.  z and u
    are made again from x, in 32 bits; the gradients at z and u are rounded to
    bfloat16 for the products that follow.  Returns GatedProjectionGrads."""
    g = (_fast or _load()).gated_projection_backward(grad_h, x, gate_weight, up_weight, activation)
    if g is not None:
        return g
    _refuse_tangents(grad_h, x, gate_weight, up_weight)
    return _projection_backward(grad_h, x, gate_weight, up_weight, activation, True, True)


# ---------------------------------------------------------------------------
# distillation from a teacher's top logits

def _distill_args(logits, teacher_logits, teacher_tokens, temperature, mask):
    """Checks; (device, the packed arguments, the tensors they point at)."""
    dev = _lead("logits", logits, 3)
    N, T, V = logits.shape
    if V == 0:
        raise ValueError("logits must have a vocabulary")
    if not isinstance(teacher_logits, torch.Tensor) or teacher_logits.dim() != 3:
        raise ValueError("teacher_logits must be a [N, T, K] tensor")
    K = teacher_logits.shape[2]
    if not 1 <= K <= MAX_TEACHER_TOKENS:
        raise ValueError(f"teacher_logits has {K} tokens: 1 to {MAX_TEACHER_TOKENS} are supported")
    if teacher_logits.dtype not in _TYPES:
        raise TypeError(f"teacher_logits: expected torch.float32 or torch.bfloat16, got {teacher_logits.dtype}")
    if not isinstance(teacher_tokens, torch.Tensor) or teacher_tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError("teacher_tokens must be an int32 or int64 tensor")
    if not 1e-6 <= temperature <= 1e6:
        raise ValueError("temperature must be between 1e-6 and 1e6")
    lp, lr, lt, logits = _act("logits", logits, logits.shape, logits.dtype, dev)
    teacher_logits = _dense("teacher_logits", teacher_logits, (N, T, K), teacher_logits.dtype, dev)
    teacher_tokens = _dense("teacher_tokens", teacher_tokens, (N, T, K), teacher_tokens.dtype, dev)
    if isinstance(mask, torch.Tensor) and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    mask = _dense("mask", mask, (N, T), torch.uint8, dev)
    packed = _DISTILL_ARGS.pack(N, T, V, K, _TYPES[logits.dtype], _TYPES[teacher_logits.dtype],
                                teacher_tokens.element_size(), lp, lr, lt, teacher_logits.data_ptr(),
                                teacher_tokens.data_ptr(), _at(mask), temperature)
    return dev, packed, (logits, teacher_logits, teacher_tokens, mask)


def _distill_forward(want_normalizers, *args):
    dev, packed, kept = _distill_args(*args)
    logits = kept[0]
    loss = torch.empty(logits.shape[:2], dtype=torch.float32, device=logits.device)
    norm = torch.empty((*logits.shape[:2], 2), dtype=torch.float32, device=logits.device) if want_normalizers else None
    with _on(dev):
        _native.check(_native.lib().rlscan_distill_loss(packed, loss.data_ptr(), _at(norm),
                                                        _stream_handle(logits.device)), "rlscan_distill_loss")
    return loss, norm


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_logits, teacher_tokens, temperature, mask):
        loss, norm = _distill_forward(True, logits, teacher_logits, teacher_tokens, temperature, mask)
        ctx.temperature = temperature
        ctx.save_for_backward(logits, teacher_logits, teacher_tokens, mask, norm)
        ctx.mark_non_differentiable(norm)
        ctx.set_materialize_grads(False)
        return loss, norm

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, _):
        if grad_loss is None:
            return (None,) * 5
        logits, teacher_logits, teacher_tokens, mask, norm = ctx.saved_tensors
        return (distill_loss_backward(grad_loss, logits, teacher_logits, teacher_tokens, norm, ctx.temperature, mask),
                None, None, None, None)


def distill_loss(logits, teacher_logits, teacher_tokens, temperature=1.0, mask=None, return_normalizers=False):
    """The divergence of a student's tokens from a teacher's top logits:

        q = softmax(teacher_logits / temperature) over the teacher's K tokens
        p = softmax(logits / temperature) over the vocabulary
        loss = sum_k q_k (log q_k - log p_k)

    logits [N,T,vocabulary] float32 or bfloat16 (any strides over rows and
    tokens); teacher_logits [N,T,K] float32 or bfloat16 and teacher_tokens
    [N,T,K] int32 or int64, K up to 256 (a token outside the vocabulary, -1
    say, is an empty place; one that comes twice counts twice); ``temperature``
    1e-6 to 1e6; ``mask`` [N,T] (uint8 or bool) is 0 where a token has no loss,
    and its logits are not read.  Returns the loss [N,T] float32, 0 where nothing is left to learn
    from; with ``return_normalizers`` also what distill_loss_backward needs,
    [N,T,2] float32.  Differentiable in the logits; the teacher has no
    gradient (one that requires it is refused).  The factor temperature^2
    that some recipes have is left to the caller."""
    if not return_normalizers:
        loss = (_fast or _load()).distill_loss(logits, teacher_logits, teacher_tokens, temperature, mask)
        if loss is not None:
            return loss
    _refuse_tangents(logits, teacher_logits)
    args = (logits, teacher_logits, teacher_tokens, temperature, mask)
    if _wants_grad(teacher_logits):
        raise ValueError("teacher_logits must not require a gradient: detach the teacher")
    out = _DistillLoss.apply(*args) if _wants_grad(logits) else _distill_forward(return_normalizers, *args)
    return out if return_normalizers else out[0]


def _grad_loss(grad_loss, logits, device):
    if grad_loss is None:
        raise TypeError("grad_loss must be a torch.Tensor")
    return _dense("grad_loss", grad_loss, logits.shape[:2], torch.float32, device)


def distill_loss_backward(grad_loss, logits, teacher_logits, teacher_tokens, normalizers, temperature=1.0, mask=None):
    """The gradient of distill_loss in the logits (dense, of their type):
    ``grad_loss`` [N,T] float32, ``normalizers`` from the forward call on the
    same inputs."""
    _refuse_tangents(grad_loss, logits, teacher_logits)
    dev, packed, kept = _distill_args(logits, teacher_logits, teacher_tokens, temperature, mask)
    logits = kept[0]
    grad_loss = _grad_loss(grad_loss, logits, dev)
    if normalizers is None:
        raise ValueError("normalizers is required (distill_loss(..., return_normalizers=True))")
    norm = _dense("normalizers", normalizers, (*logits.shape[:2], 2), torch.float32, dev)
    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_distill_loss_backward(
            packed, grad_loss.data_ptr(), norm.data_ptr(), grad.data_ptr(), _stream_handle(logits.device)),
            "rlscan_distill_loss_backward")
    return grad


def distill_loss_and_grad(grad_loss, logits, teacher_logits, teacher_tokens, temperature=1.0, mask=None):
    """(loss, gradient in the logits) in one call, for a training step that
    knows each token's weight ``grad_loss`` [N,T] float32 before its loss (a
    mask over the number of tokens, say): the logits are read once.  Not
    followed by autograd."""
    out = (_fast or _load()).distill_loss_and_grad(grad_loss, logits, teacher_logits, teacher_tokens, temperature, mask)
    if out is not None:
        return out
    _refuse_tangents(grad_loss, logits, teacher_logits)
    dev, packed, kept = _distill_args(logits, teacher_logits, teacher_tokens, temperature, mask)
    logits = kept[0]
    grad_loss = _grad_loss(grad_loss, logits, dev)
    f32 = dict(dtype=torch.float32, device=logits.device)
    loss, norm = torch.empty(logits.shape[:2], **f32), torch.empty((*logits.shape[:2], 2), **f32)
    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_distill_loss_and_grad(
            packed, grad_loss.data_ptr(), loss.data_ptr(), norm.data_ptr(), grad.data_ptr(),
            _stream_handle(logits.device)), "rlscan_distill_loss_and_grad")
    return loss, grad
