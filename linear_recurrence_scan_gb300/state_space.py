"""The state-space layer for PyTorch tensors: the selective scan, the short
causal convolution in front of it and the root-mean-square norm in front of
the layer, over prompts, in training and for single tokens.

Like the estimators, each function checks its arguments, allocates the
outputs with torch and makes one librlscan call on the current CUDA stream
of the tensors' device, without synchronising; there is no CPU path.  Unlike the estimators, tensors
live on the GPU, activations are token-major ([N, T, width], any strides over
rows and tokens) and float32 or bfloat16, and parameters and recurrent states
of the scan are float32.

``selective_scan``, ``causal_conv`` and ``add_rms_norm`` are differentiable
when an input requires a gradient (once; the gradients themselves are not);
the ``*_backward`` functions are the same gradients as plain calls.  Nothing
here has a forward-mode derivative: dual tensors are refused.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import os
import struct
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad as _forward_ad

from . import _native
from .api import _raw_stream, _stream_handle

__all__ = [
    "selective_scan", "selective_scan_backward", "selective_scan_step", "SelectiveScanGrads",
    "causal_conv", "causal_conv_backward", "causal_conv_step", "CausalConvGrads",
    "add_rms_norm", "add_rms_norm_backward", "RmsNorm", "RmsNormGrads",
]

CHECKPOINT = 16   # tokens between two checkpoints of the scan (RLSCAN_SELECTIVE_SCAN_CHECKPOINT)
MAX_STATES = 128
MAX_TAPS = 8
SCALE_BLOCK = 128  # columns that share one scale of an 8-bit output

_changed = torch.autograd.graph.increment_version   # what a graph saved of a state is then known to be stale
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_HERE = contextlib.nullcontext()
_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_SCAN_ARGS = struct.Struct("=27q")
_SCAN_GRADS = struct.Struct("=9q")
_CONV_ARGS = struct.Struct("=14q")
_ARRAY3 = struct.Struct("=3q")


# ---------------------------------------------------------------------------
# calls in the usual form (csrc_sequence/fastcall.c), where it has been built

class _NoFastCall:
    """Leaves every call to the Python way."""

    @staticmethod
    def _none(*args):
        return None

    selective_scan = selective_scan_step = causal_conv = causal_conv_step = add_rms_norm = _none


_fast = None


def _load_fast():
    """The native call layer, or one that leaves all to Python."""
    global _fast
    if _fast is None:
        path = os.path.join(_native.HERE, "_build", "_fastcall" + importlib.machinery.EXTENSION_SUFFIXES[0])
        if not os.path.exists(path) or _raw_stream is None:
            _fast = _NoFastCall
        else:
            spec = importlib.util.spec_from_file_location("_fastcall", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _setup(module)
            _fast = module
    return _fast


def _setup(module):
    module.setup(torch, RmsNorm, _raw_stream, _current_device, _forward_ad, _changed, *(
        ctypes.cast(getattr(_native.lib(), "rlscan_" + name), ctypes.c_void_p).value for name in (
            "selective_scan_workspace_bytes", "selective_scan", "selective_scan_step", "causal_conv",
            "causal_conv_step", "add_rms_norm")))


# ---------------------------------------------------------------------------
# argument checks

def _fail_type(name, t, dtypes):
    raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


def _check(name, t, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on CUDA")
    if t.dtype != dtype:
        _fail_type(name, t, (dtype,))
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _lead(name, t, dims):
    """The tensor the others are measured by: a CUDA activation of `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on CUDA")
    if t.dtype not in _TYPES:
        _fail_type(name, t, tuple(_TYPES))
    return t.get_device()


# The checks of every call cost as much as a small kernel, so the usual case
# asks a tensor for no more than what decides: its type, shape and device (-1
# for a CPU tensor).  Whatever is out of order goes through _check, which
# says what.

def _act(name, t, shape, dtype, device):
    """(address, row stride, token stride, tensor) of an activation: any strides
    over rows and tokens, element stride 1."""
    try:
        fits = t.dtype is dtype and t.shape == shape and t.get_device() == device
    except AttributeError:
        fits = False
    if not fits:
        _check(name, t, shape, dtype, device)
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        t = t.contiguous()
        strides = t.stride()
    return t.data_ptr(), strides[0], (strides[1] if len(strides) == 3 else 0), t


def _dense(name, t, shape, dtype, device):
    """A dense array or None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t
    except AttributeError:
        pass
    _check(name, t, shape, dtype, device)
    return t if t.is_contiguous() else t.contiguous()


def _flags(resets, shape, device):
    if resets is None:
        return None
    if isinstance(resets, torch.Tensor) and resets.dtype == torch.bool:
        resets = resets.view(torch.uint8)
    return _dense("resets", resets, shape, torch.uint8, device)


def _at(t):
    return 0 if t is None else t.data_ptr()


_NONE = (0, 0, 0, None)


def _wants_grad(*ts):
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and getattr(t, "requires_grad", False):
                return True
    return False


def _refuse_tangents(*ts):
    """These functions have no forward-mode derivative: dual tensors, which
    live inside a dual level only, would lose their tangents."""
    if _forward_ad._current_level >= 0:
        for t in ts:
            if isinstance(t, torch.Tensor) and _forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError("the state-space layer's functions have no forward-mode derivative")


def _on(device):
    """Plans, workspace sizes and launches are the current device's: makes it the tensors' own."""
    return _HERE if _current_device() == device else torch.cuda.device(device)


def _scratch(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


# ---------------------------------------------------------------------------
# selective scan

class SelectiveScanGrads(NamedTuple):
    """Gradients of selective_scan's inputs (None where the input was not given)."""
    x: torch.Tensor
    delta: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    C: torch.Tensor
    D: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    delta_bias: Optional[torch.Tensor]
    initial_state: torch.Tensor


def _scan_args(step, x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, resets, lengths):
    """Checks; (device, (N, T, channels, S), the packed arguments, the tensors they point at)."""
    dev = _lead("x", x, 2 if step else 3)
    dtype, shape = x.dtype, x.shape
    N, T, width = (shape[0], 1, shape[1]) if step else shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [channels, states] tensor")
    S = A.shape[1]
    if not 1 <= S <= MAX_STATES:
        raise ValueError(f"A has {S} states: 1 to {MAX_STATES} are supported")
    f32 = torch.float32
    A = _dense("A", A, (width, S), f32, dev)
    bc = (N, S) if step else (N, T, S)
    xp, xr, xt, x = _act("x", x, shape, dtype, dev)
    dp, dr, dt, delta = _act("delta", delta, shape, dtype, dev)
    Bp, Br, Bt, B = _act("B", B, bc, dtype, dev)
    Cp, Cr, Ct, C = _act("C", C, bc, dtype, dev)
    zp, zr, zt, z = _NONE if z is None else _act("z", z, shape, dtype, dev)
    D = _dense("D", D, (width,), f32, dev)
    delta_bias = _dense("delta_bias", delta_bias, (width,), f32, dev)
    if initial_state is not None:
        initial_state = _dense("initial_state", initial_state, (N, width, S), f32, dev)
    if resets is not None:
        resets = _flags(resets, (N, T), dev)
    if lengths is not None:
        lengths = _dense("lengths", lengths, (N,), torch.int32, dev)
    kept = (x, delta, z, B, C, A, D, delta_bias, initial_state, resets, lengths)
    packed = _SCAN_ARGS.pack(N, T, width, S, _TYPES[dtype], 1 if delta_softplus else 0, xp, xr, xt, dp, dr, dt, zp, zr,
                             zt, Bp, Br, Bt, Cp, Cr, Ct, A.data_ptr(), _at(D), _at(delta_bias), _at(initial_state),
                             _at(resets), _at(lengths))
    return dev, (N, T, width, S), packed, kept


def _scan_forward(want_checkpoints, *args):
    dev, (N, T, width, S), packed, kept = _scan_args(False, *args)
    x = kept[0]
    f32 = dict(dtype=torch.float32, device=x.device)
    y = torch.empty((N, T, width), dtype=x.dtype, device=x.device)
    final = torch.empty((N, width, S), **f32)
    marks = torch.empty((N, -(-T // CHECKPOINT), width, S), **f32) if want_checkpoints else None
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_selective_scan_workspace_bytes(packed), x.device)
        _native.check(lib.rlscan_selective_scan(packed, y.data_ptr(), final.data_ptr(), _at(marks), _at(ws),
                                                0 if ws is None else ws.numel(), _stream_handle(x.device)),
                      "rlscan_selective_scan")
    return y, final, marks


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, resets, lengths):
        y, final, marks = _scan_forward(True, x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state,
                                        resets, lengths)
        ctx.delta_softplus, ctx.started = delta_softplus, initial_state is not None
        ctx.save_for_backward(x, delta, A, B, C, D, z, delta_bias, resets, lengths, marks)
        ctx.mark_non_differentiable(marks)
        ctx.set_materialize_grads(False)
        return y, final, marks

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_final, _):
        x, delta, A, B, C, D, z, delta_bias, resets, lengths, marks = ctx.saved_tensors
        if grad_y is None:
            if grad_final is None:
                return (None,) * 12
            grad_y = torch.zeros_like(x)
        g = selective_scan_backward(grad_y, x, delta, A, B, C, marks, D, z, delta_bias, ctx.delta_softplus, resets,
                                    lengths, grad_final)
        return (g.x, g.delta, g.A, g.B, g.C, g.D, g.z, g.delta_bias, None,
                g.initial_state if ctx.started else None, None, None)


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True, initial_state=None,
                   resets=None, lengths=None, return_checkpoints=False):
    """The selective scan over prompts: for every channel d and state s

        dt_t = softplus(delta_t + delta_bias)     (delta_softplus=False: without softplus)
        h_t  = exp(dt_t A) h_{t-1} + dt_t x_t B_t,    h_{-1} = initial_state
        y_t  = (sum_s C_t h_t + D x_t) * silu(z_t)

    x, delta, z [N,T,channels] and B, C [N,T,S] are float32 or bfloat16 (one
    type, any strides); A [channels,S], D and delta_bias [channels] and
    initial_state [N,channels,S] float32.  ``resets`` [N,T] (uint8 or bool)
    is non-zero where an episode starts (nothing from before it reaches it);
    ``lengths`` [N] int32 is the number of tokens of each row, the rest is
    padding (not read, y = 0).  Returns (y, final_state): y like x, the
    states [N,channels,S] float32 after each row's last token.  With
    ``return_checkpoints`` a third value, what selective_scan_backward
    needs: the states before every 16th token (these carry no gradient)."""
    if not return_checkpoints:
        out = (_fast or _load_fast()).selective_scan(x, delta, A, B, C, D, z, delta_bias, delta_softplus,
                                                     initial_state, resets, lengths)
        if out is not None:
            return out
    _refuse_tangents(x, delta, A, B, C, D, z, delta_bias, initial_state)
    args = (x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, resets, lengths)
    out = (_SelectiveScan.apply(*args) if _wants_grad(x, delta, A, B, C, D, z, delta_bias, initial_state)
           else _scan_forward(return_checkpoints, *args))
    return out if return_checkpoints else out[:2]


def selective_scan_backward(grad_y, x, delta, A, B, C, checkpoints, D=None, z=None, delta_bias=None,
                            delta_softplus=True, resets=None, lengths=None, grad_final_state=None):
    """Gradients of selective_scan: ``grad_y`` like x, ``checkpoints`` from the
    forward call on the same inputs, ``grad_final_state`` [N,channels,S]
    float32 or None.  Returns SelectiveScanGrads."""
    _refuse_tangents(grad_y, x, delta, A, B, C, checkpoints, D, z, delta_bias, grad_final_state)
    dev, (N, T, width, S), packed, kept = _scan_args(False, x, delta, A, B, C, D, z, delta_bias, delta_softplus,
                                                     None, resets, lengths)
    x = kept[0]
    dtype, f32 = x.dtype, torch.float32
    gp, gr, gt, grad_y = _act("grad_y", grad_y, x.shape, dtype, dev)
    marks = _dense("checkpoints", checkpoints, (N, -(-T // CHECKPOINT), width, S), f32, dev)
    if marks is None:
        raise ValueError("checkpoints is required (selective_scan(..., return_checkpoints=True))")
    gfinal = _dense("grad_final_state", grad_final_state, (N, width, S), f32, dev)

    def like(shape, to=f32, when=True):
        return torch.empty(shape, dtype=to, device=x.device) if when else None

    acts = (N, T, width)
    g = SelectiveScanGrads(
        x=like(acts, dtype), delta=like(acts, dtype), A=like((width, S)), B=like((N, T, S), dtype),
        C=like((N, T, S), dtype), D=like((width,), when=D is not None), z=like(acts, dtype, z is not None),
        delta_bias=like((width,), when=delta_bias is not None), initial_state=like((N, width, S)))
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_selective_scan_backward_workspace_bytes(packed), x.device)
        _native.check(lib.rlscan_selective_scan_backward(
            packed, _ARRAY3.pack(gp, gr, gt), _at(gfinal), marks.data_ptr(),
            _SCAN_GRADS.pack(_at(g.x), _at(g.delta), _at(g.z), _at(g.B), _at(g.C), _at(g.A), _at(g.D),
                             _at(g.delta_bias), _at(g.initial_state)),
            _at(ws), 0 if ws is None else ws.numel(), _stream_handle(x.device)), "rlscan_selective_scan_backward")
    return g


def selective_scan_step(state, x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True, slots=None):
    """One token of each of N sequences: x, delta, z [N,channels], B, C [N,S];
    ``state`` [P,channels,S] float32 (dense) is updated in place.  Sequence n
    has the state of slot ``slots[n]`` (int32; None: slot n); a slot outside
    0..P-1 marks an idle sequence, whose y is 0.  The slots of a call are
    distinct.  Returns y [N,channels].  Not differentiable."""
    y = (_fast or _load_fast()).selective_scan_step(state, x, delta, A, B, C, D, z, delta_bias, delta_softplus, slots)
    if y is not None:
        return y
    _refuse_tangents(state, x, delta, A, B, C, D, z, delta_bias)
    dev, (N, _, width, S), packed, kept = _scan_args(True, x, delta, A, B, C, D, z, delta_bias, delta_softplus, None,
                                                     None, None)
    P = _slot_pool(state, (width, S), torch.float32, dev)
    slots = _dense("slots", slots, (N,), torch.int32, dev)
    if slots is None and P < N:
        raise ValueError(f"state holds {P} slots for {N} sequences")
    y = torch.empty((N, width), dtype=x.dtype, device=x.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_selective_scan_step(packed, state.data_ptr(), P, _at(slots), y.data_ptr(),
                                                               _stream_handle(x.device)), "rlscan_selective_scan_step")
    _changed(state)
    return y


def _slot_pool(state, shape, dtype, device):
    """The number of slots of a state that is updated in place."""
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a [slots, ...] tensor of 3 dimensions")
    whole = state.shape
    if state.dtype is not dtype or whole[1:] != shape or state.get_device() != device:
        _check("state", state, (whole[0], *shape), dtype, device)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous: it is updated in place")
    return whole[0]


# ---------------------------------------------------------------------------
# causal convolution

class CausalConvGrads(NamedTuple):
    """Gradients of causal_conv's inputs (None where the input was not given)."""
    x: torch.Tensor
    weight: torch.Tensor
    bias: Optional[torch.Tensor]
    initial_state: torch.Tensor


def _conv_args(step, x, weight, bias, activation, initial_state, resets, lengths):
    dev = _lead("x", x, 2 if step else 3)
    if activation not in ("silu", None):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    dtype, shape = x.dtype, x.shape
    N, T, width = (shape[0], 1, shape[1]) if step else shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [channels, taps] tensor")
    K = weight.shape[1]
    if not 1 <= K <= MAX_TAPS:
        raise ValueError(f"weight has {K} taps: 1 to {MAX_TAPS} are supported")
    weight = _dense("weight", weight, (width, K), torch.float32, dev)
    bias = _dense("bias", bias, (width,), torch.float32, dev)
    xp, xr, xt, x = _act("x", x, shape, dtype, dev)
    if initial_state is not None:
        initial_state = _dense("initial_state", initial_state, (N, K - 1, width), dtype, dev)
    if resets is not None:
        resets = _flags(resets, (N, T), dev)
    if lengths is not None:
        lengths = _dense("lengths", lengths, (N,), torch.int32, dev)
    packed = _CONV_ARGS.pack(N, T, width, K, _TYPES[dtype], 1 if activation else 0, xp, xr, xt, weight.data_ptr(),
                             _at(bias), _at(initial_state), _at(resets), _at(lengths))
    return dev, (N, T, width, K), packed, (x, weight, bias, initial_state, resets, lengths)


def _conv_forward(x, weight, bias, activation, initial_state, resets, lengths):
    dev, (N, T, width, K), packed, kept = _conv_args(False, x, weight, bias, activation, initial_state, resets, lengths)
    x = kept[0]
    y = torch.empty((N, T, width), dtype=x.dtype, device=x.device)
    final = torch.empty((N, K - 1, width), dtype=x.dtype, device=x.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_causal_conv(packed, y.data_ptr(), final.data_ptr(),
                                                       _stream_handle(x.device)), "rlscan_causal_conv")
    return y, final


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, initial_state, resets, lengths):
        ctx.activation = activation
        ctx.save_for_backward(x, weight, bias, initial_state, resets, lengths)
        ctx.set_materialize_grads(False)
        return _conv_forward(x, weight, bias, activation, initial_state, resets, lengths)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_final):
        x, weight, bias, initial_state, resets, lengths = ctx.saved_tensors
        if grad_y is None:
            if grad_final is None:
                return (None,) * 7
            grad_y = torch.zeros_like(x)
        g = causal_conv_backward(grad_y, x, weight, bias, ctx.activation, initial_state, resets, lengths, grad_final)
        return g.x, g.weight, g.bias, None, (None if initial_state is None else g.initial_state), None, None


def causal_conv(x, weight, bias=None, activation="silu", initial_state=None, resets=None, lengths=None):
    """The causal convolution of each channel with its own K taps (1 to 8):

        pre_t = bias + sum_k weight[:, k] x_{t-K+1+k},    y = silu(pre)  (activation=None: pre)

    x [N,T,channels] float32 or bfloat16; weight [channels,K] and bias
    [channels] float32; ``initial_state`` [N,K-1,channels] of x's type holds
    the inputs before the first token, oldest first (None: zeros).  ``resets``
    and ``lengths`` as in selective_scan: taps stay inside their token's
    episode.  Returns (y, final_state): the last K-1 inputs of each row, zero
    where they lie before its last episode."""
    out = (_fast or _load_fast()).causal_conv(x, weight, bias, activation, initial_state, resets, lengths)
    if out is not None:
        return out
    _refuse_tangents(x, weight, bias, initial_state)
    if _wants_grad(x, weight, bias, initial_state):
        return _CausalConv.apply(x, weight, bias, activation, initial_state, resets, lengths)
    return _conv_forward(x, weight, bias, activation, initial_state, resets, lengths)


def causal_conv_backward(grad_y, x, weight, bias=None, activation="silu", initial_state=None, resets=None,
                         lengths=None, grad_final_state=None):
    """Gradients of causal_conv (``grad_final_state`` [N,K-1,channels] of x's
    type or None).  Returns CausalConvGrads."""
    _refuse_tangents(grad_y, x, weight, bias, initial_state, grad_final_state)
    dev, (N, T, width, K), packed, kept = _conv_args(False, x, weight, bias, activation, initial_state, resets, lengths)
    x = kept[0]
    gp, gr, gt, grad_y = _act("grad_y", grad_y, x.shape, x.dtype, dev)
    gfinal = _dense("grad_final_state", grad_final_state, (N, K - 1, width), x.dtype, dev)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = CausalConvGrads(
        x=torch.empty((N, T, width), dtype=x.dtype, device=x.device), weight=torch.empty((width, K), **f32),
        bias=torch.empty((width,), **f32) if bias is not None else None,
        initial_state=torch.empty((N, K - 1, width), dtype=x.dtype, device=x.device))
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_causal_conv_backward_workspace_bytes(packed), x.device)
        _native.check(lib.rlscan_causal_conv_backward(
            packed, _ARRAY3.pack(gp, gr, gt), _at(gfinal), g.x.data_ptr(), g.weight.data_ptr(), _at(g.bias),
            g.initial_state.data_ptr(), _at(ws), 0 if ws is None else ws.numel(), _stream_handle(x.device)),
            "rlscan_causal_conv_backward")
    return g


def causal_conv_step(state, x, weight, bias=None, activation="silu", slots=None):
    """One token of each of N sequences: x [N,channels]; ``state``
    [P,K-1,channels] of x's type (dense) is shifted by one token in place.
    ``slots`` as in selective_scan_step.  Returns y [N,channels].  Not
    differentiable."""
    y = (_fast or _load_fast()).causal_conv_step(state, x, weight, bias, activation, slots)
    if y is not None:
        return y
    _refuse_tangents(state, x, weight, bias)
    dev, (N, _, width, K), packed, kept = _conv_args(True, x, weight, bias, activation, None, None, None)
    P = _slot_pool(state, (K - 1, width), x.dtype, dev)
    slots = _dense("slots", slots, (N,), torch.int32, dev)
    if slots is None and P < N:
        raise ValueError(f"state holds {P} slots for {N} sequences")
    y = torch.empty((N, width), dtype=x.dtype, device=x.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_causal_conv_step(packed, state.data_ptr(), P, _at(slots), y.data_ptr(),
                                                            _stream_handle(x.device)), "rlscan_causal_conv_step")
    _changed(state)
    return y


# ---------------------------------------------------------------------------
# root-mean-square norm

class RmsNorm(NamedTuple):
    """y; the sum x + residual (None without a residual); the scales of an 8-bit y (else None)."""
    y: torch.Tensor
    residual: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


class RmsNormGrads(NamedTuple):
    """Gradients of add_rms_norm's inputs; ``residual`` is ``x`` where both have one type."""
    x: torch.Tensor
    weight: torch.Tensor
    residual: torch.Tensor


def _rows(name, t, shape, dtype, device):
    """(tensor, address, row stride) of [..., D] as rows of D elements."""
    try:
        fits = t.dtype is dtype and t.shape == shape and t.get_device() == device
    except AttributeError:
        fits = False
    if not fits:
        _check(name, t, shape, dtype, device)
    if len(shape) != 2:
        t = t.reshape(t.numel() // max(shape[-1], 1), shape[-1])
    strides = t.stride()
    if strides[1] != 1 and shape[-1] > 1:
        t = t.contiguous()
        strides = t.stride()
    return t, t.data_ptr(), strides[0]


def _norm_lead(name, x, weight, eps):
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError(f"{name} must be a [..., channels] tensor of at least 2 dimensions")
    dev = x.get_device()
    if dev < 0 or x.dtype not in _TYPES:
        _lead(name, x, x.dim())
    if weight is None:
        raise TypeError("weight must be a torch.Tensor")
    if not float(eps) >= 0:
        raise ValueError("eps must not be negative")
    shape = x.shape
    width = shape[-1]
    M = shape[0] if len(shape) == 2 else (x.numel() // width if width else 0)
    return dev, M, width, _dense("weight", weight, (width,), torch.float32, dev)


def _norm_forward(x, weight, residual, eps, out_dtype):
    dev, M, width, weight = _norm_lead("x", x, weight, eps)
    eight = out_dtype == torch.float8_e4m3fn
    if not eight and out_dtype not in (None, x.dtype):
        raise ValueError("out_dtype must be x's type or torch.float8_e4m3fn")
    shape = x.shape
    xr, xp, xs = _rows("x", x, shape, x.dtype, dev)
    rp = rs = rtype = 0
    summed = None
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"residual: expected a tensor of {x.dtype} or torch.float32")
        rr, rp, rs = _rows("residual", residual, shape, residual.dtype, dev)
        rtype = _TYPES[residual.dtype]
        summed = torch.empty(shape, dtype=residual.dtype, device=x.device)
    y = torch.empty(shape, dtype=torch.float8_e4m3fn if eight else x.dtype, device=x.device)
    scales = None
    if eight:
        scales = torch.empty((*shape[:-1], -(-width // SCALE_BLOCK)), dtype=torch.float32, device=x.device)
    with _on(dev):
        _native.check(_native.lib().rlscan_add_rms_norm(
            xp, xs, rp, rs, weight.data_ptr(), M, width, eps, _TYPES[x.dtype], rtype, y.data_ptr(), _at(scales),
            _at(summed), _stream_handle(x.device)), "rlscan_add_rms_norm")
    return RmsNorm(y, summed, scales)


class _AddRmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        out = _norm_forward(x, weight, residual, eps, None)
        ctx.eps, ctx.plain = eps, residual is None
        ctx.io = x.dtype
        ctx.save_for_backward(x if residual is None else out.residual, weight)
        ctx.set_materialize_grads(False)
        return out.y, out.residual

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_y, grad_sum):
        h, weight = ctx.saved_tensors
        if grad_y is None:
            if grad_sum is None:
                return None, None, None, None
            grad_y = torch.zeros(h.shape, dtype=ctx.io, device=h.device)
        g = add_rms_norm_backward(grad_y, h, weight, grad_sum, ctx.eps)
        return g.x, g.weight, (None if ctx.plain else g.residual), None


def add_rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=None):
    """h = x + residual and y = h / sqrt(mean(h^2) + eps) * weight over the last
    dimension.  x [..., channels] float32 or bfloat16, weight [channels]
    float32, residual of x's type or float32.  Returns RmsNorm(y, residual,
    scales): ``residual`` is h in the residual's type (None without one).
    ``out_dtype=torch.float8_e4m3fn`` gives y in 8 bits with a float32 scale
    for each 128 columns of a row (y stands for y.float() * its scale); that
    form is not differentiable."""
    out = (_fast or _load_fast()).add_rms_norm(x, weight, residual, eps, out_dtype)
    if out is not None:
        return out
    _refuse_tangents(x, weight, residual)
    if out_dtype != torch.float8_e4m3fn and _wants_grad(x, weight, residual):
        if out_dtype not in (None, x.dtype):
            raise ValueError("out_dtype must be x's type or torch.float8_e4m3fn")
        y, summed = _AddRmsNorm.apply(x, weight, residual, eps)
        return RmsNorm(y, summed, None)
    return _norm_forward(x, weight, residual, eps, out_dtype)


def add_rms_norm_backward(grad_y, h, weight, grad_residual=None, eps=1e-6):
    """Gradients of add_rms_norm from ``h``, the sum it returned as ``residual``
    (x itself where there was none): ``grad_y`` float32 or bfloat16, h of its
    type or float32, ``grad_residual`` the gradient of the returned sum (h's
    type) or None.  Returns RmsNormGrads."""
    _refuse_tangents(grad_y, h, weight, grad_residual)
    dev, M, width, weight = _norm_lead("grad_y", grad_y, weight, eps)
    shape = grad_y.shape
    if not isinstance(h, torch.Tensor) or h.dtype not in (grad_y.dtype, torch.float32):
        raise TypeError(f"h: expected a tensor of {grad_y.dtype} or torch.float32")
    yr, yp, ys = _rows("grad_y", grad_y, shape, grad_y.dtype, dev)
    hr, hp, hs = _rows("h", h, shape, h.dtype, dev)
    gp = gs = 0
    if grad_residual is not None:
        gr, gp, gs = _rows("grad_residual", grad_residual, shape, h.dtype, dev)
    gx = torch.empty(shape, dtype=grad_y.dtype, device=grad_y.device)
    gh = gx if h.dtype == grad_y.dtype else torch.empty(shape, dtype=h.dtype, device=h.device)
    gw = torch.empty((width,), dtype=torch.float32, device=grad_y.device)
    lib = _native.lib()
    with _on(dev):
        ws = _scratch(lib.rlscan_add_rms_norm_backward_workspace_bytes(M, width), grad_y.device)
        _native.check(lib.rlscan_add_rms_norm_backward(
            yp, ys, hp, hs, gp, gs, weight.data_ptr(), M, width, eps, _TYPES[grad_y.dtype], _TYPES[h.dtype],
            gx.data_ptr(), 0 if gh is gx else gh.data_ptr(), gw.data_ptr(), _at(ws), 0 if ws is None else ws.numel(),
            _stream_handle(grad_y.device)), "rlscan_add_rms_norm_backward")
    return RmsNormGrads(gx, gw, gh)
