"""Torch-facing operators around the layer, with their gradients: norm, gated
feed-forward block, dropout with the residual add.

Each operator has a forward and a backward function over plain tensors
(``norm_forward`` / ``norm_backward``, ``gated_ffn_forward`` / ``gated_ffn_backward``,
``dropout_add_forward`` / ``dropout_add_backward``) and a differentiable function
(``layer_norm``, ``rms_norm``, ``gated_ffn``, ``dropout_add``) that autograd records. The
former record nothing: their outputs carry neither a graph nor a forward-mode tangent.
All arithmetic runs in libmoe_ffn.so on the tensors' device and its current stream;
outputs and workspaces are torch allocations of the call. Nothing synchronises the host,
so the calls can be captured into a CUDA graph. (A captured training step should call the
forward and backward functions themselves: autograd's own accumulation of leaf gradients
may touch streams outside the capture.)

Wrong shapes, types, strides or devices raise ``MoEError``; there is no fallback.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad

from .binding import MoEError, _check, load_library
from .build import host_path

__all__ = ["MoEError", "norm_forward", "norm_backward", "layer_norm", "rms_norm",
           "gated_ffn_forward", "gated_ffn_backward", "gated_ffn", "dropout_add_forward",
           "dropout_add_backward", "dropout_add", "gated_ffn_block", "device_status"]

_MODULE = None


def _host():
    """The module that checks, allocates and launches (raises if it has not been built)."""
    global _MODULE
    if _MODULE is None:
        path = host_path()
        if not os.path.exists(path):
            raise MoEError(4, f"module not found at {path}; build it with "
                              "`python -m mixture_experts_ffn_expert_b200.build`")
        load_library()
        loader = importlib.machinery.ExtensionFileLoader("_moe_host", path)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("_moe_host", path, loader=loader))
        loader.exec_module(module)
        module.set_error(MoEError)
        _MODULE = module
    return _MODULE


def _has_tangent(*arguments) -> bool:
    """Whether an argument carries a forward-mode tangent."""
    # outside every forward-mode level no tensor does (asking each takes 2 us)
    if getattr(forward_ad, "_current_level", 0) < 0:
        return False
    return any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None
               for t in arguments)


def _unrecorded(*arguments) -> bool:
    """Whether a call may pass its autograd function by and save nothing: grad mode is off and
    no argument carries a forward-mode tangent. A tangent does not depend on grad mode; the
    autograd functions have no such derivative and raise, where a plain call would drop it."""
    return not torch.is_grad_enabled() and not _has_tangent(*arguments)


# ------------------------------------------------------------------------ norm
def norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, eps: float = 1e-5, kind: str = "layer",
                 save: bool = False):
    """Layer norm (kind "layer") or RMS norm ("rms") over x's last dimension.

    x is bf16, fp16 or fp32 with any leading dimensions; weight and bias are (cols,) of x's
    type or fp32 (the same of both). Returns y, or with ``save`` (y, mean, rstd) for
    ``norm_backward``: fp32, one a row, mean None for an RMS norm.
    """
    return (_MODULE or _host()).norm_forward(x, weight, bias, eps, kind, save)


def norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                  mean: Optional[torch.Tensor], rstd: torch.Tensor, kind: str = "layer",
                  bias: bool = False, need_dx: bool = True, need_dweight: bool = True,
                  grad_dtype: Optional[torch.dtype] = None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor],
                             Optional[torch.Tensor]]:
    """Gradients (dx, dweight, dbias) of ``norm_forward`` from its saved mean and rstd.

    dweight is None without a weight (or ``need_dweight`` False), dbias None unless
    ``bias``; both have ``grad_dtype``, by default the weight's type (x's without a weight),
    and are summed in a fixed order.
    """
    fp32 = None
    if grad_dtype is not None:
        if grad_dtype not in ((x.dtype, torch.float32) if weight is None else (weight.dtype,)):
            raise MoEError(2, "grad_dtype must be the weight's type, or x's type or fp32 without "
                              "a weight")
        fp32 = grad_dtype == torch.float32
    return (_MODULE or _host()).norm_backward(dy, x, weight, mean, rstd, kind, bias, need_dx,
                                              need_dweight, fp32)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, kind):
        y, mean, rstd = norm_forward(x, weight, bias, eps, kind, save=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.kind, ctx.has_bias = kind, bias is not None
        ctx.bias_type = None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = norm_backward(dy, x, weight, mean, rstd, ctx.kind,
                                   bias=ctx.has_bias and need[2], need_dx=need[0],
                                   need_dweight=need[1],
                                   grad_dtype=ctx.bias_type if weight is None else None)
        return dx, dw, db, None, None


def _norm(x, weight, bias, eps, kind):
    if _unrecorded(x, weight, bias):
        return norm_forward(x, weight, bias, eps, kind)
    return _Norm.apply(x, weight, bias, eps, kind)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over x's last dimension (see ``norm_forward``)."""
    return _norm(x, weight, bias, eps, "layer")


def rms_norm(x, weight=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable RMS norm over x's last dimension (see ``norm_forward``)."""
    return _norm(x, weight, None, eps, "rms")


# ------------------------------------------------------------------------ gated feed-forward
def gated_ffn_forward(x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor,
                      activation: str = "silu", save: bool = False):
    """(act(x W1^T) * (x W3^T)) W2^T over x (..., d), bf16 or fp16.

    W1 and W3 are (f, d), W2 (d, f), contiguous and 16-byte aligned, d and f multiples of 8;
    activation is "silu" or "gelu" (tanh form). Returns out, or with ``save`` (out, gate, up):
    the (T, f) fp32 pre-activations for ``gated_ffn_backward``. Products accumulate in fp32; the
    hidden layer is rounded to x's type between them (fp16: infinite beyond 65504).
    """
    return (_MODULE or _host()).gated_ffn_forward(x, W1, W3, W2, activation, save)


def gated_ffn_backward(dout: torch.Tensor, x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor,
                       W2: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                       activation: str = "silu",
                       needs: Tuple[bool, bool, bool, bool] = (True, True, True, True)):
    """Gradients (dx, dW1, dW3, dW2) of ``gated_ffn_forward`` from its saved gate and up;
    ``needs`` leaves out those not wanted (None in their place)."""
    return (_MODULE or _host()).gated_ffn_backward(dout, x, W1, W3, W2, gate, up, activation,
                                                   *needs)


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W1, W3, W2, activation):
        if not any(ctx.needs_input_grad):
            return gated_ffn_forward(x, W1, W3, W2, activation)
        out, gate, up = gated_ffn_forward(x, W1, W3, W2, activation, save=True)
        ctx.save_for_backward(x, W1, W3, W2, gate, up)
        ctx.activation = activation
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, W1, W3, W2, gate, up = ctx.saved_tensors
        return (*gated_ffn_backward(dout, x, W1, W3, W2, gate, up, ctx.activation,
                                    ctx.needs_input_grad[:4]), None)


def gated_ffn(x, W1, W3, W2, activation: str = "silu") -> torch.Tensor:
    """Differentiable gated feed-forward block (see ``gated_ffn_forward``)."""
    if _unrecorded(x, W1, W3, W2):
        return gated_ffn_forward(x, W1, W3, W2, activation)
    return _GatedFFN.apply(x, W1, W3, W2, activation)


# ------------------------------------------------------------------------ dropout
def dropout_add_forward(x: torch.Tensor, residual: Optional[torch.Tensor], p: float,
                        rng: Optional[torch.Tensor]) -> torch.Tensor:
    """residual + dropout(x): x / (1 - p) where the generator keeps the element, else 0.

    x and residual (None: 0) have one shape and type (bf16, fp16, fp32). rng is an int64
    (2,) tensor on the device, the seed and the offset; the mask depends on them and on an
    element's position in x alone, is not stored, and is drawn again by the backward pass.
    Give every draw another offset; a captured graph reads rng at each replay.
    """
    return (_MODULE or _host()).dropout_add(x, residual, p, rng)


def dropout_add_backward(dout: torch.Tensor, p: float, rng: Optional[torch.Tensor]
                         ) -> torch.Tensor:
    """Gradient of x in ``dropout_add_forward`` with the same p and rng contents (the
    residual's gradient is dout itself)."""
    return (_MODULE or _host()).dropout_add(dout, None, p, rng)


class _DropoutAdd(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, rng):
        ctx.save_for_backward(rng)     # autograd refuses a backward after rng has changed
        ctx.p = p
        return dropout_add_forward(x, residual, p, rng)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        rng, = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dropout_add_backward(dout, ctx.p, rng) if need[0] else None
        return dx, dout if need[1] else None, None, None


def dropout_add(x, residual, p: float, rng: Optional[torch.Tensor]) -> torch.Tensor:
    """Differentiable residual + dropout(x) (see ``dropout_add_forward``). rng must hold the
    same seed and offset in the backward pass: changing it in place in between raises."""
    if _unrecorded(x, residual):
        return dropout_add_forward(x, residual, p, rng)
    return _DropoutAdd.apply(x, residual, p, rng)


def gated_ffn_block(x, W1, W3, W2, norm_weight=None, norm_bias=None, norm: str = "rms",
                    eps: float = 1e-5, activation: str = "silu", p: float = 0.0,
                    rng: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable pre-norm residual block x + dropout(gated_ffn(norm(x))): the block
    around the layer ("Shared Expert (DeepSeek-V3)", "How it works": normalised input, the
    residual added at block level) with a dense feed-forward layer in its middle."""
    h = _norm(x, norm_weight, norm_bias, eps, norm)
    return dropout_add(gated_ffn(h, W1, W3, W2, activation), x, p, rng)


def device_status(device=None) -> None:
    """Raise ``MoEError`` if one of these operators' kernels on the device (default: the
    current one) gave up a bounded wait since the last call. Synchronises."""
    lib = load_library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        torch.cuda.synchronize()
        _check(lib, lib.moe_ops_device_status())
