"""Torch-facing operators around the layer, with their gradients: norm, gated
feed-forward block, dropout with the residual add.

Each operator has a forward and a backward function over plain tensors
(``norm_forward`` / ``norm_backward``, ``gated_ffn_forward`` / ``gated_ffn_backward``,
``dropout_add_forward`` / ``dropout_add_backward``) and a differentiable function
(``layer_norm``, ``rms_norm``, ``gated_ffn``, ``dropout_add``) that autograd records.
All arithmetic runs in libmoe_ffn.so on the tensors' device and its current stream;
outputs and workspaces are torch allocations of the call. Nothing synchronises the host,
so the calls can be captured into a CUDA graph. (A captured training step should call the
forward and backward functions themselves: autograd's own accumulation of leaf gradients
may touch streams outside the capture.)

Wrong shapes, types, strides or devices raise ``MoEError``; there is no fallback.
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple

import torch

from .binding import (MOE_ACT_GELU, MOE_ACT_SILU, MOE_DTYPE_BF16, MOE_DTYPE_FP16, MOE_DTYPE_FP32,
                      MOE_NORM_LAYER, MOE_NORM_RMS, MoEError, _check, load_library)

__all__ = ["MoEError", "norm_forward", "norm_backward", "layer_norm", "rms_norm",
           "gated_ffn_forward", "gated_ffn_backward", "gated_ffn", "dropout_add_forward",
           "dropout_add_backward", "dropout_add", "gated_ffn_block", "device_status"]

_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_FP16,
           torch.float32: MOE_DTYPE_FP32}
_KINDS = {"layer": MOE_NORM_LAYER, "rms": MOE_NORM_RMS}
_ACTS = {"silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}


def _bad(message: str) -> MoEError:
    return MoEError(2, message)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _code(table, key, what: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise _bad(f"unsupported {what} {key!r}") from None


def _cuda(x: torch.Tensor, what: str) -> int:
    """Index of x's CUDA device."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise _bad(f"{what} must be a CUDA tensor")
    return x.get_device()


def _as_rows(t: torch.Tensor, what: str) -> torch.Tensor:
    """t as (rows, cols) with unit column stride, as a view where its strides allow it."""
    if t.dim() == 0:
        raise _bad(f"{what} must have at least one dimension")
    if t.shape[-1] == 0:
        raise _bad(f"{what} has an empty last dimension")
    t2 = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    # rows that overlap (an expanded tensor) or run backwards are laid out first
    if (t2.shape[1] > 1 and t2.stride(1) != 1) or \
            (t2.shape[0] > 1 and t2.stride(0) < t2.shape[1]):
        t2 = t2.contiguous()
    return t2


def _like(t: torch.Tensor, x: torch.Tensor, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.shape != x.shape or t.dtype != x.dtype \
            or t.device != x.device:
        raise _bad(f"{what} must be a {tuple(x.shape)} {x.dtype} tensor on {x.device}")
    return t


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(index: int, name: str, *args) -> None:
    """Call a C entry point with the tensors' device current and its current stream as the
    last argument."""
    lib = load_library()
    if _current_device() == index:
        status = getattr(lib, name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = getattr(lib, name)(*args, _raw_stream(index))
    if status:
        _check(lib, status)


def _is_rows(t: torch.Tensor) -> bool:
    """Whether t already is what the operators' outputs look like: contiguous (rows, cols)."""
    return t.dim() == 2 and t.is_contiguous() and t.shape[1] > 0


@lru_cache(maxsize=256)
def _norm_workspace(kind: int, rows: int, cols: int) -> int:
    return load_library().moe_norm_workspace_bytes(kind, rows, cols)


@lru_cache(maxsize=256)
def _ffn_workspace(T: int, d: int, f: int, backward: int) -> int:
    return load_library().moe_gated_ffn_workspace_bytes(T, d, f, backward)


# ------------------------------------------------------------------------ norm
def _norm_vector(t, x, cols, what):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.numel() != cols or not t.is_cuda \
            or t.get_device() != x.get_device() or t.dtype not in (x.dtype, torch.float32):
        raise _bad(f"{what} must be a ({cols},) tensor of x's type or fp32 on {x.device}")
    return t if t.is_contiguous() else t.contiguous()


def norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, eps: float = 1e-5, kind: str = "layer",
                 save: bool = False):
    """Layer norm (kind "layer") or RMS norm ("rms") over x's last dimension.

    x is bf16, fp16 or fp32 with any leading dimensions; weight and bias are (cols,) of x's
    type or fp32 (the same of both). Returns y, or with ``save`` (y, mean, rstd) for
    ``norm_backward``: fp32, one a row, mean None for an RMS norm.
    """
    index = _cuda(x, "x")
    dt, kd = _code(_DTYPES, x.dtype, "dtype"), _code(_KINDS, kind, "norm kind")
    x2 = x if _is_rows(x) else _as_rows(x, "x")
    rows, cols = x2.shape
    weight, bias = _norm_vector(weight, x, cols, "weight"), _norm_vector(bias, x, cols, "bias")
    if kd == MOE_NORM_RMS and bias is not None:
        raise _bad("an RMS norm has no bias")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise _bad("weight and bias must have the same type")
    vec = weight if weight is not None else bias
    wdt = dt if vec is None else _DTYPES[vec.dtype]
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    mean = rstd = None
    if save:
        rstd = x.new_empty((rows,), dtype=torch.float32)
        if kd == MOE_NORM_LAYER:
            mean = x.new_empty((rows,), dtype=torch.float32)
    _launch(index, "moe_norm_forward", kd, dt, wdt, rows, cols, x2.data_ptr(), x2.stride(0),
            _ptr(weight), _ptr(bias), eps, y.data_ptr(), cols, _ptr(mean), _ptr(rstd))
    return (y, mean, rstd) if save else y


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
    index = _cuda(x, "x")
    dt, kd = _code(_DTYPES, x.dtype, "dtype"), _code(_KINDS, kind, "norm kind")
    _like(dy, x, "dy")
    x2 = x if _is_rows(x) else _as_rows(x, "x")
    dy2 = dy if _is_rows(dy) else _as_rows(dy, "dy")
    rows, cols = x2.shape
    weight = _norm_vector(weight, x, cols, "weight")
    if kd == MOE_NORM_RMS and bias:
        raise _bad("an RMS norm has no bias")
    for name, t in (("rstd", rstd), ("mean", mean)):
        if name == "mean" and kd == MOE_NORM_RMS:
            continue
        if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.numel() != rows \
                or t.dtype != torch.float32 or not t.is_cuda or t.get_device() != index \
                or not t.is_contiguous():
            raise _bad(f"{name} must be the contiguous fp32 ({rows},) tensor of norm_forward")
    wtype = weight.dtype if weight is not None else grad_dtype or x.dtype
    if wtype not in (x.dtype, torch.float32) or grad_dtype not in (None, wtype):
        raise _bad("grad_dtype must be the weight's type, or x's type or fp32 without a weight")
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_dx else None
    dweight = torch.empty_like(weight) if need_dweight and weight is not None else None
    dbias = x.new_empty((cols,), dtype=wtype) if bias else None
    ws, nbytes = None, 0
    if dweight is not None or dbias is not None:
        nbytes = _norm_workspace(kd, rows, cols)
        ws = x.new_empty((max(nbytes, 16),), dtype=torch.uint8)
    _launch(index, "moe_norm_backward", kd, dt, _DTYPES[wtype], rows, cols, dy2.data_ptr(),
            dy2.stride(0), x2.data_ptr(), x2.stride(0), _ptr(weight),
            _ptr(mean) if kd == MOE_NORM_LAYER else None, rstd.data_ptr(), _ptr(dx), cols,
            _ptr(dweight), _ptr(dbias), _ptr(ws), nbytes)
    return dx, dweight, dbias


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


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over x's last dimension (see ``norm_forward``)."""
    return _Norm.apply(x, weight, bias, eps, "layer")


def rms_norm(x, weight=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable RMS norm over x's last dimension (see ``norm_forward``)."""
    return _Norm.apply(x, weight, None, eps, "rms")


# ------------------------------------------------------------------------ gated feed-forward
def _ffn_rows(t: torch.Tensor, what: str) -> torch.Tensor:
    """t as (T, d) rows the tensor maps can describe: 16-byte aligned rows and base."""
    t2 = t if _is_rows(t) else _as_rows(t, what)
    if t2.data_ptr() % 16 or (t2.shape[0] > 1 and t2.stride(0) % 8):
        t2 = t2.clone(memory_format=torch.contiguous_format)
    return t2


def _ffn_weights(x, W1, W3, W2):
    if x.dim() < 1 or not isinstance(W1, torch.Tensor) or W1.dim() != 2:
        raise _bad("x needs a last dimension d and W1 the shape (f, d)")
    d, f = x.shape[-1], W1.shape[0]
    for name, w, shape in (("W1", W1, (f, d)), ("W3", W3, (f, d)), ("W2", W2, (d, f))):
        if not isinstance(w, torch.Tensor) or w.shape != shape or w.dtype != x.dtype \
                or not w.is_cuda or w.get_device() != x.get_device() or not w.is_contiguous():
            raise _bad(f"{name} must be a contiguous {x.dtype} {shape} tensor on {x.device}")
    return d, f


def gated_ffn_forward(x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor, W2: torch.Tensor,
                      activation: str = "silu", save: bool = False):
    """(act(x W1^T) * (x W3^T)) W2^T over x (..., d), bf16 or fp16.

    W1 and W3 are (f, d), W2 (d, f), contiguous, d and f multiples of 8; activation is
    "silu" or "gelu" (tanh form). Returns out, or with ``save`` (out, gate, up): the (T, f)
    pre-activations for ``gated_ffn_backward``.
    """
    index = _cuda(x, "x")
    d, f = _ffn_weights(x, W1, W3, W2)
    dt, act = _code(_DTYPES, x.dtype, "dtype"), _code(_ACTS, activation, "activation")
    x2 = _ffn_rows(x, "x")
    T = x2.shape[0]
    out = torch.empty_like(x, memory_format=torch.contiguous_format)
    gate = up = None
    if save:
        gate, up = x.new_empty((T, f)), x.new_empty((T, f))
    nbytes = _ffn_workspace(T, d, f, 0)
    ws = x.new_empty((nbytes,), dtype=torch.uint8)
    _launch(index, "moe_gated_ffn_forward", act, dt, T, d, f, x2.data_ptr(), x2.stride(0),
            W1.data_ptr(), W3.data_ptr(), W2.data_ptr(), out.data_ptr(), d, _ptr(gate), _ptr(up),
            ws.data_ptr(), nbytes)
    return (out, gate, up) if save else out


def gated_ffn_backward(dout: torch.Tensor, x: torch.Tensor, W1: torch.Tensor, W3: torch.Tensor,
                       W2: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                       activation: str = "silu",
                       needs: Tuple[bool, bool, bool, bool] = (True, True, True, True)):
    """Gradients (dx, dW1, dW3, dW2) of ``gated_ffn_forward`` from its saved gate and up;
    ``needs`` leaves out those not wanted (None in their place)."""
    index = _cuda(x, "x")
    d, f = _ffn_weights(x, W1, W3, W2)
    dt, act = _code(_DTYPES, x.dtype, "dtype"), _code(_ACTS, activation, "activation")
    x2, dout2 = _ffn_rows(x, "x"), _ffn_rows(_like(dout, x, "dout"), "dout")
    T = x2.shape[0]
    for name, t in (("gate", gate), ("up", up)):
        if not isinstance(t, torch.Tensor) or t.shape != (T, f) or t.dtype != x.dtype \
                or not t.is_cuda or t.get_device() != index or not t.is_contiguous():
            raise _bad(f"{name} must be the contiguous ({T}, {f}) tensor of gated_ffn_forward")
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if needs[0] else None
    dW1 = torch.empty_like(W1) if needs[1] else None
    dW3 = torch.empty_like(W3) if needs[2] else None
    dW2 = torch.empty_like(W2) if needs[3] else None
    nbytes = _ffn_workspace(T, d, f, 1)
    ws = x.new_empty((nbytes,), dtype=torch.uint8)
    _launch(index, "moe_gated_ffn_backward", act, dt, T, d, f, dout2.data_ptr(), dout2.stride(0),
            x2.data_ptr(), x2.stride(0), W1.data_ptr(), W3.data_ptr(), W2.data_ptr(),
            gate.data_ptr(), up.data_ptr(), _ptr(dx), d, _ptr(dW1), _ptr(dW3), _ptr(dW2),
            ws.data_ptr(), nbytes)
    return dx, dW1, dW3, dW2


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
    return _GatedFFN.apply(x, W1, W3, W2, activation)


# ------------------------------------------------------------------------ dropout
def _rng_state(rng, p, x):
    if p == 0 and rng is None:
        return None
    if not isinstance(rng, torch.Tensor) or rng.dim() != 1 or rng.numel() != 2 \
            or not rng.is_cuda or rng.get_device() != x.get_device() \
            or rng.dtype not in (torch.int64, torch.uint64) or not rng.is_contiguous():
        raise _bad(f"rng must be a contiguous int64 (2,) tensor (seed, offset) on {x.device}")
    return rng


def dropout_add_forward(x: torch.Tensor, residual: Optional[torch.Tensor], p: float,
                        rng: Optional[torch.Tensor]) -> torch.Tensor:
    """residual + dropout(x): x / (1 - p) where the generator keeps the element, else 0.

    x and residual (None: 0) have one shape and type (bf16, fp16, fp32). rng is an int64
    (2,) tensor on the device, the seed and the offset; the mask depends on them and on an
    element's position in x alone, is not stored, and is drawn again by the backward pass.
    Give every draw another offset; a captured graph reads rng at each replay.
    """
    index = _cuda(x, "x")
    dt = _code(_DTYPES, x.dtype, "dtype")
    if x.dim() == 0:
        raise _bad("x must have at least one dimension")
    rng = _rng_state(rng, p, x)
    if residual is not None:
        _like(residual, x, "residual")
    out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.numel() == 0:
        return out
    if x.is_contiguous() and (residual is None or residual.is_contiguous()):
        # one line of all elements, whatever the shape
        n, cols = 1, x.numel()
        x2, r2, ldx, ldr = x, residual, cols, cols
    else:
        x2 = _as_rows(x, "x")
        r2 = None if residual is None else _as_rows(residual, "residual")
        n, cols = x2.shape
        ldx, ldr = x2.stride(0), 0 if r2 is None else r2.stride(0)
    _launch(index, "moe_dropout_forward", dt, n, cols, x2.data_ptr(), ldx, _ptr(r2), ldr, p,
            _ptr(rng), out.data_ptr(), cols)
    return out


def dropout_add_backward(dout: torch.Tensor, p: float, rng: Optional[torch.Tensor]
                         ) -> torch.Tensor:
    """Gradient of x in ``dropout_add_forward`` with the same p and rng contents (the
    residual's gradient is dout itself)."""
    return dropout_add_forward(dout, None, p, rng)


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
    return _DropoutAdd.apply(x, residual, p, rng)


def gated_ffn_block(x, W1, W3, W2, norm_weight=None, norm_bias=None, norm: str = "rms",
                    eps: float = 1e-5, activation: str = "silu", p: float = 0.0,
                    rng: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable pre-norm residual block x + dropout(gated_ffn(norm(x))): the block
    around the layer ("Shared Expert (DeepSeek-V3)", "How it works": normalised input, the
    residual added at block level) with a dense feed-forward layer in its middle."""
    h = _Norm.apply(x, norm_weight, norm_bias, eps, norm)
    return dropout_add(gated_ffn(h, W1, W3, W2, activation), x, p, rng)


def device_status(device=None) -> None:
    """Raise ``MoEError`` if one of these operators' kernels on the device (default: the
    current one) gave up a bounded wait since the last call. Synchronises."""
    lib = load_library()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        torch.cuda.synchronize()
        _check(lib, lib.moe_ops_device_status())
