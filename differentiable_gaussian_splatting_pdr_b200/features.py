"""From a predictor's features to Gaussian parameters: the operators before render().

    y = linear(x, weight, bias, residual, activation)      # act(x W^T + b) + r
    h = gated(x, w_gate, w_up, activation)                 # act(x Wg^T) * (x Wu^T)
    y, s = rms_norm(x, weight, residual)                   # s = x + r, y = s / rms(s) * w
    params = adapter(features, weights, base)              # the three in a row, [B, N, 5 + C]

These are differentiable (autograd).  linear_fwd / linear_bwd, gated_fwd /
gated_bwd and rms_norm_fwd / rms_norm_bwd are the single calls behind them,
quantize_rows gives rows in 8 bits with a scale each, which linear_fwd and
gated_fwd take as operands.  Rows are the flattened leading dimensions.
Products take float16 or bfloat16 (or float8_e4m3fn with scales) and add up in
fp32; rms_norm takes float32 too.  Every call enqueues the library's kernels
on the current torch stream of the tensors' device; argument meaning, numerics
and limits are in include/pdr.h.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass, replace

import torch

from . import _lib
from .api import _DTYPES

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_E4M3 = torch.float8_e4m3fn
_HALF = (torch.float16, torch.bfloat16)
_TYPE = {**_DTYPES, _E4M3: 3}
_FLOAT = tuple(_DTYPES)
_MAX_ROWS = 1 << 30  # as in include/pdr.h; sizes travel as C ints
_OPERAND = (*_HALF, _E4M3)


_raw_stream = torch._C._cuda_getCurrentRawStream  # without the Stream object of torch.cuda.current_stream
_functions = {}


def _function(name: str):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(_lib.load(), name)
    return f


def _call(name: str, device: torch.device, *args) -> None:
    """One library call on the current stream of `device`, with it current."""
    index = device.index
    if index == torch.cuda.current_device():
        status = _function(name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = _function(name)(*args, _raw_stream(index))
    if status:
        _lib.check(name, status)


@functools.lru_cache(maxsize=4096)
def _bytes(name: str, *sizes) -> int:
    """Workspace bytes: a function of the sizes and types alone."""
    return _function(name)(*sizes)


def _new(shape, dtype, device):
    """torch.empty (for matrices by the entry point that takes half the time)."""
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _workspace(n: int, device: torch.device):
    """(tensor, pointer, bytes) of a workspace of n bytes."""
    if n == 0:
        return None, None, 0
    ws = torch.empty_strided((n,), (1,), dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), n


def _ptr(t):
    return None if t is None else t.data_ptr()


def _act(activation: str) -> int:
    try:
        return ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError("activation must be one of %s, got %r" % (", ".join(ACTIVATIONS), activation)) from None


def _check(t, what: str, dtypes, shape=None, device=None):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous() and \
            (shape is None or t.shape == shape) and (device is None or t.device == device):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (what, " / ".join(str(d)[6:] for d in dtypes), t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (what, list(shape), list(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s like the first tensor, got %s" % (what, device, t.device))
    raise ValueError("%s must be contiguous" % what)


def _check_rows(t, what: str, dtypes):
    _check(t, what, dtypes)
    shape = t.shape
    if not shape or shape[-1] < 1:
        raise ValueError("%s must be [..., features] with at least one feature" % what)
    width = shape[-1]
    rows = shape[0] if len(shape) == 2 else t.numel() // width
    if rows > _MAX_ROWS or width > _MAX_ROWS:
        raise ValueError("%s has more rows or features than 2^30" % what)
    return rows, width


def _check_weight(w, what: str, dtype, width: int, device):
    _check(w, what, (dtype,), device=device)
    if w.dim() != 2 or w.shape[1] != width or not 1 <= w.shape[0] <= _MAX_ROWS:
        raise ValueError("%s must be [outputs, %d], got %s" % (what, width, list(w.shape)))
    return w.shape[0]


def _aligned(t, n: int = 16):
    """The tensor, or a copy of it where it does not start at a multiple of n bytes."""
    return t if t.data_ptr() % n == 0 else t.clone()


def _check_scales(x, weights, x_scale, scales, M: int):
    """Row scales: with 8-bit operands, and only with them."""
    if x.dtype == _E4M3:
        _check(x_scale, "x_scale", (torch.float32,), device=x.device)
        if x_scale.numel() != M:
            raise ValueError("x_scale must have one value for each of the %d rows" % M)
        for w, s, name in zip(weights, scales, ("weight scale", "up scale")):
            _check(s, name, (torch.float32,), (w.shape[0],), x.device)
    elif x_scale is not None or any(s is not None for s in scales):
        raise ValueError("scales go with float8_e4m3fn operands only")


def _out(out, shape, dtype, device):
    """`out`, or a new tensor where there is none or it does not start at 16 bytes."""
    if out is not None:
        _check(out, "out", (dtype,), shape, device)
        if out.data_ptr() % 16 == 0:
            return out
    return _new(shape, dtype, device)


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               residual: torch.Tensor | None = None, activation: str = "none",
               out_dtype: torch.dtype | None = None, x_scale: torch.Tensor | None = None,
               weight_scale: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """act(x W^T + bias) + residual: [..., N] from x [..., K] and weight [N, K].

    x and weight: float16, bfloat16, or both float8_e4m3fn with x_scale (a value
    per row of x) and weight_scale [N].  bias [N] is float32 or 16 bits; residual
    [..., N] has out_dtype (float32, float16 or bfloat16; by default x's type, or
    bfloat16 for 8-bit operands).  `out`, where given, is written and returned; it
    may not overlap the inputs."""
    act = _act(activation)
    M, K = _check_rows(x, "x", _OPERAND)
    dev = x.device
    N = _check_weight(weight, "weight", x.dtype, K, dev)
    if x_scale is not None or weight_scale is not None or x.dtype == _E4M3:
        _check_scales(x, (weight,), x_scale, (weight_scale,), M)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype == _E4M3 else x.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32, float16 or bfloat16")
    shape = (M, N) if x.dim() == 2 else (*x.shape[:-1], N)
    if bias is not None:
        _check(bias, "bias", _FLOAT, (N,), dev)
    if residual is not None:
        _check(residual, "residual", (out_dtype,), shape, dev)
    y = _out(out, shape, out_dtype, dev)
    x, weight = _aligned(x), _aligned(weight)
    if residual is not None:
        residual = _aligned(residual, 32)
    t, to = _TYPE[x.dtype], _TYPE[out_dtype]
    ws, wp, wn = _workspace(_bytes("pdr_linear_workspace_bytes", M, N, K, t, to, residual is not None), dev)
    _call("pdr_linear_fwd", dev, x.data_ptr(), weight.data_ptr(), t, _ptr(x_scale), _ptr(weight_scale),
          _ptr(bias), 0 if bias is None else _TYPE[bias.dtype], _ptr(residual), act, M, N, K,
          y.data_ptr(), to, wp, wn)
    return y if out is None or y is out else out.copy_(y)


def linear_bwd(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               activation: str = "none", need: tuple = (True, True, True)):
    """(dL/dx, dL/dweight, dL/dbias) of linear_fwd from grad = dL/dy [..., N].

    grad is float32, float16 or bfloat16; the gradients have the types of x,
    weight and bias.  `need` says which are wanted (None in the others' place;
    without a bias there is no dL/dbias).  dL/dresidual is grad itself."""
    act = _act(activation)
    M, K = _check_rows(x, "x", _HALF)
    dev = x.device
    N = _check_weight(weight, "weight", x.dtype, K, dev)
    _check(grad, "grad", _FLOAT, torch.Size((*x.shape[:-1], N)), dev)
    if bias is not None:
        _check(bias, "bias", _FLOAT, (N,), dev)
    dx = torch.empty_like(x) if need[0] else None
    dw = torch.empty_like(weight) if need[1] else None
    db = torch.empty_like(bias) if bias is not None and need[2] else None
    grad, x, weight = _aligned(grad, 32), _aligned(x), _aligned(weight)
    t, tg = _TYPE[x.dtype], _TYPE[grad.dtype]
    ws, wp, wn = _workspace(_bytes("pdr_linear_bwd_workspace_bytes", M, N, K, t, tg, act), dev)
    _call("pdr_linear_bwd", dev, grad.data_ptr(), tg, x.data_ptr(), weight.data_ptr(), t, _ptr(bias),
          0 if bias is None else _TYPE[bias.dtype], act, M, N, K, _ptr(dx), _ptr(dw), _ptr(db), wp, wn)
    return dx, dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation, out_dtype):
        ctx.save_for_backward(x, weight, bias)
        ctx.activation = activation
        return linear_fwd(x, weight, bias, residual, activation, out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        x, weight, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = linear_bwd(grad.contiguous(), x, weight, bias, ctx.activation, need[:3])
        return dx, dw, db, grad if need[3] else None, None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, activation: str = "none",
           out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Differentiable linear_fwd for 16-bit x and weight."""
    return _Linear.apply(x.contiguous(), weight.contiguous(), None if bias is None else bias.contiguous(),
                         None if residual is None else residual.contiguous(), activation, out_dtype)


def _check_gated(x, w_gate, w_up, dtypes):
    M, D = _check_rows(x, "x", dtypes)
    F = _check_weight(w_gate, "w_gate", x.dtype, D, x.device)
    _check(w_up, "w_up", (x.dtype,), w_gate.shape, x.device)
    return M, D, F


def gated_fwd(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu",
              out_dtype: torch.dtype | None = None, x_scale: torch.Tensor | None = None,
              gate_scale: torch.Tensor | None = None, up_scale: torch.Tensor | None = None,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """act(x Wg^T) * (x Wu^T): h [..., F] from x [..., D] and two weights [F, D].

    float16, bfloat16, or float8_e4m3fn with the scales (x's rows, [F], [F]).
    out_dtype: x's type, or bfloat16 for 8-bit operands, unless given.  `out` as in
    linear_fwd."""
    act = _act(activation)
    M, D, F = _check_gated(x, w_gate, w_up, _OPERAND)
    dev = x.device
    if x_scale is not None or gate_scale is not None or up_scale is not None or x.dtype == _E4M3:
        _check_scales(x, (w_gate, w_up), x_scale, (gate_scale, up_scale), M)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype == _E4M3 else x.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32, float16 or bfloat16")
    h = _out(out, (M, F) if x.dim() == 2 else (*x.shape[:-1], F), out_dtype, dev)
    x, w_gate, w_up = _aligned(x), _aligned(w_gate), _aligned(w_up)
    t, to = _TYPE[x.dtype], _TYPE[out_dtype]
    ws, wp, wn = _workspace(_bytes("pdr_gated_workspace_bytes", M, D, F, t, to), dev)
    _call("pdr_gated_fwd", dev, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), t, _ptr(x_scale),
          _ptr(gate_scale), _ptr(up_scale), act, M, D, F, h.data_ptr(), to, wp, wn)
    return h if out is None or h is out else out.copy_(h)


def gated_bwd(grad: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
              activation: str = "silu", need: tuple = (True, True)):
    """(dL/dx, dL/dw_gate, dL/dw_up) of gated_fwd from grad = dL/dh [..., F] of x's type.

    `need`: whether dL/dx, and whether the weights' gradients, are wanted."""
    act = _act(activation)
    M, D, F = _check_gated(x, w_gate, w_up, _HALF)
    dev = x.device
    _check(grad, "grad", (x.dtype,), torch.Size((*x.shape[:-1], F)), dev)
    dx = torch.empty_like(x) if need[0] else None
    dg = torch.empty_like(w_gate) if need[1] else None
    du = torch.empty_like(w_up) if need[1] else None
    grad, x, w_gate, w_up = _aligned(grad, 32), _aligned(x), _aligned(w_gate), _aligned(w_up)
    t = _TYPE[x.dtype]
    ws, wp, wn = _workspace(_bytes("pdr_gated_bwd_workspace_bytes", M, D, F, t), dev)
    _call("pdr_gated_bwd", dev, grad.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), t, act,
          M, D, F, _ptr(dx), _ptr(dg), _ptr(du), wp, wn)
    return dx, dg, du


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation):
        ctx.save_for_backward(x, w_gate, w_up)
        ctx.activation = activation
        return gated_fwd(x, w_gate, w_up, activation)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        n = ctx.needs_input_grad
        dx, dg, du = gated_bwd(grad.contiguous(), *ctx.saved_tensors, ctx.activation, (n[0], n[1] or n[2]))
        return dx, dg, du, None


def gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu") -> torch.Tensor:
    """Differentiable gated_fwd for 16-bit x and weights."""
    return _Gated.apply(x.contiguous(), w_gate.contiguous(), w_up.contiguous(), activation)


def _check_norm(x, weight):
    M, D = _check_rows(x, "x", _FLOAT)
    _check(weight, "weight", (x.dtype, torch.float32), (D,), x.device)
    return M, D


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                 eps: float = 1e-6, out_dtype: torch.dtype | None = None):
    """(y, s, scale): s = x + residual (x itself without one), y = s / sqrt(mean s^2 + eps) * weight.

    x [..., D] float32, float16 or bfloat16, residual like x, weight [D] of x's
    type or float32.  out_dtype float8_e4m3fn gives y in 8 bits and scale [...],
    y * scale[..., None] being the value; otherwise y has x's type and scale is None."""
    M, D = _check_norm(x, weight)
    dev = x.device
    if residual is not None:
        _check(residual, "residual", (x.dtype,), x.shape, dev)
    if out_dtype is None:
        out_dtype = x.dtype
    if out_dtype not in (x.dtype, _E4M3):
        raise ValueError("out_dtype must be x's type or float8_e4m3fn")
    y = _new(x.shape, out_dtype, dev)
    s = x if residual is None else torch.empty_like(x)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev) if out_dtype == _E4M3 else None
    rows = _aligned(x)
    residual = None if residual is None else _aligned(residual)
    _call("pdr_rms_norm_fwd", dev, rows.data_ptr(), _ptr(residual), _TYPE[x.dtype], weight.data_ptr(),
          _TYPE[weight.dtype], eps, M, D, None if residual is None else s.data_ptr(),
          y.data_ptr(), _TYPE[out_dtype], _ptr(scale))
    return y, s, scale


def rms_norm_bwd(grad: torch.Tensor, s: torch.Tensor, weight: torch.Tensor, grad_s: torch.Tensor | None = None,
                 eps: float = 1e-6, need: tuple = (True, True)):
    """(dL/dx, dL/dweight) from grad = dL/dy, the norm's input s and grad_s = dL/ds of s's other uses.

    grad and grad_s are like s; dL/dx is the residual's gradient too."""
    M, D = _check_norm(s, weight)
    dev = s.device
    _check(grad, "grad", (s.dtype,), s.shape, dev)
    if grad_s is not None:
        _check(grad_s, "grad_s", (s.dtype,), s.shape, dev)
    dx = torch.empty_like(s) if need[0] else None
    dw = torch.empty_like(weight) if need[1] else None
    grad, s, grad_s = _aligned(grad), _aligned(s), None if grad_s is None else _aligned(grad_s)
    ws, wp, wn = _workspace(_bytes("pdr_rms_norm_bwd_workspace_bytes", M, D), dev) if need[1] else (None, None, 0)
    _call("pdr_rms_norm_bwd", dev, grad.data_ptr(), s.data_ptr(), _TYPE[s.dtype], weight.data_ptr(),
          _TYPE[weight.dtype], _ptr(grad_s), eps, M, D, _ptr(dx), _ptr(dw), wp, wn)
    return dx, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, s, _ = rms_norm_fwd(x, weight, residual, eps)
        ctx.save_for_backward(s, weight)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, s)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_s=None):
        s, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        if grad is None:  # only the sum was used
            dx, dw = grad_s, torch.zeros_like(weight) if need[1] else None
        else:
            dx, dw = rms_norm_bwd(grad.contiguous(), s, weight, None if grad_s is None else grad_s.contiguous(),
                                  ctx.eps, (need[0] or need[2], need[1]))
        return dx if need[0] else None, dw, dx if need[2] else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """Differentiable rms_norm_fwd: y, or (y, s) with a residual."""
    return _RmsNorm.apply(x.contiguous(), weight.contiguous(),
                          None if residual is None else residual.contiguous(), eps)


def quantize_rows(x: torch.Tensor):
    """(q, scale): x [..., D] as float8_e4m3fn and one fp32 scale per row, q * scale[..., None] ~ x."""
    M, D = _check_rows(x, "x", _FLOAT)
    q = torch.empty(x.shape, dtype=_E4M3, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    x = _aligned(x)
    _call("pdr_quantize_rows", x.device, x.data_ptr(), _TYPE[x.dtype], M, D, q.data_ptr(), scale.data_ptr())
    return q, scale


@dataclass
class AdapterWeights:
    """Weights of adapter(): width D, hidden width F, 5 + C parameters per Gaussian."""
    norm_in: torch.Tensor    # [D]
    gate: torch.Tensor       # [F, D]
    up: torch.Tensor         # [F, D]
    down: torch.Tensor       # [D, F]
    norm_out: torch.Tensor   # [D]
    head: torch.Tensor       # [5 + C, D]
    head_bias: torch.Tensor  # [5 + C]
    gate_scale: torch.Tensor | None = None  # [F], of 8-bit gate and up (inference)
    up_scale: torch.Tensor | None = None

    def quantized(self) -> "AdapterWeights":
        """The same weights with gate and up in 8 bits, for inference."""
        gate, gs = quantize_rows(self.gate.detach().contiguous())
        up, us = quantize_rows(self.up.detach().contiguous())
        return replace(self, gate=gate, up=up, gate_scale=gs, up_scale=us)


def adapter(features: torch.Tensor, weights: AdapterWeights, base: torch.Tensor,
            update: torch.Tensor | None = None, activation: str = "silu", eps: float = 1e-6) -> torch.Tensor:
    """Gaussian parameters [B, N, 5 + C] (fp32, for render()) from features [B, N, D].

        s = features + update,  h = gated(rms_norm(s)),  t = h Wdown^T + s,
        params = rms_norm(t) Whead^T + head_bias + base

    base [B, N, 5 + C] fp32 holds the parameters that the head corrects (means on
    a grid, for instance); update (like features, or None) is the predictor's last
    residual update.  Differentiable in everything; with 8-bit gate and up
    (AdapterWeights.quantized) the normalised features go to 8 bits too, and
    there are no gradients."""
    w = weights
    if w.gate.dtype == _E4M3:
        with torch.no_grad():
            n, s, scale = rms_norm_fwd(features.contiguous(), w.norm_in.contiguous(),
                                       None if update is None else update.contiguous(), eps, out_dtype=_E4M3)
            h = gated_fwd(n, w.gate, w.up, activation, features.dtype, scale, w.gate_scale, w.up_scale)
            t = linear(h, w.down, residual=s)
            return linear(rms_norm(t, w.norm_out, eps=eps), w.head, w.head_bias, base, out_dtype=torch.float32)
    if update is None:
        s, n = features, rms_norm(features, w.norm_in, eps=eps)
    else:
        n, s = rms_norm(features, w.norm_in, update, eps)
    t = linear(gated(n, w.gate, w.up, activation), w.down, residual=s)
    return linear(rms_norm(t, w.norm_out, eps=eps), w.head, w.head_bias, base, out_dtype=torch.float32)


def check_wait_error(device=None) -> None:
    """Synchronise the current stream and raise if a product's kernel gave up a wait since the last call.

    A wait that gives up (after seconds) leaves wrong results.  linear, gated and adapter calls
    made on that device after the kernel's end raise too, without synchronising, until
    this call has reported it; this call waits for the work so far."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.index is None:
        device = torch.device(device.type, torch.cuda.current_device())
    _call("pdr_check_wait_error", device)
