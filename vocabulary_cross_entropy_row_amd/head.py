"""The operators around the cross-entropy: norm, matrix product with an epilogue, rules on logits.

Argument marshalling for the C entry points of the same names (include/lce.h), and the autograd
forms.  Like the rest of the binding, every function runs on ``stream`` (default: the current
stream of the first argument's device) and allocates what is not passed in with that stream
current.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from . import LCE_BF16, LCE_E4M3, LCE_F32, _buf, _check, _on_gpu, _ptr, _torch_stream, lib

_CODES = {torch.float32: LCE_F32, torch.bfloat16: LCE_BF16, torch.float8_e4m3fn: LCE_E4M3}
# The current stream's handle, without the stream object around it (3 us of a 10 us call).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call_stream(fn):
    """Runs a binding function with its call stream and device current; the function receives the
    stream's handle as ``stream``.  The common call -- no stream named, tensors of the current
    device -- switches nothing."""
    name = fn.__code__.co_varnames[0]   # of the operand whose device it is, which may come by name

    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not (isinstance(first, torch.Tensor) and first.is_cuda):
            return fn(*args, stream=0, **kw)   # the function's own checks raise
        device = first.device
        if stream is None and device.index == torch.cuda.current_device():
            return fn(*args, stream=_current_stream(device.index), **kw)
        st = _torch_stream(stream, device)
        with torch.cuda.device(device), torch.cuda.stream(st):
            return fn(*args, stream=st.cuda_stream, **kw)
    return wrapper


def _float_code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None or code == LCE_E4M3:
        raise TypeError(f"{name} must be bfloat16 or float32 (got {t.dtype})")
    return code


def _rows(t, name: str, dtype, n: int, width: int, device, required: bool = False) -> int:
    """Checks a [n, width] operand with unit column stride; returns its row stride."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return width
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.shape != (n, width):
        raise ValueError(f"{name} must be [{n}, {width}] (got {list(t.shape)})")
    row, column = t.stride()
    if column != 1 and width > 1:
        raise ValueError(f"{name} must have unit column stride")
    return row if n > 1 else width


# ---- root-mean-square norm -------------------------------------------------------------------

@dataclass
class NormResult:
    y: object       # [n, H], the rows' type or e4m3
    sum: object     # [n, H] x + residual, or None without a residual
    rstd: object    # fp32 [n], or None
    scale: object   # fp32 [n] with an e4m3 y, or None


def _norm_weight(weight, H: int, device):
    if weight is None:
        return LCE_F32
    if not torch.is_tensor(weight):
        raise TypeError("weight must be a torch tensor")
    if weight.device != device:
        raise ValueError(f"weight must be on {device} (got {weight.device})")
    if weight.dim() != 1 or weight.shape[0] != H or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{H}] tensor")
    return _float_code(weight, "weight")


@_call_stream
def lce_rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, out_dtype=None,
                 want_rstd: bool = False, y=None, sum_out=None, rstd=None, scale=None, stream=None) -> NormResult:
    """y = s / sqrt(mean(s^2) + eps) * (weight + weight_offset) of the rows of s = x + residual (in x's
    type; x without a residual).  ``x`` is a [n, H] view with unit column stride.  With ``out_dtype``
    torch.float8_e4m3fn, y holds y / scale with one scale per row.  Outputs not passed in are
    allocated; ``sum_out`` may be ``x`` or ``residual`` itself."""
    if not torch.is_tensor(x) or x.dim() != 2:
        raise ValueError("x must be a 2-D tensor")
    dev = _on_gpu(x, "x")
    n, H = x.shape
    code = _float_code(x, "x")
    ldx = _rows(x, "x", x.dtype, n, H, dev)
    ldr = _rows(residual, "residual", x.dtype, n, H, dev)
    wcode = _norm_weight(weight, H, dev)
    if out_dtype is None:
        out_dtype = x.dtype if y is None else y.dtype
    ycode = _CODES.get(out_dtype)
    if out_dtype != x.dtype and ycode != LCE_E4M3:
        raise TypeError(f"out_dtype must be {x.dtype} or torch.float8_e4m3fn (got {out_dtype})")
    ldy = lds = H
    plain = ldx == H   # x is contiguous: its like is the cheapest allocation
    if y is not None:
        ldy = _rows(y, "y", out_dtype, n, H, dev)
    elif plain and out_dtype == x.dtype:
        y = torch.empty_like(x)
    else:
        y = torch.empty((n, H), dtype=out_dtype, device=dev)
    if sum_out is not None:
        lds = _rows(sum_out, "sum_out", x.dtype, n, H, dev)
    elif residual is not None:
        sum_out = torch.empty_like(x) if plain else torch.empty((n, H), dtype=x.dtype, device=dev)
    if rstd is None and want_rstd:
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
    if ycode != LCE_E4M3:
        scale = None
    elif scale is None:
        scale = torch.empty(n, dtype=torch.float32, device=dev)
    _buf(rstd, "rstd", torch.float32, n, dev)
    _buf(scale, "scale", torch.float32, n, dev)
    _check(lib().lce_rms_norm(x.data_ptr(), ldx, code, _ptr(residual), ldr, _ptr(weight), wcode, float(weight_offset),
                              float(eps), n, H, _ptr(sum_out), lds, y.data_ptr(), ldy, ycode, _ptr(scale), _ptr(rstd),
                              stream))
    return NormResult(y, sum_out, rstd, scale)


def lce_rms_norm_workspace_bytes(n: int, H: int) -> int:
    return int(lib().lce_rms_norm_workspace_bytes(int(n), int(H)))


def _norm_backward(gy, ldg, s, lds, code, n, H, weight, wcode, offset, rstd, gs, ldgs, gx, ldgx, gw, gwcode, workspace,
                   stream):
    """The call, its operands checked: allocates the workspace that a weight's gradient needs."""
    bytes_ = 0
    if gw is not None:
        bytes_ = lib().lce_rms_norm_workspace_bytes(n, H)
        if workspace is None:   # clobbered by the call
            workspace = torch.empty(max(bytes_, 1), dtype=torch.uint8, device=s.device)
    _check(lib().lce_rms_norm_backward(gy.data_ptr(), ldg, s.data_ptr(), lds, code, _ptr(weight), wcode, offset,
                                       rstd.data_ptr(), _ptr(gs), ldgs, n, H, gx.data_ptr(), ldgx, _ptr(gw), gwcode,
                                       _ptr(workspace), bytes_, stream))


@_call_stream
def lce_rms_norm_backward(grad_y, s, weight, rstd, *, grad_sum=None, weight_offset: float = 0.0, grad_x=None,
                          grad_weight=None, want_grad_weight: bool = True, workspace=None, stream=None):
    """(grad_x, grad_weight) of lce_rms_norm from its ``s`` (the sum; x without a residual) and ``rstd``.
    grad_x is the gradient of x and of the residual alike; grad_weight has the weight's type (None
    without a weight or with ``want_grad_weight`` false)."""
    if not torch.is_tensor(s) or s.dim() != 2:
        raise ValueError("s must be a 2-D tensor")
    dev = _on_gpu(grad_y, "grad_y")
    n, H = s.shape
    code = _float_code(s, "s")
    ldg = _rows(grad_y, "grad_y", s.dtype, n, H, dev)
    lds = _rows(s, "s", s.dtype, n, H, dev)
    ldgs = _rows(grad_sum, "grad_sum", s.dtype, n, H, dev)
    wcode = _norm_weight(weight, H, dev)
    _buf(rstd, "rstd", torch.float32, n, dev, required=True)
    if grad_x is None:
        grad_x = torch.empty((n, H), dtype=s.dtype, device=dev)
    ldgx = _rows(grad_x, "grad_x", s.dtype, n, H, dev)
    gwcode = LCE_F32
    if weight is None or not want_grad_weight:
        grad_weight = None
    else:
        if grad_weight is None:
            grad_weight = torch.empty(H, dtype=weight.dtype, device=dev)
        gwcode = _float_code(grad_weight, "grad_weight")
        _buf(grad_weight, "grad_weight", grad_weight.dtype, H, dev)
        if workspace is not None:
            _buf(workspace, "workspace", torch.uint8, lce_rms_norm_workspace_bytes(n, H), dev)
    _norm_backward(grad_y, ldg, s, lds, code, n, H, weight, wcode, float(weight_offset), rstd, grad_sum, ldgs, grad_x,
                   ldgx, grad_weight, gwcode, workspace, stream)
    return grad_x, grad_weight


def _rows_of(t, H: int):
    """t with its leading dimensions as rows of H, unit column stride, no two rows overlapping."""
    if t.dim() != 2:
        t = t.reshape(-1, H)
    row, column = t.stride()
    if (H > 1 and column != 1) or (t.shape[0] > 1 and row < H):
        t = t.contiguous()
    return t


def _ld(rows) -> int:
    return rows.stride(0) if rows.shape[0] > 1 else rows.shape[1]


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, offset):
        _on_gpu(x, "x")
        if x.dim() < 1:
            raise ValueError("x must have at least one dimension")
        H = x.shape[-1]
        x2, r2, total, sum2 = _rows_of(x, H), None, None, None
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        if residual is not None:
            if residual.shape != x.shape:
                raise ValueError(f"residual must have the shape of x, {list(x.shape)} (got {list(residual.shape)})")
            r2 = _rows_of(residual, H)
            total = torch.empty_like(y)
            sum2 = _rows_of(total, H)
        rstd = lce_rms_norm(x2, weight, residual=r2, eps=eps, weight_offset=offset, want_rstd=True, y=_rows_of(y, H),
                            sum_out=sum2).rstd
        ctx.set_materialize_grads(False)
        ctx.offset = offset
        if residual is None:
            ctx.save_for_backward(x, weight, rstd)
            return y
        ctx.save_for_backward(total, weight, rstd)
        return y, total

    @staticmethod
    def backward(ctx, gy, gs=None):
        return (_norm_backward_twice if torch.is_grad_enabled() else _norm_backward_once)(ctx, gy, gs)


def _norm_backward_once(ctx, gy, gs):
    """The backward on autograd's own thread, where every interpreted line costs twice what it does on
    the caller's.  Autograd hands gradients of the outputs' shape, type and device, on the stream the
    forward ran on and with its device current; the saved tensors were checked in the forward."""
    s, weight, rstd = ctx.saved_tensors
    need_x, need_w, need_r = ctx.needs_input_grad[:3]
    if gy is None:   # nothing came through the norm
        return (gs if need_x else None), None, (gs if need_r else None), None, None
    H = s.shape[-1]
    lds = ldg = ldgs = H
    rows = s
    if not (s.is_contiguous() and gy.is_contiguous() and (gs is None or gs.is_contiguous())):
        rows, gy = _rows_of(s, H), _rows_of(gy, H)
        lds, ldg = _ld(rows), _ld(gy)
        if gs is not None:
            gs = _rows_of(gs, H)
            ldgs = _ld(gs)
    gx = torch.empty_like(s, memory_format=torch.contiguous_format)
    gw = None if weight is None or not need_w else torch.empty_like(weight)
    code = _CODES[s.dtype]
    wcode = code if weight is None else _CODES[weight.dtype]
    _norm_backward(gy, ldg, rows, lds, code, s.numel() // H, H, weight, wcode, ctx.offset, rstd, gs, ldgs, gx, H, gw,
                   wcode, None, _current_stream(s.device.index))
    return (gx if need_x else None), gw, (gx if need_r else None), None, None


# with create_graph: first-order gradients, and an error for those of higher order
_norm_backward_twice = torch.autograd.function.once_differentiable(_norm_backward_once)


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """Autograd form of the norm over the last dimension of ``x``.

    Without a residual returns y; with one (x's shape and type) returns (y, sum), sum = x + residual
    being the stream that goes on.  Gradients: x, weight and residual; the gradient that reaches
    ``sum`` is added in the same kernel.  Under capture, what ``linear`` says of it holds here too.
    """
    return _RmsNorm.apply(x, weight, residual, float(eps), float(weight_offset))


# ---- matrix product with an epilogue ---------------------------------------------------------

_MAX_LD = (1 << 23) - 512   # elements between the rows of a bf16 operand, as the product reads them


def _operand_rows(x, K: int):
    """x's rows as the product reads them; copied where they lie too far apart."""
    rows = _rows_of(x, K)
    return rows.contiguous() if _ld(rows) > _MAX_LD else rows


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


@dataclass
class LinearResult:
    out: object      # [n, M]
    preact: object   # bf16 [n, M], or None


@dataclass
class LinearGrads:
    grad_x: object        # bf16 [n, K], or None
    grad_weight: object   # [M, K], or None
    grad_bias: object     # [M], or None


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"unknown activation {name!r} (one of {', '.join(ACTIVATIONS)})")
    return ACTIVATIONS[name]


def _operand(t, name: str, dtype, width: int | None, device):
    """Checks a 2-D operand of the product; returns (rows, row stride)."""
    if not torch.is_tensor(t) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape[0], _rows(t, name, dtype, t.shape[0], t.shape[1] if width is None else width, device)


def lce_linear_workspace_bytes(n: int, K: int, M: int, e4m3: bool = False) -> int:
    return int(lib().lce_linear_workspace_bytes(int(n), int(K), int(M), LCE_E4M3 if e4m3 else LCE_BF16))


def lce_linear_backward_workspace_bytes(n: int, K: int, M: int) -> int:
    return int(lib().lce_linear_backward_workspace_bytes(int(n), int(K), int(M)))


@_call_stream
def lce_linear(x, weight, *, bias=None, activation: str = "none", residual=None, scale_x=None, scale_w=None,
               out_dtype=None, want_preact: bool = False, out=None, preact=None, workspace=None,
               stream=None) -> LinearResult:
    """act(x weight^T + bias) + residual for x [n, K] and weight [M, K], both bfloat16 or both
    float8_e4m3fn (then with ``scale_x`` [n] and ``scale_w`` [M], as lce_rms_norm's e4m3 output has).
    The output is bfloat16, or (bfloat16 operands) float32 with ``out_dtype``; a residual has its
    type.  ``want_preact``
    keeps the activation's input in bf16 for the backward.  Outputs not passed in are allocated."""
    if not torch.is_tensor(x) or x.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError("x must be a bfloat16 or float8_e4m3fn tensor")
    dev = _on_gpu(x, "x")
    act = _activation(activation)
    n, ldx = _operand(x, "x", x.dtype, None, dev)
    K = x.shape[1]
    M, ldw = _operand(weight, "weight", x.dtype, K, dev)
    e4m3 = x.dtype == torch.float8_e4m3fn
    if not e4m3 and (scale_x is not None or scale_w is not None):
        raise ValueError("scales go with float8_e4m3fn operands")
    _buf(scale_x, "scale_x", torch.float32, n, dev)
    _buf(scale_w, "scale_w", torch.float32, M, dev)
    bcode = LCE_F32
    if bias is not None:
        bcode = _float_code(bias, "bias")
        if bias.dim() != 1 or bias.shape[0] != M:
            raise ValueError(f"bias must be [{M}] (got {list(bias.shape)})")
        _buf(bias, "bias", bias.dtype, M, dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
    ldo = ldp = M
    if out is not None:
        ldo = _rows(out, "out", out_dtype, n, M, dev)
    else:
        out = torch.empty((n, M), dtype=out_dtype, device=dev)
    if preact is not None:
        ldp = _rows(preact, "preact", torch.bfloat16, n, M, dev)
    elif want_preact:
        preact = torch.empty((n, M), dtype=torch.bfloat16, device=dev)
    ldr = M if residual is None else _rows(residual, "residual", out_dtype, n, M, dev)
    need = lce_linear_workspace_bytes(n, K, M, e4m3)
    if workspace is not None:
        _buf(workspace, "workspace", torch.uint8, need, dev)
    elif need:   # clobbered by the call
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().lce_linear(x.data_ptr(), ldx, weight.data_ptr(), ldw, LCE_E4M3 if e4m3 else LCE_BF16, _ptr(scale_x),
                            _ptr(scale_w), _ptr(bias), bcode, act, _ptr(residual), ldr, n, K, M, out.data_ptr(), ldo,
                            _CODES[out_dtype], _ptr(preact), ldp, _ptr(workspace),
                            0 if workspace is None else workspace.numel(), stream))
    return LinearResult(out, preact)


@_call_stream
def lce_linear_backward(grad_out, x, weight, *, activation: str = "none", preact=None, want_grad_x: bool = True,
                        want_grad_weight: bool = True, want_grad_bias: bool = False, grad_weight_dtype=None,
                        grad_bias_dtype=None, grad_x=None, grad_weight=None, grad_bias=None, workspace=None,
                        stream=None) -> LinearGrads:
    """Gradients of lce_linear (bfloat16 operands) from grad_out [n, M] and, with an activation, the
    forward's ``preact``; the residual's gradient is grad_out itself.  grad_x is bf16, grad_weight and
    grad_bias bf16 unless another type is named."""
    if not torch.is_tensor(x):
        raise TypeError("x must be a torch tensor")
    dev = _on_gpu(grad_out, "grad_out")
    act = _activation(activation)
    n, ldx = _operand(x, "x", torch.bfloat16, None, dev)
    K = x.shape[1]
    M, ldw = _operand(weight, "weight", torch.bfloat16, K, dev)
    gcode = _float_code(grad_out, "grad_out")
    ldg = _rows(grad_out, "grad_out", grad_out.dtype, n, M, dev)
    ldp = _rows(preact, "preact", torch.bfloat16, n, M, dev, required=act != 0)
    if grad_x is None and want_grad_x:
        grad_x = torch.empty((n, K), dtype=torch.bfloat16, device=dev)
    ldgx = _rows(grad_x, "grad_x", torch.bfloat16, n, K, dev)
    if grad_weight is None and want_grad_weight:
        grad_weight = torch.empty((M, K), dtype=grad_weight_dtype or torch.bfloat16, device=dev)
    wcode = bcode = LCE_F32
    if grad_weight is not None:
        wcode = _float_code(grad_weight, "grad_weight")
        _buf(grad_weight, "grad_weight", grad_weight.dtype, M * K, dev)
    if grad_bias is None and want_grad_bias:
        grad_bias = torch.empty(M, dtype=grad_bias_dtype or torch.bfloat16, device=dev)
    if grad_bias is not None:
        bcode = _float_code(grad_bias, "grad_bias")
        _buf(grad_bias, "grad_bias", grad_bias.dtype, M, dev)
    need = lce_linear_backward_workspace_bytes(n, K, M)
    if workspace is not None:
        _buf(workspace, "workspace", torch.uint8, need, dev)
    _linear_backward(grad_out, ldg, gcode, x, ldx, weight, ldw, preact if act else None, ldp, act, n, K, M, grad_x, ldgx,
                     grad_weight, wcode, grad_bias, bcode, workspace, stream)
    return LinearGrads(grad_x, grad_weight, grad_bias)


def _linear_backward(g, ldg, gcode, x, ldx, weight, ldw, preact, ldp, act, n, K, M, gx, ldgx, gw, wcode, gb, bcode,
                     workspace, stream):
    """The call, its operands checked: allocates the workspace if there is none."""
    if workspace is None:   # clobbered by the call
        bytes_ = lib().lce_linear_backward_workspace_bytes(n, K, M)
        workspace = torch.empty(max(bytes_, 1), dtype=torch.uint8, device=x.device)
    else:
        bytes_ = workspace.numel()
    _check(lib().lce_linear_backward(g.data_ptr(), ldg, gcode, x.data_ptr(), ldx, weight.data_ptr(), ldw, _ptr(preact), ldp,
                                     act, n, K, M, _ptr(gx), ldgx, _ptr(gw), wcode, _ptr(gb), bcode, workspace.data_ptr(),
                                     bytes_, stream))


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation, differentiate):
        _on_gpu(x, "x")
        if x.dim() < 1 or not torch.is_tensor(weight) or weight.dim() != 2:
            raise ValueError("x must have at least one dimension, and weight two")
        for t, name in ((x, "x"), (weight, "weight")):   # the backward takes them as bf16, unchecked
            if t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be torch.bfloat16 (got {t.dtype})")
        M = weight.shape[0]
        shape = (*x.shape[:-1], M)
        if residual is not None and residual.shape != shape:
            raise ValueError(f"residual must be {list(shape)} (got {list(residual.shape)})")
        wanted = differentiate and any(ctx.needs_input_grad[:3])
        if wanted and M % 8:
            raise ValueError(f"gradients need a weight whose rows are a multiple of 8 (got {M})")
        keep = wanted and _activation(activation) != 0
        out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
        preact = lce_linear(_operand_rows(x, x.shape[-1]), weight, bias=bias, activation=activation,
                            residual=None if residual is None else _rows_of(residual, M), want_preact=keep,
                            out=_rows_of(out, M)).preact
        ctx.save_for_backward(x, weight, preact)
        ctx.activation, ctx.bias_dtype = activation, None if bias is None else bias.dtype
        return out

    @staticmethod
    def backward(ctx, g):
        return (_linear_backward_twice if torch.is_grad_enabled() else _linear_backward_once)(ctx, g)


def _linear_backward_once(ctx, g):   # on autograd's thread, as _norm_backward_once
    x, weight, preact = ctx.saved_tensors
    need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
    gx = gw = gb = None
    if need_x or need_w or need_b:
        M, K = weight.shape
        bcode = LCE_F32
        if need_x:
            gx = torch.empty_like(x, memory_format=torch.contiguous_format)
        if need_w:
            gw = torch.empty_like(weight, memory_format=torch.contiguous_format)
        if need_b:
            gb = torch.empty(M, dtype=ctx.bias_dtype, device=x.device)
            bcode = _CODES[ctx.bias_dtype]
        rows, g2, ldx, ldg = x, g, K, M
        if not (x.is_contiguous() and g.is_contiguous()):
            rows, g2 = _operand_rows(x, K), _rows_of(g, M)
            ldx, ldg = _ld(rows), _ld(g2)
        _linear_backward(g2, ldg, LCE_BF16, rows, ldx, weight, _ld(weight), preact, M, ACTIVATIONS[ctx.activation],
                         x.numel() // K, K, M, gx, K, gw, LCE_BF16, gb, bcode, None, _current_stream(x.device.index))
    return gx, gw, gb, (g if need_r else None), None, None


_linear_backward_twice = torch.autograd.function.once_differentiable(_linear_backward_once)


def linear(x, weight, bias=None, *, activation: str = "none", residual=None):
    """Autograd form of the product over the last dimension of ``x``: act(x weight^T + bias) + residual,
    all of x, weight and residual bfloat16 (bias bfloat16 or float32), the output bfloat16 with x's
    leading dimensions.  Gradients have their inputs' types; sums are fp32.  Where x, weight or bias asks
    for one, weight must have a multiple of 8 rows.

    Captured into a graph, forward and backward belong to one capture, and no graph of the same leaves
    built outside it may be alive: autograd would wait on the stream that one was built on.
    """
    # inside no_grad needs_input_grad still says what the tensors ask for, and inside forward grad is off
    return _Linear.apply(x, weight, bias, residual, activation, torch.is_grad_enabled())


# ---- rules on logits -------------------------------------------------------------------------

def _ids(t, name: str, n: int, device):
    """Checks a [n, L] list of token ids (int32 or int64); returns (row stride, length).  A row stride
    of 0 (one list expanded over the rows) is kept."""
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{name} must be int32 or int64 (got {t.dtype})")
    return _list(t, name, n)


def _list(t, name: str, n: int):
    if t.dim() != 2 or t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}, length] (got {list(t.shape)})")
    L = t.shape[1]
    if L > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return (t.stride(0) if n > 1 else L), L


@_call_stream
def lce_logits_process(logits, *, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
                       frequency=None, bias_ids=None, bias_values=None, temperature=None, allowed=None,
                       mask_rows=None, mask_value: float = float("-inf"), softcap: float = 0.0, out=None, stream=None):
    """The rules a serving step puts on ``logits`` ([n, V] view, unit column stride) before a token is
    drawn, in one pass: softcap, penalties for the tokens of ``history`` ([n, L] ids; the first
    ``prompt_lens`` of a row's ``history_lens`` are its prompt), ``bias_values`` at ``bias_ids`` ([n, B],
    the last entry of a token counts), ``temperature`` and the grammar masks ``allowed`` (int32 [masks,
    ceil(V / 32)], one bit per token; ``mask_rows`` names each row's mask, -1 none).  repetition,
    presence, frequency and temperature are fp32 [n].  Writes to ``out``, or in place, and returns it;
    lce_ce_argmax reads it from there, and with ``mask_value`` -1e4 (the losses need finite logits)
    lce_ce_stats and lce_ce_combine."""
    if not torch.is_tensor(logits) or logits.dim() != 2:
        raise ValueError("logits must be a 2-D view with unit column stride")
    dev = _on_gpu(logits, "logits")
    n, V = logits.shape
    code = _float_code(logits, "logits")
    ldx = _rows(logits, "logits", logits.dtype, n, V, dev)
    if out is None:
        out = logits
    ldo = _rows(out, "out", logits.dtype, n, V, dev)
    ldh = L = ldbi = ldbv = B = ldm = masks = 0
    wide = True
    if history is not None:
        ldh, L = _ids(history, "history", n, dev)
        wide = history.dtype == torch.int64
    elif history_lens is not None or prompt_lens is not None:
        raise ValueError("history_lens and prompt_lens go with history")
    if (bias_ids is None) != (bias_values is None):
        raise ValueError("bias_ids and bias_values go together")
    if bias_ids is not None:
        ldbi, B = _ids(bias_ids, "bias_ids", n, dev)
        if history is not None and bias_ids.dtype != history.dtype:
            raise TypeError("history and bias_ids must have the same type")
        wide = bias_ids.dtype == torch.int64
        if not torch.is_tensor(bias_values) or bias_values.dtype != torch.float32 or bias_values.device != dev:
            raise TypeError(f"bias_values must be a float32 tensor on {dev}")
        ldbv, values = _list(bias_values, "bias_values", n)
        if values != B:
            raise ValueError(f"bias_ids has {B} entries a row, bias_values {values}")
    if allowed is not None:
        if not torch.is_tensor(allowed) or allowed.dtype != torch.int32 or allowed.device != dev:
            raise TypeError(f"allowed must be an int32 tensor on {dev}")
        if allowed.dim() != 2 or allowed.shape[1] < (V + 31) // 32:
            raise ValueError(f"allowed must be [masks, {(V + 31) // 32}] (got {list(allowed.shape)})")
        if allowed.shape[1] > 1 and allowed.stride(1) != 1:
            raise ValueError("allowed must have unit column stride")
        masks = allowed.shape[0]
        ldm = allowed.stride(0) if masks > 1 else allowed.shape[1]
    elif mask_rows is not None:
        raise ValueError("mask_rows goes with allowed")
    for t, name in ((history_lens, "history_lens"), (prompt_lens, "prompt_lens"), (mask_rows, "mask_rows")):
        _buf(t, name, torch.int64, n, dev)
    for t, name in ((repetition, "repetition"), (presence, "presence"), (frequency, "frequency"),
                    (temperature, "temperature")):
        _buf(t, name, torch.float32, n, dev)
    _check(lib().lce_logits_process(logits.data_ptr(), ldx, code, n, V, _ptr(history), ldh, L, _ptr(history_lens),
                                    _ptr(prompt_lens), _ptr(bias_ids), ldbi, _ptr(bias_values), ldbv, B, int(wide),
                                    _ptr(repetition), _ptr(presence), _ptr(frequency), _ptr(temperature),
                                    _ptr(allowed), ldm, masks, _ptr(mask_rows), float(mask_value), float(softcap),
                                    out.data_ptr(), ldo, stream))
    return out
