"""8-bit products with a scale for each block of 128 (the quantiser, the product, the product's training
form), and the orthogonalised update of a weight.

Argument marshalling for the C entry points of the same names (include/lce.h), in the manner of head.py.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import LCE_BF16, LCE_E8M0, LCE_F32, _buf, _check, _on_gpu, _ptr, lib
from .head import (LinearGrads, LinearResult, _CODES, _activation, _call_stream, _current_stream, _float_code, _ld,
                   _operand, _rows, _rows_of)

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_SCALES = {torch.float32: LCE_F32, E8M0: LCE_E8M0}
BLOCKS = {"row": 0, "tile": 1}


@dataclass
class BlocksResult:
    values: object     # e4m3 [n, K], or None
    scale: object      # [n, ceil(K / 128)], or [ceil(n / 128), ceil(K / 128)] for tiles
    values_t: object   # e4m3 [K, n] of the transpose, or None
    scale_t: object


def _blocks(name, what: str) -> int:
    if name not in BLOCKS:
        raise ValueError(f"unknown {what} {name!r} (one of {', '.join(BLOCKS)})")
    return BLOCKS[name]


def _up(v: int, unit: int) -> int:
    return -(-v // unit) * unit


def _scale_shape(n: int, K: int, tile: bool):
    return (-(-n // 128) if tile else n), -(-K // 128)


def _new_values(n: int, K: int, device):
    """(values [n, K], their row stride): rows on 16 bytes."""
    ld = _up(K, 16)
    return torch.empty_strided((n, K), (ld, 1), dtype=E4M3, device=device), ld


def _new_scale(n: int, K: int, tile: bool, dtype, device):
    """(scales, their strides): those of row blocks block by block, for the product reads those of 16 rows together."""
    rows, cols = shape = _scale_shape(n, K, tile)
    order = (cols, 1) if tile else (1, rows)
    return torch.empty_strided(shape, order, dtype=dtype, device=device), *order


def _scale(t, name: str, n: int, K: int, tile: bool, device):
    """Checks the scales of an [n, K] operand; returns (row stride, block stride, code)."""
    shape = _scale_shape(n, K, tile)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    code = _SCALES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or float8_e8m0fnu (got {t.dtype})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    row, col = t.stride()
    return row, col, code


def _outputs(values, scale, names, n: int, K: int, tile: bool, dtype, device):
    """(values, their row stride, scales, their strides): those that the caller brought, checked, and new ones."""
    if values is None:
        values, ld = _new_values(n, K, device)
    else:
        ld = _rows(values, names[0], E4M3, n, K, device)
    if scale is None:
        return values, ld, *_new_scale(n, K, tile, dtype, device)
    *order, code = _scale(scale, names[1], n, K, tile, device)
    if code != _SCALES[dtype]:
        raise TypeError(f"{names[1]} must be {dtype} (got {scale.dtype})")
    return values, ld, scale, *order


@_call_stream
def lce_quantize_blocks(x, *, blocks: str | None = "row", transposed: str | None = None, scale_dtype=None, values=None,
                        scale=None, values_t=None, scale_t=None, stream=None) -> BlocksResult:
    """x [n, K] (bfloat16 or float32, unit column stride) in e4m3 with a scale, a power of two, for each
    block of 128 values of a row (``blocks`` "row") or of 128 x 128 ("tile"); None: only the transpose.
    ``transposed`` asks for the transpose [K, n] in blocks of its own.  Scales are float8_e8m0fnu, or the
    same numbers as float32 with ``scale_dtype``.  Outputs not passed in are allocated, as
    lce_linear_blocks reads them best: rows on 16 bytes, scales of row blocks block by block."""
    if not torch.is_tensor(x) or x.dim() != 2:
        raise ValueError("x must be a 2-D tensor")
    dev = _on_gpu(x, "x")
    n, K = x.shape
    code = _float_code(x, "x")
    ldx = _rows(x, "x", x.dtype, n, K, dev)
    if blocks is None and transposed is None:
        raise ValueError("blocks and transposed are both None: nothing is asked for")
    if blocks is None and (values is not None or scale is not None):
        raise ValueError("values and scale go with blocks")
    if transposed is None and (values_t is not None or scale_t is not None):
        raise ValueError("values_t and scale_t go with transposed")
    if scale_dtype is None:
        first = scale if scale is not None else scale_t
        scale_dtype = first.dtype if torch.is_tensor(first) else E8M0
    if scale_dtype not in _SCALES:
        raise TypeError(f"scale_dtype must be float8_e8m0fnu or float32 (got {scale_dtype})")
    kind = kind_t = ldv = ldvt = s_row = s_col = st_row = st_col = 0
    scode = _SCALES[scale_dtype]
    if blocks is not None:
        kind = _blocks(blocks, "blocks")
        values, ldv, scale, s_row, s_col = _outputs(values, scale, ("values", "scale"), n, K, kind == 1, scale_dtype, dev)
    if transposed is not None:
        kind_t = _blocks(transposed, "transposed")
        values_t, ldvt, scale_t, st_row, st_col = _outputs(values_t, scale_t, ("values_t", "scale_t"), K, n, kind_t == 1,
                                                           scale_dtype, dev)
    _check(lib().lce_quantize_blocks(x.data_ptr(), ldx, code, n, K, _ptr(values), ldv, kind, _ptr(scale), s_row, s_col,
                                     _ptr(values_t), ldvt, kind_t, _ptr(scale_t), st_row, st_col, scode, stream))
    return BlocksResult(values, scale, values_t, scale_t)


def lce_linear_blocks_workspace_bytes(n: int, K: int, M: int) -> int:
    return int(lib().lce_linear_blocks_workspace_bytes(int(n), int(K), int(M)))


def lce_linear_blocks_backward_workspace_bytes(n: int, K: int, M: int) -> int:
    return int(lib().lce_linear_blocks_backward_workspace_bytes(int(n), int(K), int(M)))


@_call_stream
def lce_linear_blocks(x, scale_x, weight, scale_w, *, bias=None, activation: str = "none", residual=None,
                      want_preact: bool = False, out=None, preact=None, workspace=None, stream=None) -> LinearResult:
    """act(x weight^T + bias) + residual for float8_e4m3fn x [n, K] with ``scale_x`` [n, ceil(K / 128)] (row
    blocks) and weight [M, K] with ``scale_w`` [ceil(M / 128), ceil(K / 128)] (tiles), scales float32 or
    float8_e8m0fnu with any strides; the output and a residual are bfloat16.  Rows of x and weight
    start on 16 bytes, as lce_quantize_blocks lays them; K may be any.  ``want_preact`` keeps the
    activation's input in bf16.  Outputs not passed in are allocated."""
    dev = _on_gpu(x, "x")
    act = _activation(activation)
    n, ldx = _operand(x, "x", E4M3, None, dev)
    K = x.shape[1]
    M, ldw = _operand(weight, "weight", E4M3, K, dev)
    if n == 1:   # a single row has no stride
        ldx = _up(K, 16)
    if M == 1:
        ldw = _up(K, 16)
    sx_row, sx_col, sx_code = _scale(scale_x, "scale_x", n, K, False, dev)
    sw_row, sw_col, sw_code = _scale(scale_w, "scale_w", M, K, True, dev)
    bcode = LCE_F32
    if bias is not None:
        bcode = _float_code(bias, "bias")
        if bias.dim() != 1 or bias.shape[0] != M:
            raise ValueError(f"bias must be [{M}] (got {list(bias.shape)})")
        _buf(bias, "bias", bias.dtype, M, dev)
    ldo = ldp = M
    if out is not None:
        ldo = _rows(out, "out", torch.bfloat16, n, M, dev)
    else:
        out = torch.empty((n, M), dtype=torch.bfloat16, device=dev)
    if preact is not None:
        ldp = _rows(preact, "preact", torch.bfloat16, n, M, dev)
    elif want_preact:
        preact = torch.empty((n, M), dtype=torch.bfloat16, device=dev)
    ldr = M if residual is None else _rows(residual, "residual", torch.bfloat16, n, M, dev)
    need = lib().lce_linear_blocks_workspace_bytes(n, K, M)
    if workspace is not None:
        _buf(workspace, "workspace", torch.uint8, need, dev)
    elif need:   # clobbered by the call
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().lce_linear_blocks(x.data_ptr(), ldx, scale_x.data_ptr(), sx_row, sx_col, sx_code, weight.data_ptr(), ldw,
                                   scale_w.data_ptr(), sw_row, sw_col, sw_code, _ptr(bias), bcode, act, _ptr(residual),
                                   ldr, n, K, M, out.data_ptr(), ldo, _ptr(preact), ldp, _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), stream))
    return LinearResult(out, preact)


def _transposed(t, scale, names, K: int, width: int, device):
    """Checks a transposed operand of the backward [K, width] in tiles; returns what the call takes."""
    rows, ld = _operand(t, names[0], E4M3, width, device)
    if rows != K:
        raise ValueError(f"{names[0]} must have {K} rows (got {rows})")
    if K == 1:
        ld = _up(width, 16)
    s_row, s_col, code = _scale(scale, names[1], K, width, True, device)
    if code != LCE_E8M0:
        raise TypeError(f"{names[1]} must be float8_e8m0fnu (got {scale.dtype})")
    return t.data_ptr(), ld, scale.data_ptr(), s_row, s_col


@_call_stream
def lce_linear_blocks_backward(grad_out, xt=None, scale_xt=None, wt=None, scale_wt=None, *, want_grad_bias: bool = False,
                               grad_bias_dtype=None, grad_x=None, grad_weight=None, grad_bias=None, workspace=None,
                               stream=None) -> LinearGrads:
    """Gradients of a product of quantised x [n, K] and weight [M, K] from grad_out [n, M] (bfloat16 or
    float32), straight through the operands' rounding: grad_weight with ``xt``, ``scale_xt`` (the transposed
    x in tiles, ``values_t`` and ``scale_t`` of lce_quantize_blocks) and grad_x with ``wt``, ``scale_wt`` (the
    transposed weight in tiles).  grad_x and grad_weight are bf16, grad_bias too unless another type is named."""
    dev = _on_gpu(grad_out, "grad_out")
    if grad_out.dim() != 2:
        raise ValueError("grad_out must be a 2-D tensor")
    n, M = grad_out.shape
    gcode = _float_code(grad_out, "grad_out")
    ldg = _rows(grad_out, "grad_out", grad_out.dtype, n, M, dev)
    if xt is None and wt is None:
        raise ValueError("xt (for grad_weight) or wt (for grad_x) is required")
    if not torch.is_tensor(xt if xt is not None else wt) or (xt if xt is not None else wt).dim() != 2:
        raise ValueError("xt and wt must be 2-D tensors")
    K = (xt if xt is not None else wt).shape[0]
    none = (None, 0, None, 0, 0)
    x_args = none if xt is None else _transposed(xt, scale_xt, ("xt", "scale_xt"), K, n, dev)
    w_args = none if wt is None else _transposed(wt, scale_wt, ("wt", "scale_wt"), K, M, dev)
    if wt is None and grad_x is not None:
        raise ValueError("grad_x goes with wt")
    if xt is None and grad_weight is not None:
        raise ValueError("grad_weight goes with xt")
    ldgx = K
    if grad_x is not None:
        ldgx = _rows(grad_x, "grad_x", torch.bfloat16, n, K, dev)
    elif wt is not None:
        grad_x = torch.empty((n, K), dtype=torch.bfloat16, device=dev)
    if grad_weight is not None:
        _buf(grad_weight, "grad_weight", torch.bfloat16, M * K, dev)
    elif xt is not None:
        grad_weight = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    bcode = LCE_F32
    if grad_bias is None and want_grad_bias:
        grad_bias = torch.empty(M, dtype=grad_bias_dtype or torch.bfloat16, device=dev)
    if grad_bias is not None:
        bcode = _float_code(grad_bias, "grad_bias")
        _buf(grad_bias, "grad_bias", grad_bias.dtype, M, dev)
    if workspace is not None:
        _buf(workspace, "workspace", torch.uint8, lce_linear_blocks_backward_workspace_bytes(n, K, M), dev)
    _blocks_backward(grad_out, ldg, gcode, x_args, w_args, n, K, M, grad_x, ldgx, grad_weight, grad_bias, bcode, workspace,
                     stream)
    return LinearGrads(grad_x, grad_weight, grad_bias)


def _blocks_backward(g, ldg, gcode, x_args, w_args, n, K, M, gx, ldgx, gw, gb, bcode, workspace, stream):
    """The call, its operands checked: allocates the workspace if there is none."""
    if workspace is None:   # clobbered by the call
        bytes_ = lib().lce_linear_blocks_backward_workspace_bytes(n, K, M)
        workspace = torch.empty(max(bytes_, 1), dtype=torch.uint8, device=g.device)
    else:
        bytes_ = workspace.numel()
    _check(lib().lce_linear_blocks_backward(g.data_ptr(), ldg, gcode, *x_args, *w_args, n, K, M, _ptr(gx), ldgx, _ptr(gw),
                                            _ptr(gb), bcode, workspace.data_ptr(), bytes_, stream))


def _kept(need: bool, K: int, width: int, at: int):
    """Where a transposed operand [K, width] and its scales lie in what the forward keeps: (row stride, offset of
    the scales, end), all bytes, from ``at`` on."""
    if not need:
        return 0, at, at
    ld = _up(width, 16)
    scales = _up(at + K * ld, 256)
    return ld, scales, _up(scales + -(-K // 128) * -(-width // 128), 256)


class _LinearBlocks(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, differentiate):
        dev = _on_gpu(x, "x")
        if x.dim() < 1 or not torch.is_tensor(weight) or weight.dim() != 2:
            raise ValueError("x must have at least one dimension, and weight two")
        for t, name in ((x, "x"), (weight, "weight"), (residual, "residual")):
            if t is not None and t.dtype != torch.bfloat16:
                raise TypeError(f"{name} must be torch.bfloat16 (got {t.dtype})")
            if t is not None and t.device != dev:
                raise ValueError(f"{name} must be on {dev} (got {t.device})")
        M, K = weight.shape
        if x.shape[-1] != K:
            raise ValueError(f"weight must be [{M}, {x.shape[-1]}] (got {list(weight.shape)})")
        shape = (*x.shape[:-1], M)
        if residual is not None and residual.shape != shape:
            raise ValueError(f"residual must be {list(shape)} (got {list(residual.shape)})")
        bcode = LCE_F32
        if bias is not None:
            bcode = _float_code(bias, "bias")
            if bias.dim() != 1 or bias.shape[0] != M:
                raise ValueError(f"bias must be [{M}] (got {list(bias.shape)})")
            _buf(bias, "bias", bias.dtype, M, dev)
        x2, w2 = _rows_of(x, K), _rows_of(weight, K)
        r2 = None if residual is None else _rows_of(residual, M)
        n = x2.shape[0]
        keep_x, keep_w = (differentiate and need for need in (ctx.needs_input_grad[1], ctx.needs_input_grad[0]))
        ldxt, sxt, wt = _kept(keep_x, K, n, 0)
        ldwt, swt, end = _kept(keep_w, K, M, wt)
        _forward(x2, w2, bias, bcode, r2, out := torch.empty(shape, dtype=torch.bfloat16, device=dev),
                 kept := torch.empty(end, dtype=torch.uint8, device=dev), n, K, M, (ldxt, 0, sxt) if keep_x else None,
                 (ldwt, wt, swt) if keep_w else None, stream=None)
        ctx.save_for_backward(kept)
        ctx.sizes, ctx.places, ctx.x_shape = (n, K, M), (ldxt, 0, sxt, ldwt, wt, swt), x.shape
        ctx.bias_dtype = None if bias is None else bias.dtype
        return out

    @staticmethod
    def backward(ctx, g):
        return (_blocks_backward_twice if torch.is_grad_enabled() else _blocks_backward_once)(ctx, g)


@_call_stream
def _forward(x, w, bias, bcode, residual, out, kept, n, K, M, xt, wt, stream):
    """The call, its operands checked; ``xt`` and ``wt``: (row stride, offset, offset of the scales) in ``kept``."""
    bytes_ = lib().lce_linear_blocks_forward_workspace_bytes(n, K, M)
    workspace = torch.empty(max(bytes_, 1), dtype=torch.uint8, device=x.device)
    base = kept.data_ptr()

    def place(p):
        return (None, 0, None) if p is None else (base + p[1], p[0], base + p[2])

    _check(lib().lce_linear_blocks_forward(x.data_ptr(), _ld(x), w.data_ptr(), _ld(w), _ptr(bias), bcode, _ptr(residual),
                                           M if residual is None else _ld(residual), n, K, M, out.data_ptr(), M, *place(xt),
                                           *place(wt), workspace.data_ptr(), bytes_, stream))


def _blocks_backward_once(ctx, g):   # on autograd's thread, as the norm's in head.py
    kept, = ctx.saved_tensors
    need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
    gx = gw = gb = None
    if need_x or need_w or need_b:
        n, K, M = ctx.sizes
        ldxt, xt, sxt, ldwt, wt, swt = ctx.places
        dev = g.device
        bcode = LCE_F32
        if need_x:
            gx = torch.empty(ctx.x_shape, dtype=torch.bfloat16, device=dev)
        if need_w:
            gw = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        if need_b:
            gb = torch.empty(M, dtype=ctx.bias_dtype, device=dev)
            bcode = _CODES[ctx.bias_dtype]
        g2 = _rows_of(g, M)
        base = kept.data_ptr()
        none = (None, 0, None, 0, 0)
        x_args = (base + xt, ldxt, base + sxt, -(-n // 128), 1) if need_w else none
        w_args = (base + wt, ldwt, base + swt, -(-M // 128), 1) if need_x else none
        _blocks_backward(g2, _ld(g2), LCE_BF16, x_args, w_args, n, K, M, gx, K, gw, gb, bcode, None,
                         _current_stream(dev.index))
    return gx, gw, gb, (g if need_r else None), None


_blocks_backward_twice = torch.autograd.function.once_differentiable(_blocks_backward_once)


def linear_blocks(x, weight, bias=None, *, residual=None):
    """Autograd form of the product over the last dimension of ``x`` with all three of its matrix products
    in 8 bits: x weight^T + bias + residual, x, weight and residual bfloat16 (bias bfloat16 or float32), the
    output bfloat16 with x's leading dimensions.  x is quantised in row blocks of 128 and weight in tiles;
    the gradients take grad_out in row blocks along what each sums over, and go straight through the
    roundings: grad_x = Q(g) Q(weight), grad_weight = Q(g^T) Q(x) with x in tiles.  grad_bias is the sum of g
    itself.  Any sizes; what the backward keeps of x and weight is their 8-bit transposes.

    Under capture, what ``linear`` says of it holds here too.
    """
    return _LinearBlocks.apply(x, weight, bias, residual, torch.is_grad_enabled())


# ---- orthogonalised update -------------------------------------------------------------------

def lce_orthogonalise_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return int(lib().lce_orthogonalise_workspace_bytes(int(batch), int(rows), int(cols)))


def _matrices(t, name: str, dtype, shape, device):
    """Checks a [batch, rows, cols] or [rows, cols] operand; returns (row stride, batch stride)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} (got {list(t.shape)})")
    rows, cols = t.shape[-2:]
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return (t.stride(-2) if rows > 1 else cols), (t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else 0)


@_call_stream
def lce_orthogonalise(g, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, out=None,
                      workspace=None, stream=None):
    """The orthogonalised update of a matrix ``g`` [rows, cols], or of each of a batch [batch, rows, cols]
    (bfloat16 or float32, unit column stride): X = g / (its norm + eps), then ``steps`` times
    X <- a X + (b A + c A A) X with A = X X^T (X^T X of a matrix taller than wide) and ``coefficients``
    (a, b, c), refused where they can take singular values of 0 to 1 past 256 before the last step.
    Returns bfloat16 of g's shape, ``out`` if it is given."""
    dev = _on_gpu(g, "g")
    if g.dim() not in (2, 3):
        raise ValueError(f"g must be [rows, cols] or [batch, rows, cols] (got {list(g.shape)})")
    a, b, c = (float(v) for v in coefficients)
    code = _float_code(g, "g")
    ldg, batch_stride = _matrices(g, "g", g.dtype, g.shape, dev)
    batch, (rows, cols) = (g.shape[0] if g.dim() == 3 else 1), g.shape[-2:]
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=dev)
    ldo, out_stride = _matrices(out, "out", torch.bfloat16, g.shape, dev)
    need = lib().lce_orthogonalise_workspace_bytes(batch, rows, cols)
    if workspace is not None:
        _buf(workspace, "workspace", torch.uint8, need, dev)
    elif need:   # clobbered by the call
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().lce_orthogonalise(g.data_ptr(), ldg, batch_stride, code, batch, rows, cols, int(steps), a, b, c, float(eps),
                                   out.data_ptr(), ldo, out_stride, _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), stream))
    return out
