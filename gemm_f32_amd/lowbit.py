"""Products on 4-bit weights and 8-bit activation checkpoints for torch device tensors.

Argument marshalling only, like `matmul`: every step runs in libgemm's HIP kernels
(include/gemm.h, "Low-bit operands"), on the tensors' device and its current stream.

    w = w4_quantize(weight, group=128)            # weight (N, K), bf16 or fp16 -> W4
    y = w4_linear(x, w, bias=b, out=y)            # act(x . W^T + bias)
    dx = w4_dgrad(dy, w)                          # dy . W
    saved = x8_quantize(x)                        # x kept for the backward pass, 8 bits a value
    dw = x8_wgrad(dy, saved)                      # dy^T . x

No gradients are recorded; the calls are the forward and backward passes of a layer.
"""
from __future__ import annotations

import ctypes

from . import binding
from .binding import Act, EpilogueStruct, Order, Out, W4Struct, X8Struct

# (libgemm's name of a 16-bit type, C's element code) by torch dtype; filled on first use, since torch
# is imported only then
_NAMES: dict = {}
_OUTS: dict = {}
_FUNCTIONS: dict = {}
# the epilogue of a call without a bias, alpha 1 and beta 0, by activation and element code of C
_PLAIN: dict = {}
_module = None


def _torch():
    global _module
    if _module is None:
        import torch
        _NAMES.update({torch.bfloat16: "bf16", torch.float16: "f16"})
        _OUTS.update({torch.float32: Out.F32, torch.bfloat16: Out.BF16, torch.float16: Out.F16})
        _module = torch
    return _module


def _name(dtype) -> str:
    _torch()
    try:
        return _NAMES[dtype]
    except KeyError:
        raise TypeError(f"expected bfloat16 or float16, got {dtype}") from None


def _ld(t, what: str) -> int:
    """Leading dimension of a 2-D row-major tensor on a GPU."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a GPU")
    rows, cols = t.shape
    step, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{what} must be contiguous along its rows, got strides {t.stride()}")
    if rows <= 1:
        return max(1, cols)
    if step < max(1, cols):
        raise ValueError(f"{what} has overlapping rows, strides {t.stride()}")
    return step


def _same_device(index: int, *tensors) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on cuda:{index} and {t.device}")


def _call(name: str, index: int, *args) -> None:
    """lib.<name>(*args, current stream) with GPU `index` current."""
    torch = _torch()
    fn = _FUNCTIONS.get(name)
    if fn is None:
        fn = _FUNCTIONS[name] = getattr(binding.lib_handle(), name)
    # (the stream's handle without an object around it: 0.06 us against 1.7 us of a call that takes about 6)
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        raise binding.GemmError(rc, name)


class W4:
    """A rows x cols matrix in 4-bit codes (gemm_w4_t), rows x ceil(cols / 2) uint8; `scales` bfloat16 or
    float16 and `zeros` uint8 or None, both rows x ceil(cols / group)."""

    __slots__ = ("codes", "scales", "zeros", "group", "rows", "cols", "dtype", "device", "index", "name", "ref")

    def __init__(self, codes, scales, zeros, group: int, cols: int):
        torch = _torch()
        rows, groups = codes.shape[0], -(-cols // group) if group in (32, 64, 128) else None
        if groups is None:
            raise ValueError(f"group must be 32, 64 or 128, got {group}")
        if codes.dtype != torch.uint8 or tuple(codes.shape) != (rows, (cols + 1) // 2):
            raise ValueError(f"codes must be uint8 of shape (rows, {(cols + 1) // 2})")
        name = _name(scales.dtype)
        if tuple(scales.shape) != (rows, groups):
            raise ValueError(f"scales must have shape {(rows, groups)}")
        if zeros is not None and (zeros.dtype != torch.uint8 or tuple(zeros.shape) != (rows, groups)):
            raise ValueError(f"zeros must be uint8 of shape {(rows, groups)}")
        ld, lds, ldz = _ld(codes, "codes"), _ld(scales, "scales"), _ld(zeros, "zeros") if zeros is not None else 0
        _same_device(codes.get_device(), scales, zeros)
        self._fill(codes, scales, zeros, group, rows, cols, name, ld, lds, ldz)

    def _fill(self, codes, scales, zeros, group, rows, cols, name, ld, lds, ldz):
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, group
        self.rows, self.cols, self.dtype, self.device, self.name = rows, cols, scales.dtype, codes.device, name
        self.index = codes.get_device()
        self.ref = ctypes.byref(W4Struct(codes.data_ptr() or None, ld, scales.data_ptr() or None, lds,
                                           zeros.data_ptr() if zeros is not None else None, ldz, group))


class X8:
    """A rows x cols matrix in E4M3 codes (gemm_x8_t), uint8, with `exponents` uint8, rows x
    ceil(cols / 32); `dtype` (bfloat16 or float16) is the type its values are numbers of."""

    __slots__ = ("codes", "exponents", "rows", "cols", "dtype", "device", "index", "name", "ref")

    def __init__(self, codes, exponents, dtype):
        torch = _torch()
        rows, cols = codes.shape
        if codes.dtype != torch.uint8 or exponents.dtype != torch.uint8:
            raise TypeError("codes and exponents must be uint8")
        if tuple(exponents.shape) != (rows, -(-cols // 32)):
            raise ValueError(f"exponents must have shape {(rows, -(-cols // 32))}")
        name, ld, lde = _name(dtype), _ld(codes, "codes"), _ld(exponents, "exponents")
        _same_device(codes.get_device(), exponents)
        self._fill(codes, exponents, dtype, rows, cols, name, ld, lde)

    def _fill(self, codes, exponents, dtype, rows, cols, name, ld, lde):
        self.codes, self.exponents, self.dtype, self.device, self.name = codes, exponents, dtype, codes.device, name
        self.rows, self.cols, self.index = rows, cols, codes.get_device()
        self.ref = ctypes.byref(X8Struct(codes.data_ptr() or None, ld, exponents.data_ptr() or None, lde))


def w4_quantize(w, group: int = 128, zero_points: bool = False, out: W4 | None = None) -> W4:
    """`w` (bfloat16 or float16) rounded to 4 bits, with a scale for every `group` columns of a row."""
    torch = _torch()
    name, ldw = _name(w.dtype), _ld(w, "w")
    rows, cols = w.shape
    if out is None:
        if group not in (32, 64, 128):
            raise ValueError(f"group must be 32, 64 or 128, got {group}")
        groups = -(-cols // group)
        device, packed = w.device, (cols + 1) // 2
        out = W4.__new__(W4)
        out._fill(torch.empty((rows, packed), dtype=torch.uint8, device=device),
                  torch.empty((rows, groups), dtype=w.dtype, device=device),
                  torch.empty((rows, groups), dtype=torch.uint8, device=device) if zero_points else None, group,
                  rows, cols, name, max(1, packed), max(1, groups), max(1, groups) if zero_points else 0)
    elif (out.rows, out.cols, out.dtype) != (rows, cols, w.dtype):
        raise ValueError(f"out is {out.rows} x {out.cols} {out.dtype}, w {rows} x {cols} {w.dtype}")
    elif (out.group, out.zeros is not None) != (group, zero_points):
        raise ValueError("out has another group or zero points")
    index = w.get_device()
    _same_device(index, out.codes)
    _call(f"gemm_{name}_w4_quantize", index, rows, cols, w.data_ptr() or None, ldw, out.ref)
    return out


def w4_dequantize(w: W4, out=None):
    """The matrix that `w` stands for, of its scales' type."""
    return _dequantize(w, out, "w4")


def x8_quantize(x, out: X8 | None = None) -> X8:
    """`x` (bfloat16 or float16) in 8 bits a value, with an exponent for every 32 columns of a row."""
    torch = _torch()
    name, ldx = _name(x.dtype), _ld(x, "x")
    rows, cols = x.shape
    if out is None:
        device, groups = x.device, -(-cols // 32)
        out = X8.__new__(X8)
        out._fill(torch.empty((rows, cols), dtype=torch.uint8, device=device),
                  torch.empty((rows, groups), dtype=torch.uint8, device=device), x.dtype, rows, cols, name,
                  max(1, cols), max(1, groups))
    elif (out.rows, out.cols, out.dtype) != (rows, cols, x.dtype):
        raise ValueError(f"out is {out.rows} x {out.cols} {out.dtype}, x {rows} x {cols} {x.dtype}")
    index = x.get_device()
    _same_device(index, out.codes)
    _call(f"gemm_{name}_x8_quantize", index, rows, cols, x.data_ptr() or None, ldx, out.ref)
    return out


def x8_dequantize(q: X8, out=None):
    """The matrix that `q` stands for, of q.dtype."""
    return _dequantize(q, out, "x8")


def _dequantize(q, out, kind: str):
    torch = _torch()
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=q.dtype, device=q.device)
        ld = max(1, q.cols)
    elif out.dtype != q.dtype or tuple(out.shape) != (q.rows, q.cols):
        raise ValueError(f"out must be {q.dtype} of shape {(q.rows, q.cols)}")
    else:
        ld = _ld(out, "out")
        _same_device(q.index, out)
    _call(f"gemm_{q.name}_{kind}_dequantize", q.index, q.rows, q.cols, q.ref, out.data_ptr() or None, ld)
    return out


def _out(out, shape, device, beta):
    """C and its element code; allocated as float32 if None."""
    torch = _torch()
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out = torch.empty(shape, dtype=torch.float32, device=device)
    kind = _OUTS.get(out.dtype)
    if kind is None or out.shape != shape:
        raise ValueError(f"out must be float32, bfloat16 or float16 of shape {shape}")
    return out, kind


def _workspace(workspace, size: int, device):
    """(pointer, bytes, the tensor to keep until the call is enqueued)."""
    torch = _torch()
    if workspace is None:
        if size == 0:
            return None, 0, None
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr() or None, workspace.nbytes, workspace


def _epilogue(alpha, beta, bias, activation, kind):
    if bias is None and alpha == 1.0 and beta == 0.0:
        e = _PLAIN.get((activation, kind))
        if e is None:
            e = _PLAIN[activation, kind] = ctypes.byref(EpilogueStruct(1.0, 0.0, None, activation, kind))
        return e
    return ctypes.byref(EpilogueStruct(alpha, beta, bias.data_ptr() if bias is not None else None, activation, kind))


def w4_workspace_size(w: W4, rows: int, transposed: bool = False) -> int:
    """Workspace bytes of w4_linear (or, transposed, w4_dgrad) for `rows` rows; 0: it uses none."""
    n, k = (w.cols, w.rows) if transposed else (w.rows, w.cols)
    return binding.gemm_w4_workspace_size(rows, n, k, Order.ROW_MAJOR if transposed else Order.COL_MAJOR)


def _w4_product(x, w: W4, order, n, k, bias, activation, alpha, beta, out, workspace):
    if x.dtype != w.dtype:
        raise TypeError(f"activations are {x.dtype}, the weights' scales {w.dtype}")
    lda = _ld(x, "activations")
    m, inner = x.shape
    if inner != k:
        raise ValueError(f"inner dimensions differ: activations {tuple(x.shape)}, weights {w.rows} x {w.cols}")
    out, kind = _out(out, (m, n), w.device, beta)
    ldc = _ld(out, "out")
    if bias is not None:
        torch = _torch()
        if bias.dtype != torch.float32 or tuple(bias.shape) != (n,) or (n > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be contiguous float32 of shape ({n},)")
    size = binding.lib_handle().gemm_w4_workspace_size(m, n, k, order) if workspace is None else 0
    ptr, nbytes, keep = _workspace(workspace, size, w.device)
    _same_device(w.index, x, out, bias, keep)
    _call("gemm_bf16_w4" if w.name == "bf16" else "gemm_f16_w4", w.index, m, n, k, x.data_ptr() or None, lda, w.ref,
          order, out.data_ptr() or None, ldc, _epilogue(alpha, beta, bias, activation, kind), ptr, nbytes)
    return out


def w4_linear(x, w: W4, bias=None, activation: Act = Act.NONE, alpha: float = 1.0, beta: float = 0.0, out=None,
              workspace=None):
    """out = act(alpha * x . W^T + beta * out + bias): x (M, w.cols) of the type of w's scales, out (M, w.rows)
    float32, bfloat16 or float16 (allocated as float32 if None), bias (w.rows,) float32.

    workspace: a tensor of w4_workspace_size(w, M) bytes, allocated if None; an empty tensor runs
    without one."""
    return _w4_product(x, w, Order.COL_MAJOR, w.rows, w.cols, bias, activation, alpha, beta, out, workspace)


def w4_dgrad(dy, w: W4, alpha: float = 1.0, beta: float = 0.0, out=None, workspace=None):
    """out = alpha * dy . W + beta * out: the input gradient of w4_linear, dy (M, w.rows), out (M, w.cols); the
    rest as w4_linear (workspace: w4_workspace_size(w, M, transposed=True))."""
    return _w4_product(dy, w, Order.ROW_MAJOR, w.cols, w.rows, None, Act.NONE, alpha, beta, out, workspace)


def x8_wgrad_workspace_size(q: X8, n: int) -> int:
    """Workspace bytes of x8_wgrad for a dy of n columns."""
    return binding.gemm_x8_wgrad_workspace_size(q.rows, n, q.cols)


def x8_wgrad(dy, q: X8, alpha: float = 1.0, beta: float = 0.0, out=None, workspace=None):
    """out = alpha * dy^T . X + beta * out: the weight gradient of a layer from its output gradient dy
    (tokens, N) of q's type and its input kept in 8 bits (tokens, K); out (N, K) float32, bfloat16 or
    float16 (allocated as float32 if None).

    workspace: a tensor of at least x8_wgrad_workspace_size(q, N) bytes, allocated if None."""
    if dy.dtype != q.dtype:
        raise TypeError(f"dy is {dy.dtype}, the activations {q.dtype}")
    lddy = _ld(dy, "dy")
    if dy.shape[0] != q.rows:
        raise ValueError(f"dy has {dy.shape[0]} rows, the activations {q.rows}")
    n = dy.shape[1]
    out, kind = _out(out, (n, q.cols), q.device, beta)
    ldc = _ld(out, "out")
    size = binding.lib_handle().gemm_x8_wgrad_workspace_size(q.rows, n, q.cols) if workspace is None else 0
    ptr, nbytes, keep = _workspace(workspace, size, q.device)
    _same_device(q.index, dy, out, keep)
    _call(f"gemm_{q.name}_x8_wgrad", q.index, q.rows, n, q.cols, dy.data_ptr() or None, lddy, q.ref,
          out.data_ptr() or None, ldc, alpha, beta, kind, ptr, nbytes)
    return out
