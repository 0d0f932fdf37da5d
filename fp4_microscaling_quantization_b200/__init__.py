"""B200 (sm_100a) microscaling FP4: MXFP4 / NVFP4 quantization with a fused
block-diagonal Hadamard rotation, and the block-scaled W4A4 GEMM.

Python front end of the C ABI in include/fp4.h.  Tensors are torch CUDA
tensors (device memory and the current stream come from torch); all
arithmetic runs in libfp4.so.
"""
from __future__ import annotations

import ctypes
import functools

from . import _lib
from ._lib import (FP4_MX_SCALE_CEIL, FP4_MX_SCALE_FLOOR, FP4_MXFP4, FP4_MXFP4_16, FP4_NVFP4, FP4_OUT_BF16,
                   FP4_OUT_F32, FP4_ROUND_AWAY, FP4_ROUND_EVEN, FP4_SCALE_ABSMAX, FP4_SCALE_MSE, Fp4Error)

__all__ = [
    "quantize", "dequantize", "gemm", "gemm_quantized", "linear", "linear_residual", "linear_workspace_size",
    "quantize_sizes", "linear_w4a16", "linear_w4a16_workspace_size", "KVCache", "kv_cache_sizes", "kv_append", "kv_gather", "paged_attention",
    "paged_attention_workspace_size",
    "gemm_workspace_size", "check_device_status", "kernel_launches",
    "FP4_MXFP4", "FP4_NVFP4", "FP4_MXFP4_16", "FP4_ROUND_EVEN", "FP4_ROUND_AWAY", "FP4_MX_SCALE_CEIL",
    "FP4_MX_SCALE_FLOOR", "FP4_OUT_F32", "FP4_OUT_BF16", "FP4_SCALE_ABSMAX", "FP4_SCALE_MSE",
    "Fp4Error", "block_of",
]


def block_of(fmt: int) -> int:
    """Elements per block: 32 for MXFP4, 16 for NVFP4 and MXFP4_16."""
    return 32 if fmt == FP4_MXFP4 else 16


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return {"mxfp4": FP4_MXFP4, "nvfp4": FP4_NVFP4, "mxfp4_16": FP4_MXFP4_16}[fmt.lower()]
    return int(fmt)


def _stream_handle(torch, device) -> int:
    """The current stream of a device (a tensor's, or an ordinal)."""
    index = device if isinstance(device, int) else device.index
    # Without the stream object that the public call makes (2.2 us of a call's
    # 10), where this torch has that.
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _run(name: str, device, *args) -> None:
    """Calls entry point `name` of the library with `device` current.  The
    library launches on the current device and takes the SM count and the
    scratch it uses from it, so that must be the device whose memory and
    stream the call is given."""
    import torch

    if torch.cuda.current_device() == device.index:
        code = getattr(_lib._lib or _lib.lib(), name)(*args)
        if code:
            _lib.check(name, code)
        return
    with torch.cuda.device(device):
        _lib.check(name, getattr(_lib.lib(), name)(*args))


@functools.lru_cache(maxsize=64)
def _opts(round: int, mx_scale_rule: int, gscale_given: int, scale_search: int, weights_static: int):
    """A pointer to an fp4_opts of these values (only ever read)."""
    return ctypes.byref(_lib.Fp4Opts(round, mx_scale_rule, gscale_given, scale_search, weights_static))


def _dev(t, name: str, device, dtype=None, min_bytes: int = 0, contiguous: bool = True):
    """Checks a tensor whose device pointer goes to the library: a CUDA tensor
    on `device`, of `dtype`, contiguous, holding at least `min_bytes` bytes.
    The library sees only the pointer, so a host tensor or a short buffer
    would otherwise be read or written out of bounds on the device."""
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if min_bytes and t.nbytes < min_bytes:
        raise ValueError(f"{name} holds {t.nbytes} bytes, {min_bytes} needed")
    return t


def _operand(t3, rows: int, cols: int, fmt: int, name: str, device):
    """A quantized operand (q, s, g) of a rows x cols tensor in format fmt."""
    import torch

    q, s, g = t3
    qb, sb = _quantize_sizes(rows, cols, fmt)
    try:  # the checks of _dev in one expression: a decode step's call takes as long as its checks
        if (q.is_cuda and q.device == device and s.device == device and g.device == device
                and q.dtype is torch.uint8 and s.dtype is torch.uint8 and g.dtype is torch.float32
                and q.is_contiguous() and s.is_contiguous() and g.is_contiguous()
                and q.nbytes >= qb and s.nbytes >= sb and g.nbytes >= 4):
            return q, s, g
    except AttributeError:  # not a tensor: named below
        pass
    _dev(q, name + " elements", device, torch.uint8, qb)
    _dev(s, name + " scales", device, torch.uint8, sb)
    _dev(g, name + " tensor scale", device, torch.float32, 4)
    return q, s, g


def _out2d(out, rows: int, cols: int, dtype, name: str, device):
    """A row-major output of at least rows x cols (its row stride is passed on)."""
    _dev(out, name, device, dtype, contiguous=False)
    if out.dim() != 2 or out.shape[0] < rows or out.shape[1] < cols or (out.numel() and out.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D tensor of at least {rows} x {cols}, contiguous along its rows")
    return out


def quantize_sizes(rows: int, cols: int, fmt) -> tuple[int, int]:
    return _quantize_sizes(rows, cols, _fmt(fmt))


@functools.lru_cache(maxsize=4096)
def _quantize_sizes(rows: int, cols: int, fmt: int) -> tuple[int, int]:
    qb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check("fp4_quantize_sizes",
               _lib.lib().fp4_quantize_sizes(rows, cols, fmt, block_of(fmt), ctypes.byref(qb), ctypes.byref(sb)))
    return qb.value, sb.value


def quantize(x, fmt, hadamard_k: int = 0, round: int = FP4_ROUND_EVEN,
             mx_scale_rule: int = FP4_MX_SCALE_CEIL, gscale=None, out=None,
             scale_search: int = FP4_SCALE_ABSMAX):
    """Quantize a 2-D bf16 CUDA tensor along its last axis.

    Returns (q, s, g): q uint8 (rows, cols/2) packed nibbles, s uint8 scales in
    the tensor-core tile layout, g a 1-element fp32 tensor holding s_g (NVFP4;
    for MXFP4 a tensor holding 1).  If ``gscale`` is given (NVFP4) it is used
    as s_g instead of computing it.  ``out`` = (q, s, g) reuses buffers.
    ``scale_search`` = FP4_SCALE_MSE picks each block scale by the MSE search.
    """
    import torch

    fmt = _fmt(fmt)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a 2-D bf16 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("x must be contiguous along its last axis")
    rows, cols = x.shape
    qb, sb = quantize_sizes(rows, cols, fmt)
    if out is None:
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty((sb,), dtype=torch.uint8, device=x.device)
        g = torch.ones((1,), dtype=torch.float32, device=x.device)
    else:
        q, s, g = out
        _dev(q, "q", x.device, torch.uint8, qb)
        _dev(s, "s", x.device, torch.uint8, sb)
        _dev(g, "g", x.device, torch.float32, 4)
    given = gscale is not None
    if given:
        g.copy_(gscale.reshape(1).to(torch.float32))
    opts = _lib.Fp4Opts(int(round), int(mx_scale_rule), int(given), int(scale_search))
    gp = g.data_ptr() if fmt == FP4_NVFP4 else None
    _run("fp4_quantize", x.device,
        x.data_ptr(), rows, cols, x.stride(0), fmt, block_of(fmt), int(hadamard_k), ctypes.byref(opts),
        q.data_ptr(), s.data_ptr(), gp, _stream_handle(torch, x.device))
    return q, s, g


def dequantize(q, s, g, fmt, hadamard_k: int = 0, out_dtype: int = FP4_OUT_F32, out=None):
    """Inverse of :func:`quantize`; returns a (rows, cols) fp32 or bf16 tensor."""
    import torch

    fmt = _fmt(fmt)
    rows, half = q.shape
    cols = half * 2
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    _operand((q, s, g), rows, cols, fmt, "x", q.device)
    if out is None:
        out = torch.empty((rows, cols), dtype=dt, device=q.device)
    _dev(out, "out", q.device, dt, rows * cols * (4 if dt == torch.float32 else 2))
    gp = g.data_ptr() if fmt == FP4_NVFP4 else None
    _run("fp4_dequantize", q.device,
        q.data_ptr(), s.data_ptr(), gp, rows, cols, fmt, block_of(fmt), int(hadamard_k), int(out_dtype),
        out.data_ptr(), _stream_handle(torch, q.device))
    return out


def gemm_workspace_size(M: int, N: int, K: int, fmt) -> int:
    b = ctypes.c_size_t()
    _lib.check("fp4_gemm_workspace_size",
               _lib.lib().fp4_gemm_workspace_size(M, N, K, _fmt(fmt), ctypes.byref(b)))
    return b.value


def gemm(a, w, M: int, N: int, K: int, fmt, out_dtype: int = FP4_OUT_BF16, out=None, workspace=None):
    """C = A W^T from quantized operands a = (Aq, As, gA), w = (Wq, Ws, gW)."""
    import torch

    fmt = _fmt(fmt)
    dev = a[0].device
    Aq, As, gA = _operand(a, M, K, fmt, "A", dev)
    Wq, Ws, gW = _operand(w, N, K, fmt, "W", dev)
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=Aq.device)
    _out2d(out, M, N, dt, "out", dev)
    need = gemm_workspace_size(M, N, K, fmt)
    if need and workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=Aq.device)
    if workspace is not None:
        _dev(workspace, "workspace", dev, torch.uint8)
    wp = workspace.data_ptr() if workspace is not None else None
    wb = workspace.numel() if workspace is not None else 0
    _run("fp4_gemm", Aq.device,
        Aq.data_ptr(), As.data_ptr(), gA.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), gW.data_ptr(),
        M, N, K, fmt, int(out_dtype), out.data_ptr(), out.stride(0), wp, wb,
        _stream_handle(torch, Aq.device))
    return out


def gemm_quantized(a, w, M: int, N: int, K: int, fmt, out_fmt, gscale=None, round: int = FP4_ROUND_EVEN,
                   mx_scale_rule: int = FP4_MX_SCALE_CEIL, out=None):
    """C = A W^T quantized along N for the next layer, in the GEMM's epilogue.

    a = (Aq, As, gA), w = (Wq, Ws, gW) as for :func:`gemm`.  Returns
    (Cq, Cs, gC) like :func:`quantize`: Cq (M, N/2) packed nibbles, Cs the
    tile-layout scales, gC the NVFP4 tensor scale of C, which must be given
    (``gscale``) for an NVFP4 output.
    """
    import torch

    fmt, out_fmt = _fmt(fmt), _fmt(out_fmt)
    dev = a[0].device
    Aq, As, gA = _operand(a, M, K, fmt, "A", dev)
    Wq, Ws, gW = _operand(w, N, K, fmt, "W", dev)
    qb, sb = quantize_sizes(M, N, out_fmt)
    if out is None:
        Cq = torch.empty((M, N // 2), dtype=torch.uint8, device=Aq.device)
        Cs = torch.empty((sb,), dtype=torch.uint8, device=Aq.device)
        gC = torch.ones((1,), dtype=torch.float32, device=Aq.device)
    else:
        Cq, Cs, gC = out
        _operand(out, M, N, out_fmt, "C", dev)
    if gscale is not None:
        gC.copy_(gscale.reshape(1).to(torch.float32))
    opts = _lib.Fp4Opts(int(round), int(mx_scale_rule), int(gscale is not None))
    _run("fp4_gemm_quantized", Aq.device,
        Aq.data_ptr(), As.data_ptr(), gA.data_ptr(), Wq.data_ptr(), Ws.data_ptr(), gW.data_ptr(),
        M, N, K, fmt, out_fmt, ctypes.byref(opts), gC.data_ptr() if out_fmt == FP4_NVFP4 else None,
        Cq.data_ptr(), Cs.data_ptr(), _stream_handle(torch, Aq.device))
    return Cq, Cs, gC


def quantize_residual(x, fmt, hadamard_k: int = 0, round: int = FP4_ROUND_EVEN,
                      mx_scale_rule: int = FP4_MX_SCALE_CEIL, gscale=None):
    """:func:`quantize` with the sparse residual lane (TransFP4 Eq.(3), one
    value per 32): returns (q, s, g, res), res (rows, cols/32) int32 words =
    bf16 bits | index << 16."""
    import torch

    fmt = _fmt(fmt)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 CUDA tensor, contiguous along its last axis")
    rows, cols = x.shape
    _, sb = quantize_sizes(rows, cols, fmt)
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
    s = torch.empty((sb,), dtype=torch.uint8, device=x.device)
    g = torch.ones((1,), dtype=torch.float32, device=x.device)
    res = torch.empty((rows, cols // 32), dtype=torch.int32, device=x.device)
    given = gscale is not None
    if given:
        g.copy_(gscale.reshape(1).to(torch.float32))
    opts = _lib.Fp4Opts(int(round), int(mx_scale_rule), int(given), 0, 0)
    _run("fp4_quantize_residual", x.device,
        x.data_ptr(), rows, cols, x.stride(0), fmt, block_of(fmt), int(hadamard_k), ctypes.byref(opts),
        q.data_ptr(), s.data_ptr(), g.data_ptr() if fmt == FP4_NVFP4 else None, res.data_ptr(),
        _stream_handle(torch, x.device))
    return q, s, g, res


def dequantize_residual(q, s, g, res, fmt, hadamard_k: int = 0, out_dtype: int = FP4_OUT_F32):
    """Inverse of :func:`quantize_residual`."""
    import torch

    fmt = _fmt(fmt)
    rows, cols = q.shape[0], q.shape[1] * 2
    _operand((q, s, g), rows, cols, fmt, "x", q.device)
    _dev(res, "res", q.device, None, rows * (cols // 32) * 4)
    out = torch.empty((rows, cols), dtype=torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16,
                      device=q.device)
    _run("fp4_dequantize_residual", q.device,
        q.data_ptr(), s.data_ptr(), g.data_ptr() if fmt == FP4_NVFP4 else None, res.data_ptr(), rows, cols, fmt,
        block_of(fmt), int(hadamard_k), int(out_dtype), out.data_ptr(), _stream_handle(torch, q.device))
    return out


def nv_refine_gscale(x, hadamard_k: int = 0, rounds: int = 4, round: int = FP4_ROUND_EVEN):
    """The NVFP4 tensor scale of x refined by alternating MSE group steps and
    least-squares global steps (see fp4_nv_refine_gscale); returns a
    1-element fp32 tensor for ``quantize(..., gscale=...,
    scale_search=FP4_SCALE_MSE)``."""
    import torch

    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 CUDA tensor, contiguous along its last axis")
    rows, cols = x.shape
    qb, sb = quantize_sizes(rows, cols, FP4_NVFP4)
    q = torch.empty((max(qb, 16),), dtype=torch.uint8, device=x.device)
    s = torch.empty((max(sb, 16),), dtype=torch.uint8, device=x.device)
    nb = ctypes.c_size_t()
    _lib.check("fp4_nv_refine_gscale_workspace_size",
               _lib.lib().fp4_nv_refine_gscale_workspace_size(rows, cols, ctypes.byref(nb)))
    ws = torch.empty((nb.value,), dtype=torch.uint8, device=x.device)
    g = torch.empty((1,), dtype=torch.float32, device=x.device)
    opts = _lib.Fp4Opts(int(round), 0, 0, 0, 0)
    _run("fp4_nv_refine_gscale", x.device,
        x.data_ptr(), rows, cols, x.stride(0), int(hadamard_k), ctypes.byref(opts), int(rounds), q.data_ptr(),
        s.data_ptr(), ws.data_ptr(), nb.value, g.data_ptr(), _stream_handle(torch, x.device))
    return g


def mx_to_nv(w):
    """An MXFP4 tensor w = (q, s, g) in the NVFP4 scale form (q, s_nv, s_g)
    with the same dequantized elements (see fp4_mx_to_nv_scales); q is shared."""
    import torch

    q, s, _ = w
    rows, cols = q.shape[0], q.shape[1] * 2
    _dev(s, "MXFP4 scales", q.device, torch.uint8, quantize_sizes(rows, cols, FP4_MXFP4)[1])
    _, sb = quantize_sizes(rows, cols, FP4_NVFP4)
    s_nv = torch.empty((sb,), dtype=torch.uint8, device=q.device)
    g = torch.empty((1,), dtype=torch.float32, device=q.device)
    _run("fp4_mx_to_nv_scales", q.device,
        s.data_ptr(), rows, cols, s_nv.data_ptr(), g.data_ptr(), _stream_handle(torch, q.device))
    return q, s_nv, g


def linear_workspace_size(M: int, N: int, K: int, fmt) -> int:
    b = ctypes.c_size_t()
    _lib.check("fp4_linear_workspace_size",
               _lib.lib().fp4_linear_workspace_size(M, N, K, _fmt(fmt), ctypes.byref(b)))
    return b.value


def linear(x, w, fmt, hadamard_k: int = 0, out_dtype: int = FP4_OUT_BF16, gscale=None,
           round: int = FP4_ROUND_EVEN, mx_scale_rule: int = FP4_MX_SCALE_CEIL, out=None, workspace=None,
           weights_static: bool = False):
    """W4A4 linear from bf16 activations x (M x K) and a pre-quantized weight
    w = (Wq, Ws, gW) (N x K): quantizes x online, returns C = x W^T.
    ``weights_static``: w is written by no kernel still in flight (inference
    weights), so the decode kernel may stream it early."""
    import torch

    fmt = _fmt(fmt)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor, contiguous along K")
    _dev(x, "x", None, torch.bfloat16, contiguous=False)
    M, K = x.shape
    N = w[0].shape[0]
    Wq, Ws, gW = _operand(w, N, K, fmt, "W", x.device)
    if gscale is not None:
        _dev(gscale, "gscale", x.device, torch.float32, 4)
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=x.device)
    _out2d(out, M, N, dt, "out", x.device)
    if workspace is None:
        workspace = torch.empty((linear_workspace_size(M, N, K, fmt),), dtype=torch.uint8, device=x.device)
    _dev(workspace, "workspace", x.device, torch.uint8)
    opts = _lib.Fp4Opts(int(round), int(mx_scale_rule), 0, 0, int(bool(weights_static)))
    _run("fp4_linear", x.device,
        x.data_ptr(), M, K, x.stride(0), fmt, int(hadamard_k), ctypes.byref(opts),
        gscale.data_ptr() if gscale is not None else None, Wq.data_ptr(), Ws.data_ptr(), gW.data_ptr(), N,
        int(out_dtype), out.data_ptr(), out.stride(0), workspace.data_ptr(), workspace.numel(),
        _stream_handle(torch, x.device))
    return out


def linear_residual(x, w, fmt, hadamard_k: int = 0, out_dtype: int = FP4_OUT_BF16, gscale=None,
                    round: int = FP4_ROUND_EVEN, mx_scale_rule: int = FP4_MX_SCALE_CEIL, out=None,
                    weights_static: bool = False):
    """The decode linear (M <= 16) with the sparse residual lane of TransFP4
    Eq.(3) in the activations (see fp4_linear_residual): each 32-value unit's
    largest rotated value (bf16) stays out of the FP4 stream and its product
    with W is added in the same launch.  w = (Wq, Ws, gW) as for
    :func:`linear`; no workspace."""
    import torch

    fmt = _fmt(fmt)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor, contiguous along K")
    _dev(x, "x", None, torch.bfloat16, contiguous=False)
    M, K = x.shape
    N = w[0].shape[0]
    Wq, Ws, gW = _operand(w, N, K, fmt, "W", x.device)
    if gscale is not None:
        _dev(gscale, "gscale", x.device, torch.float32, 4)
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=x.device)
    _out2d(out, M, N, dt, "out", x.device)
    opts = _lib.Fp4Opts(int(round), int(mx_scale_rule), 0, 0, int(bool(weights_static)))
    _run("fp4_linear_residual", x.device,
         x.data_ptr(), M, K, x.stride(0), fmt, int(hadamard_k), ctypes.byref(opts),
         gscale.data_ptr() if gscale is not None else None, Wq.data_ptr(), Ws.data_ptr(), gW.data_ptr(), N,
         int(out_dtype), out.data_ptr(), out.stride(0), _stream_handle(torch, x.device))
    return out


def linear_w4a16_workspace_size(M: int, N: int, K: int, fmt) -> int:
    """Scratch bytes of a linear_w4a16 call of these sizes on the current device."""
    b = ctypes.c_size_t()
    _lib.check("fp4_linear_w4a16_workspace_size",
               _lib.lib().fp4_linear_w4a16_workspace_size(M, N, K, _fmt(fmt), ctypes.byref(b)))
    return b.value


@functools.lru_cache(maxsize=4096)
def _w4a16_scratch(device: int, *sizes) -> int:
    import torch

    with torch.cuda.device(device):
        return linear_w4a16_workspace_size(*sizes)


def linear_w4a16(x, w, fmt, hadamard_k: int = 0, out_dtype: int = FP4_OUT_BF16, out=None, workspace=None,
                 weights_static: bool = False):
    """The weight-only decode linear (M <= 16, see fp4_linear_w4a16): C = x W^T
    with FP4 weights w = (Wq, Ws, gW) as for :func:`linear` and bf16
    activations that are not quantized.  ``hadamard_k``: the rotation that w
    was quantized with (x is rotated in the kernel)."""
    import torch

    fmt = _fmt(fmt)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor, contiguous along K")
    device = x.device
    _dev(x, "x", None, torch.bfloat16, contiguous=False)
    M, K = x.shape
    N = w[0].shape[0]
    Wq, Ws, gW = _operand(w, N, K, fmt, "W", device)
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = x.new_empty((M, N)) if dt is torch.bfloat16 else x.new_empty((M, N), dtype=dt)
    else:
        _out2d(out, M, N, dt, "out", x.device)
    need = _w4a16_scratch(device.index, M, N, K, fmt)
    if need and workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    if workspace is not None:
        _dev(workspace, "workspace", x.device, torch.uint8)
    _run("fp4_linear_w4a16", device,
         x.data_ptr(), M, K, x.stride(0) if M > 1 else (K + 7) // 8 * 8, fmt, int(hadamard_k),
         _opts(0, 0, 0, 0, int(bool(weights_static))),
         Wq.data_ptr(), Ws.data_ptr(), gW.data_ptr(), N, int(out_dtype), out.data_ptr(), out.stride(0) if M > 1 else N,
         workspace.data_ptr() if workspace is not None else None, workspace.numel() if workspace is not None else 0,
         _stream_handle(torch, device))
    return out


# ---- the paged FP4 key-value cache ------------------------------------------
def kv_cache_sizes(num_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt) -> tuple[int, int]:
    """Bytes of the elements and of the scales of K (and of V) of a cache."""
    qb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check("fp4_kv_cache_sizes",
               _lib.lib().fp4_kv_cache_sizes(num_pages, page_size, kv_heads, head_dim, _fmt(fmt), ctypes.byref(qb),
                                             ctypes.byref(sb)))
    return qb.value, sb.value


class KVCache:
    """One layer's paged key-value cache in FP4 (fp4_kv_cache).

    ``k`` and ``v`` are (q, s, g) as elsewhere: q uint8 (num_pages, kv_heads,
    page_size, head_dim / 2) packed nibbles, s uint8 (num_pages, kv_heads,
    page_size, head_dim / block) scales, g a 1-element fp32 tensor (NVFP4's
    tensor scale, static for the cache's life; not used by the other formats).
    ``hadamard_k``: keys and values are held rotated by H_k.
    A slot is page * page_size + position.  The tensors are checked here, once,
    and must not be resized afterwards."""

    def __init__(self, k, v, fmt, hadamard_k: int = 0):
        import torch

        fmt = _fmt(fmt)
        if not isinstance(k[0], torch.Tensor) or k[0].dim() != 4:
            raise ValueError("K elements must be a (num_pages, kv_heads, page_size, head_dim / 2) tensor")
        pages, heads, page, half = k[0].shape
        dev = k[0].device
        qb, sb = kv_cache_sizes(pages, page, heads, 2 * half, fmt)
        for name, (q, s, g) in (("K", k), ("V", v)):
            _dev(q, name + " elements", dev, torch.uint8, qb)
            _dev(s, name + " scales", dev, torch.uint8, sb)
            _dev(g, name + " tensor scale", dev, torch.float32, 4)
            if tuple(q.shape) != (pages, heads, page, half):
                raise ValueError(f"{name} elements are {tuple(q.shape)}, K's {(pages, heads, page, half)}")
        if hadamard_k not in (0, 16, 32, 64, 128) or (hadamard_k and 2 * half % hadamard_k):
            raise ValueError("hadamard_k must be 0, 16, 32, 64 or 128 and divide head_dim")
        self.k, self.v, self.fmt, self.hadamard_k = tuple(k), tuple(v), fmt, int(hadamard_k)
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.device = dev
        self._c = _lib.Fp4KvCache(k[0].data_ptr(), k[1].data_ptr(), v[0].data_ptr(), v[1].data_ptr(), k[2].data_ptr(),
                                  v[2].data_ptr(), pages, page, heads, 2 * half, fmt, int(hadamard_k))
        self._p = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, fmt, k_gscale: float = 1.0,
              v_gscale: float = 1.0, hadamard_k: int = 0, device="cuda"):
        """A zeroed cache.  ``k_gscale``, ``v_gscale``: NVFP4's tensor scales,
        amax / 2688 of the keys and values to come (calibrated)."""
        import torch

        fmt = _fmt(fmt)
        kv_cache_sizes(num_pages, page_size, kv_heads, head_dim, fmt)
        shape = (num_pages, kv_heads, page_size)

        def one(g):
            return (torch.zeros(shape + (head_dim // 2,), dtype=torch.uint8, device=device),
                    torch.zeros(shape + (head_dim // block_of(fmt),), dtype=torch.uint8, device=device),
                    torch.full((1,), float(g), dtype=torch.float32, device=device))

        return cls(one(k_gscale), one(v_gscale), fmt, hadamard_k)


def _is(t, device, dtype, shape) -> bool:
    """Whether t is a tensor of these (all that _dev checks and the shape, in one go)."""
    import torch

    return isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and t.dtype is dtype and t.shape == shape


def _slots(slots, device):
    import torch

    _dev(slots, "slots", device, torch.int64)
    if slots.dim() != 1:
        raise ValueError("slots must be a 1-D int64 tensor")
    return slots.shape[0]


def kv_append(cache: KVCache, k, v, slots, round: int = FP4_ROUND_EVEN, mx_scale_rule: int = FP4_MX_SCALE_CEIL) -> None:
    """Quantizes new tokens' keys and values (bf16, (tokens, kv_heads,
    head_dim), contiguous along head_dim) into the cache at ``slots`` (int64).
    Tokens whose slot is negative or past the cache are dropped; every other
    token needs a slot of its own."""
    import torch

    tokens = _slots(slots, cache.device)
    shape = (tokens, cache.kv_heads, cache.head_dim)
    for name, t in (("k", k), ("v", v)):
        if not _is(t, cache.device, torch.bfloat16, shape) or (tokens and t.stride(2) != 1):
            _dev(t, name, cache.device, torch.bfloat16, contiguous=False)
            raise ValueError(f"{name} must be {shape}, contiguous along its last axis")
    ks, vs = k.stride(), v.stride()
    many, heads = tokens > 1, cache.kv_heads > 1
    _run("fp4_kv_append", cache.device,
         cache._p, k.data_ptr(), ks[0] if many else 0, ks[1] if heads else 0, v.data_ptr(), vs[0] if many else 0,
         vs[1] if heads else 0, slots.data_ptr(), tokens,
         _opts(int(round), int(mx_scale_rule), 1, 0, 0), _stream_handle(torch, cache.device))


def kv_gather(cache: KVCache, slots, out_dtype: int = FP4_OUT_BF16, out=None):
    """The keys and values at ``slots`` (int64), dequantized and turned back:
    (k, v), each (tokens, kv_heads, head_dim).  A slot that is negative or past
    the cache reads as zeros.  ``out`` = (k, v) reuses buffers."""
    import torch

    tokens = _slots(slots, cache.device)
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    shape = (tokens, cache.kv_heads, cache.head_dim)
    if out is None:
        k = slots.new_empty(shape, dtype=dt)
        v = torch.empty_like(k)
    else:
        k, v = out
        for name, t in (("k", k), ("v", v)):
            _dev(t, name, cache.device, dt, tokens * cache.kv_heads * cache.head_dim * (4 if dt == torch.float32 else 2))
    _run("fp4_kv_gather", cache.device,
         cache._p, slots.data_ptr(), tokens, int(out_dtype), k.data_ptr(), v.data_ptr(),
         _stream_handle(torch, cache.device))
    return k, v


def paged_attention_workspace_size(batch: int, q_heads: int, kv_heads: int, head_dim: int, max_seq_len: int,
                                   window: int = 0) -> int:
    """Scratch bytes of a paged_attention call of these sizes on the current device."""
    b = ctypes.c_size_t()
    _lib.check("fp4_paged_attention_workspace_size",
               _lib.lib().fp4_paged_attention_workspace_size(batch, q_heads, kv_heads, head_dim, max_seq_len, window,
                                                             ctypes.byref(b)))
    return b.value


@functools.lru_cache(maxsize=4096)
def _attention_scratch(device: int, *sizes) -> int:
    import torch

    with torch.cuda.device(device):
        return paged_attention_workspace_size(*sizes)


def paged_attention(q, cache: KVCache, page_table, seq_lens, max_seq_len: int | None = None, scale: float | None = None,
                    window: int = 0, out_dtype: int = FP4_OUT_BF16, out=None, return_lse: bool = False, workspace=None):
    """Attention of one new token per sequence over the paged FP4 cache (see
    fp4_paged_attention): q (batch, q_heads, head_dim) bf16, page_table (batch,
    pages) int32, seq_lens (batch,) int32, all on the device.

    ``max_seq_len`` bounds the lengths on the host (default: what the table
    reaches) and sizes the work split.  ``scale`` defaults to 1/sqrt(head_dim);
    ``window`` > 0 attends to the last so many tokens.  Returns (batch,
    q_heads, head_dim), with ``return_lse`` also the fp32 log-sum-exp of the
    scores, (batch, q_heads)."""
    import torch

    dev = cache.device
    _dev(q, "q", dev, torch.bfloat16, contiguous=False)
    if q.dim() != 3:
        raise ValueError(f"q must be (batch, q_heads, {cache.head_dim}), contiguous along its last axis")
    (batch, heads, dim), qs = q.shape, q.stride()
    if dim != cache.head_dim or (batch and heads and qs[2] != 1):
        raise ValueError(f"q must be (batch, q_heads, {cache.head_dim}), contiguous along its last axis")
    _dev(page_table, "page_table", dev, torch.int32, contiguous=False)
    if page_table.dim() != 2 or page_table.shape[0] != batch or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError(f"page_table must be ({batch}, pages), contiguous along its rows")
    if not _is(seq_lens, dev, torch.int32, (batch,)) or not seq_lens.is_contiguous():
        _dev(seq_lens, "seq_lens", dev, torch.int32)
        raise ValueError(f"seq_lens must be ({batch},)")
    cols = page_table.shape[1]
    if max_seq_len is None:
        max_seq_len = max(1, cols * cache.page_size)
    dt = torch.float32 if out_dtype == FP4_OUT_F32 else torch.bfloat16
    need = _attention_scratch(dev.index, batch, heads, cache.kv_heads, cache.head_dim, int(max_seq_len), int(window))
    if out is None:
        if dt is torch.bfloat16 and q.is_contiguous():
            out = torch.empty_like(q)
        else:
            out = q.new_empty((batch, heads, dim), dtype=dt)
    else:
        _dev(out, "out", dev, dt, batch * heads * cache.head_dim * (4 if dt == torch.float32 else 2))
    lse = torch.empty((batch, heads), dtype=torch.float32, device=dev) if return_lse else None
    if need and workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _dev(workspace, "workspace", dev, torch.uint8)
    _run("fp4_paged_attention", dev,
         cache._p, q.data_ptr(), batch, heads, qs[0] if batch > 1 else 0, qs[1] if heads > 1 else 0,
         page_table.data_ptr(), page_table.stride(0) if batch > 1 else cols, cols, seq_lens.data_ptr(), int(max_seq_len),
         cache.head_dim ** -0.5 if scale is None else float(scale), int(window), int(out_dtype), out.data_ptr(),
         lse.data_ptr() if lse is not None else None, workspace.data_ptr() if workspace is not None else None,
         workspace.numel() if workspace is not None else 0, _stream_handle(torch, dev))
    return (out, lse) if return_lse else out


def kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(_lib.lib().fp4_kernel_launches())


def check_device_status() -> None:
    import torch

    _lib.check("fp4_check_device_status",
               _lib.lib().fp4_check_device_status(_stream_handle(torch, torch.cuda.current_device())))
