"""8-bit floating point with one fp32 scale per block of 128: packing and the product.

    xq, xs = fp8_pack(x)                     # x: [.., K] fp32 / bf16 / fp16 -> e4m3 codes, [.., ceil(K / 128)] scales
    wq, ws = fp8_pack_weights(w)             # w: [.., N, K] -> codes, [.., ceil(N / 128), ceil(K / 128)] scales
    y = fp8_gemm(xq, xs, wq, ws)             # [.., N], bf16 unless out_dtype says otherwise
    y = fp8_gemm_grouped(xq, xs, wq, ws, offsets)   # rows sorted by expert, wq: [E, N, K]

Codes are torch.float8_e4m3fn tensors. This module only marshals arguments for libq4's entry
points q4_fp8_pack, q4_fp8_pack_weights, q4_fp8_gemm and q4_fp8_gemm_grouped (include/q4.h
has the definitions); there is no CPU fallback. None of them registers with autograd.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _check, _cuda, lib

E4M3 = torch.float8_e4m3fn
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # q4_dtype
FP8_PACK_SILU_MUL = 1


def _dtype(t: torch.dtype, name: str) -> int:
    if t not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t}")
    return _DTYPES[t]


def _arg(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """Device pointer of a contiguous CUDA tensor of this dtype and shape (None: any) on this device."""
    # get_device() is -1 off the GPU, and half as dear as comparing devices
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous() or t.get_device() != device.index or (
            shape is not None and t.shape != shape):
        _cuda(t, name, dtype)
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")
        raise ValueError(f"{name} must have the shape {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _new(shape, dtype, device) -> torch.Tensor:
    """A contiguous tensor, uninitialised (strided: the quickest of torch's ways to make one)."""
    if len(shape) == 2:
        stride = (shape[1] or 1, 1)
    else:
        stride, n = [], 1
        for d in reversed(shape):
            stride.append(n)
            n *= d or 1
        stride.reverse()
    return torch.empty_strided(shape, stride, dtype=dtype, device=device)


def _out(t: Optional[torch.Tensor], name: str, dtype, shape, device) -> Tuple[torch.Tensor, int]:
    """An output and its device pointer: the caller's, checked, or a new one."""
    if t is None:
        t = _new(shape, dtype, device)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, device)


_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice


def _call(device: torch.device, what: str, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, with the device current."""
    i = device.index
    if _current() == i:
        code = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            code = fn(*args, _raw_stream(i))
    if code:
        _check(code, what)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _status(status: Optional[torch.Tensor], device) -> Optional[int]:
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    return _arg(status, "status", torch.int32, None, device)


def fp8_pack(x: torch.Tensor, rows: Optional[torch.Tensor] = None, count: Optional[torch.Tensor] = None,
             silu_mul: bool = False, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of activations [.., K] -> (e4m3 codes, fp32 scales of blocks of 128 values).

    rows      [R] int32: output row i takes row rows[i] of x (x: [T, K]); entries outside
              0 .. T - 1 leave their output row as it was
    count     one int32 on the device: output rows from there on are left as they were
    silu_mul  x is [.., 2K], gate then up; the values packed are silu(gate) * up
    """
    _cuda(x, "x")
    xt = _dtype(x.dtype, "x")
    if x.dim() < 1 or x.shape[-1] < 1 or (silu_mul and x.shape[-1] % 2):
        raise ValueError("x must be [.., K], or [.., 2K] with silu_mul, with K >= 1")
    dev = x.device
    K = x.shape[-1] // (2 if silu_mul else 1)
    n = x.numel() // x.shape[-1]
    if rows is None:
        lead, R, rp = tuple(x.shape[:-1]), n, None
    else:
        if x.dim() != 2 or rows.dim() != 1:
            raise ValueError("with rows, x must be [T, K] and rows [R]")
        rp = _arg(rows, "rows", torch.int32, None, dev)
        R = rows.shape[0]
        lead = (R,)
    cp = None
    if count is not None:
        cp = _arg(count, "count", torch.int32, None, dev)
        if count.numel() < 1:
            raise ValueError("count must hold one int32")
    codes, qp = _out(codes, "codes", E4M3, (*lead, K), dev)
    scales, sp = _out(scales, "scales", torch.float32, (*lead, _blocks(K)), dev)
    _call(dev, "fp8_pack", lib().q4_fp8_pack, x.data_ptr(), xt, n, K, rp, R, cp, FP8_PACK_SILU_MUL if silu_mul else 0,
          qp, sp, _status(status, dev))
    return codes, scales


def fp8_pack_weights(w: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Weights [.., N, K] -> (e4m3 codes, fp32 scales of blocks of 128 x 128 of each matrix)."""
    _cuda(w, "w")
    wt = _dtype(w.dtype, "w")
    if w.dim() < 2 or w.shape[-1] < 1:
        raise ValueError("w must be [.., N, K] with K >= 1")
    dev = w.device
    N, K = w.shape[-2:]
    E = 1
    for d in w.shape[:-2]:
        E *= d
    sshape = (*w.shape[:-2], _blocks(N), _blocks(K))
    codes, qp = _out(codes, "codes", E4M3, w.shape, dev)
    scales, sp = _out(scales, "scales", torch.float32, sshape, dev)
    _call(dev, "fp8_pack_weights", lib().q4_fp8_pack_weights, w.data_ptr(), wt, E, N, K, qp, sp, _status(status, dev))
    return codes, scales


def fp8_gemm(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
             out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
             status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[.., N] = x @ w^T from codes and scales (x: [.., K], w: [N, K]; K a multiple of 16)."""
    _cuda(x, "x", E4M3)
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1] or w.shape[1] < 1:
        raise ValueError("x must be [.., K] and w [N, K]")
    dev = x.device
    N, K = w.shape
    lead = tuple(x.shape[:-1])
    out, yp = _out(out, "out", out_dtype if out is None else out.dtype, (*lead, N), dev)
    yt = _dtype(out.dtype, "out")
    kb = _blocks(K)
    _call(dev, "fp8_gemm", lib().q4_fp8_gemm, x.data_ptr(),
          _arg(x_scales, "x_scales", torch.float32, (*lead, kb), dev), x.numel() // K, _arg(w, "w", E4M3, None, dev),
          _arg(w_scales, "w_scales", torch.float32, (_blocks(N), kb), dev), N, K,
          yp, yt, _status(status, dev))
    return out


def fp8_gemm_grouped(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                     offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                     out_dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[R, N]: rows offsets[e] .. offsets[e + 1] - 1 of x [R, K] times w[e] (w: [E, N, K]).

    offsets [E + 1] int32 on the device (moe_sort). Rows of y that no expert has are left as
    they were (undefined where `out` is not given).
    """
    _cuda(x, "x", E4M3)
    if x.dim() != 2 or w.dim() != 3 or x.shape[1] != w.shape[2] or w.shape[2] < 1:
        raise ValueError("x must be [R, K] and w [E, N, K]")
    dev = x.device
    R = x.shape[0]
    E, N, K = w.shape
    out, yp = _out(out, "out", out_dtype if out is None else out.dtype, (R, N), dev)
    yt = _dtype(out.dtype, "out")
    kb = _blocks(K)
    _call(dev, "fp8_gemm_grouped", lib().q4_fp8_gemm_grouped, x.data_ptr(),
          _arg(x_scales, "x_scales", torch.float32, (R, kb), dev), R,
          _arg(offsets, "offsets", torch.int32, (E + 1,), dev), E, _arg(w, "w", E4M3, None, dev),
          _arg(w_scales, "w_scales", torch.float32, (E, _blocks(N), kb), dev), N, K,
          yp, yt, _status(status, dev))
    return out
