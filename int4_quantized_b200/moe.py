"""Routed experts: tokens sorted by expert and back, the gradients, and a layer of experts
with 8-bit weights.

    tokens, pos, offsets = moe_sort(ids, E)       # ids: [T, k] expert of each choice
    xs = moe_gather(x, tokens)                    # rows by expert
    out = moe_combine(ys, pos, weights)           # out[t] = sum over j of weights[t, j] * ys[pos[t, j]]
    dys, dweights = moe_combine_backward(dout, ys, pos, weights)
    dx = moe_combine(dxs, pos)                    # the gradient of moe_gather

    experts = Fp8Experts.pack(gate_up, down)      # [E, 2F, D] and [E, D, F] weights
    out = experts(x, ids, weights)                # x: [T, D]

The functions marshal arguments for libq4's q4_moe_* entry points (include/q4.h has the
definitions); there is no CPU fallback. None of them registers with autograd: their results
carry no gradient, which is had by the calls above.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _cuda, lib
from .fp8 import E4M3, _arg, _blocks, _call, _dtype, _new, _out, fp8_gemm_grouped, fp8_pack, fp8_pack_weights


def moe_sort(ids: torch.Tensor, num_experts: int) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Choices [T, k] (int32 or int64) -> (tokens [T * k], pos [T, k], offsets [E + 1]), int32.

    Stable. An id outside 0 .. E - 1 drops its choice (pos = -1); tokens is -1 from
    offsets[E] on.
    """
    _cuda(ids, "ids")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError("ids must be [T, k] with k >= 1")
    T, k = ids.shape
    E = int(num_experts)
    if E < 1:
        raise ValueError("num_experts must be at least 1")
    dev = ids.device
    tokens, pos, offsets = _new((T * k,), torch.int32, dev), _new((T, k), torch.int32, dev), _new((E + 1,), torch.int32, dev)
    _call(dev, "moe_sort", lib().q4_moe_sort, ids.data_ptr(), 32 if ids.dtype == torch.int32 else 64, T, k, E,
          tokens.data_ptr(), pos.data_ptr(), offsets.data_ptr())
    return tokens, pos, offsets


def moe_gather(x: torch.Tensor, tokens: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """xs[i] = x[tokens[i]] (x: [T, D]); entries outside 0 .. T - 1 leave row i as it was."""
    _cuda(x, "x")
    xt = _dtype(x.dtype, "x")
    if x.dim() != 2 or x.shape[1] < 1 or tokens.dim() != 1:
        raise ValueError("x must be [T, D] and tokens [R]")
    dev = x.device
    T, D = x.shape
    R = tokens.shape[0]
    out, op = _out(out, "out", x.dtype, (R, D), dev)
    _call(dev, "moe_gather", lib().q4_moe_gather, x.data_ptr(), xt, T, D, _arg(tokens, "tokens", torch.int32, None, dev),
          R, op)
    return out


def moe_combine(ys: torch.Tensor, pos: torch.Tensor, weights: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] * ys[pos[t, j]] (ys: [R, D]; no weights: all ones)."""
    _cuda(ys, "ys")
    yt = _dtype(ys.dtype, "ys")
    if ys.dim() != 2 or ys.shape[1] < 1 or pos.dim() != 2 or pos.shape[1] < 1:
        raise ValueError("ys must be [R, D] and pos [T, k]")
    dev = ys.device
    R, D = ys.shape
    T, k = pos.shape
    out, op = _out(out, "out", ys.dtype, (T, D), dev)
    _call(dev, "moe_combine", lib().q4_moe_combine, ys.data_ptr(), yt, R, D, _arg(pos, "pos", torch.int32, None, dev),
          None if weights is None else _arg(weights, "weights", torch.float32, (T, k), dev), T, k,
          op)
    return out


def moe_combine_backward(dout: torch.Tensor, ys: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                         dys: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dys [R, D], dweights [T, k] fp32) of moe_combine for dout [T, D].

    Rows of dys that pos does not name are left as they were (undefined where `dys` is not
    given); the entries of pos inside 0 .. R - 1 must differ from one another.
    """
    _cuda(ys, "ys")
    yt = _dtype(ys.dtype, "ys")
    if ys.dim() != 2 or ys.shape[1] < 1 or pos.dim() != 2 or pos.shape[1] < 1:
        raise ValueError("ys must be [R, D] and pos [T, k]")
    if weights is None:
        raise TypeError("weights must be a CUDA tensor")
    dev = ys.device
    R, D = ys.shape
    T, k = pos.shape
    dys, dp = _out(dys, "dys", ys.dtype, (R, D), dev)
    dweights = _new((T, k), torch.float32, dev)
    _call(dev, "moe_combine_backward", lib().q4_moe_combine_backward, _arg(dout, "dout", ys.dtype, (T, D), dev),
          ys.data_ptr(), yt, R, D, _arg(pos, "pos", torch.int32, None, dev),
          _arg(weights, "weights", torch.float32, (T, k), dev), T, k, dp, dweights.data_ptr())
    return dys, dweights


class Fp8Experts:
    """E gated MLPs with e4m3 weights: down[e] (silu(gate[e] x) * (up[e] x)) for the experts of each token.

    gate_up [E, 2F, D] (the gate's rows, then up's) and down [E, D, F] are codes with scales
    as fp8_pack_weights gives them (D and F multiples of 16). A call sorts the tokens by
    expert, packs their rows in that order, multiplies, packs silu(gate) * up, multiplies and
    adds the weighted answers: six kernels (eight for many rows), nothing read back to the host.
    """

    def __init__(self, gate_up: torch.Tensor, gate_up_scales: torch.Tensor, down: torch.Tensor,
                 down_scales: torch.Tensor):
        _cuda(gate_up, "gate_up", E4M3)
        if gate_up.dim() != 3 or gate_up.shape[1] % 2 or gate_up.shape[1] < 2:
            raise ValueError("gate_up must be [E, 2F, D]")
        E, F2, D = gate_up.shape
        F = F2 // 2
        if D % 16 or F % 16:
            raise ValueError("D and F must be multiples of 16")
        dev = gate_up.device
        _arg(gate_up_scales, "gate_up_scales", torch.float32, (E, _blocks(F2), _blocks(D)), dev)
        _arg(down, "down", E4M3, (E, D, F), dev)
        _arg(down_scales, "down_scales", torch.float32, (E, _blocks(D), _blocks(F)), dev)
        self.gate_up, self.gate_up_scales, self.down, self.down_scales = gate_up, gate_up_scales, down, down_scales
        self.E, self.D, self.F = E, D, F

    @classmethod
    def pack(cls, gate_up: torch.Tensor, down: torch.Tensor) -> "Fp8Experts":
        """From fp32, bf16 or fp16 weights [E, 2F, D] and [E, D, F]."""
        return cls(*fp8_pack_weights(gate_up), *fp8_pack_weights(down))

    @staticmethod
    def sorted_rows(x: torch.Tensor, tokens: torch.Tensor, status: Optional[torch.Tensor] = None,
                    pos: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(codes, scales) of x[tokens]: fp8_pack(x, rows=tokens), by the shorter way.

        The status word takes what the rows in `tokens` give, whichever way is taken; the way by
        each row once needs `pos` (moe_sort's) for that, to leave the other rows of x out.
        """
        T, D = x.shape
        R = tokens.shape[0]
        # Packing in sorted order rounds a token's row once for each of its experts; from 2^25 values
        # on it is sooner done to round each row once and gather codes and scales, below one launch is
        # sooner than three. Measured in bf16, in sorted order and this way: 2^23 values 6.5 us and 7.5
        # to 10, 2^24 11.3 and 9.2 to 12.9, 2^25 21 and 13 (8 experts a token, rows of 2048 and 4096),
        # 15 (4, of 7168), 18 (8, of 512), 21 to 22 (2); 2^27 77 and 37 to 56, with 2 a token 80 and 76
        # to 85. In fp32 the same, but for 2 a token 26 and 28 to 29 at 2^25, 111 and 94 to 103 at 2^27.
        # (codes are gathered two by two, as 16-bit values)
        if R * D < 1 << 25 or R <= T or D % 2 or (status is not None and pos is None):
            return fp8_pack(x, rows=tokens, status=status)
        rows = None
        if status is not None:  # tokens without a place (padding) report nothing
            own = torch.arange(T, dtype=torch.int32, device=x.device)
            rows = torch.where(pos.amax(1) >= 0, own, -1)
        xq, xs = fp8_pack(x, rows=rows, status=status)
        return moe_gather(xq.view(torch.bfloat16), tokens).view(E4M3), moe_gather(xs, tokens)

    def __call__(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                 status: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [T, D], ids and weights [T, k] -> [T, D] of x's type.

        A choice with an id outside 0 .. E - 1 adds nothing. status: one int32 that takes
        Q4_STATUS_NONFINITE (of rows that an expert takes) and Q4_STATUS_TIMEOUT.
        """
        _cuda(x, "x")
        if x.dim() != 2 or x.shape[1] != self.D or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
            raise ValueError(f"x must be [T, {self.D}] and ids [T, k]")
        if x.device != self.gate_up.device or ids.device != x.device:
            raise ValueError(f"x and ids must be on {self.gate_up.device}")
        tokens, pos, offsets = moe_sort(ids, self.E)
        live = offsets[self.E:]  # rows that have an expert
        xq, xs = self.sorted_rows(x, tokens, status, pos)
        # gate and up become codes of 4 bits next: bf16 keeps enough of them, and unlike fp16 their range
        between = torch.bfloat16 if x.dtype == torch.float16 else x.dtype
        h = fp8_gemm_grouped(xq, xs, self.gate_up, self.gate_up_scales, offsets, out_dtype=between, status=status)
        hq, hs = fp8_pack(h, count=live, silu_mul=True, status=status)
        ys = fp8_gemm_grouped(hq, hs, self.down, self.down_scales, offsets, out_dtype=x.dtype, status=status)
        return moe_combine(ys, pos, weights)
