"""Python binding of the expert feed-forward block: the gated product, its
gradients, and the products with 4-bit weights (argument marshalling only; the
work is done by the library's HIP kernels).

For every expert e and row r with offsets[e] <= r < offsets[e+1]:
    g, u = x[r] @ Wg[e].T, x[r] @ Wu[e].T
    h[r] = act(g) * u
    y[r] = h[r] @ Wd[e].T
The calls take the expert-major rows dispatch() returns and the offsets of
layout(), both on the device; nothing is read back, so they can be captured in
a graph. Where a call allocates its output, the rows of no segment (from
offsets[E] on, and before offsets[0], which is 0 in a layout) are zero; an
output the caller passes keeps what it held there. None of them records a
gradient or follows a tangent; expert_ffn is the differentiable block.
"""
from __future__ import annotations

from typing import Optional, Union

import torch

from . import _lib as L
from .moe import (Mxfp4ExpertWeights, Mxfp4Rows, _DTYPES, _call, _check_mxfp4_rows, _check_rows,
                  _refuse_tangents)

ACTIVATIONS = {"silu": L.MOE_ACT_SILU, "gelu": L.MOE_ACT_GELU_TANH}


def _activation(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}") from None


def _weights(name: str, w: torch.Tensor, dev: torch.device):
    _check_rows(name, w, torch.bfloat16, 3, dev)
    return w.shape


def _rows(name: str, t: torch.Tensor, width: int, dev: torch.device, rows: Optional[int] = None,
          dtype: torch.dtype = torch.bfloat16):
    _check_rows(name, t, dtype, 2, dev)
    if t.shape[1] != width or (rows is not None and t.shape[0] != rows):
        want = "R" if rows is None else rows
        raise ValueError(f"{name} must be [{want}, {width}], got {tuple(t.shape)}")


def _offsets(offsets: torch.Tensor, E: int, dev: torch.device) -> None:
    _check_rows("offsets", offsets, torch.int32, 1, dev)
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets must have {E + 1} entries, got {offsets.shape[0]}")


def _out(out: Optional[torch.Tensor], rows: int, width: int, dev: torch.device, name: str = "out"):
    """The output and its flags: a fresh one is zero outside the segments."""
    if out is None:
        return torch.empty((rows, width), dtype=torch.bfloat16, device=dev), L.MOE_GEMM_ZERO_OUTSIDE
    _rows(name, out, width, dev, rows)
    return out, 0


def mxfp4_expert_weights(values: torch.Tensor, scales: torch.Tensor) -> Mxfp4ExpertWeights:
    """One-time packing of 4-bit expert weights (moe_pack_mxfp4_weights).

    values uint8 [E, n_out, k_in / 2]: e2m1 numbers, input 2i in the low half
    of byte i; scales uint8 [E, n_out, k_in / 32]: each byte b scales 32
    consecutive inputs of a row by 2^(b - 127) (255 is NaN). k_in is a multiple
    of 32, n_out of 8. For gated_grouped_gemm the rows are the gate's n_hidden,
    then the up projection's."""
    dev = values.device
    _check_rows("values", values, torch.uint8, 3, dev)
    _check_rows("scales", scales, torch.uint8, 3, dev)
    E, n_out, half = values.shape
    k_in = 2 * half
    if k_in % 32 != 0 or tuple(scales.shape) != (E, n_out, k_in // 32):
        raise ValueError("shapes: values [E, n_out, k_in / 2], scales [E, n_out, k_in / 32], "
                         f"k_in a multiple of 32; got {tuple(values.shape)}, {tuple(scales.shape)}")
    nbytes = int(L.load().moe_mxfp4_weights_bytes(E, n_out, k_in))
    if nbytes < 0:
        raise ValueError(f"unsupported expert weight shape ({E}, {n_out}, {k_in})")
    data = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _call("moe_pack_mxfp4_weights", dev, values.data_ptr(), scales.data_ptr(), E, n_out, k_in,
          data.data_ptr())
    return Mxfp4ExpertWeights(data, E, n_out, k_in)


def quantize_mxfp4(x: torch.Tensor) -> Mxfp4Rows:
    """x in MXFP4 along its last axis (moe_quantize_mxfp4): for each 32
    elements the scale 2^e, e = max(floor(log2(largest magnitude)) - 2, -127),
    and the e2m1 numbers nearest to x / 2^e (ties to even, at most 6).

    x fp32 or bf16 [..., k], contiguous, k a multiple of 32: expert-major rows
    for grouped_gemm and gated_grouped_gemm, or weights [E, n_out, k_in] for
    mxfp4_expert_weights(*quantize_mxfp4(w)). A block with a NaN or an infinity
    becomes NaN. Records no gradient; forward-mode derivatives are refused."""
    if x.dtype not in _DTYPES:
        raise TypeError(f"x must be one of {list(_DTYPES)}, got {x.dtype}")
    dev = x.device
    _check_rows("x", x, x.dtype, max(x.dim(), 1), dev)
    k = x.shape[-1]
    if k == 0 or k % 32 != 0:
        raise ValueError(f"the last axis must be a multiple of 32, got {k}")
    _refuse_tangents("quantize_mxfp4", x)
    values = torch.empty((*x.shape[:-1], k // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((*x.shape[:-1], k // 32), dtype=torch.uint8, device=dev)
    _call("moe_quantize_mxfp4", dev, x.data_ptr(), _DTYPES[x.dtype], x.numel() // k, k,
          values.data_ptr(), scales.data_ptr())
    return Mxfp4Rows(values, scales)


def dequantize_mxfp4(rows: Mxfp4Rows, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The numbers that rows stand for (moe_dequantize_mxfp4), fp32 or bf16
    [..., k], exact in both but for those past their range, which become
    infinities (scale bytes 253 and 254)."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be one of {list(_DTYPES)}, got {dtype}")
    dev = rows.values.device
    rows.check(dev, max(rows.values.dim(), 1))
    k = 2 * rows.values.shape[-1]
    if k == 0:
        raise ValueError("the last axis is empty")
    x = torch.empty((*rows.values.shape[:-1], k), dtype=dtype, device=dev)
    _call("moe_dequantize_mxfp4", dev, rows.values.data_ptr(), rows.scales.data_ptr(),
          _DTYPES[dtype], x.numel() // k, k, x.data_ptr())
    return x


def gated_grouped_gemm(x_expert: Union[torch.Tensor, Mxfp4Rows],
                       weights: Union[torch.Tensor, Mxfp4ExpertWeights],
                       offsets: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                       activation: str = "silu",
                       pre: Optional[torch.Tensor] = None) -> torch.Tensor:
    """First half of the expert block, one launch (moe_gated_grouped_gemm):
    for the rows r of expert e, out[r] = act(x[r] @ Wg[e].T) * (x[r] @ Wu[e].T).

    x_expert bf16 [R, k_in]; weights bf16 [E, 2 n_hidden, k_in], the gate's
    rows first, or the Mxfp4ExpertWeights of such rows (n_hidden a multiple of
    16), which x_expert in 4 bits (quantize_mxfp4) needs; offsets int32 [E+1];
    out bf16 [R, n_hidden]. activation "silu" or "gelu" (tanh form). pre, fp32
    [R, 2 n_hidden], receives the projections [g | u] of the segments' rows for
    the backward (bf16 weights only). Not differentiable by itself; see
    expert_ffn."""
    act = _activation(activation)
    if isinstance(x_expert, Mxfp4Rows):
        dev = _check_mxfp4_rows(x_expert, weights, offsets)
        n2, R = weights.n_out, x_expert.values.shape[0]
        if n2 % 32 != 0:
            raise ValueError(f"packed gate and up rows must be 2 * a multiple of 16, got {n2}")
        if pre is not None:
            raise ValueError("pre needs bf16 weights (4-bit weights have no backward)")
        out, flags = _out(out, R, n2 // 2, dev)
        _call("moe_gated_grouped_gemm_mxfp4_rows", dev, x_expert.values.data_ptr(),
              x_expert.scales.data_ptr(), weights.data.data_ptr(), offsets.data_ptr(),
              weights.num_experts, R, weights.k_in, n2 // 2, act, out.data_ptr(), flags)
        return out
    dev = x_expert.device
    packed = isinstance(weights, Mxfp4ExpertWeights)
    if packed:
        E, n2, k_in = weights.num_experts, weights.n_out, weights.k_in
        weights.check(dev)
        if n2 % 32 != 0:
            raise ValueError(f"packed gate and up rows must be 2 * a multiple of 16, got {n2}")
        if pre is not None:
            raise ValueError("pre needs bf16 weights (4-bit weights have no backward)")
    else:
        E, n2, k_in = _weights("weights", weights, dev)
        if n2 % 2 != 0:
            raise ValueError(f"weights must hold gate and up rows in equal number, got {n2}")
    _rows("x_expert", x_expert, k_in, dev)
    _offsets(offsets, E, dev)
    R, hidden = x_expert.shape[0], n2 // 2
    if pre is not None:
        _rows("pre", pre, n2, dev, R, torch.float32)
    out, flags = _out(out, R, hidden, dev)
    if packed:
        _call("moe_gated_grouped_gemm_mxfp4", dev, x_expert.data_ptr(), weights.data.data_ptr(),
              offsets.data_ptr(), E, R, k_in, hidden, act, out.data_ptr(), flags)
    else:
        _call("moe_gated_grouped_gemm", dev, x_expert.data_ptr(), weights.data_ptr(),
              offsets.data_ptr(), E, R, k_in, hidden, act, out.data_ptr(),
              0 if pre is None else pre.data_ptr(), flags)
    return out


def grouped_gemm_forward(x_expert: torch.Tensor, weights: torch.Tensor, offsets: torch.Tensor,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Second half of the expert block (moe_grouped_gemm_forward): out[r] =
    x[r] @ W[e].T with bf16 [E, n_out, k_in] weights.

    The same product as grouped_gemm's, summed in another order, and the faster
    one for row-major weights (MI355X, against grouped_gemm with row-major and
    with tiled weights: 256 experts of 7168 -> 4096 at one token x 8 79 us
    against 80 and 186, at 4096 tokens 3.34 ms against 4.03 and 3.23, at 32768
    13.8 ms against 21.2 and 14.3; 128 of 2048 -> 4096 at 8192 tokens 1.16 ms
    against 1.66 and 1.22). grouped_gemm is for weights in their tiled or 4-bit
    form, and where its results have to stay what they were."""
    dev = x_expert.device
    E, n_out, k_in = _weights("weights", weights, dev)
    _rows("x_expert", x_expert, k_in, dev)
    _offsets(offsets, E, dev)
    R = x_expert.shape[0]
    out, flags = _out(out, R, n_out, dev)
    _call("moe_grouped_gemm_forward", dev, x_expert.data_ptr(), weights.data_ptr(),
          offsets.data_ptr(), E, R, k_in, n_out, out.data_ptr(), flags)
    return out


def grouped_gemm_backward_input(grad_out: torch.Tensor, weights: torch.Tensor,
                                offsets: torch.Tensor,
                                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of x[r] @ W[e].T with respect to x (moe_grouped_gemm_backward_input):
    grad_out bf16 [R, n_out], weights bf16 [E, n_out, k_in], result [R, k_in]."""
    dev = grad_out.device
    E, n_out, k_in = _weights("weights", weights, dev)
    _rows("grad_out", grad_out, n_out, dev)
    _offsets(offsets, E, dev)
    R = grad_out.shape[0]
    out, flags = _out(out, R, k_in, dev)
    _call("moe_grouped_gemm_backward_input", dev, grad_out.data_ptr(), weights.data_ptr(),
          offsets.data_ptr(), E, R, k_in, n_out, out.data_ptr(), flags)
    return out


def gated_grouped_gemm_backward(grad_out: torch.Tensor, w_down: torch.Tensor, pre: torch.Tensor,
                                offsets: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                                activation: str = "silu") -> torch.Tensor:
    """Gradient of [g | u] (moe_gated_grouped_gemm_backward): grad_out bf16
    [R, n_out] of the block's output, w_down bf16 [E, n_out, n_hidden], pre
    fp32 [R, 2 n_hidden] from gated_grouped_gemm; result bf16 [R, 2 n_hidden]."""
    dev = grad_out.device
    act = _activation(activation)
    E, n_out, hidden = _weights("w_down", w_down, dev)
    _rows("grad_out", grad_out, n_out, dev)
    R = grad_out.shape[0]
    _rows("pre", pre, 2 * hidden, dev, R, torch.float32)
    _offsets(offsets, E, dev)
    out, flags = _out(out, R, 2 * hidden, dev)
    _call("moe_gated_grouped_gemm_backward", dev, grad_out.data_ptr(), w_down.data_ptr(),
          pre.data_ptr(), offsets.data_ptr(), E, R, hidden, n_out, act, out.data_ptr(), flags)
    return out


def grouped_gemm_backward_weight(grad_out: torch.Tensor, x_expert: torch.Tensor,
                                 offsets: torch.Tensor, out: Optional[torch.Tensor] = None, *,
                                 accumulate: bool = False) -> torch.Tensor:
    """Gradient of x[r] @ W[e].T with respect to W
    (moe_grouped_gemm_backward_weight): out[e] = the sum over e's rows of
    grad_out[r] x[r]^T, zero for an expert without rows.

    grad_out bf16 [R, n_out], x_expert bf16 [R, k_in]; out [E, n_out, k_in]
    bf16 or fp32 (allocated as bf16 if None). accumulate adds to what out
    holds."""
    dev = grad_out.device
    _check_rows("grad_out", grad_out, torch.bfloat16, 2, dev)
    _check_rows("offsets", offsets, torch.int32, 1, dev)
    R, n_out = grad_out.shape
    _check_rows("x_expert", x_expert, torch.bfloat16, 2, dev)
    if x_expert.shape[0] != R:
        raise ValueError("grad_out and x_expert need the same number of rows")
    E, k_in = offsets.shape[0] - 1, x_expert.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((E, n_out, k_in), dtype=torch.bfloat16, device=dev)
    else:
        if out.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"out must be bf16 or fp32, got {out.dtype}")
        _check_rows("out", out, out.dtype, 3, dev)
        if tuple(out.shape) != (E, n_out, k_in):
            raise ValueError(f"out must be [{E}, {n_out}, {k_in}], got {tuple(out.shape)}")
    _call("moe_grouped_gemm_backward_weight", dev, grad_out.data_ptr(), x_expert.data_ptr(),
          offsets.data_ptr(), E, R, k_in, n_out,
          L.MOE_F32 if out.dtype == torch.float32 else L.MOE_BF16, out.data_ptr(),
          L.MOE_GEMM_ACCUMULATE if accumulate else 0)
    return out
