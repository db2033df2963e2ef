"""Torch-level calls of the microscaled operators: they check shapes, types and
devices, allocate the outputs and call the library on the tensors' device and
that device's current stream (or `stream`).  No arithmetic happens here.

A tensor that is used on another stream than the one it was made on is the
caller's to order and to keep alive, as with any asynchronous call.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import torch

from . import _binding as B
from .layer import ExpertWeights

_DTYPES = {torch.float32: B.DTYPE_F32, torch.float16: B.DTYPE_F16, torch.bfloat16: B.DTYPE_BF16}


def _dtype(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"dtype {dtype}: float32, float16 or bfloat16 is wanted")
    return _DTYPES[dtype]


def _device(*tensors):
    """The one CUDA device of the tensors."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("the tensors must be on a CUDA device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on {dev} and on {t.device}")
    return dev


def _on(dev):
    """Makes `dev` the current device for a call (nothing to do where it is)."""
    if dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


def _row_bytes(fmt: int, K: int) -> int:
    return K // 2 if fmt == B.MX_FP4 else K


@dataclass
class MXTensor:
    """A microscaled matrix [rows, K] on the device: uint8 codes [rows, K/2]
    (MX_FP4) or [rows, K] (MX_FP8) and uint8 scales, [rows, K/32] (MX_ROWS) or
    the flat plane of tiles that mx_linear reads (MX_TILES)."""
    codes: torch.Tensor
    scales: torch.Tensor
    fmt: int
    rows: int
    K: int
    layout: int

    def __post_init__(self):
        if self.fmt not in (B.MX_FP4, B.MX_FP8) or self.layout not in (B.MX_ROWS, B.MX_TILES):
            raise ValueError("fmt must be MX_FP4 or MX_FP8, layout MX_ROWS or MX_TILES")
        if self.rows < 0 or self.K < 32 or self.K % 32:
            raise ValueError("rows must be >= 0 and K a positive multiple of 32")
        for t, n, what in ((self.codes, self.rows * _row_bytes(self.fmt, self.K), "codes"),
                           (self.scales, _scale_bytes(self.rows, self.K, self.layout), "scales")):
            if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{what} must be contiguous uint8 of {n} bytes")

    def dequantize(self, dtype=torch.float32, stream=None) -> torch.Tensor:
        """The matrix's values: [rows, K] of `dtype`."""
        dt, dev = _dtype(dtype), _device(self.codes, self.scales)
        with _on(dev):
            out = torch.empty(self.rows, self.K, dtype=dtype, device=dev)
            B.moe_mx_dequantize(self.codes, 0, self.scales, self.layout, 0, self.fmt, 1, self.rows,
                                self.K, out, dt, self.K, 0, stream)
        return out


def _scale_bytes(rows: int, K: int, layout: int) -> int:
    if layout == B.MX_TILES:
        return -(-rows // 128) * -(-K // 128) * 512
    return rows * (K // 32)


def _empty_mx(rows: int, K: int, fmt: int, layout: int, dev) -> MXTensor:
    shape = (rows, K // 32) if layout == B.MX_ROWS else (_scale_bytes(rows, K, layout),)
    return MXTensor(torch.empty(rows, _row_bytes(fmt, K), dtype=torch.uint8, device=dev),
                    torch.empty(shape, dtype=torch.uint8, device=dev), fmt, rows, K, layout)


def _rows_of(x: torch.Tensor, what: str) -> torch.Tensor:
    """x as the library reads rows: elements contiguous, each row on a 16-byte
    boundary.  Other strides are refused, not copied."""
    if x.dim() != 2:
        raise ValueError(f"{what} must be a matrix, got shape {tuple(x.shape)}")
    el = x.element_size()
    if x.numel() and ((x.shape[1] > 1 and x.stride(1) != 1) or x.data_ptr() % 16
                      or (x.shape[0] > 1 and x.stride(0) * el % 16)):
        raise ValueError(f"{what} must have contiguous rows that start on 16-byte boundaries")
    return x


def mx_quantize(x: torch.Tensor, fmt: int, layout: int = B.MX_TILES, stream=None) -> MXTensor:
    """x [rows, K] (rows may be strided) in the microscaled format `fmt`."""
    _rows_of(x, "x")
    rows, K = x.shape
    if K < 32 or K % 32:
        raise ValueError(f"K = {K}: a positive multiple of 32 is wanted")
    dt, dev = _dtype(x.dtype), _device(x)
    with _on(dev):
        q = _empty_mx(rows, K, fmt, layout, dev)
        B.moe_mx_quantize(x, dt, 1, rows, K, x.stride(0), 0, fmt, q.codes, 0, q.scales, layout, 0,
                          stream)
    return q


def mx_tile_scales(q: MXTensor, stream=None) -> MXTensor:
    """The same matrix with its scales in tiles, as mx_linear reads them."""
    if q.layout == B.MX_TILES:
        return q
    dev = _device(q.codes, q.scales)
    with _on(dev):
        tiles = torch.empty(_scale_bytes(q.rows, q.K, B.MX_TILES), dtype=torch.uint8, device=dev)
        B.moe_mx_tile_scales(q.scales, q.rows, q.K, tiles, stream)
    return MXTensor(q.codes, tiles, q.fmt, q.rows, q.K, B.MX_TILES)


@dataclass
class AddNorm:
    """What add_rmsnorm gives: the new residual stream (x itself where there
    was nothing to add), the normalised rows in 16 or 32 bits and in the
    microscaled format, each None where it was not asked for."""
    residual: torch.Tensor
    out: torch.Tensor | None
    mx: MXTensor | None


def add_rmsnorm(x: torch.Tensor, delta: torch.Tensor | None = None,
                gain: torch.Tensor | None = None, eps: float = 1e-6, out_dtype=None, fmt: int = 0,
                layout: int = B.MX_TILES, residual_out: torch.Tensor | None = None,
                stream=None) -> AddNorm:
    """r = x + delta; h = r / sqrt(mean r^2 + eps) * gain, per row of x [T, H];
    h as out_dtype (None: not written) and as microscaled `fmt` (0: not
    written).  r goes to residual_out (x for in place) or a new tensor."""
    T, H = x.shape
    for t, what in ((x, "x"), (delta, "delta"), (residual_out, "residual_out")):
        if t is not None and (t.shape != x.shape or not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous [T, H]")
    if residual_out is not None and residual_out.dtype != x.dtype:
        raise TypeError("residual_out must have the dtype of x")
    if gain is not None and (gain.dtype != torch.float32 or gain.shape != (H,)
                             or not gain.is_contiguous()):
        raise ValueError("gain must be contiguous float32 [H]")
    if out_dtype is None and not fmt:
        raise ValueError("ask for out_dtype, fmt or both")
    dev = _device(x, delta, gain, residual_out)
    xd, dd = _dtype(x.dtype), 0 if delta is None else _dtype(delta.dtype)
    od = 0 if out_dtype is None else _dtype(out_dtype)
    with _on(dev):
        res = residual_out
        if res is None and delta is not None:
            res = torch.empty_like(x)
        out = None if out_dtype is None else torch.empty(T, H, dtype=out_dtype, device=dev)
        q = _empty_mx(T, H, fmt, layout, dev) if fmt else None
        B.moe_add_rmsnorm(x, xd, delta, dd, gain, T, H, eps, res, out, od, fmt,
                          q and q.codes, q and q.scales, layout, stream)
    return AddNorm(x if res is None else res, out, q)


def mx_linear(x: MXTensor, w: MXTensor, bias: torch.Tensor | None = None,
              out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
              dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [T, K] times w [N, K] transposed, plus bias [N]: [T, N] of out_dtype
    (or of `out`, whose rows may be further apart than N)."""
    if x.K != w.K:
        raise ValueError(f"x has K = {x.K}, w K = {w.K}")
    if x.layout != B.MX_TILES or w.layout != B.MX_TILES:
        raise ValueError("mx_linear reads scales in tiles: see mx_tile_scales")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (w.rows,)
                             or not bias.is_contiguous()):
        raise ValueError("bias must be contiguous float32 [N]")
    if dev_status is not None and (dev_status.dtype != torch.int32 or not dev_status.numel()):
        raise ValueError("dev_status must be an int32 tensor")
    if out is not None:
        if out.shape != (x.rows, w.rows) or (w.rows > 1 and out.stride(1) != 1) or \
                (x.rows > 1 and out.stride(0) < w.rows):
            raise ValueError("out must be [T, N] with contiguous rows that do not overlap")
        out_dtype = out.dtype
    dt = _dtype(out_dtype)
    dev = _device(x.codes, x.scales, w.codes, w.scales, bias, out, dev_status)
    with _on(dev):
        if out is None:
            out = torch.empty(x.rows, w.rows, dtype=out_dtype, device=dev)
        ldy = out.stride(0) if x.rows > 1 else w.rows
        B.moe_mx_linear(x.codes, x.fmt, x.scales, x.rows, w.codes, w.fmt, w.scales, w.rows, w.K,
                        bias, out, dt, ldy, dev_status, stream)
    return out


def _blob_planes(H: int, I: int):
    """(codes offset, scales offset, rows, K) of gate, up and down in an MXFP4
    expert blob: each plane on a 256-byte boundary."""
    off, planes = 0, []
    for rows, K in ((I, H), (I, H), (H, I)):
        codes = off
        off = (off + rows * K // 2 + 255) & ~255
        planes.append((codes, off, rows, K))
        off = (off + rows * K // 32 + 255) & ~255
    return planes


def pack_experts(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                 stream=None) -> ExpertWeights:
    """Quantises E experts' weights, gate and up [E, I, H], down [E, H, I], to
    the MXFP4 blobs that moe_experts reads."""
    if gate.dim() != 3 or up.shape != gate.shape:
        raise ValueError("gate and up must be [E, I, H]")
    E, I, H = gate.shape
    if down.shape != (E, H, I) or H % 128 or I % 128 or not gate.numel():
        raise ValueError("down must be [E, H, I], H and I positive multiples of 128")
    ws = (gate, up, down)
    for w in ws:
        if w.stride(2) != 1 or any(w.stride(i) * w.element_size() % 16 for i in (0, 1)) or \
                w.data_ptr() % 16:
            raise ValueError("weights must have contiguous rows that start on 16-byte boundaries")
    dts, dev = [_dtype(w.dtype) for w in ws], _device(*ws)
    stride = B.strata_expert_bytes(B.FMT_MXFP4_32, H, I)
    with _on(dev):
        blobs = torch.empty(E, stride, dtype=torch.uint8, device=dev)
        for w, dt, (c, s, rows, K) in zip(ws, dts, _blob_planes(H, I)):
            B.moe_mx_quantize(w, dt, E, rows, K, w.stride(1), w.stride(0), B.MX_FP4,
                              blobs.data_ptr() + c, stride, blobs.data_ptr() + s, B.MX_ROWS,
                              stride, stream)
    return ExpertWeights(blobs, B.FMT_MXFP4_32, H, I)


def unpack_experts(w: ExpertWeights, dtype=torch.float32, stream=None):
    """(gate, up, down) that MXFP4 blobs stand for: [E, I, H] twice, [E, H, I]."""
    if w.fmt != B.FMT_MXFP4_32:
        raise ValueError("only MXFP4 blobs are read back")
    dt, dev, E = _dtype(dtype), _device(w.blobs), w.num_experts
    with _on(dev):
        outs = []
        for c, s, rows, K in _blob_planes(w.hidden, w.inter):
            o = torch.empty(E, rows, K, dtype=dtype, device=dev)
            B.moe_mx_dequantize(w.blobs.data_ptr() + c, w.blobs.stride(0), w.blobs.data_ptr() + s,
                                B.MX_ROWS, w.blobs.stride(0), B.MX_FP4, E, rows, K, o, dt, K,
                                rows * K, stream)
            outs.append(o)
    return tuple(outs)
