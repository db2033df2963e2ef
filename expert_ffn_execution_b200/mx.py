"""Torch-level calls of the microscaled operators: they check shapes, types and
devices, allocate the outputs and call the library on the tensors' device and
that device's current stream (or `stream`).  No arithmetic happens here, and
nothing is recorded for a backward pass.

What a call makes belongs to the stream that it runs on, also where that is
given by `stream`.  A tensor that is used on another stream than the one it was
made on is the caller's to order and to keep alive, as with any asynchronous call.

A decode step's kernels take a few microseconds, so the host's part of a call
counts.  The codes and scales that a call makes share one allocation, their
tensors are made when they are asked for, and calls that need nothing from
this file but its checks are made by native/mxcalls.cpp (quantising 4 rows: 10.1
us here, 3.4 us there, 2.1 of them the launch); it returns None for every other
call, which then runs here.
"""
from __future__ import annotations

import ctypes
import operator
from typing import NamedTuple

import torch

from . import _binding as B
from .layer import ExpertWeights

try:
    from . import _mxcalls
    if getattr(_mxcalls, "torch_version", None) != torch.__version__:
        _mxcalls = None
except ImportError:  # not built, or for another torch: every call runs here
    _mxcalls = None

_DTYPES = {torch.float32: B.DTYPE_F32, torch.float16: B.DTYPE_F16, torch.bfloat16: B.DTYPE_BF16}
_fast = None  # _mxcalls, once it has been given the library


def _library():
    """The loaded library; the first call arms the native one."""
    global _fast
    lib = B._lib or B.load()
    if _fast is None and _mxcalls is not None:
        names = ("moe_mx_quantize", "moe_mx_dequantize", "moe_add_rmsnorm", "moe_mx_linear",
                 "moe_mx_pack_experts", "moe_mx_unpack_experts", "strata_expert_bytes")
        _mxcalls.setup(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names),
                       torch.Tensor, torch.nn.Parameter, MXTensor, AddNorm)
        _fast = _mxcalls
    return lib


def _dtype(dtype) -> int:
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"dtype {dtype}: float32, float16 or bfloat16 is wanted")
    return dt


def _device(first, *others):
    """The one CUDA device of the tensors (None among the others is passed over)."""
    dev = first.device
    for t in (first, *others):
        if isinstance(t, torch.Tensor) and t.is_neg():
            raise ValueError("a view that negates its memory: see Tensor.resolve_neg()")
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and on {t.device}")
    return dev


def _place(dev, stream):
    """A context in which `dev` and `stream` (a stream, its handle, or None)
    are current, or None where they are.  What a call allocates is then the
    stream's that writes it: memory that another stream has given back may
    still be that stream's to use."""
    if stream is None:
        return None if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if dev.index == torch._C._cuda_getDevice() and \
            handle == torch._C._cuda_getCurrentRawStream(dev.index):
        return None
    if getattr(stream, "device", dev) != dev:
        raise ValueError(f"tensors on {dev} and a stream of {stream.device}")
    if handle in (0, 1):  # the default stream, by its two handles
        return torch.cuda.stream(torch.cuda.default_stream(dev))
    if handle == 2:
        raise ValueError("the threads' default stream is not one that torch allocates for")
    return torch.cuda.stream(torch.cuda.ExternalStream(handle, dev))


def _enter(dev):
    """(library, stream handle) for a call on `dev`, which is current."""
    return _library(), torch._C._cuda_getCurrentRawStream(dev.index)


def _check(name, rc):
    if rc:
        raise B.StrataError(name, rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _code_bytes(rows: int, fmt: int, K: int) -> int:
    return rows * (K // 2 if fmt == B.MX_FP4 else K)


def _scale_bytes(rows: int, K: int, layout: int) -> int:
    if layout == B.MX_TILES:
        return -(-rows // 128) * -(-K // 128) * 512
    return rows * (K // 32)


def _check_format(fmt, rows, K, layout):
    if fmt not in (B.MX_FP4, B.MX_FP8) or layout not in (B.MX_ROWS, B.MX_TILES):
        raise ValueError("fmt must be MX_FP4 or MX_FP8, layout MX_ROWS or MX_TILES")
    if not 0 <= rows < 1 << 31 or not 32 <= K < 1 << 31 or K % 32:
        raise ValueError(f"rows = {rows}, K = {K}: rows >= 0 and K a positive multiple of 32, "
                         "both below 2^31, are wanted")


_FIELDS = ("_fmt", "_layout", "_rows", "_K", "_both", "_codes", "_scales")
if _mxcalls is not None:
    _Matrix = _mxcalls.Matrix  # these fields, natively
else:
    class _Matrix:
        __slots__ = _FIELDS


class MXTensor(_Matrix):
    """A microscaled matrix [rows, K] on the device: uint8 codes [rows, K/2]
    (MX_FP4) or [rows, K] (MX_FP8) and uint8 scales, [rows, K/32] (MX_ROWS) or
    the flat plane of tiles that mx_linear reads (MX_TILES).

    It holds the two tensors, not their addresses: every call looks at where
    they are when it is made, and refuses them if they no longer fit.  Copies
    and pickles have tensors of their own."""

    __slots__ = ()

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, fmt: int, rows: int, K: int,
                 layout: int):
        if _fast and _fast.wrap(self, codes, scales, fmt, rows, K, layout):
            return
        _check_format(fmt, rows, K, layout)
        self._fmt, self._rows, self._K, self._layout = fmt, rows, K, layout
        self._codes, self._scales, self._both = codes, scales, None
        _planes(self)

    @classmethod
    def _empty(cls, fmt: int, rows: int, K: int, layout: int, dev) -> MXTensor:
        """One to be written by a call: both planes in one allocation."""
        _check_format(fmt, rows, K, layout)
        q = cls.__new__(cls)
        q._fmt, q._rows, q._K, q._layout = fmt, rows, K, layout
        n = _scales_at(q) + _scale_bytes(rows, K, layout)
        q._both = torch.empty(n, dtype=torch.uint8, device=dev)
        q._codes = q._scales = None
        return q

    def __reduce__(self):
        return type(self), (self.codes, self.scales, self.fmt, self.rows, self.K, self.layout)

    fmt, layout, rows, K = (property(operator.attrgetter(n)) for n in _FIELDS[:4])

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            n = _code_bytes(self.rows, self.fmt, self.K)
            self._codes = self._both[:n].view(self.rows, _code_bytes(1, self.fmt, self.K))
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            n = _scale_bytes(self.rows, self.K, self.layout)
            s = self._both[_scales_at(self):][:n]
            self._scales = s.view(self.rows, self.K // 32) if self.layout == B.MX_ROWS else s
        return self._scales

    @property
    def device(self) -> torch.device:
        return (self._both if self._codes is None else self._codes).device

    @property
    def index(self) -> int:
        """Of the CUDA device, -1: none."""
        return (self._both if self._codes is None else self._codes).get_device()

    codes_ptr = property(lambda self: _planes(self)[0])
    scales_ptr = property(lambda self: _planes(self)[1])

    def dequantize(self, dtype=torch.float32, stream=None) -> torch.Tensor:
        """The matrix's values: [rows, K] of `dtype`."""
        if _fast and (out := _fast.dequantize(self, dtype, stream)) is not None:
            return out
        dt, dev = _dtype(dtype), _device(self)
        if (place := _place(dev, stream)) is not None:
            with place:
                return self.dequantize(dtype)
        codes, scales = _planes(self)
        lib, stream = _enter(dev)
        out = torch.empty(self.rows, self.K, dtype=dtype, device=dev)
        rc = lib.moe_mx_dequantize(codes, 0, scales, self.layout, 0, self.fmt, 1, self.rows, self.K,
                                   out.data_ptr(), dt, self.K, 0, stream)
        _check("moe_mx_dequantize", rc)
        return out


def _scales_at(q: MXTensor) -> int:
    """Where the scales are in one allocation of both planes."""
    return (_code_bytes(q._rows, q._fmt, q._K) + 255) & ~255


def _planes(q: MXTensor):
    """Where the codes and the scales are now.  The tensors may have been given
    other memory since the last call (`t.data = ...`, Module.to())."""
    codes, scales = q._codes, q._scales
    if codes is None and scales is None:
        at = q._both.data_ptr()
        return at, at + _scales_at(q)
    n = _code_bytes(q._rows, q._fmt, q._K)
    if codes is None:
        codes = q._both
    elif codes.dtype != torch.uint8 or not codes.is_contiguous() or codes.numel() != n:
        raise ValueError(f"codes must be contiguous uint8 of {n} bytes")
    n, at = _scale_bytes(q._rows, q._K, q._layout), 0
    if scales is None:
        scales, at = q._both, _scales_at(q)
    elif scales.dtype != torch.uint8 or not scales.is_contiguous() or scales.numel() != n:
        raise ValueError(f"scales must be contiguous uint8 of {n} bytes")
    if codes.device != scales.device:
        raise ValueError(f"codes on {codes.device} and scales on {scales.device}")
    return codes.data_ptr(), scales.data_ptr() + at


def mx_quantize(x: torch.Tensor, fmt: int, layout: int = B.MX_TILES, stream=None) -> MXTensor:
    """x [rows, K] in the microscaled format `fmt`.  Rows may be further apart
    than they are long; other strides are refused, not copied."""
    if _fast and (q := _fast.quantize(x, fmt, layout, stream)) is not None:
        return q
    if x.dim() != 2:
        raise ValueError(f"x must be a matrix, got shape {tuple(x.shape)}")
    rows, K = x.shape
    stride, step = x.stride()
    dt, ptr = _dtype(x.dtype), x.data_ptr()
    if rows and (step != 1 or ptr % 16 or (rows > 1 and stride * x.element_size() % 16)):
        raise ValueError("x must have contiguous rows that start on 16-byte boundaries")
    if K < 32 or K % 32:
        raise ValueError(f"K = {K}: a positive multiple of 32 is wanted")
    dev = _device(x)
    if (place := _place(dev, stream)) is not None:
        with place:
            return mx_quantize(x, fmt, layout)
    lib, stream = _enter(dev)
    q = MXTensor._empty(fmt, rows, K, layout, dev)
    codes, scales = _planes(q)
    rc = lib.moe_mx_quantize(ptr, dt, 1, rows, K, stride, 0, fmt, codes, 0, scales, layout, 0,
                             stream)
    _check("moe_mx_quantize", rc)
    return q


def mx_tile_scales(q: MXTensor, stream=None) -> MXTensor:
    """The same matrix with its scales in tiles, as mx_linear reads them."""
    if q.layout == B.MX_TILES:
        return q
    dev = _device(q)
    if (place := _place(dev, stream)) is not None:
        with place:
            return mx_tile_scales(q)
    lib, stream = _enter(dev)
    tiles = torch.empty(_scale_bytes(q.rows, q.K, B.MX_TILES), dtype=torch.uint8, device=dev)
    rc = lib.moe_mx_tile_scales(_planes(q)[1], q.rows, q.K, tiles.data_ptr(), stream)
    _check("moe_mx_tile_scales", rc)
    return MXTensor(q.codes, tiles, q.fmt, q.rows, q.K, B.MX_TILES)


class AddNorm(NamedTuple):
    """What add_rmsnorm gives: the new residual stream (x itself where there
    was nothing to add and no residual_out), the normalised rows in 16 or 32
    bits and in the microscaled format, each None where it was not asked for."""
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
    if _fast and (n := _fast.add_rmsnorm(x, delta, gain, eps, out_dtype, fmt, layout, residual_out,
                                         stream)) is not None:
        return n
    shape = x.shape
    if len(shape) != 2 or shape[0] >= 1 << 31 or shape[1] >= 1 << 31:
        raise ValueError(f"x must be a matrix [T, H] of sizes below 2^31, got {tuple(shape)}")
    T, H = shape
    for t, what in ((x, "x"), (delta, "delta"), (residual_out, "residual_out")):
        if t is not None and (t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous [T, H]")
    if residual_out is not None and residual_out.dtype != x.dtype:
        raise TypeError("residual_out must have the dtype of x")
    if gain is not None and (gain.dtype != torch.float32 or gain.shape != (H,)
                             or not gain.is_contiguous()):
        raise ValueError("gain must be contiguous float32 [H]")
    if out_dtype is None and not fmt:
        raise ValueError("ask for out_dtype, fmt or both")
    xd, dd = _dtype(x.dtype), 0 if delta is None else _dtype(delta.dtype)
    od = 0 if out_dtype is None else _dtype(out_dtype)
    dev = _device(x, delta, gain, residual_out)
    if (place := _place(dev, stream)) is not None:
        with place:
            return add_rmsnorm(x, delta, gain, eps, out_dtype, fmt, layout, residual_out)
    lib, stream = _enter(dev)
    res = residual_out
    if res is None and delta is not None:
        res = torch.empty_like(x)
    out = None if out_dtype is None else torch.empty(T, H, dtype=out_dtype, device=dev)
    q = MXTensor._empty(fmt, T, H, layout, dev) if fmt else None
    codes, scales = _planes(q) if fmt else (None, None)
    rc = lib.moe_add_rmsnorm(x.data_ptr(), xd, _ptr(delta), dd, _ptr(gain), T, H, eps, _ptr(res),
                             _ptr(out), od, fmt, codes, scales, layout, stream)
    _check("moe_add_rmsnorm", rc)
    return AddNorm(x if res is None else res, out, q)


def mx_linear(x: MXTensor, w: MXTensor, bias: torch.Tensor | None = None,
              out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
              dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [T, K] times w [N, K] transposed, plus bias [N]: [T, N] of out_dtype
    (or of `out`, whose rows may be further apart than N).  K is a multiple of
    128."""
    if _fast and (y := _fast.linear(x, w, bias, out_dtype, out, dev_status, stream)) is not None:
        return y
    T, N, K = x.rows, w.rows, w.K
    if x.K != K:
        raise ValueError(f"x has K = {x.K}, w K = {K}")
    if x.layout != B.MX_TILES or w.layout != B.MX_TILES:
        raise ValueError("mx_linear reads scales in tiles: see mx_tile_scales")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (N,)
                             or not bias.is_contiguous()):
        raise ValueError("bias must be contiguous float32 [N]")
    if dev_status is not None and (dev_status.dtype != torch.int32 or not dev_status.numel()):
        raise ValueError("dev_status must be an int32 tensor")
    ldy = N
    if out is not None:
        if out.shape != (T, N) or (N > 1 and out.stride(1) != 1) or \
                (T > 1 and out.stride(0) < N):
            raise ValueError("out must be [T, N] with contiguous rows that do not overlap")
        out_dtype = out.dtype
        if T > 1:
            ldy = out.stride(0)
    dt = _dtype(out_dtype)
    dev = _device(x, w, bias, out, dev_status)
    if (place := _place(dev, stream)) is not None:
        with place:
            return mx_linear(x, w, bias, out_dtype, out, dev_status)
    lib, stream = _enter(dev)
    if out is None:
        out = torch.empty(T, N, dtype=out_dtype, device=dev)
    (xc, xs), (wc, ws) = _planes(x), _planes(w)
    rc = lib.moe_mx_linear(xc, x.fmt, xs, T, wc, w.fmt, ws, N, K, _ptr(bias), out.data_ptr(), dt,
                           ldy, _ptr(dev_status), stream)
    _check("moe_mx_linear", rc)
    return out


def pack_experts(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                 stream=None) -> ExpertWeights:
    """Quantises E experts' weights, gate and up [E, I, H], down [E, H, I], all
    of one dtype, to the MXFP4 blobs that moe_experts reads."""
    if _fast and (blobs := _fast.pack(gate, up, down, stream)) is not None:
        return ExpertWeights(blobs, B.FMT_MXFP4_32, gate.shape[2], gate.shape[1])
    if gate.dim() != 3 or up.shape != gate.shape:
        raise ValueError("gate and up must be [E, I, H]")
    E, I, H = gate.shape
    if down.shape != (E, H, I) or H % 128 or I % 128 or not gate.numel():
        raise ValueError("down must be [E, H, I], H and I positive multiples of 128")
    ws = (gate, up, down)
    dt, dev, el = _dtype(gate.dtype), _device(*ws), gate.element_size()
    rows, experts = [], []
    for w in ws:
        expert, row, step = w.stride()
        if w.dtype != gate.dtype:
            raise TypeError("gate, up and down must have one dtype")
        if step != 1 or row * el % 16 or (E > 1 and expert * el % 16) or w.data_ptr() % 16:
            raise ValueError("weights must have contiguous rows that start on 16-byte boundaries")
        rows.append(row)
        experts.append(expert)
    if (place := _place(dev, stream)) is not None:
        with place:
            return pack_experts(gate, up, down)
    _, stream = _enter(dev)
    blobs = torch.empty(E, B.strata_expert_bytes(B.FMT_MXFP4_32, H, I), dtype=torch.uint8, device=dev)
    B.moe_mx_pack_experts(gate, up, down, dt, rows, experts, E, H, I, blobs, blobs.stride(0),
                          stream)
    return ExpertWeights(blobs, B.FMT_MXFP4_32, H, I)


def unpack_experts(w: ExpertWeights, dtype=torch.float32, stream=None):
    """(gate, up, down) that MXFP4 blobs stand for: [E, I, H] twice, [E, H, I]."""
    if w.fmt != B.FMT_MXFP4_32:
        raise ValueError("only MXFP4 blobs are read back")
    if _fast and (made := _fast.unpack(w.blobs, w.hidden, w.inter, dtype, stream)) is not None:
        return made
    dt, dev, E, H, I = _dtype(dtype), _device(w.blobs), w.num_experts, w.hidden, w.inter
    if (place := _place(dev, stream)) is not None:
        with place:
            return unpack_experts(w, dtype)
    _, stream = _enter(dev)
    gate = torch.empty(E, I, H, dtype=dtype, device=dev)
    up = torch.empty(E, I, H, dtype=dtype, device=dev)
    down = torch.empty(E, H, I, dtype=dtype, device=dev)
    B.moe_mx_unpack_experts(w.blobs, w.blobs.stride(0), E, H, I, gate, up, down, dt, stream)
    return gate, up, down
