"""ctypes binding of libnf4's operators around the quantized linear layers.

The 8-bit block-scaled format (:class:`FP8Tensor`), its quantizer and product,
the RMS norm with its gradient, and the AdamW step.  As in ``_lib``: argument
checks and marshalling only, the work runs in the library's kernels on torch's
current stream, and a problem raises before anything is launched.  The calls of
a step go through the native module ``_host`` (``csrc/host_binding.cpp``).
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from ._lib import AdamWTensorStruct, FP8TensorStruct, _check, _dtype_enum, _require_device, lib

FP8_BLOCK = 128          # columns (and, for weights, rows) per scale
ADAM_BLOCK = 256         # elements per scale of an 8-bit optimizer state
FP8_FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FORMAT_ENUM = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


def _up(n: int, m: int) -> int:
    return -(-n // m) * m


def nf4_fp8_sizes(rows: int, cols: int, block_rows: int) -> dict:
    p, r, s = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().nf4_fp8_sizes(rows, cols, block_rows, ctypes.byref(p), ctypes.byref(r), ctypes.byref(s)),
           "nf4_fp8_sizes")
    return {"pitch": p.value, "scale_rows": r.value, "scale_pitch": s.value}


@dataclass
class FP8Tensor:
    """An 8-bit matrix [rows, cols] with a scale per 1 x 128 (activations) or 128 x 128 (weights) block.

    ``data``: float8_e4m3fn or float8_e5m2 [rows, cols rounded up to 128];
    ``scale``: fp32 [ceil(rows / block_rows), blocks of a row rounded up to 4].
    Both are contiguous, with zeros past the matrix.  Element (r, c) is
    ``data[r, c] * scale[r // block_rows, c // 128]``.
    """
    rows: int
    cols: int
    block_rows: int
    data: torch.Tensor
    scale: torch.Tensor

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.data.device

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int, fmt: str = "e4m3", device="cuda") -> "FP8Tensor":
        """Uninitialised buffers for the quantizers to fill."""
        if fmt not in FP8_FORMATS:
            raise ValueError(f"fmt must be one of {tuple(FP8_FORMATS)} (got {fmt!r})")
        if block_rows not in (1, FP8_BLOCK) or rows < 0 or cols < 1:
            raise ValueError(f"an 8-bit tensor needs rows >= 0, cols >= 1 and block_rows 1 or {FP8_BLOCK}")
        pitch = _up(cols, FP8_BLOCK)
        return cls(rows, cols, block_rows, torch.empty((rows, pitch), dtype=FP8_FORMATS[fmt], device=device),
                   torch.empty((-(-rows // block_rows), _up(pitch // FP8_BLOCK, 4)), dtype=torch.float32, device=device))

    @classmethod
    def from_parts(cls, data: torch.Tensor, scale: torch.Tensor, block_rows: int = FP8_BLOCK) -> "FP8Tensor":
        """Codes [rows, cols] and scales [ceil(rows / block_rows), ceil(cols / 128)], laid out once."""
        if data.dim() != 2 or data.dtype not in _FORMAT_ENUM:
            raise ValueError("data must be a 2-D float8_e4m3fn or float8_e5m2 tensor")
        rows, cols = data.shape
        fmt = "e4m3" if data.dtype == torch.float8_e4m3fn else "e5m2"
        t = cls.empty(rows, cols, block_rows, fmt, data.device)
        want = (-(-rows // block_rows), -(-cols // FP8_BLOCK))
        if tuple(scale.shape) != want or scale.device != data.device:
            raise ValueError(f"scale must be {want} on {data.device} (got {tuple(scale.shape)} on {scale.device})")
        t.data.view(torch.uint8).zero_()
        t.data.view(torch.uint8)[:, :cols].copy_(data.view(torch.uint8))
        t.scale.zero_()
        t.scale[:, :want[1]].copy_(scale)
        return t

    def t(self) -> "FP8Tensor":
        """The transpose of a 128 x 128-block tensor, laid out anew (a layer keeps it for its backward pass)."""
        if self.block_rows != FP8_BLOCK:
            raise ValueError("only a tensor with 128 x 128 blocks transposes without re-quantizing")
        data = self.data.view(torch.uint8)[:, :self.cols].t().contiguous().view(self.data.dtype)
        return FP8Tensor.from_parts(data, self.scale[:, :-(-self.cols // FP8_BLOCK)].t(), FP8_BLOCK)

    def dequantize(self, dtype: torch.dtype = torch.float32) -> torch.Tensor:
        """The values it stands for (for inspection; the product never forms them)."""
        s = self.scale.repeat_interleave(FP8_BLOCK, 1)[:, :self.cols].repeat_interleave(self.block_rows, 0)[:self.rows]
        return (self.data[:, :self.cols].float() * s).to(dtype)

    def nbytes(self) -> int:
        return self.data.numel() + 4 * self.scale.numel()

    def struct(self) -> FP8TensorStruct:
        """Descriptor for the C calls, after checking the buffers."""
        pitch = _up(self.cols, FP8_BLOCK)
        if self.block_rows not in (1, FP8_BLOCK):
            raise ValueError(f"FP8Tensor.block_rows must be 1 or {FP8_BLOCK} (got {self.block_rows})")
        if self.data.dtype not in _FORMAT_ENUM:
            raise ValueError(f"FP8Tensor.data must be float8_e4m3fn or float8_e5m2 (got {self.data.dtype})")
        if tuple(self.data.shape) != (self.rows, pitch):
            raise ValueError(f"FP8Tensor.data must be {(self.rows, pitch)} (got {tuple(self.data.shape)})")
        want = (-(-self.rows // self.block_rows), _up(pitch // FP8_BLOCK, 4))
        if tuple(self.scale.shape) != want or self.scale.dtype != torch.float32:
            raise ValueError(f"FP8Tensor.scale must be fp32 {want} (got {self.scale.dtype} {tuple(self.scale.shape)})")
        _require_device(self.data, "FP8Tensor.data")
        _require_device(self.scale, "FP8Tensor.scale")
        if self.scale.device != self.data.device:
            raise ValueError(f"FP8Tensor.scale is on {self.scale.device}, data on {self.data.device}")
        return FP8TensorStruct(self.rows, self.cols, self.block_rows, _FORMAT_ENUM[self.data.dtype],
                               self.data.data_ptr(), self.scale.data_ptr())


_host_module = None


def _host():
    """The module that checks, allocates and calls in one step (raises if it has not been built)."""
    global _host_module
    if _host_module is None:
        lib()
        try:
            from . import _host as m
        except ImportError as e:
            raise RuntimeError(f"dequant_gemm_amd/_host.so: {e}; build it with `python -m dequant_gemm_amd.build`") from e
        _host_module = m
    return _host_module


def _raw_stream(t: torch.Tensor) -> int:
    """torch's current stream on the tensor's device (a host tensor is refused by the callee)."""
    i = t.get_device()
    return 0 if i < 0 else torch._C._cuda_getCurrentRawStream(i)


def _status(out, where: str):
    if type(out) is int:
        _check(out, where)
    return out


def nf4_fp8_quantize(x: torch.Tensor, block_rows: int = 1, fmt: str = "e4m3",
                     out: Optional[FP8Tensor] = None) -> FP8Tensor:
    """8-bit codes of a 2-D bf16/fp32 device tensor with contiguous rows: activations (``block_rows`` 1)
    or weights (128).  ``out``: buffers to fill (their ``block_rows`` and type then hold)."""
    if out is not None:
        if out.shape != tuple(x.shape):
            raise ValueError(f"out is {out.shape}, x {tuple(x.shape)}")
        _status(_host().fp8_quantize(x, out.block_rows, 0, _raw_stream(x), out.data, out.scale), "nf4_fp8_quantize")
        return out
    if fmt not in FP8_FORMATS:
        raise ValueError(f"fmt must be one of {tuple(FP8_FORMATS)} (got {fmt!r})")
    data, scale = _status(_host().fp8_quantize(x, block_rows, 1 if fmt == "e5m2" else 0, _raw_stream(x), None, None),
                          "nf4_fp8_quantize")
    return FP8Tensor(x.shape[0], x.shape[1], block_rows, data, scale)


def nf4_fp8_matmul(x: FP8Tensor, w: FP8Tensor, out_dtype: torch.dtype = torch.float32,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X W^T of an 8-bit activation [M, K] and an 8-bit weight [N, K] (e4m3), fp32 accumulation.

    ``out_dtype`` float32 adds every product in fp32; bfloat16 runs on the fp8
    matrix cores, whose sums are good to about 1e-5 before the rounding.  A
    block's two scales are multiplied first: their product should stay below
    2^128, and below 2^-126 its rounding is worth up to 2^-118 of Y.
    """
    return _status(_host().fp8_matmul(x.rows, x.cols, x.block_rows, x.data, x.scale, w.rows, w.cols, w.block_rows,
                                      w.data, w.scale, out, _dtype_enum(out_dtype), _raw_stream(x.data)),
                   "nf4_fp8_matmul")


def nf4_rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, out_dtype: Optional[torch.dtype] = None):
    """(y, h, rstd): h = x + residual (x itself without one), y = h / rms(h) * weight.

    x and residual: [T, H] bf16 or fp32 with contiguous rows; weight [H]; y in
    ``out_dtype`` (x's by default); rstd fp32 [T].
    """
    y, h, rstd = _status(_host().rmsnorm_fwd(x, weight, residual, eps, -1 if out_dtype is None else _dtype_enum(out_dtype),
                                             _raw_stream(x)), "nf4_rmsnorm_fwd")
    return y, x if h is None else h, rstd


def nf4_rmsnorm_fwd_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                        eps: float = 1e-6):
    """(y, h, rstd) as :func:`nf4_rmsnorm_fwd`, y an e4m3 :class:`FP8Tensor` with a scale per 128 columns."""
    data, scale, h, rstd = _status(_host().rmsnorm_fwd(x, weight, residual, eps, 2, _raw_stream(x)), "nf4_rmsnorm_fwd")
    return FP8Tensor(x.shape[0], x.shape[1], 1, data, scale), x if h is None else h, rstd


def nf4_rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                    dh: Optional[torch.Tensor] = None):
    """(dx, dweight) of the norm: dx [T, H] in h's type, with ``dh`` (the residual stream's gradient) added."""
    return _status(_host().rmsnorm_bwd(dy, h, weight, rstd, dh, _raw_stream(h)), "nf4_rmsnorm_bwd")


class AdamWState:
    """The two moments of a list of tensors in flat buffers, fp32 or 8-bit.

    Each tensor's part starts at a multiple of 256 elements and is padded to one
    (with zeros).  fp32: ``m`` and ``v``.  8-bit: ``m`` and ``v`` are e4m3 codes,
    ``v`` those of the second moment's square root, with an fp32 scale per 256
    elements in ``m_scale`` and ``v_scale``.
    """

    def __init__(self, sizes: Sequence[int], bits: int = 32, device="cuda"):
        if bits not in (8, 32):
            raise ValueError(f"state bits must be 8 or 32 (got {bits})")
        total = sum(_up(n, ADAM_BLOCK) for n in sizes)
        if bits == 8:
            codes = [torch.zeros(total, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
            scales = [torch.zeros(total // ADAM_BLOCK, dtype=torch.float32, device=device) for _ in range(2)]
            self._init(sizes, *codes, *scales)
        else:
            self._init(sizes, torch.zeros(total, dtype=torch.float32, device=device),
                       torch.zeros(total, dtype=torch.float32, device=device), None, None)

    @classmethod
    def from_flat(cls, sizes: Sequence[int], m: torch.Tensor, v: torch.Tensor,
                  m_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> "AdamWState":
        """Around existing buffers laid out as above."""
        self = cls.__new__(cls)
        self._init(sizes, m, v, m_scale, v_scale)
        return self

    def _init(self, sizes, m, v, m_scale, v_scale):
        self.sizes = [int(n) for n in sizes]
        if any(n < 0 for n in self.sizes):
            raise ValueError("sizes must not be negative")
        self.bits = 32 if m_scale is None else 8
        self.m, self.v, self.m_scale, self.v_scale = m, v, m_scale, v_scale
        self.starts, at = [], 0
        for n in self.sizes:
            self.starts.append(at)
            at += _up(n, ADAM_BLOCK)
        dt = torch.float32 if self.bits == 32 else torch.float8_e4m3fn
        want = [("m", m, dt, at), ("v", v, dt, at)]
        if self.bits == 8:
            want += [("m_scale", m_scale, torch.float32, at // ADAM_BLOCK),
                     ("v_scale", v_scale, torch.float32, at // ADAM_BLOCK)]
        for name, t, d, n in want:
            if t is None or t.dtype != d or t.numel() != n or not t.is_contiguous() or t.device != m.device:
                raise ValueError(f"AdamWState.{name} must be contiguous {d} with {n} elements on {m.device}")
        e = m.element_size()
        self._structs = (AdamWTensorStruct * len(self.sizes))()
        self._address = ctypes.addressof(self._structs)
        for st, n, lo in zip(self._structs, self.sizes, self.starts):
            st.n = n
            st.exp_avg = m.data_ptr() + e * lo
            st.exp_avg_sq = v.data_ptr() + e * lo
            if self.bits == 8:
                st.exp_avg_scale = m_scale.data_ptr() + 4 * (lo // ADAM_BLOCK)
                st.exp_avg_sq_scale = v_scale.data_ptr() + 4 * (lo // ADAM_BLOCK)
        # what the kernel needs to find many tensors in the flat buffers, beside them on the device
        self.layout = self._layout().to(m.device) if m.is_cuda else None

    def _layout(self) -> torch.Tensor:
        n = (ctypes.c_int64 * len(self.sizes))(*self.sizes)
        size = ctypes.c_size_t()
        _check(lib().nf4_adamw_layout_bytes(n, len(self.sizes), ctypes.byref(size)), "nf4_adamw_layout_bytes")
        out = torch.zeros(size.value, dtype=torch.uint8)
        _check(lib().nf4_adamw_layout(n, len(self.sizes), out.data_ptr(), size.value), "nf4_adamw_layout")
        return out

    def subset(self, indexes: Sequence[int]) -> "AdamWState":
        """Some of the tensors, over the same buffers."""
        part = AdamWState.__new__(AdamWState)
        part.layout = None
        part.bits, part.m, part.v, part.m_scale, part.v_scale = self.bits, self.m, self.v, self.m_scale, self.v_scale
        part.sizes, part.starts = [self.sizes[i] for i in indexes], [self.starts[i] for i in indexes]
        part._structs = (AdamWTensorStruct * len(part.sizes))(*[self._structs[i] for i in indexes])
        part._address = ctypes.addressof(part._structs)
        return part

    def moments(self, i: int):
        """The fp32 first and second moment of tensor ``i`` (flat; for inspection)."""
        n, lo = self.sizes[i], self.starts[i]
        hi = lo + _up(n, ADAM_BLOCK)
        if self.bits == 32:
            return self.m[lo:lo + n], self.v[lo:lo + n]
        s = slice(lo // ADAM_BLOCK, hi // ADAM_BLOCK)
        m = (self.m[lo:hi].float().reshape(-1, ADAM_BLOCK) * self.m_scale[s, None]).reshape(-1)[:n]
        r = (self.v[lo:hi].float().reshape(-1, ADAM_BLOCK) * self.v_scale[s, None]).reshape(-1)[:n]
        return m, r * r


def nf4_adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], state: AdamWState, *, lr: float,
                   beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                   step: int = 1, grad_scale: Optional[torch.Tensor] = None, seed: int = 0) -> None:
    """One AdamW step over all ``params`` in place (bf16 or fp32, one type; grads likewise).

    ``step`` counts from 1 and is taken by value: a captured graph would repeat
    one step's bias correction, so capture is refused.  ``seed`` (32 bits)
    drives the random rounding of 8-bit states and should differ every step.
    ``grad_scale``: fp32 device scalar that multiplies every gradient (a clipping
    factor, an inverse loss scale).
    """
    _require_device(state.m, "state")
    if torch._C._cuda_isCurrentStreamCapturing():
        raise RuntimeError("nf4_adamw_step takes its step count by value and cannot be captured into a graph")
    _status(_host().adamw_step(params, grads, state._address, len(state.sizes), state.m.get_device(), lr, beta1, beta2, eps,
                               weight_decay, step, grad_scale, seed & 0xFFFFFFFF, state.bits, state.layout, _raw_stream(state.m)),
            "nf4_adamw_step")
