"""Scaled int8 layers on torch tensors: argument checks, outputs and workspaces around the C calls
(include/bq.h, "Scaled int8"). Reached as ``bq.ScaledLinear`` and ``bq.scaled_quantize``.

A decoding loop makes these calls every few microseconds, so the checks read each tensor's attributes
once and the calls go to the library directly.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import bq

_TYPE = {torch.float32: bq.BQ_TYPE_F32, torch.bfloat16: bq.BQ_TYPE_BF16, torch.float16: bq.BQ_TYPE_F16}
_quantize, _gemm = bq._lib.bq_scaled_quantize, bq._lib.bq_scaled_gemm
_gemm_grouped, _linear = bq._lib.bq_scaled_gemm_grouped, bq._lib.bq_scaled_linear
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device


_INT32 = 0x7FFFFFFF  # sizes are passed as int32, which ctypes cuts without a word


def _refuse(where: str, what: str):
    raise bq.BQError(bq.BQ_ERR_INVALID_ARG, f"{where}: {what}")


def _too_large(where: str, what: str):
    raise bq.BQError(bq.BQ_ERR_SIZE, f"{where}: {what} has more than 2^31 - 1 rows or columns")


@contextlib.contextmanager
def _on(device, stream, *tensors):
    """`device` current, and `stream` (a torch stream of it) torch's current one: what is allocated inside
    belongs to the stream that uses it. `tensors` belong to the streams they were made on, so their memory is
    marked as used by `stream`: freed by the caller, it is not handed out again before `stream` has come past
    this call. (What is None or no tensor of `device` is left to the call's own checks.)"""
    if stream is not None and not (isinstance(stream, torch.cuda.Stream) and stream.device == device):
        _refuse("stream", "needs a torch.cuda.Stream of the tensors' device")
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                for t in tensors:
                    if isinstance(t, torch.Tensor) and t.device == device:
                        t.record_stream(stream)
                yield


def _finish(device):
    """Waits for what the current stream of `device` holds (not in a capture, whose order is the graph's)."""
    with torch.cuda.device(device):
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()


def _elsewhere(device, stream) -> bool:
    return stream is not None or _current_device() != device.index


def _matrix(t, name, where, columns, device):
    """(rows, row stride) of a CUDA matrix [rows, columns] whose columns are adjacent."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        _refuse(where, f"{name} is a 2-D CUDA tensor")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols != columns or (step != 1 and cols > 1) or t.device != device:
        _refuse(where, f"{name} has {cols} columns ({columns} wanted), column stride {step}, on {t.device} ({device})")
    if rows > _INT32 or cols > _INT32:
        _too_large(where, name)
    return rows, (ld if rows > 1 else max(ld, cols))


def _vector(t, name, where, n, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.numel() == n and
            t.is_contiguous()):
        _refuse(where, f"{name} is {n} contiguous {dtype} on {device}")
    return t.data_ptr()


def _up(K: int) -> int:
    return (K + 15) & -16


def empty_codes(rows: int, K: int, device):
    """An int8 matrix [rows, K] whose rows start on 16-byte boundaries."""
    return torch.empty_strided((rows, K), (_up(K), 1), dtype=torch.int8, device=device)


def scaled_quantize(x, gate=None, rows=None, q=None, scale=None, stream=None):
    """Per-row int8 codes and scales of x [*, K] (f32, bf16 or f16; see bq_scaled_quantize in include/bq.h):
    of all rows, or with `rows` (int32 [M]) of row rows[i] for every i (negative: an empty slot); with `gate`
    of x * SiLU(gate). Returns (q [M, K] int8, scale [M] f32), written to `q` and `scale` where given.
    `stream`: as for ScaledLinear."""
    where = "scaled_quantize"
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in _TYPE:
        _refuse(where, "x is a 2-D f32, bf16 or f16 tensor")
    dev, K = x.device, x.shape[1]
    R, ldx = _matrix(x, "x", where, K, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream, x, gate, rows, q, scale):
            return scaled_quantize(x, gate, rows, q, scale)
    ldg, gp, rp, M = 0, None, None, R
    if gate is not None:
        n, ldg = _matrix(gate, "gate", where, K, dev)
        if n != R or gate.dtype != x.dtype:
            _refuse(where, f"gate is {R} rows of {x.dtype}")
        gp = gate.data_ptr()
    if rows is not None:
        if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
            _refuse(where, "rows is a 1-D int32 tensor")
        M = rows.shape[0]
        rp = _vector(rows, "rows", where, M, torch.int32, dev)
        if M > _INT32:
            _too_large(where, "rows")
    if q is None:
        q, ldq = x.new_empty_strided((M, K), (_up(K), 1), dtype=torch.int8), _up(K)
    else:
        n, ldq = _matrix(q, "q", where, K, dev)
        if n != M or q.dtype != torch.int8:
            _refuse(where, f"q is {M} rows of int8")
        ldq = ldq if M > 1 else _up(K)
    if scale is None:
        scale = x.new_empty(M, dtype=torch.float32)
        sp = scale.data_ptr()
    else:
        sp = _vector(scale, "scale", where, M, torch.float32, dev)
    st = _quantize(x.data_ptr(), _TYPE[x.dtype], ldx, R, gp, ldg, rp, M, K, q.data_ptr(), ldq, sp,
                   _raw_stream(dev.index))
    if st:
        raise bq.BQError(st, "bq_scaled_quantize")
    return q, scale


class ScaledLinear:
    """A layer (or one per expert) of int8 codes [N, K] (or [E, N, K]) with a scale per output channel.

    Holds references to the tensors it is given; `codes` whose rows do not start on 16-byte boundaries
    are copied once into rows that do. Weights that are made here (that copy, and those of `quantize`) are
    complete when the layer is: calls on any stream may read them.

    Nothing is kept between calls: outputs and workspaces are allocated per call on the stream that runs
    it (or given, `y`), so calls on several streams and several captured graphs do not share memory.
    `stream` (a torch stream) defaults to torch's current one on the layer's device. As with torch's own
    calls the caller orders the streams: what is passed has to be complete on `stream`
    (Stream.wait_stream), and what is returned belongs to it. Memory passed to a call with `stream` may be
    freed as soon as the call has returned."""

    def __init__(self, codes, scale, bias=None):
        where = "ScaledLinear"
        if not (isinstance(codes, torch.Tensor) and codes.is_cuda and codes.dtype == torch.int8 and
                codes.dim() in (2, 3) and min(codes.shape) >= 1):
            _refuse(where, "codes is a CUDA int8 tensor [N, K] or [E, N, K]")
        c3 = codes if codes.dim() == 3 else codes[None]
        E, N, K = c3.shape
        if max(E, N, K) > _INT32:
            _too_large(where, "codes")
        se, sn, sk = c3.stride()
        sn, se = (sn if N > 1 else _up(K)), (se if E > 1 else 0)
        if (sk != 1 and K > 1) or sn % 16 or sn < K or se % 16 or se < 0 or c3.data_ptr() % 16:
            sn, se = _up(K), N * _up(K)
            c3 = empty_codes(E * N, K, codes.device).as_strided((E, N, K), (se, sn, 1)).copy_(c3)
            _finish(codes.device)
        sp = _vector(scale, "scale", where, E * N, torch.float32, codes.device)
        bp = None if bias is None else _vector(bias, "bias", where, E * N, torch.float32, codes.device)
        self.codes, self.scale, self.bias, self.device = c3, scale, bias, codes.device
        self.experts, self.N, self.K = E, N, K
        self._held = (c3, scale, bias)
        self.weights = bq.bq_scaled_weights(c3.data_ptr(), sp, bp, sn, se, N, K, E)
        self._w = ctypes.byref(self.weights)
        self._workspace = {}  # tokens -> workspace bytes (sizes only; the memory is allocated per call)

    @classmethod
    def quantize(cls, W, bias=None):
        """Codes and scales of W [N, K] or [E, N, K] (f32, bf16 or f16), one scale per output channel."""
        if not isinstance(W, torch.Tensor) or W.dim() not in (2, 3):
            _refuse("ScaledLinear.quantize", "W is a tensor [N, K] or [E, N, K]")
        q, s = scaled_quantize(W.reshape(-1, W.shape[-1]))
        ld = _up(W.shape[-1])
        q = q.as_strided(W.shape, (W.shape[-2] * ld, ld, 1)[-W.dim():])
        _finish(W.device)
        return cls(q, s.view(W.shape[:-1]), bias)

    def _out(self, y, M, dtype, where):
        """(y, its type, its row stride), allocated where it is not given."""
        if y is None:
            if dtype not in _TYPE:
                _refuse(where, f"y cannot have dtype {dtype}")
            return self.scale.new_empty((M, self.N), dtype=dtype), _TYPE[dtype], self.N
        n, ldy = _matrix(y, "y", where, self.N, self.device)
        if n != M or y.dtype not in _TYPE:
            _refuse(where, f"y is {M} rows of f32, bf16 or f16")
        return y, _TYPE[y.dtype], ldy

    def _codes(self, q, scale, where):
        M, ldq = _matrix(q, "q", where, self.K, self.device)
        if q.dtype != torch.int8:
            _refuse(where, "q is int8")
        return M, (ldq if M > 1 else _up(self.K)), _vector(scale, "scale", where, M, torch.float32, self.device)

    def linear(self, x, y=None, dtype=None, stream=None):
        """x [M, K] (f32, bf16 or f16) quantized per token, then the layer: y [M, N] of `dtype` (x's by default)."""
        where, dev = "ScaledLinear.linear", self.device
        M, ldx = _matrix(x, "x", where, self.K, dev)
        if x.dtype not in _TYPE:
            _refuse(where, "x is f32, bf16 or f16")
        if _elsewhere(dev, stream):
            with _on(dev, stream, x, y, *self._held):
                return self.linear(x, y, dtype)
        y, kind, ldy = self._out(y, M, dtype or x.dtype, where)
        n = self._workspace.get(M)
        if n is None:
            n = self._workspace[M] = bq.bq_scaled_workspace_bytes(self.weights, M)
        ws = x.new_empty(n, dtype=torch.uint8) if n else None
        st = _linear(self._w, x.data_ptr(), _TYPE[x.dtype], ldx, M, y.data_ptr(), kind, ldy,
                     ws.data_ptr() if n else None, n, _raw_stream(dev.index))
        if st:
            raise bq.BQError(st, "bq_scaled_linear")
        return y

    def gemm(self, q, scale, y=None, dtype=torch.bfloat16, stream=None):
        """The layer on quantized rows (scaled_quantize): y [M, N] of `dtype` (or `y`'s)."""
        where, dev = "ScaledLinear.gemm", self.device
        M, ldq, sp = self._codes(q, scale, where)
        if _elsewhere(dev, stream):
            with _on(dev, stream, q, scale, y, *self._held):
                return self.gemm(q, scale, y, dtype)
        y, kind, ldy = self._out(y, M, dtype, where)
        st = _gemm(self._w, q.data_ptr(), ldq, sp, M, y.data_ptr(), kind, ldy, _raw_stream(dev.index))
        if st:
            raise bq.BQError(st, "bq_scaled_gemm")
        return y

    def gemm_grouped(self, q, scale, offsets, y=None, dtype=torch.bfloat16, stream=None):
        """Expert e's layer on the rows offsets[e] .. offsets[e + 1] - 1 (offsets: int32 [E + 1] on the device).
        Rows outside every group keep what `y` held (undefined in a `y` that is allocated here)."""
        where, dev = "ScaledLinear.gemm_grouped", self.device
        M, ldq, sp = self._codes(q, scale, where)
        op = _vector(offsets, "offsets", where, self.experts + 1, torch.int32, dev)
        if _elsewhere(dev, stream):
            with _on(dev, stream, q, scale, offsets, y, *self._held):
                return self.gemm_grouped(q, scale, offsets, y, dtype)
        y, kind, ldy = self._out(y, M, dtype, where)
        st = _gemm_grouped(self._w, q.data_ptr(), ldq, sp, M, op, y.data_ptr(), kind, ldy, _raw_stream(dev.index))
        if st:
            raise bq.BQError(st, "bq_scaled_gemm_grouped")
        return y
