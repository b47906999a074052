"""Thin ctypes binding of the C ABI in ``libbq.so`` (declared in include/bq.h).

Argument marshalling only: every computation runs in the library's CUDA
kernels. Torch tensors may be passed wherever the C call takes a device
pointer (their ``data_ptr()`` is used); the stream defaults to torch's current
CUDA stream. If the shared library is missing this module raises at import.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libbq.so not built at {LIB_PATH}; run bit_weight_quantization_b200.build.build()")
_lib = ctypes.CDLL(LIB_PATH)

BQ_OK, BQ_ERR_INVALID_ARG, BQ_ERR_UNSUPPORTED, BQ_ERR_SIZE = 0, 1, 2, 3
BQ_ERR_CUDA, BQ_ERR_BAD_PACKED, BQ_ERR_DEVICE_CHECK = 4, 5, 6
BQ_FMT_RABIT2, BQ_FMT_BITNET_W1A8, BQ_FMT_TERNARY_A8, BQ_FMT_ABQ, BQ_FMT_BVSR4, BQ_FMT_RABIT3 = 1, 2, 3, 4, 5, 6
FORMATS = {"rabit": 1, "bitnet": 2, "ternary": 3, "abq": 4, "bvsr": 5, "rabit3": 6}


class bq_pack_desc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("w_bits", ctypes.c_int32), ("a_bits", ctypes.c_int32),
                ("lora_rank", ctypes.c_int32), ("lora_alpha", ctypes.c_float), ("h2", ctypes.c_void_p),
                ("lora_A", ctypes.c_void_p), ("lora_B", ctypes.c_void_p), ("rabit_svid_rounds", ctypes.c_int32),
                ("abq_bit_balance", ctypes.c_int32), ("abq_comp_a", ctypes.c_void_p),
                ("abq_comp_b", ctypes.c_void_p), ("h3", ctypes.c_void_p), ("bvsr_cluster_rounds", ctypes.c_int32)]


class bq_plan_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens_per_cta", "token_groups", "ctas_per_group",
                                              "warps_per_row_block", "tiles_per_warp", "ring_stages",
                                              "tiles_per_stage", "x_chunks_per_thread")] + \
               [("shared_bytes", ctypes.c_uint32)]


class bq_layer(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("N_pad", ctypes.c_int32), ("K_pad", ctypes.c_int32), ("w_bits", ctypes.c_int32),
                ("a_bits", ctypes.c_int32), ("lora_rank", ctypes.c_int32),
                ("packed_bytes", ctypes.c_uint64), ("packed", ctypes.c_void_p)]


class bq_scaled_weights(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("ld", ctypes.c_int64), ("expert_stride", ctypes.c_int64), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("experts", ctypes.c_int32)]


_P = ctypes.c_void_p
_I, _L = ctypes.c_int32, ctypes.c_int64
_SW = ctypes.POINTER(bq_scaled_weights)
_SIGS = {
    "bq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "bq_version": (ctypes.c_int32, []),
    "bq_packed_bytes": (ctypes.c_int, [ctypes.POINTER(bq_pack_desc), ctypes.c_int32, ctypes.c_int32,
                                       ctypes.POINTER(ctypes.c_size_t)]),
    "bq_pack_weights": (ctypes.c_int, [ctypes.POINTER(bq_pack_desc), _P, ctypes.c_int32, ctypes.c_int32, _P,
                                       ctypes.c_size_t, _P, ctypes.POINTER(bq_layer)]),
    "bq_packed_validate": (ctypes.c_int, [_P, ctypes.c_size_t, _P, ctypes.POINTER(bq_layer)]),
    "bq_act_bytes": (ctypes.c_int, [ctypes.POINTER(bq_layer), ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "bq_quantize_act": (ctypes.c_int, [ctypes.POINTER(bq_layer), _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "bq_gemv": (ctypes.c_int, [ctypes.POINTER(bq_layer), _P, _P, _P, _P]),
    "bq_gemm": (ctypes.c_int, [ctypes.POINTER(bq_layer), _P, ctypes.c_int32, _P, _P, _P]),
    "bq_linear_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(bq_layer), ctypes.c_int32,
                                                 ctypes.POINTER(ctypes.c_size_t)]),
    "bq_linear": (ctypes.c_int, [ctypes.POINTER(bq_layer), _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]),
    "bq_linear_static_scratch": (ctypes.c_int, [ctypes.POINTER(bq_layer), _P, ctypes.c_int32, _P, _P, _P]),
    "bq_linear_plan": (ctypes.c_int, [ctypes.POINTER(bq_layer), ctypes.c_int32, ctypes.c_int32,
                                      ctypes.POINTER(bq_plan_info)]),
    "bq_linear_group": (ctypes.c_int, [ctypes.POINTER(bq_layer), ctypes.c_int32, _P, ctypes.c_int32,
                                       ctypes.POINTER(_P), ctypes.POINTER(_P), _P]),
    "bq_device_check": (ctypes.c_int, []),
    "bq_scaled_quantize": (ctypes.c_int, [_P, _I, _L, _I, _P, _L, _P, _I, _I, _P, _L, _P, _P]),
    "bq_scaled_gemm": (ctypes.c_int, [_SW, _P, _L, _P, _I, _P, _I, _L, _P]),
    "bq_scaled_gemm_grouped": (ctypes.c_int, [_SW, _P, _L, _P, _I, _P, _P, _I, _L, _P]),
    "bq_scaled_workspace_bytes": (ctypes.c_int, [_SW, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "bq_scaled_linear": (ctypes.c_int, [_SW, _P, _I, _L, _I, _P, _I, _L, _P, ctypes.c_size_t, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args

EXPORTED = tuple(_SIGS)

# the struct layouts below are those of this ABI version of include/bq.h
BQ_ABI_VERSION = 4
if _lib.bq_version() != BQ_ABI_VERSION:
    raise ImportError(f"{LIB_PATH} has ABI version {_lib.bq_version()}, this binding needs {BQ_ABI_VERSION}; "
                      "rebuild it with bit_weight_quantization_b200.build.build(force=True)")


class BQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bq_status_str(status)} (status {status})")


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else int(stream.cuda_stream)
    import torch
    return int(torch.cuda.current_stream().cuda_stream)


def _check(st: int, where: str):
    if st != BQ_OK:
        raise BQError(st, where)


def bq_status_str(status: int) -> str:
    return _lib.bq_status_str(status).decode()


def bq_version() -> int:
    return _lib.bq_version()


def make_desc(fmt, w_bits=0, a_bits=0, lora_rank=0, lora_alpha=0.1, h2=None, lora_A=None, lora_B=None,
              rabit_svid_rounds=0, abq_bit_balance=0, abq_comp_a=None, abq_comp_b=None, h3=None,
              bvsr_cluster_rounds=0):
    return bq_pack_desc(FORMATS.get(fmt, fmt), w_bits, a_bits, lora_rank, lora_alpha,
                        _ptr(h2), _ptr(lora_A), _ptr(lora_B), rabit_svid_rounds, abq_bit_balance,
                        _ptr(abq_comp_a), _ptr(abq_comp_b), _ptr(h3), bvsr_cluster_rounds)


def bq_packed_bytes(desc: bq_pack_desc, N: int, K: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.bq_packed_bytes(ctypes.byref(desc), N, K, ctypes.byref(out)), "bq_packed_bytes")
    return out.value


def bq_pack_weights(desc: bq_pack_desc, W, N: int, K: int, packed, packed_bytes: int, stream=None) -> bq_layer:
    layer = bq_layer()
    _check(_lib.bq_pack_weights(ctypes.byref(desc), _ptr(W), N, K, _ptr(packed), packed_bytes,
                                _stream(stream), ctypes.byref(layer)), "bq_pack_weights")
    return layer


def bq_packed_validate(packed_host: bytes, packed_dev) -> bq_layer:
    layer = bq_layer()
    buf = ctypes.create_string_buffer(bytes(packed_host), len(packed_host))
    _check(_lib.bq_packed_validate(buf, len(packed_host), _ptr(packed_dev), ctypes.byref(layer)),
           "bq_packed_validate")
    return layer


def bq_act_bytes(layer: bq_layer, M: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.bq_act_bytes(ctypes.byref(layer), M, ctypes.byref(out)), "bq_act_bytes")
    return out.value


def bq_quantize_act(layer: bq_layer, x_bf16, M: int, act, act_bytes: int, stream=None) -> None:
    _check(_lib.bq_quantize_act(ctypes.byref(layer), _ptr(x_bf16), M, _ptr(act), act_bytes, _stream(stream)),
           "bq_quantize_act")


def bq_gemv(layer: bq_layer, act, y, acc_dbg=None, stream=None) -> None:
    _check(_lib.bq_gemv(ctypes.byref(layer), _ptr(act), _ptr(y), _ptr(acc_dbg), _stream(stream)), "bq_gemv")


def bq_gemm(layer: bq_layer, act, M: int, y, acc_dbg=None, stream=None) -> None:
    _check(_lib.bq_gemm(ctypes.byref(layer), _ptr(act), M, _ptr(y), _ptr(acc_dbg), _stream(stream)), "bq_gemm")


def bq_linear_workspace_bytes(layer: bq_layer, M: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.bq_linear_workspace_bytes(ctypes.byref(layer), M, ctypes.byref(out)), "bq_linear_workspace_bytes")
    return out.value


def bq_linear_plan(layer: bq_layer, M: int, fused: bool = True) -> dict:
    """The work split of bq_linear (fused) or bq_gemm for `layer` and M tokens (host only)."""
    info = bq_plan_info()
    _check(_lib.bq_linear_plan(ctypes.byref(layer), M, int(fused), ctypes.byref(info)), "bq_linear_plan")
    return {n: getattr(info, n) for n, _ in bq_plan_info._fields_}


BQ_STATIC_SCRATCH_BYTES = 1 << 20
BQ_MAX_GROUP = 4


def bq_linear_group(layers, x_bf16, M: int, ys, accs=None, stream=None) -> None:
    """Several layers sharing the input x in one launch (bq_linear_group)."""
    n = len(layers)
    arr = (bq_layer * n)(*layers)
    yp = (_P * n)(*[_ptr(y) for y in ys])
    ap = None if accs is None else (_P * n)(*[_ptr(a) for a in accs])
    _check(_lib.bq_linear_group(arr, n, _ptr(x_bf16), M, yp, ap, _stream(stream)), "bq_linear_group")


def bq_linear_static_scratch(layer: bq_layer, x_bf16, M: int, y, acc_dbg=None, stream=None) -> None:
    """bq_linear with the library's fixed scratch array instead of a workspace."""
    _check(_lib.bq_linear_static_scratch(ctypes.byref(layer), _ptr(x_bf16), M, _ptr(y), _ptr(acc_dbg),
                                         _stream(stream)), "bq_linear_static_scratch")


def bq_linear(layer: bq_layer, x_bf16, M: int, y, acc_dbg=None, workspace=None, workspace_bytes: int = 0,
              stream=None) -> None:
    _check(_lib.bq_linear(ctypes.byref(layer), _ptr(x_bf16), M, _ptr(y), _ptr(acc_dbg), _ptr(workspace),
                          workspace_bytes, _stream(stream)), "bq_linear")


def bq_device_check() -> None:
    _check(_lib.bq_device_check(), "bq_device_check")


BQ_TYPE_F32, BQ_TYPE_BF16, BQ_TYPE_F16 = 0, 1, 2
BQ_MAX_EXPERTS = 1024


def bq_scaled_quantize(x, x_type: int, ldx: int, x_rows: int, gate, ldg: int, rows, M: int, K: int, q, ldq: int,
                       scale, stream=None) -> None:
    _check(_lib.bq_scaled_quantize(_ptr(x), x_type, ldx, x_rows, _ptr(gate), ldg, _ptr(rows), M, K, _ptr(q), ldq,
                                   _ptr(scale), _stream(stream)), "bq_scaled_quantize")


def bq_scaled_gemm(w: bq_scaled_weights, q, ldq: int, scale, M: int, y, y_type: int, ldy: int, stream=None) -> None:
    _check(_lib.bq_scaled_gemm(ctypes.byref(w), _ptr(q), ldq, _ptr(scale), M, _ptr(y), y_type, ldy,
                               _stream(stream)), "bq_scaled_gemm")


def bq_scaled_gemm_grouped(w: bq_scaled_weights, q, ldq: int, scale, M: int, offsets, y, y_type: int, ldy: int,
                           stream=None) -> None:
    _check(_lib.bq_scaled_gemm_grouped(ctypes.byref(w), _ptr(q), ldq, _ptr(scale), M, _ptr(offsets), _ptr(y), y_type,
                                       ldy, _stream(stream)), "bq_scaled_gemm_grouped")


def bq_scaled_workspace_bytes(w: bq_scaled_weights, M: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.bq_scaled_workspace_bytes(ctypes.byref(w), M, ctypes.byref(out)), "bq_scaled_workspace_bytes")
    return out.value


def bq_scaled_linear(w: bq_scaled_weights, x, x_type: int, ldx: int, M: int, y, y_type: int, ldy: int, workspace,
                     workspace_bytes: int, stream=None) -> None:
    _check(_lib.bq_scaled_linear(ctypes.byref(w), _ptr(x), x_type, ldx, M, _ptr(y), y_type, ldy, _ptr(workspace),
                                 workspace_bytes, _stream(stream)), "bq_scaled_linear")


def raw_status(name: str, *args) -> int:
    """Call an ABI function and return its status code without raising (for fault tests)."""
    return getattr(_lib, name)(*args)


class QuantLinear:
    """Device buffers (torch allocations) for one packed layer plus the calls on them.

    Owns: the packed buffer. Per call: an activation buffer for M tokens and y.
    All arithmetic happens in the library."""

    def __init__(self, fmt, W, *, w_bits=0, a_bits=0, lora_rank=0, lora_alpha=0.1, h2=None,
                 lora_A=None, lora_B=None, rabit_svid_rounds=0, abq_bit_balance=0, abq_comp_a=None,
                 abq_comp_b=None, h3=None, bvsr_cluster_rounds=0, stream=None):
        import torch
        N, K = W.shape
        self.desc = make_desc(fmt, w_bits, a_bits, lora_rank, lora_alpha, h2, lora_A, lora_B, rabit_svid_rounds,
                              abq_bit_balance, abq_comp_a, abq_comp_b, h3, bvsr_cluster_rounds)
        nbytes = bq_packed_bytes(self.desc, N, K)
        self.packed = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
        self.layer = bq_pack_weights(self.desc, W, N, K, self.packed, nbytes, stream)
        # the pack reads W, h2, h3, the LoRA matrices and a, b asynchronously: wait before the caller may free them
        torch.cuda.synchronize(W.device)
        self.N, self.K = N, K
        self._acts = {}

    def act_buffer(self, M):
        import torch
        if M not in self._acts:
            n = bq_act_bytes(self.layer, M)
            self._acts[M] = torch.empty(n, dtype=torch.uint8, device=self.packed.device)
        return self._acts[M]

    def quantize_act(self, x_bf16, stream=None):
        M = x_bf16.shape[0]
        act = self.act_buffer(M)
        bq_quantize_act(self.layer, x_bf16, M, act, act.numel(), stream)
        return act

    def workspace(self, M):
        import torch
        key = ("ws", M)
        if key not in self._acts:
            n = bq_linear_workspace_bytes(self.layer, M)
            self._acts[key] = torch.empty(max(n, 256), dtype=torch.uint8, device=self.packed.device)
        return self._acts[key]

    def linear(self, x_bf16, y=None, acc_dbg=None, stream=None):
        """Fused activation quantization + layer (bq_linear)."""
        import torch
        M = x_bf16.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float32, device=x_bf16.device)
        ws = self.workspace(M)
        bq_linear(self.layer, x_bf16, M, y, acc_dbg, ws, ws.numel(), stream)
        return y

    def forward(self, x_bf16, y=None, acc_dbg=None, stream=None):
        import torch
        M = x_bf16.shape[0]
        act = self.quantize_act(x_bf16, stream)
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float32, device=x_bf16.device)
        if M == 1:
            bq_gemv(self.layer, act, y, acc_dbg, stream)
        else:
            bq_gemm(self.layer, act, M, y, acc_dbg, stream)
        return y


class StepGraph:
    """A fixed sequence of this library's calls, captured once into a CUDA graph and replayed.

    This is how a decode loop avoids paying the host cost of every call on every step: the
    calls in ``issue()`` (which enqueue on torch's current stream, the default of every call
    here) are captured on ``stream`` after ``warmup`` eager runs. The buffers they read and
    write are fixed in the graph, so a step refreshes their contents (e.g. one copy into the
    input buffer), calls ``replay()``, and reads the outputs. ``replay()`` enqueues the whole
    step on torch's current stream. The library allocates nothing and never synchronizes in
    its compute calls, which is what makes them capturable. ``issue()`` may fork work onto other
    streams and join it back before returning (e.g. read each call's outputs back to pinned host
    memory on a copy stream while the later calls run)."""

    def __init__(self, issue, stream=None, warmup: int = 1):
        import torch
        s = stream if stream is not None else torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(warmup):
                issue()
        s.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=s):
            issue()
        s.synchronize()

    def replay(self) -> None:
        self.graph.replay()


# ---------------------------------------------------------------------------------------------------
# scaled int8 layers on torch tensors
# ---------------------------------------------------------------------------------------------------

def _types():
    import torch
    return {torch.float32: BQ_TYPE_F32, torch.bfloat16: BQ_TYPE_BF16, torch.float16: BQ_TYPE_F16}


def _need(ok, where, what):
    if not ok:
        raise BQError(BQ_ERR_INVALID_ARG, f"{where}: {what}")


class _On:
    """Makes a tensor's device current, and `stream` (a torch stream) torch's current one, so that outputs
    and workspaces allocated inside belong to the stream that uses them."""

    def __init__(self, device, stream):
        import torch
        self._ctx = [] if torch.cuda.current_device() == device.index else [torch.cuda.device(device)]
        if stream is not None:
            _need(isinstance(stream, torch.cuda.Stream) and stream.device == device, "stream",
                  "a torch.cuda.Stream of the tensors' device")
            self._ctx.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self._ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._ctx):
            c.__exit__(*exc)


def _rows_of(t, name, where, K=None, dtypes=None, device=None):
    """A 2-D CUDA matrix with unit column stride: its row stride in elements."""
    import torch
    _need(isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2, where, f"{name} is a 2-D CUDA tensor")
    _need(dtypes is None or t.dtype in dtypes, where, f"{name} has dtype {t.dtype}")
    _need(device is None or t.device == device, where, f"{name} is on {t.device}")
    _need(K is None or t.shape[1] == K, where, f"{name} has {t.shape[1]} columns, not {K}")
    _need(t.shape[1] <= 1 or t.stride(1) == 1, where, f"{name} has column stride {t.stride(1)}")
    return max(t.stride(0), t.shape[1]) if t.shape[0] <= 1 else t.stride(0)


def _vector(t, name, where, n, dtype, device):
    import torch
    _need(isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.is_contiguous() and
          t.numel() == n, where, f"{name} is {n} contiguous {dtype} on {device}")


def empty_codes(rows: int, K: int, device):
    """An int8 matrix [rows, K] whose rows start on 16-byte boundaries."""
    import torch
    return torch.empty((rows, (K + 15) // 16 * 16), dtype=torch.int8, device=device)[:, :K]


def scaled_quantize(x, gate=None, rows=None, q=None, scale=None, stream=None):
    """Per-row int8 codes and scales of x [*, K] (f32, bf16 or f16; see bq_scaled_quantize in include/bq.h):
    of all rows, or with `rows` (int32 [M]) of row rows[i] for every i (negative: an empty slot); with `gate`
    of x * SiLU(gate). Returns (q [M, K] int8, scale [M] f32), written to `q` and `scale` where given."""
    import torch
    where, types = "scaled_quantize", _types()
    ldx = _rows_of(x, "x", where, dtypes=types)
    dev, K, ldg = x.device, x.shape[1], 0
    if gate is not None:
        ldg = _rows_of(gate, "gate", where, K, (x.dtype,), dev)
        _need(gate.shape[0] == x.shape[0], where, f"gate has {gate.shape[0]} rows, x {x.shape[0]}")
    M = x.shape[0]
    if rows is not None:
        _need(rows.dim() == 1, where, "rows is 1-D")
        M = rows.shape[0]
        _vector(rows, "rows", where, M, torch.int32, dev)
    with _On(dev, stream):
        if q is None:
            q = empty_codes(M, K, dev)
        else:
            _rows_of(q, "q", where, K, (torch.int8,), dev)
            _need(q.shape[0] == M, where, f"q has {q.shape[0]} rows, not {M}")
        if scale is None:
            scale = torch.empty(M, dtype=torch.float32, device=dev)
        else:
            _vector(scale, "scale", where, M, torch.float32, dev)
        ldq = q.stride(0) if M > 1 else (K + 15) // 16 * 16
        bq_scaled_quantize(x, types[x.dtype], ldx, x.shape[0], gate, ldg, rows, M, K, q, ldq, scale)
    return q, scale


class ScaledLinear:
    """A layer (or one per expert) of int8 codes [N, K] (or [E, N, K]) with a scale per output channel.

    Holds references to the tensors it is given; `codes` whose rows do not start on 16-byte boundaries
    are copied once into rows that do. Nothing is kept between calls: outputs and workspaces are
    allocated per call on the stream that runs it (or given, `y`), so calls on several streams and
    several captured graphs do not share memory."""

    def __init__(self, codes, scale, bias=None):
        import torch
        where = "ScaledLinear"
        _need(codes.is_cuda and codes.dtype == torch.int8 and codes.dim() in (2, 3) and min(codes.shape) >= 1, where,
              "codes is a CUDA int8 tensor [N, K] or [E, N, K]")
        c3 = codes if codes.dim() == 3 else codes[None]
        E, N, K = c3.shape
        se, sn, sk = c3.stride()
        sn, se = (sn if N > 1 else (K + 15) // 16 * 16), (se if E > 1 else 0)
        if (sk != 1 and K > 1) or sn % 16 or sn < K or se % 16 or se < 0 or c3.data_ptr() % 16:
            buf = torch.zeros((E, N, (K + 15) // 16 * 16), dtype=torch.int8, device=codes.device)
            buf[:, :, :K] = c3
            c3 = buf[:, :, :K]
            sn, se = buf.stride(1), buf.stride(0)
        _vector(scale, "scale", where, E * N, torch.float32, codes.device)
        if bias is not None:
            _vector(bias, "bias", where, E * N, torch.float32, codes.device)
        self.codes, self.scale, self.bias, self.device = c3, scale, bias, codes.device
        self.experts, self.N, self.K = E, N, K
        self.grouped = codes.dim() == 3
        self.weights = bq_scaled_weights(c3.data_ptr(), scale.data_ptr(), _ptr(bias), sn, se, N, K, E)

    @classmethod
    def quantize(cls, W, bias=None):
        """Codes and scales of W [N, K] or [E, N, K] (f32, bf16 or f16), one scale per output channel."""
        q, s = scaled_quantize(W.reshape(-1, W.shape[-1]))
        ld = q.stride(0) if q.shape[0] > 1 else (W.shape[-1] + 15) // 16 * 16
        q = q.as_strided(W.shape, (W.shape[-2] * ld, ld, 1)[-W.dim():])
        return cls(q, s.view(W.shape[:-1]), bias)

    def _out(self, y, M, dtype, where):
        import torch
        if y is None:
            return torch.empty((M, self.N), dtype=dtype, device=self.device), self.N
        ldy = _rows_of(y, "y", where, self.N, _types(), self.device)
        _need(y.shape[0] == M and (dtype is None or y.dtype == dtype), where, f"y is {M} rows of {dtype or y.dtype}")
        return y, ldy

    def _codes_in(self, q, scale, where):
        import torch
        _rows_of(q, "q", where, self.K, (torch.int8,), self.device)
        M = q.shape[0]
        _vector(scale, "scale", where, M, torch.float32, self.device)
        return M, q.stride(0) if M > 1 else (self.K + 15) // 16 * 16

    def linear(self, x, y=None, dtype=None, stream=None):
        """x [M, K] (f32, bf16 or f16) quantized per token, then the layer: y [M, N] of `dtype` (x's by default)."""
        import torch
        where, types = "ScaledLinear.linear", _types()
        ldx = _rows_of(x, "x", where, self.K, types, self.device)
        M = x.shape[0]
        with _On(self.device, stream):
            y, ldy = self._out(y, M, dtype if y is not None else dtype or x.dtype, where)
            _need(y.dtype in types, where, f"y has dtype {y.dtype}")
            n = bq_scaled_workspace_bytes(self.weights, M)
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
            bq_scaled_linear(self.weights, x, types[x.dtype], ldx, M, y, types[y.dtype], ldy, ws, n)
        return y

    def gemm(self, q, scale, y=None, dtype=None, stream=None):
        """The layer on quantized rows (scaled_quantize): y [M, N] of `dtype` (bf16 by default)."""
        import torch
        where, types = "ScaledLinear.gemm", _types()
        M, ldq = self._codes_in(q, scale, where)
        with _On(self.device, stream):
            y, ldy = self._out(y, M, dtype if y is not None else dtype or torch.bfloat16, where)
            _need(y.dtype in types, where, f"y has dtype {y.dtype}")
            bq_scaled_gemm(self.weights, q, ldq, scale, M, y, types[y.dtype], ldy)
        return y

    def gemm_grouped(self, q, scale, offsets, y=None, dtype=None, stream=None):
        """Expert e's layer on the rows offsets[e] .. offsets[e + 1] - 1 (offsets: int32 [E + 1] on the device).
        Rows outside every group keep what `y` held (undefined in a `y` that is allocated here)."""
        import torch
        where, types = "ScaledLinear.gemm_grouped", _types()
        M, ldq = self._codes_in(q, scale, where)
        _vector(offsets, "offsets", where, self.experts + 1, torch.int32, self.device)
        with _On(self.device, stream):
            y, ldy = self._out(y, M, dtype if y is not None else dtype or torch.bfloat16, where)
            _need(y.dtype in types, where, f"y has dtype {y.dtype}")
            bq_scaled_gemm_grouped(self.weights, q, ldq, scale, M, offsets, y, types[y.dtype], ldy)
        return y
