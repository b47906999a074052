"""The scaled int8 layers in plain numpy: codes by the f32 roundings of their definition, everything
else in 64 bits, and the error each output may have. No code of the library is used."""
import numpy as np

U = 2.0 ** -24                                     # half a step of f32, relative
HALF_STEP = {"fp32": 0.0, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # of the last rounding, relative to the value
SMALLEST = {"fp32": 2.0 ** -150, "bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half a subnormal step


def gated(x, gate):
    x, g = np.asarray(x, np.float64), np.asarray(gate, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return x * (g / (1 + np.exp(-g)))


def quantize(v, rows=None):
    """(codes int8, scale f64) of f32 values v [R, K], without the gate."""
    v = np.asarray(v, np.float32)
    if rows is not None:
        v = np.stack([v[r] if r >= 0 else np.zeros(v.shape[1], np.float32) for r in rows]) if len(rows) else v[:0]
    with np.errstate(all="ignore"):
        gamma = np.abs(v).max(1)
        bad = ~np.isfinite(v).all(1)
        some = ~bad & (gamma >= np.float32(2.0 ** -100))
        inverse = np.float32(1) / np.where(some, gamma, np.float32(1)).astype(np.float32)
        s = np.where(some, np.float32(127) * inverse, np.float32(0)).astype(np.float32)
        prod = np.where(some[:, None], v, np.float32(0)) * s[:, None]
        assert prod.dtype == np.float32
        q = np.rint(prod).astype(np.int8)
        scale = np.where(bad, np.nan, np.where(some, gamma.astype(np.float64) / 127, 0.0))
    return q, scale


def gemm(q, sa, w, sw, bias=None):
    """(y f64, |product| f64) with y = (q w^T) sa sw + bias."""
    acc = np.asarray(q, np.float64) @ np.asarray(w, np.float64).T  # whole numbers below 2^53: exact
    p = acc * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
    return (p if bias is None else p + np.asarray(bias, np.float64)[None, :]), np.abs(p)


def tolerance(y, p, kind, bias):
    """Three f32 roundings of the product (the sum, the two scales, their product with it), or two and the
    fused sum's own, then one to the output type; 1.01 covers their second-order terms."""
    first = 2 * U * p + U * np.abs(y) if bias else 3 * U * p
    return 1.01 * (first + HALF_STEP[kind] * (np.abs(y) + first)) + SMALLEST[kind]
