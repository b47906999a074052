"""The scaled int8 layers on the GPU against plain numpy in 64 bits (tests/scaled_ref.py)."""
import numpy as np
import pytest

from tests import scaled_ref as R

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp16", "fp32"]


def mods():
    import torch
    from bit_weight_quantization_b200 import bq
    return torch, bq


def kind(torch, name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def host(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def codes(torch, rng, rows, K, pad=0, lo=-128, hi=127, offset=0):
    """Random codes and their device copy in rows of a stride that is a multiple of 16 (+ pad rows of 16),
    the bytes around them set to 77."""
    h = rng.integers(lo, hi + 1, (rows, K)).astype(np.int8)
    ld = (K + 15) // 16 * 16 + 16 * pad
    buf = torch.full((rows + offset, ld), 77, dtype=torch.int8, device="cuda")
    buf[offset:, :K] = torch.from_numpy(h).cuda()
    return h, buf[offset:, :K]


def scales(torch, rng, n):
    h = (rng.random(n) * 2e-3 + 1e-4).astype(np.float32)
    return h, torch.from_numpy(h).cuda()


def check(bq, y, y_ref, p, name, bias):
    bq.bq_device_check()
    got = host(y).astype(np.float64)
    off = np.abs(got - y_ref)
    tol = R.tolerance(y_ref, p, name, bias)
    assert np.all(off <= tol), (float((off / tol).max()), np.argwhere(off > tol)[:4].tolist())


# ---------------------------------------------------------------------------------------------------
# quantization
# ---------------------------------------------------------------------------------------------------

def check_quantize(bq, torch, q, s, v):
    bq.bq_device_check()
    qr, sr = R.quantize(v)
    assert np.array_equal(host(q), qr)
    sg = host(s).astype(np.float64)
    assert np.array_equal(np.isnan(sg), np.isnan(sr))
    ok = ~np.isnan(sr)
    assert np.all(np.abs(sg[ok] - sr[ok]) <= R.U * sr[ok])  # one rounding


@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (2, 8), (3, 15), (5, 16), (1, 128), (33, 129), (2, 1000), (1, 4096),
                                 (300, 512), (7, 4095), (3, 11008), (2, 16384), (1, 30001), (2, 65536), (2000, 96)])
def test_quantize(M, K, name):
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(M * 70001 + K)
    x = (torch.randn(M, K, generator=g, device="cuda") * 3).to(kind(torch, name))
    q, s = bq.scaled_quantize(x)
    assert q.shape == (M, K) and q.dtype == torch.int8 and s.shape == (M,)
    check_quantize(bq, torch, q, s, host(x))


@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("K,ld,start", [(40, 41, 0), (40, 48, 1), (1001, 1003, 3), (4096, 4104, 8), (512, 1024, 512),
                                        (2048, 2049, 0)])
def test_quantize_strides_and_untouched_bytes(K, ld, start, name):
    torch, bq = mods()
    M = 9
    g = torch.Generator(device="cuda").manual_seed(K + ld)
    flat = torch.randn(start + M * ld + 16, generator=g, device="cuda").to(kind(torch, name))
    x = flat.as_strided((M, K), (ld, 1), start)
    big = torch.full((M + 2, (K + 15) // 16 * 16 + 32), 55, dtype=torch.int8, device="cuda")
    scale = torch.full((M + 2,), 5.0, device="cuda")
    q, s = bq.scaled_quantize(x, q=big[1:M + 1, :K], scale=scale[1:M + 1])
    check_quantize(bq, torch, q, s, host(x))
    assert torch.all(big[0] == 55) and torch.all(big[-1] == 55) and torch.all(big[:, K:] == 55)
    assert scale[0] == 5 and scale[-1] == 5


def test_quantize_special_rows():
    torch, bq = mods()
    K = 264
    x = torch.randn(12, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[1] = 0
    x[2] = -0.0
    x[3, 5] = float("nan")
    x[4, 263] = float("inf")
    x[5, 0] = float("-inf")
    x[6] *= 1e-36           # below 2^-100: a zero row
    x[7] = 0
    x[7, 200] = 2.0 ** -100  # the smallest that counts
    x[8] *= 1e37
    x[9] = 3.0e38
    x[10] = torch.arange(K, device="cuda") % 128 - 0.5   # near ties: s is about 127 / 126.5
    x[11] = (torch.arange(K, device="cuda") % 255 - 127).float()
    for t in (x, x.bfloat16()):
        q, s = bq.scaled_quantize(t)
        check_quantize(bq, torch, q, s, host(t))
    assert torch.equal(q[11, :255].cpu(), torch.arange(-127, 128, dtype=torch.int8))


@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("M,K", [(1, 1), (4, 100), (65, 1024), (3, 11008)])
def test_quantize_gated(M, K, name):
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(M + K)
    both = (torch.randn(M, 2 * K + 1, generator=g, device="cuda") * 3).to(kind(torch, name))
    gate, up = both[:, :K], both[:, K:2 * K]
    q, s = bq.scaled_quantize(up, gate=gate)
    bq.bq_device_check()
    v = R.gated(host(up), host(gate))
    gamma = np.abs(v).max(1)
    # v in f32: exp within 2 units (4 half steps of 1 + exp(-g) at most), one half step each for the sum, the
    # quotient and the product: 7 U. Codes carry v's and gamma's, and the half steps of 1 / gamma, 127 / gamma and v s.
    rel = 7 * R.U
    assert np.all(np.abs(host(s) - gamma / 127) <= 1.01 * (rel + R.U) * gamma / 127)
    live = gamma > 0
    exact = v[live] * (127 / gamma[live])[:, None]
    assert np.all(np.abs(host(q)[live] - exact) <= 0.5 + 1.01 * 127 * (2 * rel + 3 * R.U))


def test_quantize_gate_extremes():
    torch, bq = mods()
    inf = float("inf")
    gate = torch.tensor([[-100.0, 100.0, 0.0, -200.0], [inf, 1, 1, 1], [-inf, 1, 1, 1], [1, 1, 1, 1]], device="cuda")
    up = torch.tensor([[1.0, 2.0, 3.0, 4.0], [1, 1, 1, 1], [1, 1, 1, 1], [0, 0, inf, 0]], device="cuda")
    q, s = bq.scaled_quantize(up, gate=gate)
    bq.bq_device_check()
    # SiLU(-100) is 0 at 8 bits; SiLU(inf) = inf and SiLU(-inf) = -inf / inf are rows that cannot be represented
    assert q.cpu().tolist() == [[0, 127, 0, 0], [0] * 4, [0] * 4, [0] * 4]
    assert abs(s[0].item() - 200 / 127) < 1e-6 and torch.isnan(s[1:]).all()


@pytest.mark.parametrize("name", KINDS)
def test_quantize_rows(name):
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(10, 200, generator=g, device="cuda").to(kind(torch, name))
    rows = [3, 3, 0, 9, -1, 5, -7, 3]
    q, s = bq.scaled_quantize(x, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    bq.bq_device_check()
    qr, sr = R.quantize(host(x), rows)
    assert np.array_equal(host(q), qr)
    assert np.all(np.abs(host(s) - sr) <= R.U * sr)


def test_quantize_rows_out_of_range_raise_the_error_word():
    torch, bq = mods()
    x = torch.randn(4, 64, device="cuda")
    q, s = bq.scaled_quantize(x, rows=torch.tensor([1, 4, 2], dtype=torch.int32, device="cuda"))
    with pytest.raises(bq.BQError) as e:
        bq.bq_device_check()
    assert e.value.status == bq.BQ_ERR_DEVICE_CHECK
    bq.bq_device_check()  # cleared
    qr, sr = R.quantize(host(x))
    assert np.array_equal(host(q)[[0, 2]], qr[[1, 2]]) and torch.all(q[1] == 0) and torch.isnan(s[1])
    # an x without rows and only empty slots
    q, s = bq.scaled_quantize(x[:0], rows=torch.full((3,), -1, dtype=torch.int32, device="cuda"))
    bq.bq_device_check()
    assert torch.all(q == 0) and torch.all(s == 0)


# ---------------------------------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------------------------------

SHAPES = [(1, 1, 1), (1, 16, 16), (3, 7, 5), (1, 4096, 4096), (2, 128, 128), (7, 129, 257), (16, 300, 1000),
          (17, 1000, 33), (31, 512, 2049), (32, 64, 4096), (33, 255, 640), (63, 130, 129), (64, 2048, 2048),
          (65, 257, 127), (96, 96, 96), (127, 384, 1111), (128, 128, 128), (129, 640, 512), (200, 1025, 300),
          (256, 256, 256), (257, 257, 257), (300, 300, 5111), (333, 5120, 640), (512, 513, 64), (1000, 100, 100),
          (1, 13824, 5120), (5, 11008, 4096), (24, 40, 16400), (2049, 300, 130), (100, 16, 64), (70, 8, 32), (100, 24, 200),
          (64, 13824, 256), (8, 300, 4096), (9, 300, 4096), (33, 128, 100), (64, 128, 130), (3, 70, 65536)]


@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, name):
    torch, bq = mods()
    rng = np.random.default_rng(M * 1000003 + N * 1009 + K)
    bias = (M + N + K) % 2 == 0
    w, wd = codes(torch, rng, N, K, pad=(M + K) % 2)
    q, qd = codes(torch, rng, M, K, pad=N % 2)
    sw, swd = scales(torch, rng, N)
    sa, sad = scales(torch, rng, M)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    layer = bq.ScaledLinear(wd, swd, torch.from_numpy(b).cuda() if bias else None)
    y = layer.gemm(qd, sad, dtype=kind(torch, name))
    assert y.shape == (M, N)
    y_ref, p = R.gemm(q, sa, w, sw, b)
    check(bq, y, y_ref, p, name, bias)


@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("N,ldy,start", [(200, 201, 0), (200, 203, 1), (65, 72, 8), (384, 1024, 512), (33, 33, 3)])
def test_gemm_output_strides_and_untouched_memory(M, N, ldy, start, name):
    torch, bq = mods()
    K = 272
    rng = np.random.default_rng(N + ldy + M)
    w, wd = codes(torch, rng, N, K)
    q, qd = codes(torch, rng, M, K)
    sw, swd = scales(torch, rng, N)
    sa, sad = scales(torch, rng, M)
    flat = torch.full((start + M * ldy + 64,), 7.0, dtype=kind(torch, name), device="cuda")
    y = flat.as_strided((M, N), (ldy, 1), start)
    assert bq.ScaledLinear(wd, swd).gemm(qd, sad, y=y) is y
    y_ref, p = R.gemm(q, sa, w, sw)
    check(bq, y, y_ref, p, name, False)
    left = torch.ones(flat.shape, dtype=torch.bool, device="cuda")
    left.as_strided((M, N), (ldy, 1), start).zero_()
    assert torch.all(flat[left] == 7)


@pytest.mark.parametrize("M", [1, 48, 260])
def test_gemm_sums_are_exact_at_the_largest_k(M):
    """All codes -128 at K = 65536: every sum is 2^30; with codes +-127 the sums are whole numbers beyond f32."""
    torch, bq = mods()
    N, K = 40, 65536
    one = torch.ones(max(M, N), device="cuda")
    q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    y = bq.ScaledLinear(w, one[:N]).gemm(q, one[:M], dtype=torch.float32)
    assert torch.all(y == 2.0 ** 30)
    rng = np.random.default_rng(3)
    qh, qd = codes(torch, rng, M, K, lo=100)
    wh, wd = codes(torch, rng, N, K, lo=90)
    y = bq.ScaledLinear(wd, one[:N]).gemm(qd, one[:M], dtype=torch.float32)
    bq.bq_device_check()
    acc = qh.astype(np.int64) @ wh.astype(np.int64).T
    assert np.array_equal(host(y), acc.astype(np.float32))  # rounded once


def test_gemm_nan_scale_stays_in_its_row_and_column():
    torch, bq = mods()
    rng = np.random.default_rng(9)
    for M in (6, 200):
        w, wd = codes(torch, rng, 50, 100)
        q, qd = codes(torch, rng, M, 100)
        sw, swd = scales(torch, rng, 50)
        sa, sad = scales(torch, rng, M)
        sad[3], swd[7] = float("nan"), float("inf")
        y = host(bq.ScaledLinear(wd, swd).gemm(qd, sad, dtype=torch.float32))
        bq.bq_device_check()
        assert np.isnan(y[3]).all() and not np.isfinite(y[:, 7]).any()
        y_ref, p = R.gemm(q, sa, w, sw)
        keep = np.ones((M, 50), bool)
        keep[3], keep[:, 7] = False, False
        assert np.all(np.abs(y - y_ref)[keep] <= R.tolerance(y_ref, p, "fp32", False)[keep])


def test_empty_calls():
    torch, bq = mods()
    layer = bq.ScaledLinear(torch.ones(8, 32, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda"))
    e = torch.empty(0, 32, device="cuda")
    q, s = bq.scaled_quantize(e)
    assert q.shape == (0, 32) and s.shape == (0,)
    assert layer.gemm(q, s).shape == (0, 8) and layer.linear(e).shape == (0, 8)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert layer.gemm_grouped(q, s, off).shape == (0, 8)
    bq.bq_device_check()


# ---------------------------------------------------------------------------------------------------
# grouped by expert
# ---------------------------------------------------------------------------------------------------

def grouped_case(torch, rng, counts, N, K, before=0, after=0, bias=False, wpad=0):
    E, M = len(counts), before + sum(counts) + after
    w, wd = codes(torch, rng, E * N, K, pad=wpad)
    w = w.reshape(E, N, K)
    wd = wd.as_strided((E, N, K), (N * wd.stride(0) if E * N > 1 else (K + 15) // 16 * 16, wd.stride(0), 1))
    q, qd = codes(torch, rng, M, K)
    sw, swd = scales(torch, rng, E * N)
    sa, sad = scales(torch, rng, M)
    b = rng.standard_normal((E, N)).astype(np.float32) if bias else None
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + before
    return dict(w=w, wd=wd, q=q, qd=qd, sw=sw.reshape(E, N), swd=swd.view(E, N), sa=sa, sad=sad, b=b,
                bd=torch.from_numpy(b).cuda() if bias else None, off=off.astype(np.int32),
                offd=torch.from_numpy(off.astype(np.int32)).cuda(), M=M, N=N, E=E)


def grouped_ref(c, off=None):
    off = c["off"] if off is None else off
    y, p = np.full((c["M"], c["N"]), 7.0), np.zeros((c["M"], c["N"]))
    for e in range(c["E"]):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            y[r], p[r] = R.gemm(c["q"][r], c["sa"][r], c["w"][e], c["sw"][e], None if c["b"] is None else c["b"][e])
    return y, p


COUNTS = [[1], [0, 1], [1, 0], [3, 0, 5], [0, 0, 0], [16, 16], [17, 1, 0, 40], [64, 65, 63], [128, 1, 127, 129],
          [300, 0, 2, 513], [1] * 16, [2, 0] * 40, [5, 33, 0, 1, 0, 0, 260, 31]]


@pytest.mark.parametrize("name", ["bf16", "fp32"])
@pytest.mark.parametrize("N,K", [(100, 70), (256, 512), (640, 2064)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c))[:24])
def test_grouped(counts, N, K, name):
    torch, bq = mods()
    rng = np.random.default_rng(sum(counts) * 31 + N + K + len(counts))
    c = grouped_case(torch, rng, counts, N, K, before=len(counts) % 3, after=sum(counts) % 4, bias=N == 100,
                     wpad=len(counts) % 2)
    if c["M"] == 0:
        return
    layer = bq.ScaledLinear(c["wd"], c["swd"], c["bd"])
    y = torch.full((c["M"], N), 7.0, dtype=kind(torch, name), device="cuda")
    layer.gemm_grouped(c["qd"], c["sad"], c["offd"], y=y)
    y_ref, p = grouped_ref(c)
    check(bq, y, y_ref, p, name, c["b"] is not None)
    out = np.ones(c["M"], bool)
    out[c["off"][0]:c["off"][-1]] = False
    assert np.all(host(y)[out] == 7)  # rows outside every group


def test_grouped_many_experts_single_rows():
    torch, bq = mods()
    rng = np.random.default_rng(0)
    counts = (rng.random(1024) < 0.3).astype(int).tolist()
    c = grouped_case(torch, rng, counts, 48, 64)
    y = bq.ScaledLinear(c["wd"], c["swd"]).gemm_grouped(c["qd"], c["sad"], c["offd"], dtype=torch.float32)
    y_ref, p = grouped_ref(c)
    check(bq, y, y_ref, p, "fp32", False)


def test_grouped_equals_the_single_layer_bit_for_bit():
    torch, bq = mods()
    rng = np.random.default_rng(4)
    c = grouped_case(torch, rng, [37, 0, 150, 260], 300, 500, bias=True)
    y = bq.ScaledLinear(c["wd"], c["swd"], c["bd"]).gemm_grouped(c["qd"], c["sad"], c["offd"], dtype=torch.float32)
    for e in range(4):
        r = slice(int(c["off"][e]), int(c["off"][e + 1]))
        one = bq.ScaledLinear(c["wd"][e], c["swd"][e], c["bd"][e])
        assert torch.equal(y[r], one.gemm(c["qd"][r], c["sad"][r], dtype=torch.float32))


@pytest.mark.parametrize("off", [[0, 5, 3, 20], [-1, 5, 6, 20], [0, 5, 6, 21], [0, 30, 40, 50], [3, 2, 2, 2]])
def test_grouped_bad_offsets_leave_y_and_raise_the_error_word(off):
    torch, bq = mods()
    rng = np.random.default_rng(4)
    c = grouped_case(torch, rng, [5, 5, 10], 64, 64)
    y = torch.full((20, 64), 7.0, device="cuda")
    bq.ScaledLinear(c["wd"], c["swd"]).gemm_grouped(c["qd"], c["sad"],
                                                    torch.tensor(off, dtype=torch.int32, device="cuda"), y=y)
    with pytest.raises(bq.BQError) as e:
        bq.bq_device_check()
    assert e.value.status == bq.BQ_ERR_DEVICE_CHECK
    assert torch.all(y == 7)


def test_experts_may_share_weights():
    torch, bq = mods()
    rng = np.random.default_rng(8)
    c = grouped_case(torch, rng, [4, 9], 80, 96)
    shared = c["wd"][:1].expand(2, -1, -1)  # expert stride 0
    y = bq.ScaledLinear(shared, c["swd"]).gemm_grouped(c["qd"], c["sad"], c["offd"], dtype=torch.float32)
    c["w"] = np.stack([c["w"][0]] * 2)
    y_ref, p = grouped_ref(c)
    check(bq, y, y_ref, p, "fp32", False)


# ---------------------------------------------------------------------------------------------------
# linear, classes, streams, graphs, refusals
# ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("name", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (1, 4096, 4096), (1, 5, 3), (2, 64, 16384), (2, 513, 4100), (1, 100, 16390), (4, 2048, 2048),
                                   (7, 77, 7777), (16, 1024, 640), (40, 512, 512), (130, 260, 1030), (513, 100, 256)])
def test_linear_equals_quantize_and_gemm(M, N, K, name):
    torch, bq = mods()
    rng = np.random.default_rng(M + N + K)
    w, wd = codes(torch, rng, N, K)
    sw, swd = scales(torch, rng, N)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda().to(kind(torch, name))
    if M > 3:
        x[2] = 0
        x[3, K // 2] = float("nan")
    layer = bq.ScaledLinear(wd, swd, torch.from_numpy(rng.standard_normal(N).astype(np.float32)).cuda() if M % 2 else None)
    y = layer.linear(x)
    assert y.dtype == x.dtype
    q, s = bq.scaled_quantize(x)
    two = layer.gemm(q, s, dtype=x.dtype)
    bq.bq_device_check()
    assert torch.equal(torch.nan_to_num(y.float(), nan=1e9), torch.nan_to_num(two.float(), nan=1e9))
    qr, sr = R.quantize(host(x))
    assert np.array_equal(host(q), qr)
    assert M <= 3 or torch.isnan(y[3]).all()


def test_quantized_weights_class():
    torch, bq = mods()
    W = torch.randn(3, 50, 70, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    layer = bq.ScaledLinear.quantize(W)
    q, s = R.quantize(host(W).reshape(150, 70))
    assert np.array_equal(host(layer.codes).reshape(150, 70), q)
    assert layer.experts == 3 and layer.N == 50 and layer.K == 70
    one = bq.ScaledLinear.quantize(W[0], bias=torch.ones(50, device="cuda"))
    x = torch.randn(4, 70, device="cuda")
    near = x @ W[0].T + 1
    assert (one.linear(x) - near).abs().max() < 0.05 * near.abs().max()
    # codes whose rows do not start on 16-byte boundaries are laid out once
    odd = torch.from_numpy(q.reshape(3, 50, 70)).cuda()
    again = bq.ScaledLinear(odd, layer.scale)
    off = torch.tensor([0, 1, 4, 4], dtype=torch.int32, device="cuda")
    qx, sx = bq.scaled_quantize(x)
    assert torch.equal(again.gemm_grouped(qx, sx, off), layer.gemm_grouped(qx, sx, off))
    bq.bq_device_check()


def expert_block(torch, bq, up, down, x, ids, F):
    """Two products per expert with the gate between them: tokens [T, D] to their experts ids [T, top]."""
    T, top = ids.shape
    order = torch.argsort(ids.reshape(-1), stable=True)
    offsets = torch.searchsorted(ids.reshape(-1)[order].contiguous(),
                                 torch.arange(up.experts + 1, device="cuda")).to(torch.int32)
    rows = (order // top).to(torch.int32)
    q, s = bq.scaled_quantize(x, rows=rows)
    h = up.gemm_grouped(q, s, offsets, dtype=torch.float32)
    q, s = bq.scaled_quantize(h[:, F:], gate=h[:, :F])
    y = down.gemm_grouped(q, s, offsets, dtype=torch.float32)
    out = torch.zeros(T, down.N, device="cuda")
    return out.index_add_(0, rows.long(), y), offsets


@pytest.mark.parametrize("T,E,top,D,F", [(1, 4, 2, 256, 384), (37, 8, 2, 200, 304), (300, 5, 1, 512, 128)])
def test_expert_block(T, E, top, D, F):
    """The three operators as an expert block uses them, against the same block in 64 bits on the layers'
    dequantized weights: within the 8-bit rounding of the two quantized activations."""
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(T)
    up = bq.ScaledLinear.quantize(torch.randn(E, 2 * F, D, generator=g, device="cuda") * D ** -0.5)
    down = bq.ScaledLinear.quantize(torch.randn(E, D, F, generator=g, device="cuda") * F ** -0.5)
    x = torch.randn(T, D, generator=g, device="cuda")
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:top] for _ in range(T)])
    out, offsets = expert_block(torch, bq, up, down, x, ids, F)
    bq.bq_device_check()
    assert int(offsets[-1]) == T * top
    wu = up.codes.double() * up.scale.double()[..., None]
    wd = down.codes.double() * down.scale.double()[..., None]
    ref, room = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
    for t in range(T):
        for e in ids[t].tolist():
            xt = x[t].double()
            h = wu[e] @ xt
            gate, lin = h[:F], h[F:]
            a = lin * gate * torch.sigmoid(gate)
            # half a step of each quantized input, through the layer, the gate (slope of SiLU <= 1.1) and the next layer
            dh = 1.001 * wu[e].abs().sum(1) * xt.abs().max() / 254
            da = dh[F:] * (gate * torch.sigmoid(gate)).abs() + 1.1 * dh[:F] * (lin.abs() + dh[F:])
            ref[t] += (wd[e] @ a).cpu()
            room[t] += (wd[e].abs() @ (da + (a.abs() + da).max() / 254)).cpu() * 1.01 + 1e-6
    assert torch.all((out.double().cpu() - ref).abs() <= room)
    # and it is not a loose bound only: the typical error is that of 8 bits
    assert (out.double().cpu() - ref).norm() <= 0.05 * ref.norm()


def test_streams_and_graphs():
    """Calls on a side stream, two captured graphs replayed at once, and offsets that change under a graph."""
    torch, bq = mods()
    rng = np.random.default_rng(1)
    c = grouped_case(torch, rng, [20, 40, 4], 256, 512)
    layer = bq.ScaledLinear(c["wd"], c["swd"])
    one = bq.ScaledLinear(c["wd"][0], c["swd"][0].contiguous())
    xs = [torch.randn(8, 512, device="cuda") for _ in range(2)]
    want = [one.linear(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = one.linear(xs[0], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    outs, graphs = [torch.zeros_like(w) for w in want], []
    for i in range(2):
        graphs.append(bq.StepGraph(lambda i=i: one.linear(xs[i], y=outs[i])))
    for i in range(2):
        outs[i].zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    y = torch.full((64, 256), 7.0, device="cuda")
    graph = bq.StepGraph(lambda: layer.gemm_grouped(c["qd"], c["sad"], c["offd"], y=y))
    for off in ([0, 20, 60, 64], [0, 0, 64, 64], [10, 11, 11, 30], [64, 64, 64, 64]):
        y.fill_(7)
        c["offd"].copy_(torch.tensor(off, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        y_ref, p = grouped_ref(c, off)
        check(bq, y, y_ref, p, "fp32", False)
    bq.bq_device_check()


def test_calls_see_what_the_call_before_them_wrote():
    """Weights, tokens and scales written on the stream right before every call, in launches that may overlap:
    the products of every step are those of that step's values."""
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(3)
    N, K = 512, 2048
    q, s = bq.scaled_quantize(torch.zeros(N, K, device="cuda"))
    layer = bq.ScaledLinear(q, s)
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    grouped = bq.ScaledLinear(q[None], s[None])
    Ws = [torch.randn(N, K, generator=g, device="cuda") for _ in range(6)]
    xs = {M: [torch.randn(M, K, generator=g, device="cuda") for _ in range(6)] for M in (1, 4, 20, 40, 200)}
    got = []
    for i, W in enumerate(Ws):
        for M in (1, 4, 20, 200):
            bq.scaled_quantize(W, q=q, scale=s)
            got.append(layer.linear(xs[M][i]))
            q.zero_()
            bq.scaled_quantize(W, q=q, scale=s)
            qx, sx = bq.scaled_quantize(xs[M][i])
            got.append(layer.gemm(qx, sx, dtype=torch.float32))
        bq.scaled_quantize(W, q=q, scale=s)
        qx, sx = bq.scaled_quantize(xs[40][i])
        got.append(grouped.gemm_grouped(qx, sx, off, dtype=torch.float32))
    torch.cuda.synchronize()
    it = iter(got)
    for i, W in enumerate(Ws):
        w, sw = R.quantize(host(W))
        sw = (np.abs(host(W)).max(1) / np.float32(127)).astype(np.float32)
        for M in (1, 4, 20, 200, 40):
            x = host(xs[M][i])
            qr, _ = R.quantize(x)
            y_ref, p = R.gemm(qr, (np.abs(x).max(1) / np.float32(127)).astype(np.float32), w, sw)
            for _ in range(1 if M == 40 else 2):
                check(bq, next(it), y_ref, p, "fp32", False)


def test_results_are_the_same_every_time():
    """Split sums, atomics-free: the same bits from every run, alone and among others."""
    torch, bq = mods()
    rng = np.random.default_rng(6)
    w, wd = codes(torch, rng, 640, 4096)
    sw, swd = scales(torch, rng, 640)
    layer = bq.ScaledLinear(wd, swd)
    for M in (1, 3, 8, 9, 33, 64, 65, 300):
        x = torch.randn(M, 4096, device="cuda")
        first = layer.linear(x)
        torch.cuda.synchronize()
        many = [layer.linear(x) for _ in range(30)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, y) for y in many), M
    bq.bq_device_check()


def test_beside_the_packed_layers():
    """Scaled and packed layers alternating on one stream: each as it is alone."""
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(8)
    W = torch.randn(256, 1024, generator=g, device="cuda")
    packed = [bq.QuantLinear("abq", W, w_bits=8, a_bits=8), bq.QuantLinear("bitnet", W)]
    scaled = bq.ScaledLinear.quantize(W)
    for M in (1, 16, 40):
        x = torch.randn(M, 1024, generator=g, device="cuda").bfloat16()
        calls = [lambda: packed[0].linear(x), lambda: scaled.linear(x), lambda: packed[1].linear(x), lambda: scaled.linear(x)]
        alone = []
        for c in calls:
            torch.cuda.synchronize()
            alone.append(c())
        torch.cuda.synchronize()
        rows = [[c() for c in calls] for _ in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, y) for r in rows for a, y in zip(alone, r))
    bq.bq_device_check()


def test_long_matrices_pass_32_bit_offsets():
    """Codes and outputs of more than 2^31 elements: the last rows are right."""
    torch, bq = mods()
    rng = np.random.default_rng(2)
    M, K, N = 33000, 65536, 24          # 2.16e9 codes
    w, wd = codes(torch, rng, N, K)
    sw, swd = scales(torch, rng, N)
    q = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    tail, td = codes(torch, rng, 3, K)
    q[-3:] = td
    y = bq.ScaledLinear(wd, swd).gemm(q, torch.ones(M, device="cuda"), dtype=torch.float32)
    y_ref, p = R.gemm(tail, np.ones(3), w, sw)
    check(bq, y[-3:], y_ref, p, "fp32", False)
    assert torch.all(y[:-3] == 0)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(K, device="cuda").bfloat16()
    bq.scaled_quantize(x, q=q)
    assert np.array_equal(host(q[-1]), R.quantize(host(x[-1:]))[0][0])
    del q, x, y
    M, N, K = 150000, 15000, 32          # 2.25e9 outputs
    w, wd = codes(torch, rng, N, K)
    sw, swd = scales(torch, rng, N)
    qh, qd = codes(torch, rng, M, K)
    y = bq.ScaledLinear(wd, swd).gemm(qd, torch.ones(M, device="cuda"))
    y_ref, p = R.gemm(qh[-4:], np.ones(4), w, sw)
    check(bq, y[-4:], y_ref, p, "bf16", False)


def test_refusals():
    torch, bq = mods()
    w = torch.ones(16, 64, dtype=torch.int8, device="cuda")
    s = torch.ones(16, device="cuda")
    layer = bq.ScaledLinear(w, s)
    x = torch.ones(4, 64, device="cuda")
    q, sa = bq.scaled_quantize(x)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bad = [lambda: layer.linear(x[:, :63]), lambda: layer.linear(x.double()), lambda: layer.linear(x.cpu()),
           lambda: layer.linear(x.t().contiguous().t()), lambda: layer.linear(x[0]),
           lambda: layer.linear(x, y=torch.empty(4, 15, device="cuda")),
           lambda: layer.linear(x, y=torch.empty(3, 16, device="cuda")),
           lambda: layer.linear(x, dtype=torch.float64), lambda: layer.gemm(q, sa[:3]), lambda: layer.gemm(q, sa.double()),
           lambda: layer.gemm(q.float(), sa), lambda: layer.gemm(q[:, :32], sa),
           lambda: layer.gemm_grouped(q, sa, off.long()), lambda: layer.gemm_grouped(q, sa, off[:1]),
           lambda: layer.gemm_grouped(q, sa, off.cpu()),
           lambda: bq.scaled_quantize(x, gate=x[:3]), lambda: bq.scaled_quantize(x, gate=x.half()),
           lambda: bq.scaled_quantize(x, rows=off.long()), lambda: bq.scaled_quantize(x, q=q[:3]),
           lambda: bq.ScaledLinear(w.float(), s), lambda: bq.ScaledLinear(w, s[:3]), lambda: bq.ScaledLinear(w, s.half()),
           lambda: bq.ScaledLinear(w, s, torch.ones(3, device="cuda")),
           lambda: bq.ScaledLinear(w[None].expand(2, 16, 64), torch.ones(2, 16, device="cuda")).gemm(q, sa)]
    for i, f in enumerate(bad):
        with pytest.raises(bq.BQError) as e:
            f()
        assert e.value.status in (bq.BQ_ERR_INVALID_ARG, bq.BQ_ERR_SIZE), i
    # rows of codes that do not start on 16-byte boundaries
    with pytest.raises(bq.BQError) as e:
        layer.gemm(torch.ones(4, 72, dtype=torch.int8, device="cuda")[:, :64], sa)
    assert e.value.status == bq.BQ_ERR_INVALID_ARG
    torch.cuda.synchronize()
    bq.bq_device_check()
