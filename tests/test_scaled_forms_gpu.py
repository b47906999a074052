"""The scaled int8 layers on the GPU, the forms that single calls at few sizes do not reach: kernels of several
streams beside each other. Plain references: tests/scaled_ref.py."""
import numpy as np
import pytest

from tests import scaled_ref as R
from tests.test_scaled_gpu import check, codes, host, kind, mods, scales

pytestmark = pytest.mark.gpu


def test_two_streams_share_the_tensor_memory():
    """Cluster kernels of few tokens and pairs that take all of an SM's tensor memory, on two streams at once:
    each as it is alone."""
    torch, bq = mods()
    rng = np.random.default_rng(11)
    few = []
    for M, N, K in [(1, 2048, 1024), (8, 1100, 640), (40, 1024, 1024)]:
        w, wd = codes(torch, rng, N, K)
        q, qd = codes(torch, rng, M, K)
        sw, swd = scales(torch, rng, N)
        sa, sad = scales(torch, rng, M)
        few.append((bq.ScaledLinear(wd, swd), qd, sad, R.gemm(q, sa, w, sw)))
    M, N, K = 2048, 5000, 512  # 192 tokens a tile: all of the SM's tensor memory
    w, wd = codes(torch, rng, N, K)
    q, qd = codes(torch, rng, M, K)
    sw, swd = scales(torch, rng, N)
    sa, sad = scales(torch, rng, M)
    many = (bq.ScaledLinear(wd, swd), qd, sad, R.gemm(q, sa, w, sw))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        with torch.cuda.stream(streams[0]):
            got[0].append(many[0].gemm(many[1], many[2], dtype=torch.float32))
        with torch.cuda.stream(streams[1]):
            for layer, qx, sx, _ in few:
                got[1].append(layer.gemm(qx, sx, dtype=torch.float32))
    torch.cuda.synchronize()
    check(bq, got[0][0], *many[3], "fp32", False)
    for i, f in enumerate(few):
        check(bq, got[1][i], *f[3], "fp32", False)
    assert all(torch.equal(y, got[0][0]) for y in got[0])
    assert all(torch.equal(y, got[1][i % 3]) for i, y in enumerate(got[1]))


def test_few_tokens_with_channels_cut_inside_a_warp():
    """Warps whose lanes part (channels past N, the last tokens) between reads of the tensor memory. Enough
    channels that k is not split, and few enough that it is."""
    torch, bq = mods()
    for M, N, K in [(64, 40 * 1024 + 13, 256), (37, 38 * 1024 + 5, 130), (64, 205, 1024), (12, 77, 640), (100, 333, 640)]:
        rng = np.random.default_rng(M + N + K)
        w, wd = codes(torch, rng, N, K)
        q, qd = codes(torch, rng, M, K)
        sw, swd = scales(torch, rng, N)
        sa, sad = scales(torch, rng, M)
        y_ref, p = R.gemm(q, sa, w, sw)
        layer = bq.ScaledLinear(wd, swd)
        for name, t in (("bf16", torch.bfloat16), ("fp32", torch.float32)):
            check(bq, layer.gemm(qd, sad, dtype=t), y_ref, p, name, False)


@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K,ld,start", [(1, 1001, 1001, 0), (2, 1001, 1001, 1), (1, 4099, 4104, 8), (2, 4099, 4099, 3),
                                          (2, 8200, 8201, 0), (1, 16383, 16383, 5), (2, 16384, 16385, 1), (1, 9, 9, 7)])
def test_one_launch_from_unaligned_rows(M, K, ld, start, name):
    """The quantization inside the product, from rows that its wide loads do not cover: a part of the lanes takes
    element after element before the warp meets again."""
    torch, bq = mods()
    rng = np.random.default_rng(M + K + ld)
    w, wd = codes(torch, rng, 300, K)
    sw, swd = scales(torch, rng, 300)
    flat = torch.from_numpy(rng.standard_normal(start + M * ld).astype(np.float32)).cuda().to(kind(torch, name))
    x = flat.as_strided((M, K), (ld, 1), start)
    layer = bq.ScaledLinear(wd, swd)
    q, s = bq.scaled_quantize(x)
    assert np.array_equal(host(q), R.quantize(host(x))[0])
    y_ref, p = R.gemm(host(q), host(s), w, sw)
    check(bq, layer.linear(x, dtype=torch.float32), y_ref, p, "fp32", False)


def side_calls(torch, bq):
    """Every call that takes a stream, as (name, call of fresh inputs on the stream, its inputs)."""
    g = torch.Generator(device="cuda").manual_seed(21)
    M, K, N = 200, 1024, 512
    W = torch.randn(2, N, K, generator=g, device="cuda")
    one, two = bq.ScaledLinear.quantize(W[0], bias=torch.ones(N, device="cuda")), bq.ScaledLinear.quantize(W)
    x = torch.randn(M, K, generator=g, device="cuda")
    q, s = bq.scaled_quantize(x)
    rows = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 77, M], dtype=torch.int32, device="cuda")
    y = lambda: torch.zeros(M, N, device="cuda")  # noqa: E731
    held = lambda layer: [layer.codes, layer.scale] + ([] if layer.bias is None else [layer.bias])  # noqa: E731
    return [
        ("quantize", lambda st, x, gate, rows, q, s: bq.scaled_quantize(x, gate, rows, q, s, stream=st)[0],
         lambda: [x.clone(), x.clone(), rows.clone(), torch.zeros_like(q), torch.zeros_like(s)], []),
        ("linear", lambda st, x, y: one.linear(x, y=y, stream=st), lambda: [x.clone(), y()], held(one)),
        ("gemm", lambda st, q, s, y: one.gemm(q, s, y=y, stream=st), lambda: [q.clone(), s.clone(), y()], held(one)),
        ("grouped", lambda st, q, s, off, y: two.gemm_grouped(q, s, off, y=y, stream=st),
         lambda: [q.clone(), s.clone(), off.clone(), y()], held(two))]


@pytest.mark.parametrize("which", range(4))
def test_memory_passed_to_another_stream_is_recorded_there(which, monkeypatch):
    torch, bq = mods()
    name, call, make, held = side_calls(torch, bq)[which]
    side, seen = torch.cuda.Stream(), []
    args = make()
    torch.cuda.synchronize()
    record = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, st: (seen.append((t.data_ptr(), st)), record(t, st))[1])
    call(side, *args)
    side.synchronize()
    assert {(t.data_ptr(), side) for t in args + held} <= set(seen), name


@pytest.mark.parametrize("which", range(4))
def test_inputs_freed_behind_a_call_on_another_stream(which):
    """Inputs that the caller drops while the other stream has not come to the call yet, and new tensors of their
    sizes that are written at once on the inputs' own stream."""
    torch, bq = mods()
    name, call, make, _ = side_calls(torch, bq)[which]
    side = torch.cuda.Stream()
    args = make()
    torch.cuda.synchronize()
    want = call(side, *args).clone() if name != "quantize" else call(side, *args)
    side.synchronize()
    want = want.clone()
    args = make()
    sizes = [(a.shape, a.dtype) for a in args[:-1]]  # the last one is an output
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    got = call(side, *args)
    del args
    new = [torch.empty(shape, dtype=dtype, device="cuda").fill_(1) for shape, dtype in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(new) == 2 * len(sizes)
    bq.bq_device_check()


@pytest.mark.parametrize("made", ["quantize", "laid out"])
def test_weights_made_by_a_layer_are_complete_for_every_stream(made):
    """A layer made behind other work on the current stream, and called on a stream that does not wait for it."""
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randn(300, 1001, generator=g, device="cuda")
    x = torch.randn(5, 1001, generator=g, device="cuda")
    q, s = bq.scaled_quantize(W)
    tight = q.contiguous()  # rows of 1001 bytes
    want = bq.ScaledLinear(q, s).linear(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    layer = bq.ScaledLinear.quantize(W) if made == "quantize" else bq.ScaledLinear(tight, s)
    assert torch.cuda.current_stream().query()
    y = layer.linear(x, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    bq.bq_device_check()


def test_a_layer_can_be_made_in_a_captured_graph():
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(3, 77, generator=g, device="cuda")
    W = torch.randn(40, 77, generator=g, device="cuda")
    want = bq.ScaledLinear.quantize(W).linear(x)
    q, s = bq.scaled_quantize(W)
    tight, y, z = q.contiguous(), torch.zeros(3, 40, device="cuda"), torch.zeros(3, 40, device="cuda")

    def step():
        bq.ScaledLinear.quantize(W).linear(x, y=y)
        bq.ScaledLinear(tight, s).linear(x, y=z)
    graph = bq.StepGraph(step)
    y.zero_(), z.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want)
    bq.bq_device_check()


def test_calls_on_another_stream_refuse_what_others_refuse():
    torch, bq = mods()
    side = torch.cuda.Stream()
    layer = bq.ScaledLinear(torch.ones(16, 64, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda"))
    x = torch.ones(4, 64, device="cuda")
    q, s = bq.scaled_quantize(x)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    bad = [lambda st: bq.scaled_quantize(x, gate=1, stream=st), lambda st: bq.scaled_quantize(x, rows=[0], stream=st),
           lambda st: bq.scaled_quantize(x, q=q.cpu(), stream=st), lambda st: bq.scaled_quantize(x, scale=s.cpu(), stream=st),
           lambda st: layer.linear(x, y=torch.empty(4, 16), stream=st), lambda st: layer.linear(x, y=5, stream=st),
           lambda st: layer.gemm(q, s, y=[], stream=st), lambda st: layer.gemm_grouped(q, s, off.cpu(), stream=st)]
    for i, call in enumerate(bad):
        for st in (None, side):
            with pytest.raises(bq.BQError) as e:
                call(st)
            assert e.value.status == bq.BQ_ERR_INVALID_ARG, i
    for st in (0, torch.cuda.current_stream().cuda_stream, "side"):
        with pytest.raises(bq.BQError):
            layer.linear(x, stream=st)
    torch.cuda.synchronize()
    bq.bq_device_check()


def rounded_sum(p, b):
    """p + b (f64 arrays) rounded once to f32: the f64 sum is rounded to odd, so that no tie of f32 is made."""
    s = p + b
    bb = s - p
    err = (p - (s - bb)) + (b - bb)  # the exact remainder
    odd = (s.view(np.int64) & 1).astype(bool)
    s = np.where((err != 0) & ~odd, np.nextafter(s, np.where(err > 0, np.inf, -np.inf)), s)
    return s.astype(np.float32)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [1, 7, 40, 100, 300])
def test_products_take_the_documented_roundings(M, bias):
    """Bit for bit in f32, and its nearest value in the 16-bit types: fl(fl(sum) * fl(sa sw)), or with a bias
    fl(fl(sum) * fl(sa sw) + bias) from the unrounded product."""
    torch, bq = mods()
    rng = np.random.default_rng(M)
    N, K = 333, 2000
    w, wd = codes(torch, rng, N, K)
    q, qd = codes(torch, rng, M, K)
    q[0, :], w[0, :] = 127, 127  # a sum past 2^24 among them
    qd[0], wd[0] = 127, 127
    sw, swd = scales(torch, rng, N)
    sa, sad = scales(torch, rng, M)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    acc = (q.astype(np.int64) @ w.astype(np.int64).T).astype(np.float32)
    s = sa[:, None] * sw[None, :]
    assert s.dtype == np.float32
    want = rounded_sum(acc.astype(np.float64) * s.astype(np.float64), np.broadcast_to(b.astype(np.float64), acc.shape)) \
        if bias else acc * s
    layer = bq.ScaledLinear(wd, swd, torch.from_numpy(b).cuda() if bias else None)
    whole = layer.gemm(qd, sad, dtype=torch.float32)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    by_expert = layer.gemm_grouped(qd, sad, off, dtype=torch.float32)
    assert np.array_equal(host(whole), want) and torch.equal(whole, by_expert)
    for t in (torch.bfloat16, torch.float16):
        assert torch.equal(layer.gemm(qd, sad, dtype=t), whole.to(t))
        assert torch.equal(layer.gemm_grouped(qd, sad, off, dtype=t), whole.to(t))
    bq.bq_device_check()


def test_c_calls_by_their_own_names():
    """The C calls of the binding, on pointers and sizes, give what the torch layer gives."""
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(31)
    M, N, K = 9, 50, 100
    W = torch.randn(2, N, K, generator=g, device="cuda")
    two, one = bq.ScaledLinear.quantize(W), bq.ScaledLinear.quantize(W[0])
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, s = bq.scaled_quantize(x)
    q2, s2 = bq.empty_codes(M, K, x.device), torch.zeros(M, device="cuda")
    assert q2.stride(0) == 112
    bq.bq_scaled_quantize(x, bq.BQ_TYPE_BF16, K, M, None, 0, None, M, K, q2, 112, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(bq.scaled_quantize(x, q=bq.empty_codes(M, K, x.device))[0], q)
    y = torch.zeros(M, N, device="cuda")
    bq.bq_scaled_gemm(one.weights, q, 112, s, M, y, bq.BQ_TYPE_F32, N)
    assert torch.equal(y, one.gemm(q, s, dtype=torch.float32))
    off = torch.tensor([0, 4, M], dtype=torch.int32, device="cuda")
    bq.bq_scaled_gemm_grouped(two.weights, q, 112, s, M, off, y, bq.BQ_TYPE_F32, N)
    assert torch.equal(y, two.gemm_grouped(q, s, off, dtype=torch.float32))
    n = bq.bq_scaled_workspace_bytes(one.weights, M)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    bq.bq_scaled_linear(one.weights, x, bq.BQ_TYPE_BF16, K, M, y, bq.BQ_TYPE_F32, N, ws, n)
    assert torch.equal(y, one.linear(x, dtype=torch.float32))
    with pytest.raises(bq.BQError):
        bq.bq_scaled_linear(one.weights, x, bq.BQ_TYPE_BF16, K, M, y, bq.BQ_TYPE_F32, N, ws, n - 1)
    bq.bq_device_check()


# ---------------------------------------------------------------------------------------------------
# quantization of many rows
# ---------------------------------------------------------------------------------------------------

# rows x K, each more than 148 * 1024 runs of eight elements: the kernels with several runs a thread, for K up to
# 1024, up to 16384, up to 32768 and above
MANY = [(1300, 1000), (2400, 513), (1185, 1024), (1180, 1025), (300, 4096), (297, 4099), (120, 11008), (150, 16384), (64, 20001),
        (40, 32768), (20, 40000), (5, 65536)]


def special(torch, x):
    """Rows of every kind among ordinary ones, in x."""
    K = x.shape[1]
    x[1] = 0
    x[2, K // 3] = float("nan")
    x[3, K - 1] = float("inf")
    x[-1, 0] = float("-inf")
    x[4] *= 2.0 ** -20
    if x.dtype != torch.float16:
        x[0] *= 2.0 ** -110
        x[-2] *= 2.0 ** 100
    return x


def rows_of(torch, M, K, name, seed, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or K
    return (torch.randn(M, ld, generator=g, device="cuda") * 3).to(kind(torch, name))[:, :K]


def same_codes(torch, bq, q, s, v, rows=None):
    bq.bq_device_check()
    qr, sr = R.quantize(v, rows)
    assert np.array_equal(host(q), qr)
    sg = host(s).astype(np.float64)
    assert np.array_equal(np.isnan(sg), np.isnan(sr))
    ok = ~np.isnan(sr)
    assert np.all(np.abs(sg[ok] - sr[ok]) <= R.U * sr[ok])


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", MANY)
def test_quantize_many_rows(M, K, name, odd):
    torch, bq = mods()
    x = special(torch, rows_of(torch, M, K, name, M + K, K + 3 if odd else (K + 7) // 8 * 8))
    q, s = bq.scaled_quantize(x)
    same_codes(torch, bq, q, s, host(x))


@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", MANY[::2] + [(9, 100)])
def test_quantize_many_gathered_rows(M, K, name):
    torch, bq = mods()
    x = special(torch, rows_of(torch, max(M // 3, 8), K, name, M + K))
    rng = np.random.default_rng(M)
    rows = rng.integers(-1, x.shape[0], M).astype(np.int32)  # repeated ones and empty slots
    q, s = bq.scaled_quantize(x, rows=torch.from_numpy(rows).cuda())
    same_codes(torch, bq, q, s, host(x), rows)


def check_gated(bq, q, s, up, gate, rows=None):
    """The bounds of the gated codes: v = x (g / (1 + exp(-g))) in f32 is within 7 half steps (four for 1 + exp(-g),
    one each for the sum, the quotient and the product), a code carries v's and gamma's and three more."""
    bq.bq_device_check()
    v = R.gated(up, gate)
    if rows is not None:
        v = np.where((rows >= 0)[:, None], v[np.maximum(rows, 0)], 0)
    bad = ~np.isfinite(v).all(1)
    q, s = host(q).astype(np.float64), host(s).astype(np.float64)
    assert np.array_equal(np.isnan(s), bad) and np.all(q[bad] == 0)
    v, q, s = v[~bad], q[~bad], s[~bad]
    gamma, rel = np.abs(v).max(1), 7 * R.U
    assert np.all(np.abs(s - gamma / 127) <= 1.01 * (rel + R.U) * gamma / 127)
    live = gamma > 0
    assert np.all(q[~live] == 0)
    exact = v[live] * (127 / gamma[live])[:, None]
    assert np.all(np.abs(q[live] - exact) <= 0.5 + 1.01 * 127 * (2 * rel + 3 * R.U))


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", MANY + [(5, 33)])
def test_quantize_many_gated_rows(M, K, name, odd):
    """Gate and up side by side in one matrix, whole and (rows with gate) gathered."""
    torch, bq = mods()
    both = rows_of(torch, M, 2 * K + (1 if odd else 0), name, M * 3 + K)
    gate, up = both[:, :K], both[:, K:2 * K]
    up[1] = 0
    up[2, K // 2] = float("nan")
    gate[3, K - 1] = float("inf")
    gate[-1, 0] = float("-inf")  # -inf / (1 + inf) is no number
    q, s = bq.scaled_quantize(up, gate=gate)
    check_gated(bq, q, s, host(up), host(gate))
    rng = np.random.default_rng(K)
    rows = rng.integers(-1, M, M).astype(np.int32)
    q, s = bq.scaled_quantize(up, gate=gate, rows=torch.from_numpy(rows).cuda())
    check_gated(bq, q, s, host(up), host(gate), rows)


# ---------------------------------------------------------------------------------------------------
# special rows in one launch
# ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 200), (2, 200), (1, 4096), (2, 4099), (1, 16384), (2, 16384), (2, 16385)])
def test_special_rows_in_one_launch(M, K, name):
    torch, bq = mods()
    rng = np.random.default_rng(K)
    w, wd = codes(torch, rng, 300, K)
    sw, swd = scales(torch, rng, 300)
    b = rng.standard_normal(300).astype(np.float32)
    layer = bq.ScaledLinear(wd, swd, torch.from_numpy(b).cuda())
    base = rows_of(torch, M, K, name, K)

    def put(v, at):
        return lambda x: x[-1].__setitem__(at, v)
    kinds = [lambda x: x[-1].zero_(), lambda x: x[-1].fill_(-0.0), put(float("nan"), K // 2), put(float("inf"), 0),
             put(float("-inf"), K - 1), lambda x: x[-1].zero_()[K - 1:].fill_(2.0 ** -24), lambda x: x[-1].mul_(2.0 ** -15)]
    if name != "fp16":
        kinds += [lambda x: x[-1].mul_(2.0 ** -110), lambda x: x[-1].zero_()[3:4].fill_(2.0 ** -100),
                  lambda x: x[-1].zero_()[3:4].fill_(2.0 ** -101), lambda x: x[-1].mul_(2.0 ** 120)]
    for i, change in enumerate(kinds):
        x = base.clone()
        change(x)
        y = layer.linear(x, dtype=torch.float32)
        q, s = bq.scaled_quantize(x)
        same_codes(torch, bq, q, s, host(x))
        two = layer.gemm(q, s, dtype=torch.float32)
        assert torch.equal(torch.nan_to_num(y, nan=1e9), torch.nan_to_num(two, nan=1e9)), i
        if torch.isnan(s[-1]):
            assert torch.isnan(y[-1]).all() and not torch.isnan(y[:-1]).any(), i
        elif s[-1] == 0:
            assert np.array_equal(host(y[-1]), b), i
    bq.bq_device_check()


# ---------------------------------------------------------------------------------------------------
# several tiles a CTA
# ---------------------------------------------------------------------------------------------------

# whole products of three tiles a pair and more, every width of a tile among them (tests/test_scaled_plan.py
# holds the list to that): M, N, K
TILES = [(4100, 4104, 640), (3000, 5000, 1111), (2048, 8200, 1800), (493, 7801, 130), (630, 14140, 1800), (5504, 2124, 2100),
         (1100, 9001, 130), (300, 30000, 400), (9000, 2056, 520)]


def near(torch, bq, y, q, sa, w, sw, b, name):
    """Every output against the exact sums in 64 bits, on the device, with the tolerance of tests/scaled_ref.py."""
    bq.bq_device_check()
    p = q.double() @ w.double().t() * sa.double()[:, None] * sw.double()
    ref = p if b is None else p + b.double()
    p, size = p.abs(), ref.abs()
    first = 2 * R.U * p + R.U * size if b is not None else 3 * R.U * p
    off = (y.double() - ref).abs() / (1.01 * (first + R.HALF_STEP[name] * (size + first)) + R.SMALLEST[name])
    assert float(off.max()) <= 1, (float(off.max()), (off > 1).nonzero()[:4].tolist())


def device_case(torch, M, N, K, seed, bias, lead=()):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def matrix(*shape):
        ld = (K + 15) // 16 * 16
        return torch.randint(-128, 128, (*shape, ld), generator=g, device="cuda", dtype=torch.int8)[..., :K]
    r = lambda *shape: torch.rand(*shape, generator=g, device="cuda") * 2e-3 + 1e-4  # noqa: E731
    return (matrix(*lead, N), r(*lead, N), torch.randn(*lead, N, generator=g, device="cuda") if bias else None, matrix(M), r(M))


@pytest.mark.parametrize("name", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", TILES)
def test_several_tiles_a_pair(M, N, K, name):
    torch, bq = mods()
    w, sw, b, q, sa = device_case(torch, M, N, K, M + N + K, (M + K) % 200 < 100)
    layer = bq.ScaledLinear(w, sw, b)
    near(torch, bq, layer.gemm(q, sa, dtype=kind(torch, name)), q, sa, w, sw, b, name)
    # rows of y that TMA does not take
    wide = torch.full((M, N + 1), 7.0, dtype=kind(torch, name), device="cuda")
    near(torch, bq, layer.gemm(q, sa, y=wide[:, :N]), q, sa, w, sw, b, name)
    assert torch.all(wide[:, N] == 7)


@pytest.mark.parametrize("M,N,K", TILES[:3])
def test_linear_of_several_tiles_a_pair(M, N, K):
    """The product behind its own quantization, whose weights are fetched ahead for a pair's first tile only."""
    torch, bq = mods()
    w, sw, b, _, _ = device_case(torch, M, N, K, M + N, True)
    x = rows_of(torch, M, K, "bf16", M)
    layer = bq.ScaledLinear(w, sw, b)
    q, s = bq.scaled_quantize(x)
    qr, _ = R.quantize(host(x))
    assert np.array_equal(host(q), qr)
    for _ in range(3):
        y = layer.linear(x)
        near(torch, bq, y, q, s, w, sw, b, "bf16")


# experts, rows an expert at most, N, K: single CTAs and pairs, three tiles each and more; few hot experts
GROUPED = [(64, 40, 5000, 1800, "even"), (64, 60, 4100, 130, "even"), (40, 30, 9000, 640, "even"), (8, 800, 3000, 1700, "even"),
           (16, 400, 4104, 640, "even"), (64, 100, 2048, 520, "one"), (128, 30, 2060, 700, "one"), (48, 200, 9000, 1000, "few")]


def counts_of(E, most, N, how):
    rng = np.random.default_rng(E + N)
    counts = rng.integers(0, most + 1, E)
    if how == "one":  # half of the rows are one expert's
        counts[E // 3] += counts.sum()
    if how == "few":
        counts[rng.random(E) < 0.8] = 0
    return counts


@pytest.mark.parametrize("name", ["bf16", "fp32"])
@pytest.mark.parametrize("E,most,N,K,how", GROUPED)
def test_grouped_of_several_tiles_a_cta(E, most, N, K, how, name):
    torch, bq = mods()
    counts = counts_of(E, most, N, how)
    before, after = 3, 5
    M = before + int(counts.sum()) + after
    w, sw, b, q, sa = device_case(torch, M, N, K, E * N, name == "fp32", (E,))
    edges = before + np.concatenate([[0], np.cumsum(counts)])
    y = torch.full((M, N), 7.0, dtype=kind(torch, name), device="cuda")
    bq.ScaledLinear(w, sw, b).gemm_grouped(q, sa, torch.from_numpy(edges.astype(np.int32)).cuda(), y=y)
    for e in range(E):
        r = slice(int(edges[e]), int(edges[e + 1]))
        if counts[e]:
            near(torch, bq, y[r], q[r], sa[r], w[e], sw[e], None if b is None else b[e], name)
    assert torch.all(y[:before] == 7) and torch.all(y[M - after:] == 7)


def test_experts_of_any_stride():
    """Experts interleaved row by row ([N, E, K]), and ones with a gap that is no whole row: views, not copied."""
    torch, bq = mods()
    E, N, K = 5, 200, 320
    g = torch.Generator(device="cuda").manual_seed(6)
    flat = torch.randint(-128, 128, (E * (N * K + 48),), generator=g, device="cuda", dtype=torch.int8)
    sw, q, sa = (torch.rand(E, N, generator=g, device="cuda"), flat[:300 * K].view(300, K).flip(1).contiguous(),
                 torch.rand(300, generator=g, device="cuda"))
    off = torch.tensor([0, 10, 10, 150, 151, 300], dtype=torch.int32, device="cuda")
    for w in (flat[:E * N * K].view(N, E, K).transpose(0, 1), flat.as_strided((E, N, K), (N * K + 48, K, 1))):
        layer = bq.ScaledLinear(w, sw)
        assert layer.codes.data_ptr() == flat.data_ptr()
        y = layer.gemm_grouped(q, sa, off, dtype=torch.float32)
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            if r.stop > r.start:
                near(torch, bq, y[r], q[r], sa[r], w[e], sw[e], None, "fp32")


def test_a_refused_launch_leaves_no_error_to_the_next_call():
    """A launch on the legacy stream is refused while a blocking stream is being captured. The call says so, and
    the next one, which looks for errors of its own launches, finds none."""
    import ctypes
    torch, bq = mods()
    rt = ctypes.CDLL("libcudart.so.12")  # torch's
    x = torch.randn(4, 64, device="cuda")
    W = torch.randn(32, 256, device="cuda")
    q, s = bq.scaled_quantize(x)
    torch.cuda.synchronize()
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    status = bq.raw_status("bq_scaled_quantize", x.data_ptr(), bq.BQ_TYPE_F32, 64, 4, None, 0, None, 4, 64, q.data_ptr(),
                           q.stride(0), s.data_ptr(), None)
    assert rt.cudaStreamEndCapture(stream, ctypes.byref(graph)) != 0  # the refused launch has ended the capture
    rt.cudaGetLastError()
    assert rt.cudaStreamDestroy(stream) == 0
    assert status == bq.BQ_ERR_CUDA
    bq.QuantLinear("bitnet", W)
    bq.bq_device_check()


def test_calls_on_a_forked_stream_of_a_captured_graph():
    """stream= inside a capture: work forked onto another stream and joined, inputs that do not outlive the step,
    replayed beside eager calls of the same layers on another stream."""
    torch, bq = mods()
    g = torch.Generator(device="cuda").manual_seed(12)
    layer = bq.ScaledLinear.quantize(torch.randn(300, 1000, generator=g, device="cuda"))
    xs = [torch.randn(M, 1000, generator=g, device="cuda") for M in (1, 40, 200)]
    want = [layer.linear(x) for x in xs]
    ys, side = [torch.zeros_like(y) for y in want], torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        tmp = [x + 0 for x in xs]
        side.wait_stream(here)
        for x, y in zip(tmp, ys):
            layer.linear(x, y=y, stream=side)
        del tmp, x
        junk = [torch.full_like(x, 3.0) for x in xs]
        here.wait_stream(side)
        return junk
    graph = bq.StepGraph(step)
    for _ in range(3):
        for y in ys:
            y.zero_()
        graph.replay()
        eager = [layer.linear(x, stream=side) for x in xs]
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, want))
        assert all(torch.equal(y, w) for y, w in zip(eager, want))
    bq.bq_device_check()
