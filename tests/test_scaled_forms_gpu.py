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
