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
