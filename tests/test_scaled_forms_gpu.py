"""The scaled int8 layers on the GPU, the forms that single calls at few sizes do not reach: kernels of several
streams beside each other. Plain references: tests/scaled_ref.py."""
import numpy as np
import pytest

from tests import scaled_ref as R
from tests.test_scaled_gpu import check, codes, mods, scales

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
