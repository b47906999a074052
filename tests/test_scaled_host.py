"""The scaled int8 calls on the host (no GPU): arguments are refused with the documented status before
anything is enqueued, workspaces have the documented size, and the plain reference holds its own definition."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from bit_weight_quantization_b200 import bq
from tests import scaled_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an address no call reads on the host
OK, INVALID, SIZE = bq.BQ_OK, bq.BQ_ERR_INVALID_ARG, bq.BQ_ERR_SIZE


def weights(**kw):
    d = dict(codes=P, scale=P, bias=None, ld=4096, expert_stride=0, N=64, K=4096, experts=1)
    d.update(kw)
    return bq.bq_scaled_weights(*[d[n] for n, _ in bq.bq_scaled_weights._fields_])


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_struct_matches_the_c_header(tmp_path):
    names = [f for f, _ in bq.bq_scaled_weights._fields_]
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bq.h"\nint main(void) {\n'
                   '  printf("%zu %d %d %d %d\\n", sizeof(bq_scaled_weights), BQ_TYPE_F32, BQ_TYPE_BF16, BQ_TYPE_F16, '
                   'BQ_MAX_EXPERTS);\n' +
                   "".join(f'  printf("%zu\\n", offsetof(bq_scaled_weights, {n}));\n' for n in names) + "  return 0;\n}\n")
    exe = tmp_path / "o"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in out] == [ctypes.sizeof(bq.bq_scaled_weights), bq.BQ_TYPE_F32, bq.BQ_TYPE_BF16,
                                     bq.BQ_TYPE_F16, bq.BQ_MAX_EXPERTS] + \
        [getattr(bq.bq_scaled_weights, n).offset for n in names]


BAD_WEIGHTS = [(dict(codes=None), INVALID), (dict(codes=P + 8), INVALID), (dict(scale=None), INVALID),
               (dict(scale=P + 2), INVALID), (dict(bias=P + 1), INVALID), (dict(ld=4104), INVALID),
               (dict(ld=4080), SIZE), (dict(ld=1 << 36), SIZE), (dict(N=0), SIZE), (dict(N=(1 << 20) + 1), SIZE),
               (dict(K=0), SIZE), (dict(K=(1 << 16) + 1, ld=1 << 17), SIZE), (dict(experts=0), SIZE),
               (dict(experts=1025), SIZE), (dict(experts=2, expert_stride=8), INVALID),
               (dict(experts=2, expert_stride=-16), SIZE), (dict(experts=2, expert_stride=1 << 39), SIZE)]


@pytest.mark.parametrize("kw,status", BAD_WEIGHTS)
def test_bad_weights_are_refused_by_every_call(kw, status):
    w = ctypes.byref(weights(**kw))
    n = ctypes.c_size_t(7)
    assert bq.raw_status("bq_scaled_workspace_bytes", w, 4, ctypes.byref(n)) == status and n.value == 7
    assert bq.raw_status("bq_scaled_gemm", w, P, 4096, P, 4, P, 1, 64, None) == status
    assert bq.raw_status("bq_scaled_gemm_grouped", w, P, 4096, P, 4, P, P, 1, 64, None) == status
    assert bq.raw_status("bq_scaled_linear", w, P, 1, 4096, 4, P, 1, 64, P, 1 << 30, None) == status


GEMM = dict(q=P, ldq=4096, scale=P, M=4, y=P, y_type=1, ldy=64)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(q=P + 4), INVALID), (dict(ldq=4100), INVALID), (dict(ldq=4080), SIZE),
    (dict(scale=None), INVALID), (dict(scale=P + 1), INVALID), (dict(M=-1), SIZE), (dict(M=2 ** 31 - 1), SIZE),
    (dict(y=None), INVALID), (dict(y=P + 1), INVALID), (dict(y=P + 2, y_type=0), INVALID), (dict(y_type=3), INVALID),
    (dict(y_type=-1), INVALID), (dict(ldy=63), SIZE), (dict(ldy=1 << 36), SIZE)])
def test_bad_product_arguments(kw, status):
    a = {**GEMM, **kw}
    w = ctypes.byref(weights())
    tail = (a["y"], a["y_type"], a["ldy"], None)
    assert bq.raw_status("bq_scaled_gemm", w, a["q"], a["ldq"], a["scale"], a["M"], *tail) == status
    assert bq.raw_status("bq_scaled_gemm_grouped", w, a["q"], a["ldq"], a["scale"], a["M"], P, *tail) == status


def test_offsets_and_expert_counts():
    one, two = ctypes.byref(weights()), ctypes.byref(weights(experts=2, expert_stride=64 * 4096))
    args = (P, 4096, P, 4)
    assert bq.raw_status("bq_scaled_gemm_grouped", two, *args, None, P, 1, 64, None) == INVALID
    assert bq.raw_status("bq_scaled_gemm_grouped", two, *args, P + 2, P, 1, 64, None) == INVALID
    # the ungrouped calls take one expert
    assert bq.raw_status("bq_scaled_gemm", two, *args, P, 1, 64, None) == INVALID
    assert bq.raw_status("bq_scaled_linear", two, P, 1, 4096, 4, P, 1, 64, P, 1 << 30, None) == INVALID
    # no rows: nothing to do, whatever the pointers
    for w in (one, two):
        assert bq.raw_status("bq_scaled_gemm_grouped", w, None, 0, None, 0, None, None, 1, 0, None) == OK
    assert bq.raw_status("bq_scaled_gemm", one, None, 0, None, 0, None, 1, 0, None) == OK
    assert bq.raw_status("bq_scaled_linear", one, None, 1, 0, 0, None, 1, 0, None, 0, None) == OK


LINEAR = dict(x=P, x_type=1, ldx=4096, M=6, y=P, y_type=1, ldy=64, ws=P, n=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(x_type=3), INVALID), (dict(ldx=4095), SIZE),
    (dict(M=-1), SIZE), (dict(y=None), INVALID), (dict(y_type=9), INVALID), (dict(ldy=10), SIZE),
    (dict(ws=None), INVALID), (dict(ws=P + 128), INVALID), (dict(n=6 * 4096 + 255), SIZE)])
def test_bad_linear_arguments(kw, status):
    a = {**LINEAR, **kw}
    assert bq.raw_status("bq_scaled_linear", ctypes.byref(weights()), *[a[k] for k in LINEAR], None) == status


QUANT = dict(x=P, x_type=1, ldx=4096, x_rows=4, gate=None, ldg=0, rows=None, M=4, K=4096, q=P, ldq=4096, scale=P)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(x=P + 1), INVALID), (dict(x=P + 2, x_type=0), INVALID), (dict(x_type=5), INVALID),
    (dict(ldx=4095), SIZE), (dict(x_rows=3), SIZE), (dict(x_rows=-1), SIZE), (dict(gate=P + 1, ldg=4096), INVALID),
    (dict(gate=P, ldg=4000), SIZE), (dict(rows=P + 2), INVALID), (dict(M=-1), SIZE), (dict(K=0), SIZE),
    (dict(K=(1 << 16) + 1), SIZE), (dict(q=None), INVALID), (dict(q=P + 8), INVALID), (dict(ldq=4104), INVALID),
    (dict(ldq=16), SIZE), (dict(scale=None), INVALID), (dict(scale=P + 2), INVALID)])
def test_bad_quantize_arguments(kw, status):
    a = {**QUANT, **kw}
    assert bq.raw_status("bq_scaled_quantize", *[a[k] for k in QUANT], None) == status


def test_workspace_bytes():
    w = weights(K=4100, ld=4112)
    assert bq.bq_scaled_workspace_bytes(w, 0) == 0
    # up to two tokens are quantized inside the product
    assert [bq.bq_scaled_workspace_bytes(w, M) for M in (1, 2)] == [0, 0]
    assert bq.bq_scaled_workspace_bytes(weights(K=16385, ld=16400), 1) == 16640 + 256
    for M in (3, 64, 70000):
        up = lambda v: (v + 255) // 256 * 256  # noqa: E731
        assert bq.bq_scaled_workspace_bytes(w, M) == up(M * 4112) + up(4 * M)


def test_host_tensors_are_refused():
    import torch
    x = torch.zeros(2, 32)
    with pytest.raises(bq.BQError) as e:
        bq.scaled_quantize(x)
    assert e.value.status == INVALID
    with pytest.raises(bq.BQError):
        bq.ScaledLinear(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))


def test_reference_quantizer_by_hand():
    v = np.array([[1.0, -2.0, 0.5, 4.0], [0.0, 0.0, -0.0, 0.0], [1e-35, 0, 0, 0], [np.nan, 1, 2, 3], [np.inf, 1, 2, 3],
                  [127.0, 0.5, 1.5, -2.5]], np.float32)
    q, s = R.quantize(v)
    assert q.tolist() == [[32, -64, 16, 127], [0] * 4, [0] * 4, [0] * 4, [0] * 4, [127, 0, 2, -2]]  # ties to even
    assert s[0] == 4 / 127 and s[1] == 0 and s[2] == 0 and np.isnan(s[3]) and np.isnan(s[4]) and s[5] == 1
    q, s = R.quantize(v, [5, -1, 0])
    assert q[1].tolist() == [0] * 4 and s[1] == 0 and q[2].tolist() == [32, -64, 16, 127]


def test_reference_product_by_hand():
    y, p = R.gemm([[1, -2]], [0.5], [[3, 4], [-128, 127]], [2.0, 1.0], [10.0, 0.0])
    assert y.tolist() == [[5.0, -191.0]] and p.tolist() == [[5.0, 191.0]]


def test_header_documents_every_scaled_call():
    src = open(os.path.join(ROOT, "include", "bq.h")).read()
    code = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    for n in bq.EXPORTED:
        if n.startswith("bq_scaled"):
            assert re.search(rf"\b{n}\s*\(", code)


@pytest.fixture
def cuda_like():
    """Tensors that say they are on a GPU and have no memory: what the calls check before they use one."""
    import torch
    from torch._subclasses import FakeTensorMode

    def make(*shape, dtype=torch.bfloat16):
        with FakeTensorMode():
            return torch.empty(shape, device="cuda", dtype=dtype)
    return make


@pytest.mark.parametrize("shape", [(2 ** 32 + 4, 1), (2 ** 31, 8), (1, 2 ** 32 + 64), (3, 2 ** 31)])
def test_sizes_past_32_bits_are_refused(shape, cuda_like):
    """Sizes go to the library as int32: cut to it, 2^32 + 4 rows would be 4."""
    import torch
    with pytest.raises(bq.BQError) as e:
        bq.scaled_quantize(cuda_like(*shape))
    assert e.value.status == SIZE
    with pytest.raises(bq.BQError) as e:
        bq.ScaledLinear(cuda_like(*shape, dtype=torch.int8), cuda_like(shape[0], dtype=torch.float32))
    assert e.value.status == SIZE
    with pytest.raises(bq.BQError) as e:
        bq.ScaledLinear(cuda_like(2 ** 32 + 1, 1, 1, dtype=torch.int8), cuda_like(2 ** 32 + 1, dtype=torch.float32))
    assert e.value.status == SIZE


def test_gathers_past_32_bits_are_refused(cuda_like, monkeypatch):
    import torch
    from bit_weight_quantization_b200 import scaled
    monkeypatch.setattr(scaled, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(scaled, "_vector", lambda *a: 256)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 256)
    with pytest.raises(bq.BQError) as e:
        bq.scaled_quantize(cuda_like(4, 16), rows=cuda_like(2 ** 32 + 4, dtype=torch.int32))
    assert e.value.status == SIZE


def test_arguments_of_another_kind_are_refused(cuda_like, monkeypatch):
    import torch
    from bit_weight_quantization_b200 import scaled
    monkeypatch.setattr(scaled, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 256)
    x = cuda_like(4, 16)
    for call in (lambda: bq.scaled_quantize(x, rows=[0, 1]), lambda: bq.scaled_quantize(x, rows=cuda_like(2, 2, dtype=torch.int32)),
                 lambda: bq.scaled_quantize(x, rows=cuda_like(dtype=torch.int32)), lambda: bq.scaled_quantize(x, gate=1.0),
                 lambda: bq.scaled_quantize(None), lambda: bq.ScaledLinear.quantize(cuda_like(16)),
                 lambda: bq.ScaledLinear.quantize(cuda_like(1, 2, 4, 16)), lambda: bq.ScaledLinear.quantize(None),
                 lambda: bq.ScaledLinear(cuda_like(4, 16, dtype=torch.int8), 1.0)):
        with pytest.raises(bq.BQError) as e:
            call()
        assert e.value.status == INVALID
