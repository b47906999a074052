"""Launch plans of the scaled int8 products (no GPU): what every plan has to fit into, over the range of sizes."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "bq_scaled_plan.h"
using namespace bqi;
int main() {
  char op[8];
  int M, N, K, E, flag, tma;
  const int clusters[9] = {0, 148, 74, 48, 36, 28, 24, 20, 18};
  while (std::scanf("%7s %d %d %d %d %d %d", op, &M, &N, &K, &E, &flag, &tma) == 7) {
    if (!std::strcmp(op, "tc")) {
      const SgPlan p = plan_scaled_gemm(M, N, K, E, flag, tma, 148);
      std::printf("%d %d %d %d %d %d %u\n", p.cg, p.bn, p.stages, p.stage_bytes, p.cols, p.acc_stride, p.smem);
    } else {
      const SsPlan p = plan_scaled_split(M, N, K, flag, clusters, 148);
      std::printf("%d %d %d %d %d %d %u\n", p.nn, p.cols, p.splits, p.slice, p.stages, p.stage_bytes, p.smem);
    }
  }
}
"""
SMEM, KB, COLS = 227 * 1024, 1024, 512  # of a CTA; what the SM keeps for itself a CTA; tensor-memory columns
REGION, SPLIT_REGION = 256 + 2 * 256 * 4, 576


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "bit_weight_quantization_b200", "csrc"),
                    "-o", str(d / "p"), str(d / "p.cpp")], check=True)

    def run(rows):
        text = "\n".join(" ".join(map(str, r)) for r in rows)
        out = subprocess.run([str(d / "p")], input=text, check=True, capture_output=True, text=True).stdout.split("\n")
        return list(zip(rows, [tuple(map(int, o.split())) for o in out[:len(rows)]]))
    return run


def log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def whole(rng, n):
    sizes = [(M, 4096, 4096) for M in list(range(65, 700)) + [1000, 2048, 8192, 1 << 20]]
    sizes += [(log(rng, 65, 1 << 20), log(rng, 1, 1 << 20), log(rng, 1, 65536)) for _ in range(n)]
    return [("tc", M, N, K, 1, 0, rng.randint(0, 1)) for M, N, K in sizes]


def grouped(rng, n):
    return [("tc", log(rng, 1, 1 << 20), log(rng, 1, 1 << 16), log(rng, 1, 65536), log(rng, 1, 1024), 1, rng.randint(0, 1))
            for _ in range(n)]


def split(rng, n):
    rows = [("split", M, N, K, 1, f, 0) for f in (0, 1) for M in range(1, 3 if f else 65)
            for N, K in [(1, 1), (128, 128), (300, 1024), (4096, 4096), (13824, 5120), (4096, 16384), (40, 16384)]]
    for _ in range(n):
        f = rng.randint(0, 1)
        rows.append(("split", rng.randint(1, 2 if f else 64), log(rng, 1, 1 << 20), log(rng, 1, 16384 if f else 65536), 1, f, 0))
    return rows


def test_plans_fit_their_shared_and_tensor_memory(plans):
    rng = random.Random(1)
    widths = set()
    for (_, M, N, K, E, by_expert, tma), (cg, bn, stages, stage, cols, stride, smem) in plans(whole(rng, 2000) + grouped(rng, 4000)):
        case = (M, N, K, E, by_expert, tma)
        assert cg in (1, 2) and bn % (16 * cg) == 0 and 16 <= bn <= (64 if cg == 1 else 256), case
        assert stage == 128 * 128 + bn // cg * 128 and stage % 1024 == 0 and 2 <= stages <= 12, case
        assert smem <= SMEM
        assert smem >= 1024 + stages * stage + (16384 if tma else 0) + REGION + (4 * (E + 1) if by_expert else 0), case
        assert stride >= bn and stride % 32 == 0 and 2 * stride <= cols <= COLS and cols & (cols - 1) == 0, case
        widths.add((cg, bn))
    assert {(2, n) for n in range(64, 257, 32)} <= widths and {(1, n) for n in (16, 32, 48, 64)} <= widths
    for (_, M, N, K, _, fused, _), (nn, cols, p, slice_, stages, stage, smem) in plans(split(rng, 4000)):
        case = (M, N, K, fused)
        kc = -(-K // 128)
        assert 1 <= p <= min(8, kc) and p * slice_ >= M and nn >= M and nn % 16 == 0 and cols >= nn, case
        fixed = 1024 + SPLIT_REGION + (-(-kc // p) * 2048 if fused else 0) + (p * slice_ * 512 if p > 1 else 0)
        assert stages >= 1 and fixed + stages * stage <= smem <= SMEM, case
        assert stages * stage >= (M + 7) // 8 * 8 * 512, case  # the sums lie over the stages before they are copied


def test_no_allocation_of_tensor_memory_has_to_wait_beside_a_pair(plans):
    """The CTAs that share an SM never ask for more columns than it has. A pair that waits for columns on one SM
    while it holds those of the other could be waited for by what holds them."""
    rng = random.Random(2)
    # columns per byte of shared memory, and the least shared memory, of the CTAs that may lie beside others
    density, least, pairs = 0.0, SMEM, []
    for _, (cg, bn, _, _, cols, _, smem) in plans(whole(rng, 2000) + grouped(rng, 4000)):
        if cg == 2:
            pairs.append((bn, cols, smem))
        else:
            density, least = max(density, cols / (smem + KB)), min(least, smem + KB)
    for _, (nn, cols, _, _, _, _, smem) in plans(split(rng, 4000)):
        density, least = max(density, cols / (smem + KB)), min(least, smem + KB)
    assert density * 228 * KB <= COLS
    assert any(cols == COLS for _, cols, _ in pairs)
    for bn, cols, smem in pairs:
        left = 228 * KB - (smem + KB)
        assert left < least or cols + density * left <= COLS, (bn, cols, smem)


def test_gpu_cases_take_a_third_tile(plans):
    """The whole-output comparisons of tests/test_scaled_forms_gpu.py: every width of a pair's tile, single CTAs
    and pairs, and more than two tiles each (an accumulator is used again from the third on)."""
    from tests.test_scaled_forms_gpu import GROUPED, TILES, counts_of
    widths, deep = set(), 0
    for (_, M, N, K, *_), (cg, bn, stages, *_) in plans([("tc", M, N, K, 1, 0, 1) for M, N, K in TILES]):
        assert cg == 2 and -(-M // bn) * -(-N // 256) > 2 * 74, (M, N, K)
        widths.add(bn)
        deep += -(-K // 128) > stages
    assert widths == set(range(64, 257, 32)) and deep >= 3
    kinds = []
    for E, most, N, K, how in GROUPED:
        counts = counts_of(E, most, N, how)
        [(_, (cg, bn, stages, *_))] = plans([("tc", int(counts.sum()) + 8, N, K, E, 1, 1)])
        tiles = sum(-(-int(c) // bn) for c in counts) * -(-N // (128 * cg))
        assert tiles > 2 * (74 if cg == 2 else 296), (E, N)
        kinds.append((cg, -(-K // 128) > stages))
    assert set(kinds) == {(1, True), (1, False), (2, True), (2, False)}
