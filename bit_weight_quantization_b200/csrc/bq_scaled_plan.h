// Scaled int8 products: sizes of their kernels' shared and tensor memory, and the plans of their launches.
// Plain C++, no device code: a plan can be looked at without a GPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace bqi {

constexpr int kSgRows = 128;       // channels per CTA
constexpr int kSgChunk = 128;      // bytes of k per stage
constexpr int kSgMaxStages = 12;
constexpr int kSgMaxTokens = 256;  // tokens per tile at most
constexpr uint32_t kSgWBytes = kSgRows * kSgChunk;
// shared memory: alignment slack, the stages (each a multiple of 1024 bytes), the outputs'
// staging where y is written by TMA, then this region:
// full[12] (0), empty[12] (96), acc_full[2] (192), acc_empty[2] (208), words[8] (224), token scales
// [2][256] (256); then, grouped, the first tile of every expert [E + 1]
constexpr uint32_t kSgYBytes = 4 * 2 * 2048;  // outputs on their way: two blocks of 32 x 32 for each epilogue warp
constexpr uint32_t kSgRegion = 256 + 2 * kSgMaxTokens * 4;

constexpr int kSsMaxTokens = 64, kSsFusedTokens = 2;
constexpr int kSsMaxSplit = 8, kSsDirect = 8;
constexpr uint32_t kSsFusedRow = 16 * kSgChunk;  // a chunk of the fused operand: 16 rows of 128 codes
// after the stages, the fused operand and the received sums: full[12] (0), empty[12] (96), acc_full
// (192), tok_full (200), sums_full (208), words[8] (224), token scales [64] (256), maxima [2][4] (512)
constexpr uint32_t kSsRegion = 576;

// shared memory of a CTA: all it can have, and what leaves room for a second one on its SM
constexpr uint32_t kSgSmemMax = 227 * 1024, kSsSmem = 113 * 1024;
constexpr int kTmemCols = 512;  // tensor-memory columns of an SM

struct SgPlan {
  int cg, bn, stages, stage_bytes;
  int cols, acc_stride;  // tensor-memory columns, and between the two accumulators
  uint32_t smem;
};

// Tokens per tile of CTA pairs, for rows of one whole product on N channels: the choice that
// takes the fewest cycles by this model. A chunk of 128 k costs a pair its four MMAs (138 cycles each at 256
// tokens, 69 at 128, 47 at 64) or the copies of its operands at 64 bytes a cycle and SM; a wave is as many
// tiles as there are pairs; the last tile's epilogue, 23 cycles a token, is not hidden. (Measured, 333 x
// 5120 x 5104: 21.9 us with 256, 17.9 with 128; 256 x 4096 x 4096: 16.8 and, with 64, 11.4.)
inline int scaled_pair_tokens(long long rows, int N, int K, int sms) {
  const long long nt = (N + 2 * kSgRows - 1) / (2 * kSgRows), kc = (K + kSgChunk - 1) / kSgChunk, pairs = sms / 2;
  int best = 256;
  double best_cost = -1;
  for (int bn = 256; bn >= 64; bn -= 32) {
    const long long tiles = (rows + bn - 1) / bn * nt, waves = (tiles + pairs - 1) / pairs;
    const double chunk = std::max(4.0 * std::max(47.0, 0.54 * bn), (double(kSgWBytes) + 64.0 * bn) / 64.0);
    const double cost = double(waves) * double(kc) * chunk + 23.0 * double(std::min<long long>(bn, rows));
    if (best_cost < 0 || cost < best_cost) { best = bn; best_cost = cost; }
  }
  return best;
}

// By expert: single CTAs, two an SM, for 64 rows an expert and fewer on average, pairs above. (Measured with
// both forced, even rows, pairs / single, in us. 64 experts of 2048 x 2048, f32: 46.5 / 46.2 at 1 row, 49.5 /
// 48.7 at 16, 51.2 / 50.8 at 32, 52.5 / 53.2 at 48, 54.4 / 54.5 at 64, 54.8 / 58.6 at 72, 57.0 / 62.2 at 96. 16
// experts of 4096 x 4096, bf16: 47.8 / 43.9, 48.4 / 45.8, 49.2 / 46.3, 51.2 / 48.0, 51.0 / 47.4, 54.0 / 59.6,
// 54.1 / 60.9. 64 experts of 4096 x 1024, bf16: 56.0 / 45.6, 59.9 / 46.5, 56.8 / 47.2, 64.0 / 49.3, 60.8 / 50.0,
// 72.5 / 61.8, 71.2 / 65.0: there single CTAs would still win above 64. Rows that differ by up to half either
// way cost single CTAs more where some pass 64: 16 experts of 56 and 64 rows, 51.5 / 55.4 and 53.3 / 53.6.) Tokens
// a tile go up to twice the average: a hotter expert takes several tiles and reads its weights again for each.
//
// A pair that takes every column of its SMs leaves 16 KB of their shared memory at most, so that no other CTA with
// tensor memory (20 KB at least) can lie on either. One could otherwise hold columns on the first SM while it waits
// for a CTA of its own cluster that waits for columns on the second, which the pair holds while it waits for the
// first. Not the whole of it, so that the next launch's first blocks, where they need little, can lie beside the
// pair's last (bq_scaled_linear of 2048 x 4096 x 4096: 30.7 us with the whole, 30.2 in bf16, 35.3 and
// 34.8 in f32).
inline SgPlan plan_scaled_gemm(int M, int N, int K, int E, bool grouped, bool y_tma, int sms) {
  SgPlan p{};
  const long long rows = grouped ? ((long long)M + E - 1) / E : M;  // of one expert, on average
  const long long most = grouped ? std::min<long long>(M, 2 * rows) : M;
  if (rows <= 64) {
    p.cg = 1;
    p.bn = int(std::min<long long>(64, (most + 15) / 16 * 16));
  } else {
    p.cg = 2;
    p.bn = int(std::min<long long>(grouped ? 256 : scaled_pair_tokens(rows, N, K, sms), (most + 31) / 32 * 32));
  }
  p.stage_bytes = int(kSgWBytes) + p.bn / p.cg * kSgChunk;
  p.acc_stride = (p.bn + 31) / 32 * 32;
  p.cols = 32;
  while (p.cols < 2 * p.acc_stride) p.cols *= 2;
  const uint32_t fixed = 1024 + kSgRegion + (y_tma ? kSgYBytes : 0u) + (grouped ? 4u * uint32_t(E + 1) : 0u);
  // single CTAs (few rows an expert) share an SM
  const uint32_t room = p.cg == 1 ? kSsSmem : kSgSmemMax;
  p.stages = std::min(kSgMaxStages, int(room - fixed) / p.stage_bytes);
  p.smem = fixed + uint32_t(p.stages * p.stage_bytes);
  if (p.cols == kTmemCols) p.smem = std::max(p.smem, kSgSmemMax - 16 * 1024);
  return p;
}

// The split kernel for M tokens (M <= kSsMaxTokens): clusters of `splits` CTAs per 128 channels, each
// CTA within half of an SM's shared memory. Two then run on an SM, or one beside the next launch's first
// (with the whole of it, one token of 4096 x 4096 took 9.7 us among others instead of 6.6).

// What p splits of `tiles` 128-channel tiles are expected to take, in ns, where `clusters` of p CTAs run at
// once. A chunk of k takes an SM 200 ns for 16 KB of weights (more with the tokens' codes beside them), or
// 900 ns over the stages in flight; all SMs together draw at most 16 KB in 2.64 ns, 2.45 where two CTAs
// share some. SMs take equal shares, so those with two CTAs finish their second one's chunks alone. 2 us for
// a further wave, 2.7 for launch, first copies and output, and the exchange of the sums grows with the tokens;
// a CTA that quantizes takes 0.1 us a chunk of its own range. (Measured, in us, for 1 / 2 / 3 / 4 / 6 / 8
// splits: one token from codes, 4096 x 4096: 9.1 / 6.8 / 5.8 / 5.7 / 6.4 / 5.6; 11008 x 4096: 10.5 / 11.2 /
// 9.4 / 12.0 / 12.3 / 13.2; 13824 x 5120: 13.8 / 13.9 / 16.1 / 15.0 / 17.6 / 17.7; 4096 x 11008: 20.7 / 12.5 /
// 10.2 / 10.0 / 9.7 / 9.4; 64 tokens, 4096 x 4096: 13.3 / 12.2 / 9.7 / 9.1 / 9.8 / 9.2.)
inline double scaled_split_ns(int p, int tiles, int clusters, int chunks, int stages, int stage_bytes, int M, bool fused,
                              int sms) {
  const double least = std::max(200.0 * stage_bytes / kSgWBytes, 900.0 / stages);
  auto wave = [&](int n) {  // n clusters at once
    const int a = n * p;
    if (a <= sms) return chunks * std::max(least, 2.64 * a);
    return chunks * (std::max(least, 2.45 * sms) + std::max(least, 2.45 * (a - sms)));
  };
  const int full = tiles / clusters, rest = tiles % clusters;
  return 2700.0 + full * wave(clusters) + (rest ? wave(rest) : 0.0) + 2000.0 * (full + (rest ? 1 : 0) - 1) +
         (p > 1 ? 25.0 * M + 0.45 * M * M : 16.0 * M) + (fused ? 50.0 * chunks * (M + 1) : 0.0);
}


struct SsPlan {
  int nn, cols;    // tokens of the MMA, tensor-memory columns
  int splits;      // 0: no split fits
  int slice;       // tokens that one CTA of the cluster finishes
  int stages, stage_bytes;
  uint32_t smem;
};

// clusters[p]: clusters of p CTAs that the device holds at once, one CTA an SM (0: none)
inline SsPlan plan_scaled_split(int M, int N, int K, bool fused, const int* clusters, int sms) {
  const int tiles = (N + kSgRows - 1) / kSgRows, kc = (K + kSgChunk - 1) / kSgChunk;
  SsPlan run{};
  run.nn = (M + 15) / 16 * 16;
  run.cols = 32;
  while (run.cols < run.nn) run.cols *= 2;
  run.stage_bytes = int(kSgWBytes) + (fused ? 0 : run.nn * kSgChunk);
  // the stages also hold the CTA's sums, 512 bytes a token, before they are copied: two at least beyond 32 tokens
  const int least = M > 32 ? 2 : 1;
  double best = -1;
  for (int p = 1; p <= kSsMaxSplit && p <= kc; p++) {
    if (clusters[p] <= 0) continue;
    const int slots = 2 * clusters[p], chunks = (kc + p - 1) / p;
    SsPlan t = run;
    t.splits = p;
    t.slice = (M + p - 1) / p;
    const uint32_t fixed = 1024 + kSsRegion + (fused ? uint32_t(chunks) * kSsFusedRow : 0u) +
                           (p > 1 ? uint32_t(p * t.slice) * kSgRows * 4u : 0u);
    const uint32_t room = fixed + uint32_t(2 * t.stage_bytes) > kSsSmem ? kSgSmemMax : kSsSmem;
    if (fixed + uint32_t(least * t.stage_bytes) > room) continue;
    t.stages = std::min(std::max(least, std::min(kSgMaxStages, chunks)), int((room - fixed) / uint32_t(t.stage_bytes)));
    t.smem = fixed + uint32_t(t.stages * t.stage_bytes);
    const double ns = scaled_split_ns(p, tiles, slots, chunks, t.stages, t.stage_bytes, M, fused, sms) +
                      (room > kSsSmem ? 5000.0 : 0.0);
    if (best < 0 || ns < best) {
      best = ns;
      run = t;
    }
  }
  return run;
}

}  // namespace bqi
