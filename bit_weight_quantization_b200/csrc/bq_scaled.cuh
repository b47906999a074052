// Scaled int8 layers: per-row int8 quantization and the int8 product with a scale per token and
// per output channel, whole or grouped by expert (include/bq.h, "Scaled int8").
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "bq_scaled_plan.h"
#include "bq_tc.cuh"

namespace bqi {

constexpr unsigned int kErrScaledIndex = 4u;  // a gathered row or a group offset out of range

// ---------------------------------------------------------------------------
// quantization
// ---------------------------------------------------------------------------

struct SqArgs {
  const void* x;
  const void* gate;     // or null
  const int* rows;      // or null
  int8_t* q;
  float* scale;
  long long ldx, ldg, ldq;
  int x_rows, M, K;
  int vec_x, vec_g;     // rows of x / gate start on 16-byte boundaries
};

// Eight elements of a row as they lie in memory (zero from K on), their largest |.|, and their
// values. The order of the bits of |.| is that of the values in all three types, with infinities and
// then NaNs above, so the maximum is taken on the bits, two 16-bit elements at a time.
template <typename T>
struct SqRun {
  static constexpr int W = int(sizeof(T)) * 2;  // 32-bit words
  uint32_t w[W];
  // vec: p is 16-byte aligned (k is a multiple of 8)
  __device__ __forceinline__ void load(const T* p, int k, int K, bool vec) {
    if (vec && k + 8 <= K) {
#pragma unroll
      for (int i = 0; i < W / 4; i++) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + k) + i);
        w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
      }
    } else {
      zero();
#pragma unroll
      for (int i = 0; i < 8; i++) {
        if (k + i < K) {
          if constexpr (sizeof(T) == 4) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + k + i);
          else w[i >> 1] |= uint32_t(__ldg(reinterpret_cast<const unsigned short*>(p) + k + i)) << (16 * (i & 1));
        }
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; i++) w[i] = 0u;
  }
  __device__ __forceinline__ uint32_t most(uint32_t m) const {  // of packed |.| bits
#pragma unroll
    for (int i = 0; i < W; i++) m = sizeof(T) == 4 ? max(m, w[i] & 0x7FFFFFFFu) : __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return m;
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    else return __half2float(__ushort_as_half((unsigned short)(w[i >> 1] >> (16 * (i & 1)))));
  }
  // the larger of the packed maxima as the bits of a float
  static __device__ __forceinline__ uint32_t as_float_bits(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    m = max(m & 0xFFFFu, m >> 16);
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
    else return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
  }
};
// the values of a run times SiLU of another's, kept in f32
template <>
struct SqRun<void> {
  float v[8];
  template <typename T>
  __device__ __forceinline__ void load(const SqArgs& a, long long r, int k) {
    SqRun<T> x, g;
    x.load(static_cast<const T*>(a.x) + r * a.ldx, k, a.K, a.vec_x != 0);
    g.load(static_cast<const T*>(a.gate) + r * a.ldg, k, a.K, a.vec_g != 0);
#pragma unroll
    for (int i = 0; i < 8; i++)
      v[i] = __fmul_rn(x.value(i), __fdiv_rn(g.value(i), __fadd_rn(1.f, expf(-g.value(i)))));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.f;
  }
  __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ float value(int i) const { return v[i]; }
  static __device__ __forceinline__ uint32_t as_float_bits(uint32_t m) { return m; }
};
template <typename T, bool GATE>
using SqHeld = SqRun<typename std::conditional<GATE, void, T>::type>;

template <typename T, bool GATE>
__device__ __forceinline__ void sq_load(const SqArgs& a, long long r, int k, SqHeld<T, GATE>& h) {
  if constexpr (GATE) h.template load<T>(a, r, k);
  else h.load(static_cast<const T*>(a.x) + r * a.ldx, k, a.K, a.vec_x != 0);
}

// Eight codes to p + k. |v s| <= 127 (1 + 2^-22), so adding 1.5 * 2^23 rounds the (already rounded)
// product to the nearest whole number, ties to even, and leaves its two's complement in the low byte.
template <typename H>
__device__ __forceinline__ void sq_store8(int8_t* p, int k, int K, const H& h, float s) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; i++) c[i] = __float_as_uint(__fadd_rn(__fmul_rn(h.value(i), s), 12582912.f));
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; i++)
    w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
  if (k + 8 <= K) {
    *reinterpret_cast<uint2*>(p + k) = make_uint2(w[0], w[1]);
  } else {
    for (int i = 0; k + i < K; i++) p[k + i] = int8_t(w[i >> 2] >> (8 * (i & 3)));
  }
}

// What a row's maximum makes of it. m: the largest |v| as bits.
struct SqScale {
  uint32_t m;
  float s;
  __device__ __forceinline__ explicit SqScale(uint32_t most) : m(most) {
    s = some() ? __fmul_rn(127.f, __frcp_rn(__uint_as_float(m))) : 0.f;
  }
  __device__ __forceinline__ bool fine() const { return m < 0x7F800000u; }
  __device__ __forceinline__ bool some() const { return fine() && m >= 0x0D800000u; }  // 2^-100: s is finite
  __device__ __forceinline__ float scale() const {
    return !fine() ? __uint_as_float(0x7FC00000u) : some() ? __fdiv_rn(__uint_as_float(m), 127.f) : 0.f;
  }
};

// A row's slot: its source row, or -1 where it is empty or out of range
__device__ __forceinline__ int sq_row(const SqArgs& a, int i, bool* bad) {
  const int r = a.rows ? __ldg(a.rows + i) : i;
  *bad = r >= a.x_rows;
  return r < 0 || *bad ? -1 : r;
}

__device__ __forceinline__ void sq_finish(const SqArgs& a, int i, const SqScale& c, bool bad) {
  if (bad) atomicOr(&g_bq_device_error, kErrScaledIndex);
  a.scale[i] = bad ? __uint_as_float(0x7FC00000u) : c.scale();
}

// A row lies in the registers of blockDim.x threads (whole warps), C runs of 8 elements each, so x is
// read once and the gate computed once; blockDim.y rows a block. Bound by memory for f32 and, with 8 runs
// a thread to spread the fixed cost of a thread over, nearly so for 16-bit types; with the gate by the
// instruction issue of its exp and divide, for which the registers are held to 40 so that 48 warps fit
// an SM (60 registers, 22 warps: 95 us for 4096 x 11008 bf16, against 65.6). That costs spills, 12 words a
// thread in 16-bit types and 30 in f32 (75.0 us for 4096 x 11008, 5.4 TB/s).
template <typename T, bool GATE, int C, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_scaled_quantize(const SqArgs a) {
  __shared__ uint32_t most[32];
  pdl_wait();     // nothing is read or written before everything ahead is complete, and only then may the
  pdl_trigger();  // next kernel start: its fetches ahead of its own wait can count on that
  const int i = int(blockIdx.x * blockDim.y + threadIdx.y);
  const bool live = i < a.M;
  bool bad = false;
  const int r = live ? sq_row(a, i, &bad) : -1;
  SqHeld<T, GATE> h[C];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int k = 8 * int(threadIdx.x + c * blockDim.x);
    if (r >= 0 && k < a.K) sq_load<T, GATE>(a, r, k, h[c]);
    else h[c].zero();
  }
#pragma unroll
  for (int c = 0; c < C; c++) m = h[c].most(m);
  m = __reduce_max_sync(0xffffffffu, SqHeld<T, GATE>::as_float_bits(m));
  if (blockDim.x > 32) {
    const int warps = blockDim.x >> 5, w0 = threadIdx.y * warps, lane = threadIdx.x & 31;
    if (lane == 0) most[w0 + (threadIdx.x >> 5)] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < warps ? most[w0 + lane] : 0u);
  }
  if (!live) return;
  const SqScale q(m);
  int8_t* out = a.q + i * a.ldq;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int k = 8 * int(threadIdx.x + c * blockDim.x);
    if (!q.some()) h[c].zero();  // infinities and NaNs must not meet the rounding
    if (k < a.K) sq_store8(out, k, a.K, h[c], q.s);
  }
  if (threadIdx.x == 0) sq_finish(a, i, q, bad);
}

// Rows too long for that: one block of 1024 per row, x read twice (the second time from the caches).
template <typename T, bool GATE>
__global__ void __launch_bounds__(1024) k_scaled_quantize_long(const SqArgs a) {
  __shared__ uint32_t most[32];
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  bool bad;
  const int r = sq_row(a, i, &bad);
  uint32_t m = 0;
  SqHeld<T, GATE> h;
  for (int k = 8 * threadIdx.x; k < a.K && r >= 0; k += 8 * 1024) {
    sq_load<T, GATE>(a, r, k, h);
    m = h.most(m);
  }
  m = __reduce_max_sync(0xffffffffu, SqHeld<T, GATE>::as_float_bits(m));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, most[threadIdx.x & 31]);
  const SqScale q(m);
  for (int k = 8 * threadIdx.x; k < a.K; k += 8 * 1024) {
    if (q.some()) sq_load<T, GATE>(a, r, k, h);
    else h.zero();
    sq_store8(a.q + i * a.ldq, k, a.K, h, q.s);
  }
  if (threadIdx.x == 0) sq_finish(a, i, q, bad);
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
//
// y^T = W q^T on the fifth-generation tensor cores: tcgen05.mma kind::i8 (s8 x s8 -> s32), the
// weights as the MMA's M (128 channels a CTA) and the tokens as its N. Channels are many and
// their number is known, tokens are few, ragged or both: a tile of n tokens costs an MMA of N = n
// rounded up to 16 (32 for a CTA pair), not a whole 128 or 256 rows.
//
// Both operands are K-major rows of codes, copied by TMA in boxes of 128 bytes of k by 128
// channels or n tokens with the 128-byte swizzle, which is the layout the MMA reads. Rows past the
// matrices and k past K read as zero, so K and N need no padding in memory. CG = 2: the two CTAs of
// a cluster hold 128 channels and half of the tokens each, and one MMA of M = 256 reads both.
//
// Warp roles, coupled only by mbarriers: warps 0-3 are the epilogue (tensor-memory lanes 32w ..),
// warp 4 copies, warp 5 issues the MMAs. Accumulators are double-buffered in tensor memory, so the
// copies and MMAs of the next tile run under this tile's epilogue; the kernel is persistent, tile t
// of the CTA (pair) c is c, c + grid, ...
//
// Large products are bound by the tensor cores and, over milliseconds, by the board's power:
// 8192 x 13824 x 5120 in 359 us (3.23 POPS; tensor pipe 93 % active), 424 us in a loop of seconds.
//
// Every wait on an mbarrier is bounded and ends when another role has stopped; then the error word is
// raised, the peer is told, copies in flight are waited for and the tensor memory is freed. Three waits have
// no bound: for the kernel before (it ends by itself), for tensor memory (whatever holds some comes to its
// end: a pair shares its SMs with nothing that leaves it too few columns, see plan_scaled_gemm, and the split
// kernel waits for no peer while it holds some), and at the cluster's barrier (its CTAs start together, and each
// arrives on every path).

constexpr int kSgThreads = 192;
constexpr int kSgCopyWarp = 4, kSgMmaWarp = 5;

struct SgArgs {
  TcTensorMap wmap, qmap, qmap16;  // weights; tokens in boxes of a whole tile, and of 16 rows
  TcTensorMap ymap;                // 16-bit y in boxes of 32 tokens x 32 channels (y_tma)
  const float* w_scale;
  const float* bias;               // or null
  const float* scale;
  const int* offsets;              // or null: one group of M rows
  void* y;
  long long ldy;
  int M, N, K, E, y_type, y_tma;
  int w_experts;                   // distinct weight matrices: E, or 1 where the experts share one
  int bn;                          // tokens per tile at most, a multiple of 16 CG
  int stages, stage_bytes, cols, acc_stride;  // tensor-memory columns, and between accumulators
  int ahead;                       // the kernel before this one is the quantization: weights may be fetched before it ends
};

// Shared-memory descriptor of a K-major operand in 128-byte swizzled rows: start address, 1024
// bytes between 8-row groups, version 1, layout type 2 (the leading offset is not used).
__device__ __forceinline__ uint64_t sg_desc(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(64) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// kind::i8 with s32 accumulators, s8 x s8, both K-major
__device__ __forceinline__ uint32_t sg_idesc(int n, int m) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void sg_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accum) {
  if constexpr (CG == 1)
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(int(accum))
                 : "memory");
  else
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(int(accum))
                 : "memory");
}
// completion of this thread's MMAs so far, on bar of this CTA (CG = 1) or of both CTAs of the pair
template <int CG>
__device__ __forceinline__ void sg_commit(uint64_t* bar, uint32_t pair_mask) {
  if constexpr (CG == 1)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(pair_mask))
        : "memory");
}
// one box into this CTA's shared memory, completing on the barrier at (cluster) address bar
template <int CG>
__device__ __forceinline__ void sg_copy_2d(void* dst, const TcTensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void sg_copy_3d(void* dst, const TcTensorMap* map, int x, int y, int z, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// Instructions that the whole warp takes together (.aligned: tcgen05.ld, alloc and dealloc, stmatrix, the named and
// the cluster barriers) stand behind a __syncwarp() or a vote wherever lanes may have gone different ways before.
//
// One lane of a converged warp. The copying and the MMA warp run their loops with all lanes and let one
// issue: addresses and descriptors then stay in uniform registers. From a branch that only lane 0 takes, an
// MMA took 76 cycles to issue and a chunk of four 594, whatever its tokens.
__device__ __forceinline__ bool sg_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// tc_wait of a converged warp
__device__ __forceinline__ bool sg_wait(uint64_t* bar, uint32_t parity, const uint32_t* stop) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, stop));
}
__device__ __forceinline__ void sg_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void sg_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void sg_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void sg_put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ uint32_t sg_pack(__nv_bfloat16, float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t sg_pack(__half, float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 16 lanes x 32 columns of tensor memory in the m16n8 fragment pattern: thread 4g + t takes columns
// 8i + 2t and + 1 of lane g in v[4i], v[4i + 1], and of lane g + 8 in v[4i + 2], v[4i + 3]
__device__ __forceinline__ void sg_ld_fragments(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void sg_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
// four transposed 8x8 blocks of 16-bit values: thread 4g + t holds rows 2t, 2t + 1 of column g of
// each, lane l gives the address of row l % 8 of block l / 8
__device__ __forceinline__ void sg_store_blocks(uint32_t saddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(saddr), "r"(r0),
               "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void sg_store_2d(const TcTensorMap* map, int x, int y, uint32_t saddr) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(saddr)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}

// One tile of work: tokens m0 .. m0 + n - 1 of expert e against the channels from n0 on.
struct SgTile {
  int e, m0, n, n0;
};

// Walks a CTA's (or pair's) tiles in order. Tiles are numbered expert by expert, and within one in
// bands of 8 token tiles that run along the channels, so that tiles in flight at the same time share
// rows of both operands in the L2.
struct SgWalk {
  const SgArgs& a;
  const int* first;  // grouped: first tile of every expert (shared memory)
  int step, total, nt, e;
  __device__ __forceinline__ SgWalk(const SgArgs& args, const int* first_tile, int channels)
      : a(args), first(first_tile), step(channels), nt((args.N + channels - 1) / channels), e(0) {
    total = a.offsets ? first[a.E] : (a.M + a.bn - 1) / a.bn * nt;
  }
  __device__ __forceinline__ bool at(int t, SgTile* o) {
    if (t >= total) return false;
    int lo = 0, hi = a.M, r = t;
    if (a.offsets) {
      while (first[e + 1] <= t) e++;
      lo = __ldg(a.offsets + e);
      hi = __ldg(a.offsets + e + 1);
      r = t - first[e];
    }
    const int mt = (hi - lo + a.bn - 1) / a.bn;
    const int band = r / (8 * nt), m_first = 8 * band, gm = min(8, mt - m_first);
    r -= band * 8 * nt;
    const int m = m_first + r % gm;
    o->e = e;
    o->n0 = r / gm * step;
    o->m0 = lo + m * a.bn;
    o->n = min(a.bn, hi - o->m0);
    return true;
  }
};

// First tile of every expert from the offsets (warp 0): first[E] is their number, or 0 and *bad = 1
// where the offsets decrease or leave [0, M].
__device__ __forceinline__ void sg_first_tiles(const SgArgs& a, int* first, int channels, uint32_t* bad, int lane) {
  const int nt = (a.N + channels - 1) / channels;
  int base = 0;
  bool wrong = false;
  for (int i0 = 0; i0 < a.E; i0 += 32) {
    const int i = i0 + lane;
    int tiles = 0;
    if (i < a.E) {
      const int lo = __ldg(a.offsets + i), hi = __ldg(a.offsets + i + 1);
      if (lo < 0 || hi < lo || hi > a.M) wrong = true;
      else tiles = (hi - lo + a.bn - 1) / a.bn * nt;
    }
    int sum = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (i < a.E) first[i] = base + sum - tiles;
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  wrong = __any_sync(0xffffffffu, wrong);
  if (lane == 0) {
    first[a.E] = wrong ? 0 : base;
    *bad = wrong;
  }
}

// y of a tile's tokens for this warp's 32 channels ch .. ch + 31 (ch + lane is the thread's). Whole
// blocks of 32 tokens of 16-bit outputs whose rows are aligned go through shared memory: fragments
// out of tensor memory, transposed by stmatrix into [token][32 channels] and written by TMA (which
// drops channels past N), 3.6 instructions an output. The rest (32-bit outputs, unaligned rows, the
// last tokens) is stored column by column, a token's 32 channels as one 64- or 128-byte store.
template <typename Y, bool BIAS>
__device__ __forceinline__ void sg_epilogue(const SgArgs& a, const SgTile& t, uint32_t acc, const float* tok,
                                            uint8_t* stage, int ch, int lane, int* turn) {
  const float* ws = a.w_scale + (long long)t.e * a.N;
  const float* wb = a.bias + (long long)t.e * a.N;
  int c = 0;
  if constexpr (sizeof(Y) == 2) {
    // a store box that N cuts is cut on 16-byte units only: with other N the last channels go below
    if (a.y_tma && ch < a.N && t.n >= 32 && (ch + 32 <= a.N || a.N % 8 == 0)) {
      const int g = lane >> 2, tt = lane & 3;
      float sw[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int n = min(ch + 8 * i + g, a.N - 1);
        sw[i] = __ldg(ws + n);
        b[i] = BIAS ? __ldg(wb + n) : 0.f;
      }
      // row l % 8 of block l / 8, the block's 16 bytes at the 64-byte swizzle's place
      const uint32_t at = uint32_t(lane & 7) * 64u + (uint32_t(lane >> 3) ^ (uint32_t(lane & 7) >> 1)) * 16u;
      for (; c + 32 <= t.n; c += 32) {
        uint32_t lo[16], hi[16];  // channels ch .. + 15, and + 16 .. + 31
        sg_ld_fragments(acc + uint32_t(c), lo);
        sg_ld_fragments(acc + (16u << 16) + uint32_t(c), hi);
        const uint32_t buf = smem_u32(stage) + uint32_t(*turn) * 2048u;
        *turn ^= 1;
        // the copy that read this buffer two blocks ago is done
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;\n" ::: "memory");
        __syncwarp();
        sg_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float2 s = *reinterpret_cast<const float2*>(tok + c + 8 * i + 2 * tt);
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t* v = (j < 2 ? lo : hi) + 4 * i + 2 * (j & 1);
            const float x0 = float(int(v[0])), x1 = float(int(v[1])), s0 = __fmul_rn(s.x, sw[j]), s1 = __fmul_rn(s.y, sw[j]);
            r[j] = BIAS ? sg_pack(Y(), __fmaf_rn(x0, s0, b[j]), __fmaf_rn(x1, s1, b[j]))
                        : sg_pack(Y(), __fmul_rn(x0, s0), __fmul_rn(x1, s1));
          }
          sg_store_blocks(buf + uint32_t(i) * 512u + at, r[0], r[1], r[2], r[3]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) sg_store_2d(&a.ymap, ch, t.m0 + c, buf);
        __syncwarp();
      }
    }
  }
  const int n = ch + lane;
  const bool live = n < a.N;
  const float sw = live ? __ldg(ws + n) : 0.f, b = BIAS && live ? __ldg(wb + n) : 0.f;
  Y* y = static_cast<Y*>(a.y) + (t.m0 + c) * a.ldy + n;
  for (; c < t.n; c += 32) {
    uint32_t v[32];
    tc_ld32(acc + uint32_t(c), v);
    const int left = live ? t.n - c : 0;
#pragma unroll
    for (int i = 0; i < 32; i++) {
      const float x = float(int(v[i])), s = __fmul_rn(tok[c + i], sw);
      if (i < left) sg_put(y, BIAS ? __fmaf_rn(x, s, b) : __fmul_rn(x, s));
      y += a.ldy;
    }
    __syncwarp();
  }
}

template <typename Y>
__device__ __forceinline__ void sg_epilogue(const SgArgs& a, const SgTile& t, uint32_t acc, const float* tok,
                                            uint8_t* stage, int ch, int lane, int* turn) {
  if (a.bias) sg_epilogue<Y, true>(a, t, acc, tok, stage, ch, lane, turn);
  else sg_epilogue<Y, false>(a, t, acc, tok, stage, ch, lane, turn);
}

template <int CG>
__global__ void __launch_bounds__(kSgThreads, 1) k_scaled_tc(const __grid_constant__ SgArgs a) {
  extern __shared__ __align__(128) uint8_t sg_smem[];
  const uint32_t pad = (1024u - (smem_u32(sg_smem) & 1023u)) & 1023u;
  uint8_t* stages = sg_smem + pad;
  uint8_t* region = stages + size_t(a.stages) * a.stage_bytes + (a.y_tma ? kSgYBytes : 0u);
  uint64_t* full = reinterpret_cast<uint64_t*>(region);
  uint64_t* empty = full + kSgMaxStages;
  uint64_t* acc_full = empty + kSgMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  // words: [0] tensor-memory address, [1] a role stopped, [2] bad offsets, [3] copies issued
  uint32_t* words = reinterpret_cast<uint32_t*>(region + 224);
  float* tok = reinterpret_cast<float*>(region + 256);
  int* first = reinterpret_cast<int*>(region + kSgRegion);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), S = a.stages;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int kc = (a.K + kSgChunk - 1) / kSgChunk;
  const int unit = blockIdx.x / CG, units = gridDim.x / CG;
  uint32_t* stop = &words[1];

  if (tid == 0) {
    for (int i = 0; i < S; i++) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4 * CG);
    }
    fence_mbar_init();
    for (int i = 1; i < 8; i++) words[i] = 0;
  }
  if (warp == kSgMmaWarp) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(words)), "r"(a.cols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(words)), "r"(a.cols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
  }
  if (a.offsets) {
    pdl_wait();
    __syncthreads();  // words[2] is zeroed before the scan may set it
    if (warp == 0) sg_first_tiles(a, first, kSgRows * CG, &words[2], lane);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // the peer's barriers and tensor memory are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, words[0], 0);
  SgWalk walk(a, first, kSgRows * CG);
  SgTile t;
  // this CTA's failure is told to its peer, whose waits then end too
  auto give_up = [&]() {
    *reinterpret_cast<volatile uint32_t*>(stop) = 1u;
    if constexpr (CG == 2)
      asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(dsmem_map(smem_u32(stop), rank ^ 1u)), "r"(1u) : "memory");
  };

  if (warp == kSgCopyWarp) {
    const bool lead = sg_elect();
    int st = 0, issued = 0, ahead = 0;
    uint32_t ph = 1;
    bool ok = true;
    // tokens of a tile's MMA, and this CTA's part of them
    auto part_of = [&](const SgTile& o) { return (o.n + 16 * CG - 1) / (16 * CG) * 16; };
    auto bar_of = [&](int i) { return CG == 2 ? dsmem_map(smem_u32(&full[i]), 0u) : smem_u32(&full[i]); };
    auto copy_weights = [&](int i, int k) {
      if (rank == 0) mbar_expect_tx(&full[i], CG * (kSgWBytes + uint32_t(part_of(t)) * kSgChunk));
      sg_copy_3d<CG>(stages + size_t(i) * a.stage_bytes, &a.wmap, k * kSgChunk, t.n0 + int(rank) * kSgRows,
                     min(t.e, a.w_experts - 1), bar_of(i));
    };
    // behind the quantization (which waits for everything before it) the first stages' weights are
    // fetched while it runs; a whole product's tiles do not hang on device data
    if (!a.ahead) pdl_wait();
    if (!a.offsets && walk.at(unit, &t)) {
      ahead = min(S, kc);
      if (lead)
        for (int k = 0; k < ahead; k++) copy_weights(k, k);
    }
    pdl_wait();
    for (int u = unit; ok && walk.at(u, &t); u += units) {
      const int part = part_of(t), m = t.m0 + int(rank) * part;
      for (int k = 0; k < kc; k++) {
        const bool fresh = issued >= ahead;
        if (fresh && !(ok = sg_wait(&empty[st], ph, stop))) break;
        if (lead) {
          if (fresh) copy_weights(st, k);
          uint8_t* dst = stages + size_t(st) * a.stage_bytes + kSgWBytes;
          if (part * CG == a.bn) {
            sg_copy_2d<CG>(dst, &a.qmap, k * kSgChunk, m, bar_of(st));
          } else {
            for (int i = 0; i < part; i += 16) sg_copy_2d<CG>(dst + i * kSgChunk, &a.qmap16, k * kSgChunk, m + i, bar_of(st));
          }
        }
        __syncwarp();
        issued++;
        if (++st == S) { st = 0; ph ^= 1; }
      }
    }
    if (lead) {
      if (!ok) give_up();
      words[3] = uint32_t(issued);
    }
    // every stage's last MMAs have read it (and their arrivals have landed) before this CTA may end
    for (int i = 0; i < min(S, issued) && ok; i++) {
      if (--st < 0) { st = S - 1; ph ^= 1; }
      ok = sg_wait(&empty[st], ph ^ 1u, stop);
    }
  } else if (warp == kSgMmaWarp) {
    pdl_wait();  // not in the bounded waits below: the kernel before may take any time
    if (rank == 0) {
      const bool lead = sg_elect();
      int st = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = unit; ok && walk.at(u, &t); u += units, i++) {
        const int nn = (t.n + 16 * CG - 1) / (16 * CG) * (16 * CG), buf = i & 1;
        const uint32_t idesc = sg_idesc(nn, kSgRows * CG), d = tmem + uint32_t(buf * a.acc_stride);
        if (!(ok = sg_wait(&acc_empty[buf], uint32_t((i >> 1) & 1) ^ 1u, stop))) break;
        tc_fence_after();
        for (int k = 0; k < kc; k++) {
          if (!(ok = sg_wait(&full[st], ph, stop))) break;
          tc_fence_after();
          const uint32_t wa = smem_u32(stages) + uint32_t(st * a.stage_bytes);
          const uint64_t da = sg_desc(wa), db = sg_desc(wa + kSgWBytes);
          if (lead) {
            // always the whole chunk (k past K reads as zero): four MMAs of 32 k issued back to back
#pragma unroll
            for (int j = 0; j < kSgChunk / 32; j++) sg_mma<CG>(d, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
            sg_commit<CG>(&empty[st], 3u);
            if (k == kc - 1) sg_commit<CG>(&acc_full[buf], 3u);
          }
          __syncwarp();
          if (++st == S) { st = 0; ph ^= 1; }
        }
      }
      if (!ok && lead) give_up();
    }
  } else {
    pdl_wait();  // the tokens' scales may be the previous kernel's
    pdl_trigger();
    bool ok = true;
    const uint32_t lanes = uint32_t(32 * warp) << 16;
    uint8_t* ystage = stages + size_t(S) * a.stage_bytes + warp * 4096;
    int i = 0, turn = 0;
    for (int u = unit; walk.at(u, &t); u += units, i++) {
      const int buf = i & 1;
      float* tk = tok + buf * kSgMaxTokens;
      for (int j = tid; j < t.n; j += 128) tk[j] = __ldg(a.scale + t.m0 + j);
      __syncwarp();
      const int ch = t.n0 + int(rank) * kSgRows + 32 * warp;
      asm volatile("bar.sync 1, 128;\n" ::: "memory");  // the scales are written (buffer i - 2 was read before tile i - 1's)
      ok = __all_sync(0xffffffffu, tc_wait(&acc_full[buf], uint32_t((i >> 1) & 1), stop));
      if (ok) {
        tc_fence_after();
        const uint32_t acc = tmem + lanes + uint32_t(buf * a.acc_stride);
        if (a.y_type == BQ_TYPE_F32) sg_epilogue<float>(a, t, acc, tk, ystage, ch, lane, &turn);
        else if (a.y_type == BQ_TYPE_BF16) sg_epilogue<__nv_bfloat16>(a, t, acc, tk, ystage, ch, lane, &turn);
        else sg_epilogue<__half>(a, t, acc, tk, ystage, ch, lane, &turn);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) sg_arrive_at(dsmem_map(smem_u32(&acc_empty[buf]), 0u));
          else mbar_arrive(&acc_empty[buf]);
        }
      } else if (lane == 0) {
        give_up();
      }
      // a warp that gave up still takes the tiles' barriers with the others, without waiting for MMAs
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
  }
  __syncthreads();
  if (tid == 0) {
    if (words[2]) atomicOr(&g_bq_device_error, kErrScaledIndex);
    if (words[1]) {  // a role gave up: copies it had issued are given time to land
      const int issued = int(words[3]);
      if (rank == 0)
        for (int j = max(0, issued - S); j < issued; j++) mbar_wait_bounded(&full[j % S], uint32_t((j / S) & 1));
      for (int j = 0; j < 1000; j++) __nanosleep(1000);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();  // no arrival of the peer is still on its way
  if (warp == kSgMmaWarp) {
    tc_fence_after();
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(a.cols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(a.cols) : "memory");
  }
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
//
// For at most 64 tokens the product is a pass over the weights, N K bytes, and N / 128 tiles are too
// few for the SMs. So a cluster of CTAs splits the k-range of one 128-channel tile; each leaves its
// s32 sums in the shared memory of the CTA that finishes those tokens (integer sums: exact in any
// order). The tensor cores keep up with the memory although an MMA of 128 channels costs the same
// 27 ns for 16 tokens as for 64 (4 KB of weights: 150 GB/s an SM, 22 TB/s in all). Bound by the memory and
// by the time until its first bytes: 1 x 4096 x 4096 from bf16 in 6.6 us (2.5 TB/s), 1 x 13824 x 5120 in
// 14.7 (4.8 TB/s); from codes 16 x 4096 x 4096 in 6.1, 1 x 13824 x 5120 in 13.8 (5.1 TB/s).
//
// T = int8_t: the tokens' codes come by TMA beside the weights. Otherwise x is quantized here, by
// every CTA the tokens of the whole row (their maximum) and the codes of its own k-range, straight
// into the operand's swizzled rows, while the weights are on their way: one launch for a decoded token.

struct SsArgs {
  TcTensorMap wmap, qmap;  // boxes of 128 channels, and of nn tokens
  SqArgs x;                // T != int8_t: the unquantized tokens
  const float* w_scale;
  const float* bias;       // or null
  const float* scale;      // T = int8_t: the tokens' scales
  void* y;
  long long ldy;
  int M, N, K, y_type;
  int nn, stages, stage_bytes, cols, splits;
  int slice;               // tokens that one CTA of the cluster finishes
  int ahead;               // the kernel before this one is the quantization: weights may be fetched before it ends
};

// shared memory of this CTA to that of a CTA of the cluster, counted by a barrier there
__device__ __forceinline__ void dsmem_copy(uint32_t rdst, uint32_t src, uint32_t bytes, uint32_t rbar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(rdst),
               "r"(src), "r"(bytes), "r"(rbar)
               : "memory");
}
// a word to the shared memory of a CTA of the cluster, counted by a barrier there
__device__ __forceinline__ void dsmem_st_async(uint32_t raddr, uint32_t v, uint32_t rbar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];\n" ::"r"(raddr), "r"(v),
               "r"(rbar)
               : "memory");
}
// 32 lanes x 8 columns of tensor memory
__device__ __forceinline__ void ss_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

// y of this thread's channel n for up to four tokens from m on, from their exact sums
template <typename Y>
__device__ __forceinline__ void ss_put(const SsArgs& a, int m, int count, int n, const float* scale, float sw, float b,
                                       const uint32_t (&v)[4]) {
  Y* y = static_cast<Y*>(a.y) + m * a.ldy + n;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (i < count) {
      const float s = __fmul_rn(scale[m + i], sw), f = float(int(v[i]));
      sg_put(y, a.bias ? __fmaf_rn(f, s, b) : __fmul_rn(f, s));
      y += a.ldy;
    }
  }
}
__device__ __forceinline__ void ss_out(const SsArgs& a, int m, int count, int n, const float* scale, float sw, float b,
                                       const uint32_t (&v)[4]) {
  if (a.y_type == BQ_TYPE_F32) ss_put<float>(a, m, count, n, scale, sw, b, v);
  else if (a.y_type == BQ_TYPE_BF16) ss_put<__nv_bfloat16>(a, m, count, n, scale, sw, b, v);
  else ss_put<__half>(a, m, count, n, scale, sw, b, v);
}

// 32 lanes x 4 columns of tensor memory
__device__ __forceinline__ void ss_ld4(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

// Warps 0-3: every token's largest |x| of this warp's share of the row, to most[4 t + warp]. The first
// loads are issued before the copying warp is let go on (barrier 2): behind the weights they would
// take three times as long.
template <typename T, int TOK>
__device__ __forceinline__ void ss_maxima(const SsArgs& a, uint32_t* most, int tid) {
  constexpr int U = 4;
  uint32_t m[TOK] = {};
  for (int k0 = 8 * tid; k0 == 8 * tid || k0 < a.K; k0 += 8 * 128 * U) {
    SqRun<T> h[U][TOK];
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int t = 0; t < TOK; t++)
        if (t < a.M && k0 + u * 8 * 128 < a.K)
          h[u][t].load(static_cast<const T*>(a.x.x) + t * a.x.ldx, k0 + u * 8 * 128, a.K, a.x.vec_x != 0);
        else h[u][t].zero();
    if (k0 == 8 * tid) {  // every lane's first pass
      __syncwarp();
      asm volatile("bar.arrive 2, 160;\n" ::: "memory");
    }
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int t = 0; t < TOK; t++) m[t] = h[u][t].most(m[t]);
  }
#pragma unroll
  for (int t = 0; t < TOK; t++) {
    m[t] = __reduce_max_sync(0xffffffffu, SqRun<T>::as_float_bits(m[t]));
    if ((tid & 31) == 0) most[4 * t + (tid >> 5)] = m[t];
  }
}

// Then the tokens' scales, and their codes of the chunks k0 .. k0 + n - 1 as rows 0 .. M - 1 of the
// operand (rows from M on hold whatever was there: their columns of the product are not read).
template <typename T, int TOK>
__device__ __forceinline__ void ss_quantize(const SsArgs& a, uint8_t* operand, float* scale, const uint32_t* most,
                                            int k0, int n, int tid) {
  auto of = [&](int t) { return SqScale(max(max(most[4 * t], most[4 * t + 1]), max(most[4 * t + 2], most[4 * t + 3]))); };
  for (int i = tid; i < 16 * n; i += 128) {  // run i: 8 codes, half a 16-byte unit of the swizzled row
    const int c = i >> 4, u = (i & 15) >> 1, k = (k0 + c) * kSgChunk + 8 * (i & 15);
#pragma unroll
    for (int t = 0; t < TOK; t++) {
      if (t < a.M) {
        const SqScale q = of(t);
        SqRun<T> h;
        if (q.some() && k < a.K) h.load(static_cast<const T*>(a.x.x) + t * a.x.ldx, k, a.K, a.x.vec_x != 0);
        else h.zero();
        sq_store8(reinterpret_cast<int8_t*>(operand) + c * kSsFusedRow + t * kSgChunk + ((u ^ t) << 4) + 8 * (i & 1), 0, 8, h,
                  q.s);
      }
    }
  }
  if (tid < a.M) scale[tid] = of(tid).scale();
}

template <typename T, int TOK>
__global__ void __launch_bounds__(kSgThreads, 2) k_scaled_split(const __grid_constant__ SsArgs a) {
  constexpr bool FUSED = !std::is_same<T, int8_t>::value;
  extern __shared__ __align__(128) uint8_t ss_smem[];
  const uint32_t pad = (1024u - (smem_u32(ss_smem) & 1023u)) & 1023u;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), S = a.stages, P = a.splits;
  const uint32_t rank = P > 1 ? cluster_rank() : 0u;
  const int n0 = int(blockIdx.x) / P * kSgRows, kc = (a.K + kSgChunk - 1) / kSgChunk;
  const int k0 = int(rank) * kc / P, nk = (int(rank) + 1) * kc / P - k0;  // this CTA's chunks
  uint8_t* stages = ss_smem + pad;
  uint8_t* operand = stages + size_t(S) * a.stage_bytes;
  // the sums of the tokens this CTA finishes, [sender][token][128 channels]
  uint32_t* sums = reinterpret_cast<uint32_t*>(operand + (FUSED ? uint32_t((kc + P - 1) / P) * kSsFusedRow : 0u));
  uint8_t* region = reinterpret_cast<uint8_t*>(sums) + (P > 1 ? size_t(P) * a.slice * kSgRows * 4 : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(region);
  uint64_t* empty = full + kSgMaxStages;
  uint64_t* acc_full = empty + kSgMaxStages;
  uint64_t* tok_full = acc_full + 1;
  uint64_t* sums_full = tok_full + 1;
  // words: [0] tensor-memory address, [1] a role stopped, [2] copies issued
  uint32_t* words = reinterpret_cast<uint32_t*>(region + 224);
  float* scale = reinterpret_cast<float*>(region + 256);
  uint32_t* most = reinterpret_cast<uint32_t*>(region + 512);
  uint32_t* stop = &words[1];
  const uint32_t bytes = kSgWBytes + (FUSED ? 0u : uint32_t(a.nn) * kSgChunk);
  const bool copier = warp == kSgCopyWarp && sg_elect();
  auto copy_weights = [&](int j, int st) {
    mbar_expect_tx(&full[st], bytes);
    sg_copy_3d<1>(stages + size_t(st) * a.stage_bytes, &a.wmap, (k0 + j) * kSgChunk, n0, 0, smem_u32(&full[st]));
  };
  auto copy_tokens = [&](int j, int st) {
    if constexpr (!FUSED)
      sg_copy_2d<1>(stages + size_t(st) * a.stage_bytes + kSgWBytes, &a.qmap, (k0 + j) * kSgChunk, 0, smem_u32(&full[st]));
  };

  auto free_tmem = [&]() {  // by the whole MMA warp
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(words[0]), "r"(a.cols) : "memory");
  };

  const int first = min(S, nk);
  if (copier) {  // before any other setup: the weights' first copies
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.wmap)) : "memory");
    for (int i = 0; i < S; i++) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(tok_full, 4);
    mbar_init(sums_full, 1);
    fence_mbar_init();
    if (P > 1) mbar_expect_tx(sums_full, uint32_t(P * max(0, min(a.slice, a.M - int(rank) * a.slice))) * kSgRows * 4u);
    if (!FUSED && !a.ahead) pdl_wait();
  }
  if (FUSED && warp == kSgCopyWarp) {
    pdl_wait();
    __syncwarp();
    asm volatile("bar.sync 2, 160;\n" ::: "memory");  // the tokens' loads are on their way
  }
  if (copier)
    for (int j = 0; j < first; j++) copy_weights(j, j);
  if (tid == 0)
    for (int i = 1; i < 8; i++) words[i] = 0;
  // Arrived once this CTA's barriers are set up (fence_mbar_init orders that for the cluster), waited for
  // before a peer is written to. Relaxed: a release here waits for the copies in flight, 2 us when the memory is
  // busy with weights. Ahead of the allocation, which waits while other kernels hold the SM's tensor memory: no
  // CTA waits for a peer while it holds columns itself (they are freed before the peers' sums are waited for), so
  // what holds them always comes to its end. Behind the copies: ahead of them one token of 4096 x 4096 takes 6.72
  // us instead of 6.59.
  if (P > 1) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  }
  if (warp == kSgMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(words)), "r"(a.cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (FUSED && warp < 4) {  // x is read before the weights fill the memory's queues
    pdl_wait();
    ss_maxima<T, TOK>(a, most, tid);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, words[0], 0);
  pdl_wait();
  pdl_trigger();  // only now: what follows may count on everything before this kernel being complete
  bool freed = false;  // the MMA warp's: the tensor memory

  if (warp == kSgCopyWarp) {
    bool ok = true;
    int j = 0, st = 0;
    uint32_t ph = 1;
    for (; j < nk; j++) {
      if (j >= first && !(ok = sg_wait(&empty[st], ph, stop))) break;
      if (copier) {
        if (j >= first) copy_weights(j, st);
        copy_tokens(j, st);
      }
      __syncwarp();
      if (++st == S) { st = 0; ph ^= 1; }
    }
    if (copier) {
      if (!ok) *reinterpret_cast<volatile uint32_t*>(stop) = 1u;
      words[2] = uint32_t(j);
    }
    for (int i = 0; i < first && ok; i++) {  // every stage's MMAs have arrived before this CTA may end
      if (--st < 0) { st = S - 1; ph ^= 1; }
      ok = sg_wait(&empty[st], ph ^ 1u, stop);
    }
  } else if (warp == kSgMmaWarp) {
    const bool lead = sg_elect();
    const uint32_t idesc = sg_idesc(a.nn, kSgRows);
    bool ok = !FUSED || sg_wait(tok_full, 0, stop);
    int st = 0;
    uint32_t ph = 0;
    for (int j = 0; j < nk && ok; j++) {
      if (!(ok = sg_wait(&full[st], ph, stop))) break;
      tc_fence_after();
      const uint32_t wa = smem_u32(stages) + uint32_t(st * a.stage_bytes);
      const uint64_t da = sg_desc(wa), db = sg_desc(FUSED ? smem_u32(operand) + uint32_t(j) * kSsFusedRow : wa + kSgWBytes);
      if (lead) {
#pragma unroll
        for (int i = 0; i < kSgChunk / 32; i++) sg_mma<1>(tmem, da + 2 * i, db + 2 * i, idesc, j > 0 || i > 0);
        tc_commit(&empty[st]);
        if (j == nk - 1) tc_commit(acc_full);
      }
      __syncwarp();
      if (++st == S) { st = 0; ph ^= 1; }
    }
    if (!ok && lead) *reinterpret_cast<volatile uint32_t*>(stop) = 1u;
    __syncwarp();
    asm volatile("bar.sync 3, 160;\n" ::: "memory");  // the accumulators are read, or a role has stopped
    freed = __all_sync(0xffffffffu, *reinterpret_cast<const volatile uint32_t*>(stop) == 0u);
    if (freed) free_tmem();
  } else {
    const int n = n0 + tid;  // this thread's channel
    const bool live = n < a.N;
    const float sw = live ? __ldg(a.w_scale + n) : 0.f, b = a.bias && live ? __ldg(a.bias + n) : 0.f;
    if constexpr (FUSED) {
      ss_quantize<T, TOK>(a, operand, scale, most, k0, nk, tid);
      fence_proxy_async();  // the codes are read by the MMA
      __syncwarp();
      if (lane == 0) mbar_arrive(tok_full);
    } else if (tid < a.M) {
      scale[tid] = __ldg(a.scale + tid);
    }
    __syncwarp();
    asm volatile("bar.sync 1, 128;\n" ::: "memory");  // the scales are written
    bool ok = __all_sync(0xffffffffu, tc_wait(acc_full, 0, stop));
    tc_fence_after();
    const uint32_t acc = tmem + (uint32_t(32 * warp) << 16);
    auto accumulators_read = [&]() {
      if (!ok && lane == 0) *reinterpret_cast<volatile uint32_t*>(stop) = 1u;
      tc_fence_before();
      __syncwarp();
      asm volatile("bar.arrive 3, 160;\n" ::: "memory");
    };
    if (P == 1) {
      for (int c = 0; ok && c < a.M; c += 4) {
        uint32_t v[4];
        ss_ld4(acc + uint32_t(c), v);
        if (live) ss_out(a, c, a.M - c, n, scale, sw, b, v);
        __syncwarp();
      }
      accumulators_read();
    } else {
      // token m's sums to CTA m / slice, at [this CTA][m % slice][channel] there
      if (a.M <= kSsDirect) {  // few: straight from the registers, and this CTA need not wait for their arrival
        uint32_t v[8];
        ss_ld8(acc, v);
        accumulators_read();
        asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
#pragma unroll
        for (int i = 0; i < kSsDirect; i++) {
          if (ok && i < a.M) {
            const uint32_t to = uint32_t(i / a.slice);
            dsmem_st_async(dsmem_map(smem_u32(sums + (int(rank) * a.slice + i % a.slice) * kSgRows + tid), to), v[i],
                           dsmem_map(smem_u32(sums_full), to));
          }
        }
      } else {  // over the stages (whose MMAs are done) as [token][channel], then a copy to each CTA
        uint32_t* mine = reinterpret_cast<uint32_t*>(stages);
        for (int c = 0; ok && c < a.M; c += 8) {
          uint32_t v[8];
          ss_ld8(acc + uint32_t(c), v);
#pragma unroll
          for (int i = 0; i < 8; i++) mine[(c + i) * kSgRows + tid] = v[i];
        }
        accumulators_read();
        fence_proxy_async();
        asm volatile("bar.sync 1, 128;\n" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        if (ok && tid < P && tid * a.slice < a.M)
          dsmem_copy(dsmem_map(smem_u32(sums + int(rank) * a.slice * kSgRows), uint32_t(tid)), smem_u32(mine + tid * a.slice * kSgRows),
                     uint32_t(min(a.slice, a.M - tid * a.slice)) * kSgRows * 4u, dsmem_map(smem_u32(sums_full), uint32_t(tid)));
        __syncwarp();
      }
      const int m0 = int(rank) * a.slice, m1 = min(m0 + a.slice, a.M);
      if (m0 < m1) {
        ok = __all_sync(0xffffffffu, ok && tc_wait(sums_full, 0, stop));
        for (int m = m0; ok && live && m < m1; m += 4) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            v[i] = 0;
#pragma unroll
            for (int q = 0; q < kSsMaxSplit; q++)
              if (q < P && m + i < m1) v[i] += sums[(q * a.slice + m + i - m0) * kSgRows + tid];
          }
          ss_out(a, m, m1 - m, n, scale, sw, b, v);
        }
      }
    }
    if (!ok && lane == 0) *reinterpret_cast<volatile uint32_t*>(stop) = 1u;
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (words[1]) {  // a role gave up: copies and MMAs it had issued are given time to land
    if (tid == 0) {
      const int issued = max(int(words[2]), first);
      for (int j = max(0, issued - S); j < issued; j++) mbar_wait_bounded(&full[j % S], uint32_t((j / S) & 1));
      for (int j = 0; j < 1000; j++) __nanosleep(1000);
    }
    __syncthreads();
  }
  if (warp == kSgMmaWarp && !freed) free_tmem();
  // no CTA leaves while its sums are being copied out of its shared memory; nor, if it did not get all that
  // it waited for, while a peer may still write to it (threads that have left count as arrived)
  if (P > 1 && (a.M > kSsDirect || words[1])) {
    __syncwarp();
    if (warp >= 4) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  }
}

}  // namespace bqi
