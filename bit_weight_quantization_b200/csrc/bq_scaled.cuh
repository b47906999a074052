// Scaled int8 layers: per-row int8 quantization and the int8 product with a scale per token and
// per output channel, whole or grouped by expert (include/bq.h, "Scaled int8").
#pragma once

#include <cuda_fp16.h>

#include "bq_gemv.cuh"

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

__device__ __forceinline__ float sq_to_float(float v) { return v; }
__device__ __forceinline__ float sq_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float sq_to_float(__half v) { return __half2float(v); }

// v[0..7] = p[k..k+7] as floats, zero from K on; vec: p is 16-byte aligned (k is a multiple of 8)
template <typename T>
__device__ __forceinline__ void sq_load8(const T* p, int k, int K, bool vec, float (&v)[8]) {
  if (vec && k + 8 <= K) {
    constexpr int W = int(sizeof(T)) / 2;  // 16-byte words of eight elements: 1 or 2
    uint4 w[W];
#pragma unroll
    for (int i = 0; i < W; i++) w[i] = __ldg(reinterpret_cast<const uint4*>(p + k) + i);
    T t[8];
    memcpy(t, w, sizeof(t));
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = sq_to_float(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = k + i < K ? sq_to_float(p[k + i]) : 0.f;
  }
}

// the quantized values of row r at k .. k + 7
template <typename T, bool GATE>
__device__ __forceinline__ void sq_values(const SqArgs& a, long long r, int k, float (&v)[8]) {
  sq_load8(static_cast<const T*>(a.x) + r * a.ldx, k, a.K, a.vec_x != 0, v);
  if constexpr (GATE) {
    float g[8];
    sq_load8(static_cast<const T*>(a.gate) + r * a.ldg, k, a.K, a.vec_g != 0, g);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __fmul_rn(v[i], __fdiv_rn(g[i], __fadd_rn(1.f, expf(-g[i]))));
  }
}

__device__ __forceinline__ void sq_store8(int8_t* p, int k, int K, const float (&v)[8], float s) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; i++)
    w[i >> 2] |= (uint32_t(__float2int_rn(__fmul_rn(v[i], s))) & 0xFFu) << (8 * (i & 3));
  if (k + 8 <= K) {
    *reinterpret_cast<uint2*>(p + k) = make_uint2(w[0], w[1]);
  } else {
    for (int i = 0; k + i < K; i++) p[k + i] = int8_t(w[i >> 2] >> (8 * (i & 3)));
  }
}

// One block per row; x is read twice (the second time from the caches).
template <typename T, bool GATE>
__global__ void __launch_bounds__(256) k_scaled_quantize(const SqArgs a) {
  __shared__ uint32_t most[8];
  for (int i = blockIdx.x; i < a.M; i += gridDim.x) {
    const int r = a.rows ? a.rows[i] : i;
    const bool in = r >= 0 && r < a.x_rows;
    uint32_t m = 0;  // |v| as bits: infinities and NaNs order above every finite value
    if (in) {
      for (int k = 8 * threadIdx.x; k < a.K; k += 8 * 256) {
        float v[8];
        sq_values<T, GATE>(a, r, k, v);
#pragma unroll
        for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; w++) m = max(m, most[w]);
    __syncthreads();
    const bool fine = m < 0x7F800000u, some = fine && m >= 0x0D800000u;  // finite; >= 2^-100
    const float gamma = __uint_as_float(m);
    const float s = some ? __fmul_rn(127.f, __frcp_rn(gamma)) : 0.f;
    for (int k = 8 * threadIdx.x; k < a.K; k += 8 * 256) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (some) sq_values<T, GATE>(a, r, k, v);
      sq_store8(a.q + i * a.ldq, k, a.K, v, s);
    }
    if (threadIdx.x == 0) {
      const bool bad = r >= a.x_rows;
      if (bad) atomicOr(&g_bq_device_error, kErrScaledIndex);
      a.scale[i] = !fine || bad ? __uint_as_float(0x7FC00000u) : some ? __fdiv_rn(gamma, 127.f) : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

struct SgArgs {
  const int8_t* w;
  const float* w_scale;
  const float* bias;    // or null
  const int8_t* q;
  const float* scale;
  const int* offsets;   // or null: one group of M rows
  void* y;
  long long ldw, expert_stride, ldq, ldy;
  int M, N, K, E, y_type;
};

__device__ __forceinline__ void sg_store(const SgArgs& a, long long at, float v) {
  if (a.y_type == BQ_TYPE_F32) static_cast<float*>(a.y)[at] = v;
  else if (a.y_type == BQ_TYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(a.y)[at] = __float2half_rn(v);
}

// 64 rows x 64 channels a block, K in pieces of 64 bytes through shared memory, four by four
// outputs a thread with 4-byte dot products. Block y is the y-th 64-row tile, counted group by group.
__global__ void __launch_bounds__(256) k_scaled_gemm(const SgArgs a) {
  __shared__ int As[16][65], Bs[16][65];
  int e = 0, m0 = blockIdx.y * 64, hi = a.M;
  if (a.offsets) {
    bool ok = a.offsets[0] >= 0 && a.offsets[a.E] <= a.M;
    int tile = blockIdx.y;
    bool found = false;
    for (int i = 0; i < a.E; i++) {
      const int lo = a.offsets[i], up = a.offsets[i + 1];
      if (up < lo) ok = false;
      const int n = (up - lo + 63) / 64;
      if (!found) {
        if (tile < n) { e = i; m0 = lo + 64 * tile; hi = up; found = true; }
        else tile -= n;
      }
    }
    if (!ok) {
      if (threadIdx.x == 0) atomicOr(&g_bq_device_error, kErrScaledIndex);
      return;
    }
    if (!found) return;
  }
  const int n0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int8_t* w = a.w + e * a.expert_stride;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 64) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int row = i >> 4, c = i & 15, k = k0 + 4 * c;
      uint32_t va = 0, vb = 0;
      for (int b = 0; b < 4 && k + b < a.K; b++) {
        if (m0 + row < hi) va |= uint32_t(uint8_t(a.q[(long long)(m0 + row) * a.ldq + k + b])) << (8 * b);
        if (n0 + row < a.N) vb |= uint32_t(uint8_t(w[(long long)(n0 + row) * a.ldw + k + b])) << (8 * b);
      }
      As[c][row] = int(va);
      Bs[c][row] = int(vb);
    }
    __syncthreads();
#pragma unroll 4
    for (int c = 0; c < 16; c++)
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = __dp4a(As[c][ty + 16 * i], Bs[c][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; i++)
    for (int j = 0; j < 4; j++) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < hi && n < a.N) {
        const long long wn = (long long)e * a.N + n;
        const float s = __fmul_rn(a.scale[m], a.w_scale[wn]);
        const float v = float(acc[i][j]);
        sg_store(a, m * a.ldy + n, a.bias ? __fmaf_rn(v, s, a.bias[wn]) : __fmul_rn(v, s));
      }
    }
}

}  // namespace bqi
