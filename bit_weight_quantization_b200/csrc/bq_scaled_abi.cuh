// C ABI of the scaled int8 layers: host-side validation and kernel launches.
#pragma once

#include "bq_abi.cuh"
#include "bq_scaled.cuh"

namespace bqi {

constexpr int kSgMaxM = 0x7FFFFFFF - (1 << 16);  // tile ends stay inside int32

inline int type_bytes(int t) { return t == BQ_TYPE_F32 ? 4 : 2; }
inline bool type_ok(int t) { return t == BQ_TYPE_F32 || t == BQ_TYPE_BF16 || t == BQ_TYPE_F16; }

inline bq_status check_codes(const void* p, int64_t ld, int K) {
  if (!p || !aligned(p, 16) || ld % 16 != 0) return BQ_ERR_INVALID_ARG;
  if (ld < K || ld >= (int64_t(1) << 36)) return BQ_ERR_SIZE;
  return BQ_OK;
}

inline bq_status check_values(const void* p, int type, int64_t ld, int width) {
  if (!type_ok(type) || !p || !aligned(p, type_bytes(type))) return BQ_ERR_INVALID_ARG;
  if (ld < width || ld >= (int64_t(1) << 36)) return BQ_ERR_SIZE;
  return BQ_OK;
}

inline bq_status check_scaled_weights(const bq_scaled_weights* w) {
  if (!w) return BQ_ERR_INVALID_ARG;
  if (w->N < 1 || w->N > BQ_MAX_N || w->K < 1 || w->K > BQ_MAX_K || w->experts < 1 || w->experts > BQ_MAX_EXPERTS)
    return BQ_ERR_SIZE;
  if (!w->scale || !aligned(w->scale, 4) || !aligned(w->bias, 4)) return BQ_ERR_INVALID_ARG;
  if (w->experts > 1) {
    if (w->expert_stride % 16 != 0) return BQ_ERR_INVALID_ARG;
    if (w->expert_stride < 0 || w->expert_stride >= (int64_t(1) << 39)) return BQ_ERR_SIZE;
  }
  return check_codes(w->codes, w->ld, w->K);
}

// rows of codes in a workspace of bq_scaled_linear
inline int64_t scaled_ld(int K) { return (int64_t(K) + 15) / 16 * 16; }

inline bool rows_aligned(const void* p, int type, int64_t ld) {
  return aligned(p, 16) && ld * type_bytes(type) % 16 == 0;
}

template <typename T>
inline cudaError_t launch_scaled_quantize(const SqArgs& a, cudaStream_t s) {
  const dim3 grid(unsigned(std::min(a.M, 148 * 8)));
  if (a.gate) k_scaled_quantize<T, true><<<grid, 256, 0, s>>>(a);
  else k_scaled_quantize<T, false><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

inline bq_status launch_scaled_gemm(const SgArgs& a, cudaStream_t s) {
  const long long tiles = (long long)(a.M + 63) / 64 + (a.offsets ? a.E : 0);
  const dim3 grid(unsigned((a.N + 63) / 64), unsigned(std::min(tiles, 65535ll)));
  if (tiles > 65535) return BQ_ERR_UNSUPPORTED;
  k_scaled_gemm<<<grid, 256, 0, s>>>(a);
  return launch_status();
}

inline bq_status scaled_gemm(const bq_scaled_weights* w, const int8_t* q, int64_t ldq, const float* scale, int32_t M,
                             const int32_t* offsets, bool grouped, void* y, int32_t y_type, int64_t ldy,
                             void* stream) {
  bq_status st = check_scaled_weights(w);
  if (st != BQ_OK) return st;
  if (!grouped && w->experts != 1) return BQ_ERR_INVALID_ARG;
  if (M < 0 || M > kSgMaxM) return BQ_ERR_SIZE;
  if (!type_ok(y_type)) return BQ_ERR_INVALID_ARG;
  if (M == 0) return BQ_OK;
  if ((st = check_codes(q, ldq, w->K)) != BQ_OK) return st;
  if ((st = check_values(y, y_type, ldy, w->N)) != BQ_OK) return st;
  if (!scale || !aligned(scale, 4) || (grouped && (!offsets || !aligned(offsets, 4)))) return BQ_ERR_INVALID_ARG;
  SgArgs a{};
  a.w = w->codes; a.w_scale = w->scale; a.bias = w->bias; a.q = q; a.scale = scale; a.offsets = offsets; a.y = y;
  a.ldw = w->ld; a.expert_stride = w->experts > 1 ? w->expert_stride : 0; a.ldq = ldq; a.ldy = ldy;
  a.M = M; a.N = w->N; a.K = w->K; a.E = w->experts; a.y_type = y_type;
  return launch_scaled_gemm(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace bqi

extern "C" {

bq_status bq_scaled_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t x_rows, const void* gate,
                             int64_t ldg, const int32_t* rows, int32_t M, int32_t K, int8_t* q, int64_t ldq,
                             float* scale, void* stream) {
  if (K < 1 || K > BQ_MAX_K || M < 0 || M > kSgMaxM || x_rows < 0) return BQ_ERR_SIZE;
  if (!type_ok(x_type)) return BQ_ERR_INVALID_ARG;
  if (M == 0) return BQ_OK;
  if (!rows && x_rows < M) return BQ_ERR_SIZE;
  bq_status st = BQ_OK;
  if (x_rows > 0 || x) {  // with `rows` an empty x may be null: every slot must then be empty
    if ((st = check_values(x, x_type, ldx, K)) != BQ_OK) return st;
  }
  if (gate && (st = check_values(gate, x_type, ldg, K)) != BQ_OK) return st;
  if ((st = check_codes(q, ldq, K)) != BQ_OK) return st;
  if (!scale || !aligned(scale, 4) || !aligned(rows, 4)) return BQ_ERR_INVALID_ARG;
  SqArgs a{};
  a.x = x; a.gate = gate; a.rows = rows; a.q = q; a.scale = scale;
  a.ldx = ldx; a.ldg = ldg; a.ldq = ldq; a.x_rows = x_rows; a.M = M; a.K = K;
  a.vec_x = rows_aligned(x, x_type, ldx);
  a.vec_g = gate && rows_aligned(gate, x_type, ldg);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = x_type == BQ_TYPE_F32 ? launch_scaled_quantize<float>(a, s)
                        : x_type == BQ_TYPE_BF16  ? launch_scaled_quantize<__nv_bfloat16>(a, s)
                                                : launch_scaled_quantize<__half>(a, s);
  return e == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
}

bq_status bq_scaled_gemm(const bq_scaled_weights* w, const int8_t* q, int64_t ldq, const float* scale, int32_t M,
                         void* y, int32_t y_type, int64_t ldy, void* stream) {
  return scaled_gemm(w, q, ldq, scale, M, nullptr, false, y, y_type, ldy, stream);
}

bq_status bq_scaled_gemm_grouped(const bq_scaled_weights* w, const int8_t* q, int64_t ldq, const float* scale,
                                 int32_t M, const int32_t* offsets, void* y, int32_t y_type, int64_t ldy,
                                 void* stream) {
  return scaled_gemm(w, q, ldq, scale, M, offsets, true, y, y_type, ldy, stream);
}

bq_status bq_scaled_workspace_bytes(const bq_scaled_weights* w, int32_t M, size_t* bytes) {
  const bq_status st = check_scaled_weights(w);
  if (st != BQ_OK) return st;
  if (!bytes) return BQ_ERR_INVALID_ARG;
  if (M < 0 || M > kSgMaxM) return BQ_ERR_SIZE;
  *bytes = size_t(align256(uint64_t(M) * scaled_ld(w->K)) + align256(4ull * M));
  return BQ_OK;
}

bq_status bq_scaled_linear(const bq_scaled_weights* w, const void* x, int32_t x_type, int64_t ldx, int32_t M,
                           void* y, int32_t y_type, int64_t ldy, void* workspace, size_t workspace_bytes,
                           void* stream) {
  size_t need = 0;
  bq_status st = bq_scaled_workspace_bytes(w, M, &need);
  if (st != BQ_OK) return st;
  if (w->experts != 1 || !type_ok(x_type) || !type_ok(y_type)) return BQ_ERR_INVALID_ARG;
  if (M == 0) return BQ_OK;
  if ((st = check_values(x, x_type, ldx, w->K)) != BQ_OK) return st;
  if ((st = check_values(y, y_type, ldy, w->N)) != BQ_OK) return st;
  if (!workspace || !aligned(workspace, 256)) return BQ_ERR_INVALID_ARG;
  if (workspace_bytes < need) return BQ_ERR_SIZE;
  const int64_t ld = scaled_ld(w->K);
  int8_t* q = static_cast<int8_t*>(workspace);
  float* scale = reinterpret_cast<float*>(q + align256(uint64_t(M) * ld));
  st = bq_scaled_quantize(x, x_type, ldx, M, nullptr, 0, nullptr, M, w->K, q, ld, scale, stream);
  return st != BQ_OK ? st : bq_scaled_gemm(w, q, ld, scale, M, y, y_type, ldy, stream);
}

}  // extern "C"
