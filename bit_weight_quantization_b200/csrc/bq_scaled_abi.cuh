// C ABI of the scaled int8 layers: host-side validation and kernel launches.
#pragma once

#include "bq_abi.cuh"
#include "bq_scaled.cuh"

namespace bqi {

static_assert(kSgSmemMax == kTcSmemMax, "shared memory of a CTA");
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

template <typename T, bool GATE, int C, int MAXT, int MINB>
inline cudaError_t launch_scaled_rows(const SqArgs& a, cudaStream_t s) {
  const int runs = (a.K + 7) / 8, per_row = ((runs + C - 1) / C + 31) / 32 * 32, rows = std::max(1, 256 / per_row);
  return launch_pdl(k_scaled_quantize<T, GATE, C, MAXT, MINB>, dim3(unsigned((a.M + (long long)rows - 1) / rows)),
                    dim3(unsigned(per_row), unsigned(rows)), 0, s, a);
}

// Runs of 8 elements a thread. Few rows are spread over as many threads as they fill (64 rows of 11008
// bf16: 2.7 us with two runs a thread, 3.3 with eight). Many rows take four, or eight where a run is
// four registers (16384 rows of 4096 bf16, gathered: 64 / 41 / 33 us with one, two and eight).
template <typename T, bool GATE>
inline cudaError_t launch_scaled_quantize(const SqArgs& a, cudaStream_t s) {
  const int runs = (a.K + 7) / 8;
  if (runs > 4096) return launch_pdl(k_scaled_quantize_long<T, GATE>, dim3(unsigned(a.M)), dim3(1024), 0, s, a);
  if ((long long)a.M * runs <= sm_count() * 1024 || runs <= 64) {
    if (runs <= 1024) return launch_scaled_rows<T, GATE, 1, 1024, 1>(a, s);
    if (runs <= 2048) return launch_scaled_rows<T, GATE, 2, 1024, 1>(a, s);
    return launch_scaled_rows<T, GATE, 4, 1024, 1>(a, s);
  }
  if (runs <= 128) return launch_scaled_rows<T, GATE, 2, 256, 1>(a, s);
  if constexpr (!GATE && sizeof(T) == 2)
    return launch_scaled_rows<T, GATE, 8, 512, 2>(a, s);
  else if (runs > 2048)
    return launch_scaled_rows<T, GATE, 4, 1024, 1>(a, s);
  else
    return launch_scaled_rows<T, GATE, 4, 512, GATE ? 3 : 2>(a, s);
}

template <typename T>
inline cudaError_t launch_scaled_quantize(const SqArgs& a, cudaStream_t s) {
  return a.gate ? launch_scaled_quantize<T, true>(a, s) : launch_scaled_quantize<T, false>(a, s);
}

// Rows of int8 codes as a TMA map with 128-byte swizzle: [experts][rows][K], boxes of 128 bytes by
// box_rows. Rows and k past the matrix read as zero.
inline bool encode_codes_map(const int8_t* p, int64_t ld, int64_t rows, int K, int E, int64_t expert_stride,
                             int box_rows, TcTensorMap* out) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[3] = {cuuint64_t(K), cuuint64_t(rows), cuuint64_t(E)};
  const cuuint64_t strides[2] = {cuuint64_t(ld), cuuint64_t(E > 1 ? expert_stride : 16)};
  const cuuint32_t box[3] = {cuuint32_t(kSgChunk), cuuint32_t(box_rows), 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  CUtensorMap m;
  if (encode(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, E > 0 ? 3 : 2, const_cast<int8_t*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  std::memcpy(out, &m, sizeof(m));
  return true;
}

// 16-bit y [M][N] as a TMA map for stores of 32 x 32 blocks (64-byte rows, 64-byte swizzle)
inline bool encode_output_map(void* y, int64_t ldy, int M, int N, TcTensorMap* out) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[2] = {cuuint64_t(N), cuuint64_t(M)};
  const cuuint64_t strides[1] = {cuuint64_t(ldy) * 2};
  const cuuint32_t box[2] = {32u, 32u};
  const cuuint32_t estr[2] = {1u, 1u};
  CUtensorMap m;
  if (encode(&m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  std::memcpy(out, &m, sizeof(m));
  return true;
}

template <int CG>
inline bq_status launch_scaled_tc(const SgArgs& a, const SgPlan& p, long long tiles, cudaStream_t s) {
  auto k = k_scaled_tc<CG>;
  static std::mutex mu;
  static unsigned long long set_ctx = 0;
  {
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (ctx == 0 || ctx != set_ctx) {
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTcSmemMax)) != cudaSuccess) {
        (void)cudaGetLastError();
        return BQ_ERR_CUDA;
      }
      set_ctx = ctx;
    }
  }
  cudaLaunchConfig_t cfg = {};
  // one CTA pair per two SMs, or two single CTAs an SM (64 rows of 64 experts, 2048 x 2048: 39.5 us with one,
  // 37.4 with two; 2000 rows: 55.3 and 47.1)
  const int ctas = CG == 2 ? sm_count() / 2 * 2 : 2 * sm_count();
  cfg.gridDim = dim3(unsigned(std::min<long long>(CG * tiles, ctas)));
  cfg.blockDim = dim3(kSgThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (CG > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = unsigned(CG);
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[n++].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, k, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return BQ_ERR_CUDA;
  }
  return BQ_OK;
}

template <typename T, int TOK>
inline bq_status launch_scaled_split(SsArgs a, cudaStream_t s) {
  constexpr bool FUSED = !std::is_same<T, int8_t>::value;
  auto k = k_scaled_split<T, TOK>;
  static std::mutex mu;
  static unsigned long long set_ctx = 0;
  static int max_clusters[kSsMaxSplit + 1];  // of one CTA an SM: the query allows a kernel with tensor memory no second
  int clusters[kSsMaxSplit + 1];
  {
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (ctx == 0 || ctx != set_ctx) {
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kTcSmemMax)) != cudaSuccess) {
        (void)cudaGetLastError();
        return BQ_ERR_CUDA;
      }
      for (int c = 1; c <= kSsMaxSplit; c++) {
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(unsigned(c));
        q.blockDim = dim3(kSgThreads);
        q.dynamicSmemBytes = kTcSmemMax;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = unsigned(c);
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        q.attrs = at;
        q.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&max_clusters[c], k, &q) != cudaSuccess) {
          (void)cudaGetLastError();
          max_clusters[c] = c == 1 ? sm_count() : 0;  // without the query: no clusters
        }
      }
      set_ctx = ctx;
    }
    std::memcpy(clusters, max_clusters, sizeof(clusters));
  }
  const SsPlan p = plan_scaled_split(a.M, a.N, a.K, FUSED, clusters, sm_count());
  a.nn = p.nn; a.cols = p.cols; a.splits = p.splits; a.slice = p.slice; a.stages = p.stages; a.stage_bytes = p.stage_bytes;
  if (p.splits == 0) return BQ_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.N + kSgRows - 1) / kSgRows * p.splits));
  cfg.blockDim = dim3(kSgThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = unsigned(p.splits);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, k, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return BQ_ERR_CUDA;
  }
  return BQ_OK;
}

template <typename T>
inline bq_status launch_scaled_fused(const SsArgs& a, cudaStream_t s) {
  static_assert(kSsFusedTokens == 2, "instantiations");
  return a.M == 1 ? launch_scaled_split<T, 1>(a, s) : launch_scaled_split<T, 2>(a, s);
}

// Whether bq_scaled_linear quantizes inside the product: up to kSsFusedTokens tokens, as every CTA reads them
// all (4096 x 4096: one token 6.6 us, two 7.5, four 8.8, in two launches 7.6; 13824 x 5120: one token 14.6, two
// 16.0, four 23.2, in two launches 15.6; at 4096 x 11008 the rule loses: 12.5 and 14.5, four in two launches
// 12.1), and K <= 16384 so that the operand of any split leaves room for stages.
inline bool scaled_fused(int M, int K) { return M <= kSsFusedTokens && K <= 16384; }

inline bool split_args(const bq_scaled_weights* w, int M, void* y, int y_type, int64_t ldy, SsArgs* a) {
  a->w_scale = w->scale; a->bias = w->bias; a->y = y; a->ldy = ldy;
  a->M = M; a->N = w->N; a->K = w->K; a->y_type = y_type;
  return encode_codes_map(w->codes, w->ld, w->N, w->K, 1, 0, kSgRows, &a->wmap);
}

inline bq_status scaled_gemm(const bq_scaled_weights* w, const int8_t* q, int64_t ldq, const float* scale, int32_t M,
                             const int32_t* offsets, bool grouped, bool after_quantize, void* y, int32_t y_type,
                             int64_t ldy, void* stream) {
  bq_status st = check_scaled_weights(w);
  if (st != BQ_OK) return st;
  if (!grouped && w->experts != 1) return BQ_ERR_INVALID_ARG;
  if (M < 0 || M > kSgMaxM) return BQ_ERR_SIZE;
  if (!type_ok(y_type)) return BQ_ERR_INVALID_ARG;
  if (M == 0) return BQ_OK;
  if ((st = check_codes(q, ldq, w->K)) != BQ_OK) return st;
  if ((st = check_values(y, y_type, ldy, w->N)) != BQ_OK) return st;
  if (!scale || !aligned(scale, 4) || (grouped && (!offsets || !aligned(offsets, 4)))) return BQ_ERR_INVALID_ARG;
  if (!grouped && M <= kSsMaxTokens) {
    SsArgs a{};
    if (!split_args(w, M, y, y_type, ldy, &a) || !encode_codes_map(q, ldq, M, w->K, 0, 0, (M + 15) / 16 * 16, &a.qmap))
      return BQ_ERR_CUDA;
    a.scale = scale;
    a.ahead = after_quantize;
    return launch_scaled_split<int8_t, 1>(a, reinterpret_cast<cudaStream_t>(stream));
  }
  // 16-bit outputs leave by TMA where their rows start on 16-byte boundaries
  const bool y_tma = y_type != BQ_TYPE_F32 && rows_aligned(y, y_type, ldy);
  const SgPlan p = plan_scaled_gemm(M, w->N, w->K, w->experts, grouped, y_tma, sm_count());
  const int channels = kSgRows * p.cg;
  const long long tiles = ((long long)(M + p.bn - 1) / p.bn + (grouped ? w->experts : 0)) * ((w->N + channels - 1) / channels);
  if (tiles > (1 << 30)) return BQ_ERR_SIZE;
  SgArgs a{};
  a.w_experts = w->experts > 1 && w->expert_stride > 0 ? w->experts : 1;
  if (!encode_codes_map(w->codes, w->ld, w->N, w->K, a.w_experts, w->expert_stride, kSgRows, &a.wmap) ||
      !encode_codes_map(q, ldq, M, w->K, 0, 0, p.bn / p.cg, &a.qmap) ||
      !encode_codes_map(q, ldq, M, w->K, 0, 0, 16, &a.qmap16) || (y_tma && !encode_output_map(y, ldy, M, w->N, &a.ymap)))
    return BQ_ERR_CUDA;
  a.w_scale = w->scale; a.bias = w->bias; a.scale = scale; a.offsets = offsets; a.y = y; a.ldy = ldy;
  a.M = M; a.N = w->N; a.K = w->K; a.E = w->experts; a.y_type = y_type; a.y_tma = y_tma; a.ahead = after_quantize;
  a.bn = p.bn; a.stages = p.stages; a.stage_bytes = p.stage_bytes; a.cols = p.cols; a.acc_stride = p.acc_stride;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return p.cg == 2 ? launch_scaled_tc<2>(a, p, tiles, s) : launch_scaled_tc<1>(a, p, tiles, s);
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
  return scaled_gemm(w, q, ldq, scale, M, nullptr, false, false, y, y_type, ldy, stream);
}

bq_status bq_scaled_gemm_grouped(const bq_scaled_weights* w, const int8_t* q, int64_t ldq, const float* scale,
                                 int32_t M, const int32_t* offsets, void* y, int32_t y_type, int64_t ldy,
                                 void* stream) {
  return scaled_gemm(w, q, ldq, scale, M, offsets, true, false, y, y_type, ldy, stream);
}

bq_status bq_scaled_workspace_bytes(const bq_scaled_weights* w, int32_t M, size_t* bytes) {
  const bq_status st = check_scaled_weights(w);
  if (st != BQ_OK) return st;
  if (!bytes) return BQ_ERR_INVALID_ARG;
  if (M < 0 || M > kSgMaxM) return BQ_ERR_SIZE;
  *bytes = scaled_fused(M, w->K) ? 0 : size_t(align256(uint64_t(M) * scaled_ld(w->K)) + align256(4ull * M));
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
  if (need > 0 && (!workspace || !aligned(workspace, 256))) return BQ_ERR_INVALID_ARG;
  if (workspace_bytes < need) return BQ_ERR_SIZE;
  if (scaled_fused(M, w->K)) {
    SsArgs a{};
    if (!split_args(w, M, y, y_type, ldy, &a)) return BQ_ERR_CUDA;
    a.x.x = x;
    a.x.ldx = ldx;
    a.x.vec_x = rows_aligned(x, x_type, ldx);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return x_type == BQ_TYPE_F32    ? launch_scaled_fused<float>(a, s)
           : x_type == BQ_TYPE_BF16 ? launch_scaled_fused<__nv_bfloat16>(a, s)
                                    : launch_scaled_fused<__half>(a, s);
  }
  const int64_t ld = scaled_ld(w->K);
  int8_t* q = static_cast<int8_t*>(workspace);
  float* scale = reinterpret_cast<float*>(q + align256(uint64_t(M) * ld));
  st = bq_scaled_quantize(x, x_type, ldx, M, nullptr, 0, nullptr, M, w->K, q, ld, scale, stream);
  return st != BQ_OK ? st : scaled_gemm(w, q, ld, scale, M, nullptr, false, true, y, y_type, ldy, stream);
}

}  // extern "C"
