// kda_ops.h -- host-side launch interface between the C ABI of the operators beside
// kda_fwd (kda_ops_api.cpp) and their kernels. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// ---- gated linear recurrence (kda_glr.hip) ----
constexpr int GLR_TILE = 128;   // tokens between two saved states (carry), of the B * T packed tokens

struct GlrParams {
  const void* x;
  const void* g;
  const void* dy;          // backward
  void* y;                 // forward
  void* dx;                // backward
  void* dg;
  int dtype;               // 1 bf16, 2 fp32, 3 fp16
  const void* init;        // initial state
  int init_dtype;          // 0 none, 1 bf16, 2 fp32
  void* fin;               // forward: final state; backward: gradient of the initial state
  int fin_dtype;
  const void* dfin;        // backward: gradient of the final state
  int dfin_dtype;
  float* carry;            // states entering every GLR_TILE tokens (written forward, read backward)
  const int64_t* cu;       // packed boundaries, or NULL: rows of T tokens
  int32_t nseq;
  int32_t T;               // tokens of a row; packed total with cu
  int32_t tokens;          // all tokens
  int32_t D;
  const int32_t* in_slots;   // step: slots of the states, or NULL: state n is row n
  const int32_t* out_slots;
  int32_t n_slots;
};

size_t glr_workspace(int64_t tokens, int64_t D, int64_t nseq);
bool glr_fits(int64_t tokens, int64_t D, int64_t nseq);   // within what a launch can hold
hipError_t launch_glr_fwd(const GlrParams& p, void* workspace, hipStream_t stream);
hipError_t launch_glr_bwd(const GlrParams& p, void* workspace, hipStream_t stream);

// ---- layer norm (kda_layernorm.hip) ----
struct NormParams {
  const void* x;
  const void* dy;
  void* out;               // y or dx
  int dtype;
  const float* weight;
  const float* bias;
  float eps;
  float* mean;
  float* rstd;
  float* dw;
  float* db;
  float* partial;          // workspace: [2][parts][D] sums of dy xhat and dy
  int64_t M;
  int32_t D;
};
size_t layernorm_parts(int64_t M, int64_t D);
hipError_t launch_layernorm_fwd(const NormParams& p, hipStream_t stream);
hipError_t launch_layernorm_bwd(const NormParams& p, hipStream_t stream);

// ---- cache slots (kda_cache.hip) ----
struct CachePool {
  void* base;
  int64_t layers, slots;
  size_t slot_bytes;
};
hipError_t launch_cache_copy(const CachePool& pool, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream);
hipError_t launch_cache_fork(const CachePool& pool, int32_t* used, const int32_t* src, int32_t* dst, int64_t n,
                             hipStream_t stream);
hipError_t launch_cache_free(int32_t* used, int64_t S, const int32_t* slots, int64_t n, hipStream_t stream);
hipError_t launch_cache_compact(const CachePool& pool, int32_t* used, int32_t* remap, int32_t* table, int64_t n,
                                int32_t* ws, hipStream_t stream);

}  // namespace kda
