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

// ---- root-mean-square norm (kda_rmsnorm.hip) ----
struct RmsParams {
  const void* x;           // backward: the sum that was normed
  const void* res;         // forward: residual; backward: gradient of residual_out
  const void* dy;
  void* out;               // y or dx
  void* res_out;
  float* scales;           // 8-bit outputs
  int32_t group;           // elements of a scale (128 or D); 0: the output has x's type
  int dtype;
  const float* weight;
  float eps;
  float* rstd;
  float* dw;
  float* partial;          // workspace: [parts][D] sums of dy s r
  int64_t M;
  int32_t D;
};
size_t rmsnorm_parts(int64_t M, int64_t D);
hipError_t launch_rmsnorm_fwd(const RmsParams& p, hipStream_t stream);
hipError_t launch_rmsnorm_bwd(const RmsParams& p, hipStream_t stream);

// ---- short causal convolution (kda_conv.hip) ----
struct ConvParams {
  const void* x;
  const void* dy;
  void* out;               // y or dx
  int dtype, W, silu;
  const float* weight;
  const float* bias;
  const void* init;        // initial states; step: the states
  int init_dtype;
  void* fin;               // final states; step: the states
  int fin_dtype;
  const void* dfin;
  int dfin_dtype;
  void* dinit;
  int dinit_dtype;
  float* dw;
  float* db;
  float* partial;          // workspace: [parts][W + 1][D], NULL where no sum is wanted
  const int64_t* cu;
  int32_t nseq, T, tokens, D;
  const int32_t* in_slots;
  const int32_t* out_slots;
  int32_t n_slots;
};
bool conv_fits(int64_t tokens, int64_t D);   // within what a launch can hold
size_t conv_workspace(int64_t tokens, int64_t D, int64_t W);
hipError_t launch_conv_fwd(const ConvParams& p, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvParams& p, hipStream_t stream);
hipError_t launch_conv_step(const ConvParams& p, hipStream_t stream);

// ---- selective state space scan (kda_ssm.hip) ----
constexpr int SSM_BLOCK = 64;   // tokens between two saved states (carry)
struct SsmParams {
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* skip;
  const void* z;
  const float* dt_bias;
  int dtype, softplus;
  void* y;                 // forward
  const void* init;
  int init_dtype;
  void* fin;
  int fin_dtype;
  float* carry;            // written forward, read backward
  const void* dy;          // backward
  const void* dfin;
  int dfin_dtype;
  void* dx;
  void* ddt;
  float* dA;
  void* dB;
  void* dC;
  float* dskip;
  void* dz;
  float* dbias;
  void* dinit;
  int dinit_dtype;
  const int64_t* cu;
  int32_t nseq, T, tokens, D, E, G;
  const int32_t* in_slots;
  const int32_t* out_slots;
  int32_t n_slots;
};
// How a call is cut up, and its workspace
struct SsmWs {
  int32_t tiles, per_group;   // workgroups across the channels, and across a group's
  int32_t len, chunks;        // tokens of a chunk
  int32_t most;               // chunks that a call of at most as many tokens can have
  float* maps;                // [chunks - 1][D][E]
  float* sums;                // [chunks - 1][D] sum of s
  int32_t* resets;            // [chunks - 1] whether a sequence begins in the chunk
  float* stage;               // forward: [chunks - 1][D][E] initial states that final_state overwrites, or NULL
  float* table;               // [G][tokens][2][EP] B and C in fp32
  float* dA;                  // backward: [chunks][D][E]
  float* dvec;                // [chunks][2][D] of d_skip and d_dt_bias
  float* bc;                  // [tiles][tokens][2][E] of dB and dC
};
bool ssm_fits(int64_t tokens, int64_t D, int64_t E, int64_t G);
size_t ssm_workspace(int64_t tokens, int64_t D, int64_t E, int64_t G, bool backward);
hipError_t launch_ssm_fwd(const SsmParams& p, void* workspace, hipStream_t stream);
hipError_t launch_ssm_bwd(const SsmParams& p, void* workspace, hipStream_t stream);
hipError_t launch_ssm_step(const SsmParams& p, hipStream_t stream);

// ---- beam search (kda_beam.hip) ----
struct BeamParams {
  const void* logits;
  int dtype;
  const float* scores;
  const int32_t* finished;
  int32_t eos;
  int32_t* tokens;
  int32_t* parents;
  float* new_scores;
  int32_t N, W, V, k;
};
size_t beam_workspace(int64_t N, int64_t W, int64_t V, int64_t k);
hipError_t launch_beam_select(const BeamParams& p, void* workspace, hipStream_t stream);

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
hipError_t launch_cache_reorder(const CachePool& pool, const int32_t* slots, const int32_t* parents, int32_t* new_slots,
                                int64_t N, int W, hipStream_t stream);

}  // namespace kda
