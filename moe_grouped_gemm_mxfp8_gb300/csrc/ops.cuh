// Parameters and launchers of the router, the few-token MoE layer and the dense product.
#pragma once
#include "common.cuh"

namespace gmmfr {

constexpr int kMaxTopk = 32;
constexpr int kMaxGroups = 64;
constexpr int kLayerMaxTokens = 64;

// The router's rule (gmmfr_gate_problem).
struct GateRule {
  int32_t E, topk;
  int32_t sigmoid;
  int32_t n_group, topk_group, group_top;
  int32_t renormalise;
  float scale;
};

struct GateParams {
  const __nv_bfloat16* x;       // [T, H], row stride ldx
  const __nv_bfloat16* weight;  // [E, H]
  const float* select_bias;     // [E] or null
  float* logits;                // [T, E]: the caller's or the workspace's
  void* ids;                    // [T, topk] int32 or int64
  float* weights;               // [T, topk]
  int64_t T, H, ldx;
  int32_t ids_i64;
  GateRule rule;
};
cudaError_t launch_gate(const GateParams& p, cudaStream_t s);

// Grouped FFN weights in MXFP8 tiles (kernels_layer.cu)
struct FfnPrepMxParams {
  const uint8_t *w13, *s13, *w2, *s2;
  uint8_t* prepared;
  int64_t H, I;
  int32_t E, NT1, KB1, NT2, KB2;
};
cudaError_t launch_ffn_prep_mx(const FfnPrepMxParams& p, cudaStream_t s);

struct LayerParams {
  GateParams gate;  // its ids are int32; ids, weights and logits may lie in the workspace
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  const uint8_t* prepared;
  const uint8_t* shared;
  float* sw;  // workspace [T][topk][I], then [T][shared_I]
  int64_t I, shared_I, ld_residual, ld_out;
  int32_t mx;
};
cudaError_t launch_layer(const LayerParams& p, cudaStream_t s);

struct LinearParams {
  const __nv_bfloat16 *x, *w, *bias, *residual;
  void* out;
  int64_t M, N, K, ldx, ldw, ldr, ldo;
  int32_t act, out_f32;
};
cudaError_t launch_linear(const LinearParams& p, cudaStream_t s);

}  // namespace gmmfr
