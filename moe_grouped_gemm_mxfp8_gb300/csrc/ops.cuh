// Parameters and launchers of the router, the few-token MoE layer and the dense product.
#pragma once
#include <cudaTypedefs.h>

#include "common.cuh"

namespace gmmfr {

// defined in api.cu
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // null when the driver has none
int sm_count();

constexpr int kMaxTopk = 32;
constexpr int kMaxGroups = 64;
constexpr int kLayerMaxTokens = 64;
// The router's cluster form up to here, one wave of its largest clusters (1024 tokens of 2048, 256 experts: 18.7 us,
// the pair form 32; 1440 tokens: 34.9 and 32)
constexpr int kGateClusterTokens = 1024;

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
  float* logits;                // [T, E] or null
  void* ids;                    // [T, topk] int32 or int64
  float* weights;               // [T, topk]
  int64_t T, H, ldx;
  int32_t ids_i64;
  GateRule rule;
  uint32_t* hdr;       // error words (pair form)
  int64_t timeout_ns;
  int32_t test_stall;  // testing aid (pair form): 1: the accumulators' barriers wait for an arrival that never comes
  // plan_gate's choice
  int32_t pair, bn, KB, n_stages, grid;
};
struct GateMaps {
  CUtensorMap x, w;
};
bool plan_gate(GateParams& p, int sms);  // whether the pair form is taken (it needs the maps)
cudaError_t launch_gate(const GateMaps& maps, const GateParams& p, cudaStream_t s);

// Grouped FFN weights in MXFP8 tiles (kernels_layer.cu)
struct FfnPrepMxParams {
  const uint8_t *w13, *s13, *w2, *s2;
  uint8_t* prepared;
  int64_t H, I;
  int32_t E, NT1, KB1, NT2, KB2;
};
cudaError_t launch_ffn_prep_mx(const FfnPrepMxParams& p, cudaStream_t s);

constexpr int kLayerMaxCtas = 160;  // the workspace has slots for so many
struct LayerParams {
  GateParams gate;  // its ids are int32; ids and weights may lie in the workspace, logits is null
  const __nv_bfloat16* residual;
  __nv_bfloat16* out;
  const uint8_t *prepared, *prepared2;  // routed experts: gate/up tiles, down tiles
  const uint8_t *shared, *shared2;      // the shared expert's
  uint32_t* hdr;                        // error words
  uint8_t *ximg, *swimg, *swimg_s;      // B operand images: tokens, SwiGLU values (routed, shared)
  float *slots_up, *slots_down;         // pieces of cut tiles: [CTA][2][T][128] each
  // counters, zeroed by the front kernel
  uint32_t *counters, *up_done, *up_cnt, *down_cnt;
  uint32_t* nan_rows;  // [T], among the counters: 1 where a token's SwiGLU values have a NaN
  int64_t ld_residual, ld_out, timeout_ns;
  int32_t test_stall;  // as GateParams'
  int32_t n_counters, npad;
  int32_t NT1, KB1, NT2, KB2;  // tiles of a routed expert
  int32_t NT1s, KB2s;          // of the shared expert (0 without one)
  int32_t mx;
};
cudaError_t launch_layer(const LayerParams& p, int sms, cudaStream_t s);
int64_t layer_image_bytes(bool mx, int64_t npad);

// The dense product's forms (kernels_linear.cu), and the most rows of x for the first two.
enum { kLinearDirect = 0, kLinearStream = 1, kLinearPair = 2 };
constexpr int kLinearDirectRows = 32;
constexpr int kLinearStreamRows = 128;

struct LinearParams {
  const __nv_bfloat16 *x, *w, *bias, *residual;  // x and w at 16-byte row pitches; nothing is read past K
  void* out;
  uint32_t* hdr;  // error words
  int64_t M, N, K, ldx, ldw, ldr, ldo;
  int64_t timeout_ns;
  int32_t test_stall;  // as GateParams' (stream and pair form)
  int32_t act, out_f32;
  int32_t vec_out;  // rows of out and residual on 16-byte boundaries
  // plan_linear's choice
  int32_t form;              // kLinearDirect, ...
  int32_t bn;                // N of the products: rows of x (stream), columns of a tile before gating (pair)
  int32_t KB, tiles_m, tiles_n, n_stages, kps, split, group_m, grid;
  int32_t beside;             // 1: started while the launch before it runs, which it has to outlast
  int32_t slot_base, slots;   // its error words, and how many the call has
};
struct LinearMaps {
  CUtensorMap x, w;
};
// Chooses p's form.  tail.M > 0: the last rows, taken out of p, are a second launch that runs beside p's.
void plan_linear(LinearParams& p, LinearParams& tail, int sms);
cudaError_t launch_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s);
cudaError_t launch_linear_repitch(const __nv_bfloat16* src, __nv_bfloat16* dst, int64_t rows, int64_t K, int64_t Kp,
                                  int64_t ld, int sms, cudaStream_t s);

}  // namespace gmmfr
