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

// The dense product's forms (linear_forms.cuh), and the most rows of x for the first two.
enum { kLinearDirect = 0, kLinearStream = 1, kLinearPair = 2 };
constexpr int kLinearDirectRows = 32;
constexpr int kLinearStreamRows = 128;
constexpr int kLoraListInts = 260;

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
  // adapters
  const int32_t* lora_ids;       // [M]: each row's adapter, -1 none
  const __nv_bfloat16* lora_b;   // second factors [count, rows, rank]
  float* lora_s;                 // [parts, M, rank]: each row's sums of its adapter's first factor, scaled, to be added up
  int64_t lora_part;             // from one part to the next
  int32_t lora_parts;
  int32_t lora_count, lora_rank;
  int64_t lora_rows;
  // of each 256 rows: kLoraListInts words, the number of adapters and from the fourth on each, in the order of their first
  // rows
  const int32_t* lora_lists;
  const uint32_t* lora_errs;  // error bits of the sums' CTAs, which the pair form passes on
  int32_t lora_err_count;
  int32_t lora_own;           // direct form: each CTA makes the sums itself, of at most two units of 16 ranks
  const __nv_bfloat16* lora_a;  // first factors and scales, for those
  const float* lora_scale;
  int32_t lora_early;  // pair form: it may start before the sums are there
};
struct LinearMaps {
  CUtensorMap x, w;
  CUtensorMap b;  // with adapters: their second factors, boxes of 64 x as many rows as a load of w has
};
// Chooses p's form.  tail.M > 0: the last rows, taken out of p, are a second launch that runs beside p's.
void plan_linear(LinearParams& p, LinearParams& tail, int sms);
cudaError_t launch_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s);
// The same with adapters, after their first factors' sums.
struct LoraParams {
  const __nv_bfloat16 *x, *a;  // [M, K], row stride ldx; first factors [count, rank, K]
  const float* scale;          // [count] or null
  const int32_t* ids;          // [M]
  float* s;                    // [parts, M, rank]
  int64_t M, K, ldx;
  int32_t count, rank;
  int32_t* lists;              // as LinearParams'
  int32_t listed;              // whether lists are wanted
  int32_t precise;             // for FP32 results
  uint32_t* errs;              // [grid], error bits of each CTA: more than kLoraFewRows rows
  int64_t timeout_ns;
  int32_t test_stall;
  // plan_lora_sums' choice: shares of the K range, CTAs to a tile (many rows), CTAs in all, and the parts that a
  // sum is left in, M rows after one another
  int32_t split, tile_ctas, grid, parts;
};
struct LoraMaps {
  CUtensorMap x, a;  // [M, K], boxes of 128 rows; first factors, boxes of 16 rows: more than kLoraFewRows rows
};
constexpr int kLoraFewRows = 128;
void plan_lora_sums(LoraParams& p, int sms);
cudaError_t launch_lora_sums(const LoraMaps& maps, const LoraParams& p, cudaStream_t s);
cudaError_t launch_lora_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s);
cudaError_t launch_linear_repitch(const __nv_bfloat16* src, __nv_bfloat16* dst, int64_t rows, int64_t K, int64_t Kp,
                                  int64_t ld, int sms, cudaStream_t s);

// Products grouped by expert (kernels_grouped.cu)
struct GroupedParams {
  const int64_t* group_list;  // [E]
  void* out;                  // [M, N]
  uint32_t* hdr;              // error words
  int64_t M, N, ldo;
  int64_t timeout_ns;
  int32_t test_stall;  // as GateParams'
  int32_t E, group_list_type, KB;
  int32_t out_f32;
  int32_t vec_out;    // pairs of BF16 outputs start on 4-byte boundaries
  int32_t zero_rest;  // 1: rows of no group are written, as zeros
};
struct GroupedMaps {
  CUtensorMap w;     // [E, N, K], or [E, K, N]: boxes of 64 x 128, or two of 64 x 64
  CUtensorMap x[4];  // [M, K], boxes of 16, 32, 64 and 128 rows
};
cudaError_t launch_grouped(const GroupedMaps& maps, const GroupedParams& p, bool transposed, int sms, cudaStream_t s);

// Their weights' gradient: out[e] [A, B] = sum over the rows of expert e of a^T b
struct GroupedGradParams {
  const int64_t* group_list;
  int32_t* ends;  // [grouped_grad_ctas, E]
  uint32_t* hdr;
  int64_t M, A, B;
  int64_t timeout_ns;
  int32_t test_stall;
  int32_t E, group_list_type;
  int32_t out_f32, accumulate;
  // more than one: each expert's rows in so many shares, whose sums a second launch adds up into out
  int32_t shares;
  const float* parts;  // [shares, E, A, B]
  void* out;
};
struct GroupedGradMaps {
  CUtensorMap a, b;  // [M, A] and [M, B], boxes of 64 columns x 64 rows
  CUtensorMap out;   // [E, A, B], boxes of 128 bytes x 32 rows; parts as [shares E, A, B]
};
int grouped_grad_shares(int64_t M, int64_t A, int64_t B, int64_t E, int sms);
int grouped_grad_ctas(int64_t A, int64_t B, int64_t slices, int sms);
cudaError_t launch_grouped_grad(const GroupedGradMaps& maps, const GroupedGradParams& p, int sms, cudaStream_t s);

}  // namespace gmmfr
