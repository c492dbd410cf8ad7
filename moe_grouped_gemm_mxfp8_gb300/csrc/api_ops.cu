// C ABI of the router, the few-token MoE layer, the dense product and the grouped products (declared in include/gmmfr.h):
// argument checks, workspace layout, launches.
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "gmmfr.h"
#include "ops.cuh"

namespace {

gmmfr_status fail(gmmfr_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return gmmfr::record_error(st, buf);
}

gmmfr_status cuda_fail(cudaError_t e, const char* what) {
  return fail(GMMFR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int64_t kMaxSize = int64_t(1) << 31;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }
int64_t stride_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

// The limit of every wait in the kernels.  Testing aid: GMMFR_TEST_STALL_NS sets it, and makes a wait run out.  Read once:
// small calls notice each look at the environment.
struct Waits {
  int64_t limit_ns;
  int32_t stall;
};
const Waits& waits() {
  static const Waits w = [] {
    const char* t = std::getenv("GMMFR_TEST_STALL_NS");
    if (!t) return Waits{4000000000ll, 0};
    const long long ns = std::atoll(t);
    return Waits{ns > 0 ? ns : 1000000, 1};
  }();
  return w;
}

gmmfr_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!workspace) return fail(GMMFR_ERR_WORKSPACE, "workspace is NULL (needs %zu bytes)", need);
  if (bytes < need) return fail(GMMFR_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  if (!aligned(workspace, 256)) return fail(GMMFR_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return GMMFR_OK;
}

// [rows, K] BF16 with boxes of `box_rows` rows of 64 elements (128 bytes, 128-byte swizzle)
bool encode_rows(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const void* base, int64_t rows, int64_t K,
                 int64_t ld, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? ld : cdiv(K, 8) * 8) * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [depth, rows, cols], dense, in boxes of one slice
bool encode_slices(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const void* base, bool f32, int64_t depth, int64_t rows,
                   int64_t cols, int box_cols, int box_rows) {
  const int64_t size = f32 ? 4 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
  cuuint64_t strides[2] = {(cuuint64_t)(cols * size), (cuuint64_t)(rows * cols * size)};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- gate
gmmfr_status validate_gate(const gmmfr_gate_problem* p) {
  if (!p) return fail(GMMFR_ERR_INVALID_ARG, "problem is NULL");
  if (p->T < 0 || p->T >= kMaxSize) return fail(GMMFR_ERR_INVALID_ARG, "T=%lld out of range [0, 2^31)", (long long)p->T);
  if (p->H < 8 || p->H % 8 || p->H >= (int64_t(1) << 24))
    return fail(GMMFR_ERR_INVALID_ARG, "H=%lld is not a multiple of 8 in [8, 2^24)", (long long)p->H);
  if (p->E < 1 || p->E > gmmfr::kMaxExperts) return fail(GMMFR_ERR_INVALID_ARG, "E=%lld out of range [1, 1024]", (long long)p->E);
  if (p->ldx != 0 && (p->ldx < p->H || p->ldx % 8))
    return fail(GMMFR_ERR_INVALID_ARG, "ldx=%lld is not 0 or a multiple of 8 >= H", (long long)p->ldx);
  if (p->scoring != GMMFR_GATE_SOFTMAX && p->scoring != GMMFR_GATE_SIGMOID)
    return fail(GMMFR_ERR_INVALID_ARG, "scoring=%d is not 0 (softmax) or 1 (sigmoid)", p->scoring);
  if (p->n_group < 1 || p->n_group > gmmfr::kMaxGroups || p->E % p->n_group)
    return fail(GMMFR_ERR_INVALID_ARG, "n_group=%d is not in [1, 64] or does not divide E=%lld", p->n_group, (long long)p->E);
  int64_t eligible = p->E;
  if (p->n_group > 1) {
    if (p->topk_group < 1 || p->topk_group > p->n_group)
      return fail(GMMFR_ERR_INVALID_ARG, "topk_group=%d out of range [1, n_group=%d]", p->topk_group, p->n_group);
    if (p->group_top < 1 || p->group_top > 2 || p->group_top > p->E / p->n_group)
      return fail(GMMFR_ERR_INVALID_ARG, "group_top=%d is not 1 or 2, or exceeds the group size", p->group_top);
    eligible = p->topk_group * (p->E / p->n_group);
  }
  if (p->topk < 1 || p->topk > gmmfr::kMaxTopk || p->topk > eligible)
    return fail(GMMFR_ERR_INVALID_ARG, "topk=%lld out of range [1, 32], or more than the %lld eligible experts",
                (long long)p->topk, (long long)eligible);
  if (p->renormalise != 0 && p->renormalise != 1) return fail(GMMFR_ERR_INVALID_ARG, "renormalise must be 0 or 1");
  if (p->ids_type != GMMFR_INDEX_I64 && p->ids_type != GMMFR_INDEX_I32)
    return fail(GMMFR_ERR_INVALID_ARG, "ids_type=%d is not 0 (int64) or 1 (int32)", p->ids_type);
  return GMMFR_OK;
}

size_t gate_ws_bytes(const gmmfr_gate_problem*) { return gmmfr::kHdrBytes; }

gmmfr::GateParams gate_params(const gmmfr_gate_problem& p, const void* x, const void* weight, const float* select_bias) {
  gmmfr::GateParams g{};
  g.x = static_cast<const __nv_bfloat16*>(x);
  g.weight = static_cast<const __nv_bfloat16*>(weight);
  g.select_bias = select_bias;
  g.T = p.T;
  g.H = p.H;
  g.ldx = stride_or(p.ldx, p.H);
  g.rule = {(int32_t)p.E, (int32_t)p.topk, p.scoring == GMMFR_GATE_SIGMOID, p.n_group, p.topk_group, p.group_top,
            p.renormalise, p.scale};
  return g;
}

// ---------------------------------------------------------------- FFN weights in MXFP8
gmmfr_status validate_ffn_sizes(int64_t H, int64_t I, int64_t E) {
  if (H < 8 || I < 8 || H % 8 || I % 8 || H >= (int64_t(1) << 24) || I >= (int64_t(1) << 24) || E < 1 ||
      E > gmmfr::kMaxExperts)
    return fail(GMMFR_ERR_INVALID_ARG, "H=%lld I=%lld E=%lld out of range (H, I multiples of 8; 1 <= E <= 1024)",
                (long long)H, (long long)I, (long long)E);
  return GMMFR_OK;
}

size_t ffn_bytes(int64_t H, int64_t I, int64_t E, bool mx) {
  const int64_t kt = mx ? 128 : 64;
  return (size_t)E * (cdiv(I, 64) * cdiv(H, kt) + cdiv(H, 128) * cdiv(I, kt)) *
         (mx ? gmmfr::kPrepTileBytes : gmmfr::kWTileBytes);
}

// ---------------------------------------------------------------- layer
gmmfr_status validate_layer(const gmmfr_layer_problem* p) {
  if (!p) return fail(GMMFR_ERR_INVALID_ARG, "problem is NULL");
  if (gmmfr_status st = validate_gate(&p->gate)) return st;
  if (p->gate.T > gmmfr::kLayerMaxTokens)
    return fail(GMMFR_ERR_INVALID_ARG, "T=%lld exceeds the layer's 64 tokens", (long long)p->gate.T);
  if (gmmfr_status st = validate_ffn_sizes(p->gate.H, p->I, p->gate.E)) return st;
  if (p->shared_I != 0)
    if (gmmfr_status st = validate_ffn_sizes(p->gate.H, p->shared_I, 1)) return st;
  if (p->ld_residual != 0 && p->ld_residual < p->gate.H)
    return fail(GMMFR_ERR_INVALID_ARG, "ld_residual=%lld is below H", (long long)p->ld_residual);
  if (p->ld_out != 0 && p->ld_out < p->gate.H) return fail(GMMFR_ERR_INVALID_ARG, "ld_out=%lld is below H", (long long)p->ld_out);
  if (p->weight_type != GMMFR_DT_BF16 && p->weight_type != GMMFR_DT_E4M3)
    return fail(GMMFR_ERR_INVALID_ARG, "weight_type=%d is not BF16 (%d) or E4M3 (%d)", p->weight_type, GMMFR_DT_BF16, GMMFR_DT_E4M3);
  // the kernel counts the tiles of a run, times its CTAs, in 32 bits
  const int64_t kt = p->weight_type == GMMFR_DT_BF16 ? 64 : 128, H = p->gate.H, E = p->gate.E;
  const int64_t up = (E * cdiv(p->I, 64) + cdiv(p->shared_I, 64)) * cdiv(H, kt);
  const int64_t down = (E * cdiv(p->I, kt) + cdiv(p->shared_I, kt)) * cdiv(H, 128);
  if (std::max(up, down) >= (int64_t(1) << 32) / gmmfr::kLayerMaxCtas)
    return fail(GMMFR_ERR_UNSUPPORTED, "the layer's weights have %lld tiles, above 2^32 / %d", (long long)std::max(up, down),
                gmmfr::kLayerMaxCtas);
  return GMMFR_OK;
}

struct LayerLayout {
  int64_t npad, NT1, KB1, NT2, KB2, NT1s, KB2s, n_counters;
  size_t ids, weights, counters, ximg, swimg, swimg_s, slots_up, slots_down, total;
};
LayerLayout layer_layout(const gmmfr_layer_problem* p) {
  LayerLayout L{};
  const bool mx = p->weight_type == GMMFR_DT_E4M3;
  const int64_t T = p->gate.T, k = p->gate.topk, H = p->gate.H, kt = mx ? 128 : 64;
  // columns of the products, a multiple of 16: BF16 npad, MXFP8 2 npad (hi and lo)
  L.npad = mx ? std::max<int64_t>(8, cdiv(T, 8) * 8) : std::max<int64_t>(16, cdiv(T, 16) * 16);
  L.NT1 = cdiv(p->I, 64);
  L.KB1 = cdiv(H, kt);
  L.NT2 = cdiv(H, 128);
  L.KB2 = cdiv(p->I, kt);
  L.NT1s = cdiv(p->shared_I, 64);
  L.KB2s = cdiv(p->shared_I, kt);
  const int64_t experts = std::min<int64_t>(p->gate.E, T * k);  // at most so many are chosen
  L.n_counters = 1 + L.NT1s + experts * L.NT1 + L.NT2 + T;
  const size_t img = (size_t)gmmfr::layer_image_bytes(mx, L.npad);
  size_t off = gmmfr::kHdrBytes;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L.ids = take(sizeof(int32_t) * (size_t)T * k);
  L.weights = take(sizeof(float) * (size_t)T * k);
  L.counters = take(sizeof(uint32_t) * (size_t)L.n_counters);
  L.ximg = take(img * L.KB1);
  L.swimg = take(img * experts * L.KB2);
  L.swimg_s = take(img * L.KB2s);
  L.slots_up = take(sizeof(float) * 128 * T * 2 * gmmfr::kLayerMaxCtas);
  L.slots_down = take(sizeof(float) * 128 * T * 2 * gmmfr::kLayerMaxCtas);
  L.total = off;
  return L;
}

// ---------------------------------------------------------------- dense product
gmmfr_status validate_linear(const gmmfr_linear_problem* p) {
  if (!p) return fail(GMMFR_ERR_INVALID_ARG, "problem is NULL");
  if (p->M < 0 || p->M >= kMaxSize || p->N < 0 || p->N >= kMaxSize / 2 || p->K < 1 || p->K >= kMaxSize)
    return fail(GMMFR_ERR_INVALID_ARG, "M=%lld N=%lld K=%lld out of range (M in [0, 2^31), N in [0, 2^30), K in [1, 2^31))",
                (long long)p->M, (long long)p->N, (long long)p->K);
  if ((p->ldx && p->ldx < p->K) || (p->ldw && p->ldw < p->K) || (p->ld_residual && p->ld_residual < p->N) ||
      (p->ld_out && p->ld_out < p->N))
    return fail(GMMFR_ERR_INVALID_ARG, "a row stride is shorter than its row (ldx=%lld ldw=%lld ld_residual=%lld ld_out=%lld)",
                (long long)p->ldx, (long long)p->ldw, (long long)p->ld_residual, (long long)p->ld_out);
  if (p->activation < GMMFR_ACT_NONE || p->activation > GMMFR_ACT_SWIGLU)
    return fail(GMMFR_ERR_INVALID_ARG, "activation=%d is not a gmmfr_activation", p->activation);
  if (p->unaligned != 0 && p->unaligned != 1) return fail(GMMFR_ERR_INVALID_ARG, "unaligned must be 0 or 1");
  if (p->out_type != GMMFR_DT_BF16 && p->out_type != GMMFR_DT_F32)
    return fail(GMMFR_ERR_INVALID_ARG, "out_type=%d is not BF16 (%d) or F32 (%d)", p->out_type, GMMFR_DT_BF16, GMMFR_DT_F32);
  return GMMFR_OK;
}

// Rows that TMA cannot read in place are copied to a pitch of K rounded up to 8: by their stride, or by where they start
// (which the size of the workspace does not depend on).
bool odd_stride_x(const gmmfr_linear_problem* p) { return p->M > 1 && stride_or(p->ldx, p->K) % 8; }
bool odd_stride_w(const gmmfr_linear_problem* p) {
  return p->N * (p->activation == GMMFR_ACT_SWIGLU ? 2 : 1) > 1 && stride_or(p->ldw, p->K) % 8;
}

// gmmfr_lora_linear's besides
struct Adapters {
  const gmmfr_lora_problem* problem;
  const void *a, *b;
  const float* scale;
  const int32_t* ids;
};

struct LinearLayout {
  size_t x, w, total;
};
LinearLayout linear_layout(const gmmfr_linear_problem* p) {
  LinearLayout L{};
  const size_t Kp = (size_t)cdiv(p->K, 8) * 8;
  size_t off = gmmfr::kHdrBytes;
  L.x = off;
  if (p->unaligned || odd_stride_x(p)) off = align256(off + 2 * Kp * p->M);
  L.w = off;
  if (p->unaligned || odd_stride_w(p)) off = align256(off + 2 * Kp * p->N * (p->activation == GMMFR_ACT_SWIGLU ? 2 : 1));
  L.total = off;
  return L;
}

gmmfr_status validate_lora(const gmmfr_lora_problem* p) {
  if (!p) return fail(GMMFR_ERR_INVALID_ARG, "problem is NULL");
  if (gmmfr_status st = validate_linear(&p->linear)) return st;
  const gmmfr_linear_problem& q = p->linear;
  if (q.K % 8 || q.ldx % 8 || q.ldw % 8)
    return fail(GMMFR_ERR_INVALID_ARG, "K=%lld, ldx=%lld and ldw=%lld must be multiples of 8 with adapters", (long long)q.K,
                (long long)q.ldx, (long long)q.ldw);
  if (q.unaligned) return fail(GMMFR_ERR_INVALID_ARG, "unaligned must be 0 with adapters");
  if (p->count < 1 || p->count >= (int64_t(1) << 24)) return fail(GMMFR_ERR_INVALID_ARG, "count=%lld out of range [1, 2^24)", (long long)p->count);
  if (p->rank < 8 || p->rank > 256 || p->rank % 8)
    return fail(GMMFR_ERR_INVALID_ARG, "rank=%lld is not a multiple of 8 in [8, 256]", (long long)p->rank);
  return GMMFR_OK;
}

// Behind the error words: the adapters' sums, for each 256 rows a list, the sums' own error bits
struct LoraLayout {
  gmmfr::LoraParams plan;
  size_t sums, lists, errs, total;
};
LoraLayout lora_layout(const gmmfr_lora_problem* p, int sms) {
  LoraLayout L{};
  const int64_t M = p->linear.M, blocks = cdiv(M, 256);
  L.plan.M = M;
  L.plan.K = p->linear.K;
  L.plan.count = (int32_t)p->count;
  L.plan.rank = (int32_t)p->rank;
  L.plan.precise = p->linear.out_type == GMMFR_DT_F32;
  L.plan.listed = 1;
  gmmfr::plan_lora_sums(L.plan, sms);
  L.sums = gmmfr::kHdrBytes;
  L.lists = align256(L.sums + sizeof(float) * (size_t)L.plan.parts * M * p->rank);
  L.errs = align256(L.lists + sizeof(int32_t) * gmmfr::kLoraListInts * (size_t)blocks);
  L.total = align256(L.errs + sizeof(uint32_t) * (size_t)L.plan.grid);
  return L;
}

// gmmfr_linear, with adapters unless null (problem and their sizes checked)
gmmfr_status run_linear(const gmmfr_linear_problem* problem, const void* x, const void* weight, const void* bias, const void* residual,
                        void* out, void* workspace, size_t workspace_bytes, void* stream, const Adapters* adapters) {
  const gmmfr_linear_problem& p = *problem;
  if (p.M == 0 || p.N == 0) return GMMFR_OK;
  if (!x || !weight || !out) return fail(GMMFR_ERR_INVALID_ARG, "x, weight and out must be non-NULL when M, N > 0");
  if (!aligned(x, 2) || !aligned(weight, 2) || !aligned(bias, 2) || !aligned(residual, 2) ||
      !aligned(out, p.out_type == GMMFR_DT_F32 ? 4 : 2))
    return fail(GMMFR_ERR_INVALID_ARG, "an input or output is not aligned to its element size");
  const bool gated = p.activation == GMMFR_ACT_SWIGLU;
  const int64_t rows_w = gated ? 2 * p.N : p.N;
  const LinearLayout L = linear_layout(problem);
  const bool copy_x = !aligned(x, 16) || odd_stride_x(problem), copy_w = !aligned(weight, 16) || odd_stride_w(problem);
  if (!p.unaligned && ((copy_x && !odd_stride_x(problem)) || (copy_w && !odd_stride_w(problem))))
    return fail(GMMFR_ERR_INVALID_ARG, "x or weight is off a 16-byte boundary: set problem.unaligned (and size the workspace with it)");
  if (adapters) {
    if (copy_x || copy_w) return fail(GMMFR_ERR_INVALID_ARG, "x and weight must be 16-byte aligned with adapters");
    if (!adapters->a || !adapters->b || !adapters->ids)
      return fail(GMMFR_ERR_INVALID_ARG, "lora_a, lora_b and adapter_ids must be non-NULL when M, N > 0");
    if (!aligned(adapters->a, 16) || !aligned(adapters->b, 16)) return fail(GMMFR_ERR_INVALID_ARG, "lora_a and lora_b must be 16-byte aligned");
    if (!aligned(adapters->scale, 4) || !aligned(adapters->ids, 4))
      return fail(GMMFR_ERR_INVALID_ARG, "lora_scale or adapter_ids is not aligned to its element size");
  }
  if (gmmfr_status st = check_workspace(workspace, workspace_bytes, adapters ? lora_layout(adapters->problem, gmmfr::sm_count()).total : L.total)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = gmmfr::sm_count();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  gmmfr::LinearParams lp{};
  lp.x = static_cast<const __nv_bfloat16*>(x);
  lp.w = static_cast<const __nv_bfloat16*>(weight);
  lp.bias = static_cast<const __nv_bfloat16*>(bias);
  lp.residual = static_cast<const __nv_bfloat16*>(residual);
  lp.out = out;
  lp.hdr = reinterpret_cast<uint32_t*>(ws);
  lp.M = p.M;
  lp.N = p.N;
  lp.K = p.K;
  lp.ldx = stride_or(p.ldx, p.K);
  lp.ldw = stride_or(p.ldw, p.K);
  lp.ldr = stride_or(p.ld_residual, p.N);
  lp.ldo = stride_or(p.ld_out, p.N);
  lp.timeout_ns = waits().limit_ns;
  lp.test_stall = waits().stall;
  lp.act = p.activation;
  lp.out_f32 = p.out_type == GMMFR_DT_F32;
  lp.vec_out = aligned(out, 16) && lp.ldo % (lp.out_f32 ? 4 : 8) == 0 && aligned(residual, 16) && lp.ldr % 8 == 0;
  const int64_t Kp = cdiv(p.K, 8) * 8;
  __nv_bfloat16 *x_copy = nullptr, *w_copy = nullptr;
  if (copy_x) {
    lp.x = x_copy = reinterpret_cast<__nv_bfloat16*>(ws + L.x);
    lp.ldx = Kp;
  }
  if (copy_w) {
    lp.w = w_copy = reinterpret_cast<__nv_bfloat16*>(ws + L.w);
    lp.ldw = Kp;
  }
  gmmfr::LoraParams sums{};
  if (adapters) {
    lp.lora_ids = adapters->ids;
    lp.lora_b = static_cast<const __nv_bfloat16*>(adapters->b);
    const LoraLayout A = lora_layout(adapters->problem, sms);
    sums = A.plan;
    lp.lora_s = sums.s = reinterpret_cast<float*>(ws + A.sums);
    lp.lora_lists = sums.lists = reinterpret_cast<int32_t*>(ws + A.lists);
    lp.lora_count = sums.count;
    lp.lora_rank = sums.rank;
    lp.lora_rows = rows_w;
    sums.x = lp.x;
    sums.ldx = lp.ldx;
    sums.a = static_cast<const __nv_bfloat16*>(adapters->a);
    lp.lora_a = sums.a;
    lp.lora_scale = sums.scale = adapters->scale;
    sums.ids = adapters->ids;
    lp.lora_parts = sums.parts;
    lp.lora_part = p.M * sums.rank;
    sums.errs = reinterpret_cast<uint32_t*>(ws + A.errs);
    lp.lora_errs = sums.errs;
    lp.lora_err_count = sums.grid;
    sums.timeout_ns = lp.timeout_ns;
    sums.test_stall = lp.test_stall;
  }
  gmmfr::LinearParams parts[2] = {lp, lp};
  gmmfr::LinearMaps maps[2];
  gmmfr::plan_linear(parts[0], parts[1], sms);
  parts[0].lora_early = parts[1].M == 0;  // what runs beside starts with it, and does not wait
  gmmfr::LoraMaps sum_maps;
  if (adapters && parts[0].form == gmmfr::kLinearDirect) {  // which needs no lists
    sums.listed = 0;
    gmmfr::plan_lora_sums(sums, sms);
    // What each CTA reads besides its weights comes from L2.  One token, rank 16, replayed: 2048 x 2048 5.8 us, with the sums'
    // launch 7.2; 4096 x 4096 9.0 and 7.3.  Rank 32 of 1024 x 4096: 7.3 and 7.6.
    const int64_t units = p.M * cdiv(sums.rank, 16);
    parts[0].lora_own = units <= 2 && units * p.K <= 2048;
  }
  if (adapters && p.M > gmmfr::kLoraFewRows) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = gmmfr::tensor_map_encoder();
    if (!encode) return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    if (!encode_rows(encode, &sum_maps.x, lp.x, p.M, p.K, lp.ldx, 128) ||
        !encode_slices(encode, &sum_maps.a, sums.a, false, sums.count, sums.rank, p.K, 64, 16))
      return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled failed (first factors)");
  }
  for (int i = 0; i < 2; ++i) {  // what can be refused, before anything is launched
    const gmmfr::LinearParams& q = parts[i];
    if (q.M == 0 || q.form == gmmfr::kLinearDirect) continue;
    PFN_cuTensorMapEncodeTiled_v12000 encode = gmmfr::tensor_map_encoder();
    if (!encode) return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const bool stream_form = q.form == gmmfr::kLinearStream;
    if (!encode_rows(encode, &maps[i].x, q.x, q.M, q.K, q.ldx, stream_form ? q.bn : 128) ||
        !encode_rows(encode, &maps[i].w, q.w, rows_w, q.K, q.ldw, stream_form ? (gated ? 64 : 128) : q.bn / 2))
      return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled failed (ldx=%lld ldw=%lld)", (long long)q.ldx, (long long)q.ldw);
    if (adapters && !encode_slices(encode, &maps[i].b, q.lora_b, false, q.lora_count, q.lora_rows, q.lora_rank, 64,
                                   stream_form ? (gated ? 64 : 128) : q.bn / 2))
      return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled failed (adapters)");
  }
  if (x_copy) {
    cudaError_t e = gmmfr::launch_linear_repitch(static_cast<const __nv_bfloat16*>(x), x_copy, p.M, p.K, Kp, stride_or(p.ldx, p.K), sms, s);
    if (e != cudaSuccess) return cuda_fail(e, "x copy launch");
  }
  if (w_copy) {
    cudaError_t e = gmmfr::launch_linear_repitch(static_cast<const __nv_bfloat16*>(weight), w_copy, rows_w, p.K, Kp, stride_or(p.ldw, p.K), sms, s);
    if (e != cudaSuccess) return cuda_fail(e, "weight copy launch");
  }
  if (adapters && !parts[0].lora_own) {
    cudaError_t e = gmmfr::launch_lora_sums(sum_maps, sums, s);
    if (e != cudaSuccess) return cuda_fail(e, "adapters' sums launch");
  }
  for (int i = 0; i < 2; ++i) {
    if (parts[i].M == 0) continue;
    cudaError_t e = adapters ? gmmfr::launch_lora_linear(maps[i], parts[i], s) : gmmfr::launch_linear(maps[i], parts[i], s);
    if (e != cudaSuccess) return cuda_fail(e, "linear launch");
  }
  return GMMFR_OK;
}

// ---------------------------------------------------------------- products grouped by expert
gmmfr_status validate_grouped(const gmmfr_grouped_problem* p) {
  if (!p) return fail(GMMFR_ERR_INVALID_ARG, "problem is NULL");
  if (p->M < 0 || p->M > kMaxSize - 1024)  // rows are counted in 32 bits, in steps of up to 256
    return fail(GMMFR_ERR_INVALID_ARG, "M=%lld out of range [0, 2^31 - 1024]", (long long)p->M);
  if (p->N < 8 || p->K < 8 || p->N % 8 || p->K % 8 || p->N >= (int64_t(1) << 24) || p->K >= (int64_t(1) << 24) ||
      p->N * p->K >= (int64_t(1) << 38))
    return fail(GMMFR_ERR_INVALID_ARG, "N=%lld K=%lld are not multiples of 8 in [8, 2^24) with a product below 2^38",
                (long long)p->N, (long long)p->K);
  if (p->E < 1 || p->E > gmmfr::kMaxExperts) return fail(GMMFR_ERR_INVALID_ARG, "E=%lld out of range [1, 1024]", (long long)p->E);
  if ((p->ldx && p->ldx < p->K) || (p->ldy && p->ldy < p->N) || p->ldx >= (int64_t(1) << 38) || p->ldy >= (int64_t(1) << 38))
    return fail(GMMFR_ERR_INVALID_ARG, "a row stride is shorter than its row, or above 2^38 (ldx=%lld ldy=%lld)", (long long)p->ldx,
                (long long)p->ldy);
  if (p->ldx % 8) return fail(GMMFR_ERR_INVALID_ARG, "ldx=%lld is not a multiple of 8", (long long)p->ldx);
  if (p->transposed != 0 && p->transposed != 1) return fail(GMMFR_ERR_INVALID_ARG, "transposed must be 0 or 1");
  if (p->group_list_type != 0 && p->group_list_type != 1)
    return fail(GMMFR_ERR_INVALID_ARG, "group_list_type=%d is not 0 (prefix sums) or 1 (counts)", p->group_list_type);
  if (p->out_type != GMMFR_DT_BF16 && p->out_type != GMMFR_DT_F32)
    return fail(GMMFR_ERR_INVALID_ARG, "out_type=%d is not BF16 (%d) or F32 (%d)", p->out_type, GMMFR_DT_BF16, GMMFR_DT_F32);
  if (p->zero_rest != 0 && p->zero_rest != 1) return fail(GMMFR_ERR_INVALID_ARG, "zero_rest must be 0 or 1");
  if (p->accumulate != 0 && p->accumulate != 1) return fail(GMMFR_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  return GMMFR_OK;
}

// Error words; the gradient's CTAs' copies of the experts' ends; sums of shares of their rows, if there are more than one
struct GroupedLayout {
  int shares;
  size_t parts, total;
};
GroupedLayout grouped_layout(const gmmfr_grouped_problem* p) {
  const int sms = gmmfr::sm_count();
  GroupedLayout L;
  L.shares = p->M ? gmmfr::grouped_grad_shares(p->M, p->N, p->K, p->E, sms) : 1;
  L.parts = align256(gmmfr::kHdrBytes + sizeof(int32_t) * (size_t)gmmfr::grouped_grad_ctas(p->N, p->K, p->E * L.shares, sms) * p->E);
  L.total = L.parts + (L.shares > 1 ? align256(sizeof(float) * (size_t)L.shares * p->E * p->N * p->K) : 0);
  return L;
}

}  // namespace

extern "C" {

gmmfr_status gmmfr_moe_gate_workspace_size(const gmmfr_gate_problem* problem, size_t* bytes) {
  if (gmmfr_status st = validate_gate(problem)) return st;
  if (!bytes) return fail(GMMFR_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = gate_ws_bytes(problem);
  return GMMFR_OK;
}

gmmfr_status gmmfr_moe_gate(const gmmfr_gate_problem* problem, const void* x, const void* weight,
                            const float* select_bias, void* topk_ids, float* topk_weights, float* logits,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (gmmfr_status st = validate_gate(problem)) return st;
  const gmmfr_gate_problem& p = *problem;
  if (p.T == 0) return GMMFR_OK;
  if (!x || !weight || !topk_ids || !topk_weights)
    return fail(GMMFR_ERR_INVALID_ARG, "x, weight, topk_ids and topk_weights must be non-NULL when T > 0");
  if (!aligned(x, 16) || !aligned(weight, 16)) return fail(GMMFR_ERR_INVALID_ARG, "x and weight must be 16-byte aligned");
  if (!aligned(topk_ids, p.ids_type == GMMFR_INDEX_I32 ? 4 : 8) || !aligned(topk_weights, 4) ||
      !aligned(select_bias, 4) || !aligned(logits, 4))
    return fail(GMMFR_ERR_INVALID_ARG, "an input or output is not aligned to its element size");
  if (gmmfr_status st = check_workspace(workspace, workspace_bytes, gate_ws_bytes(problem))) return st;
  gmmfr::GateParams g = gate_params(p, x, weight, select_bias);
  g.logits = logits;
  g.ids = topk_ids;
  g.weights = topk_weights;
  g.ids_i64 = p.ids_type == GMMFR_INDEX_I64;
  g.hdr = static_cast<uint32_t*>(workspace);
  g.timeout_ns = waits().limit_ns;
  g.test_stall = waits().stall;
  gmmfr::GateMaps maps;
  if (gmmfr::plan_gate(g, gmmfr::sm_count())) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = gmmfr::tensor_map_encoder();
    if (!encode) return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    if (!encode_rows(encode, &maps.x, x, p.T, p.H, g.ldx, 128) || !encode_rows(encode, &maps.w, weight, p.E, p.H, p.H, g.bn / 2))
      return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  }
  cudaError_t e = gmmfr::launch_gate(maps, g, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "gate launch");
  return GMMFR_OK;
}

gmmfr_status gmmfr_ffn_prepared_weights_size_mx(const gmmfr_ffn_problem* problem, size_t* bytes) {
  if (!problem) return fail(GMMFR_ERR_INVALID_ARG, "problem is NULL");
  if (gmmfr_status st = validate_ffn_sizes(problem->H, problem->I, problem->E)) return st;
  if (!bytes) return fail(GMMFR_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = ffn_bytes(problem->H, problem->I, problem->E, true);
  return GMMFR_OK;
}

gmmfr_status gmmfr_ffn_prepare_weights_mx(const gmmfr_ffn_problem* problem, const void* w13, const void* w13_scale,
                                          const void* w2, const void* w2_scale, void* prepared, size_t prepared_bytes,
                                          void* stream) {
  size_t need = 0;
  if (gmmfr_status st = gmmfr_ffn_prepared_weights_size_mx(problem, &need)) return st;
  if (!w13 || !w13_scale || !w2 || !w2_scale || !prepared)
    return fail(GMMFR_ERR_INVALID_ARG, "w13, w13_scale, w2, w2_scale and prepared must be non-NULL");
  if (prepared_bytes < need) return fail(GMMFR_ERR_WORKSPACE, "prepared buffer has %zu bytes, needs %zu", prepared_bytes, need);
  if (!aligned(prepared, 16)) return fail(GMMFR_ERR_WORKSPACE, "prepared buffer must be 16-byte aligned");
  const gmmfr_ffn_problem& p = *problem;
  gmmfr::FfnPrepMxParams pp{};
  pp.w13 = static_cast<const uint8_t*>(w13);
  pp.s13 = static_cast<const uint8_t*>(w13_scale);
  pp.w2 = static_cast<const uint8_t*>(w2);
  pp.s2 = static_cast<const uint8_t*>(w2_scale);
  pp.prepared = static_cast<uint8_t*>(prepared);
  pp.H = p.H;
  pp.I = p.I;
  pp.E = (int32_t)p.E;
  pp.NT1 = (int32_t)cdiv(p.I, 64);
  pp.KB1 = (int32_t)cdiv(p.H, 128);
  pp.NT2 = (int32_t)cdiv(p.H, 128);
  pp.KB2 = (int32_t)cdiv(p.I, 128);
  cudaError_t e = gmmfr::launch_ffn_prep_mx(pp, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "FFN weight preparation launch");
  return GMMFR_OK;
}

gmmfr_status gmmfr_moe_layer_workspace_size(const gmmfr_layer_problem* problem, size_t* bytes) {
  if (gmmfr_status st = validate_layer(problem)) return st;
  if (!bytes) return fail(GMMFR_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = layer_layout(problem).total;
  return GMMFR_OK;
}

gmmfr_status gmmfr_moe_layer(const gmmfr_layer_problem* problem, const void* x, const void* gate_weight,
                             const float* select_bias, const void* residual, void* out, const void* prepared,
                             size_t prepared_bytes, const void* shared_prepared, size_t shared_prepared_bytes,
                             int32_t* topk_ids, float* topk_weights, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (gmmfr_status st = validate_layer(problem)) return st;
  const gmmfr_layer_problem& p = *problem;
  if (p.gate.T == 0) return GMMFR_OK;
  if (!x || !gate_weight || !out || !prepared)
    return fail(GMMFR_ERR_INVALID_ARG, "x, gate_weight, out and prepared must be non-NULL when T > 0");
  if (p.shared_I > 0 && !shared_prepared) return fail(GMMFR_ERR_INVALID_ARG, "shared_prepared is NULL but shared_I > 0");
  if (!aligned(x, 16) || !aligned(gate_weight, 16) || !aligned(prepared, 16) || !aligned(shared_prepared, 16))
    return fail(GMMFR_ERR_INVALID_ARG, "x, gate_weight and the prepared weights must be 16-byte aligned");
  if (!aligned(select_bias, 4) || !aligned(residual, 2) || !aligned(out, 2) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
    return fail(GMMFR_ERR_INVALID_ARG, "an input or output is not aligned to its element size");
  const bool mx = p.weight_type == GMMFR_DT_E4M3;
  const size_t need = ffn_bytes(p.gate.H, p.I, p.gate.E, mx);
  if (prepared_bytes < need) return fail(GMMFR_ERR_WORKSPACE, "prepared buffer has %zu bytes, needs %zu", prepared_bytes, need);
  if (p.shared_I > 0) {
    const size_t s_need = ffn_bytes(p.gate.H, p.shared_I, 1, mx);
    if (shared_prepared_bytes < s_need)
      return fail(GMMFR_ERR_WORKSPACE, "shared prepared buffer has %zu bytes, needs %zu", shared_prepared_bytes, s_need);
  }
  const LayerLayout L = layer_layout(problem);
  if (gmmfr_status st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  gmmfr::LayerParams lp{};
  lp.gate = gate_params(p.gate, x, gate_weight, select_bias);
  lp.gate.ids = topk_ids ? topk_ids : reinterpret_cast<int32_t*>(ws + L.ids);
  lp.gate.weights = topk_weights ? topk_weights : reinterpret_cast<float*>(ws + L.weights);
  lp.residual = static_cast<const __nv_bfloat16*>(residual);
  lp.out = static_cast<__nv_bfloat16*>(out);
  lp.prepared = static_cast<const uint8_t*>(prepared);
  lp.shared = static_cast<const uint8_t*>(shared_prepared);
  lp.ld_residual = stride_or(p.ld_residual, p.gate.H);
  lp.ld_out = stride_or(p.ld_out, p.gate.H);
  lp.mx = mx;
  const int64_t tile = mx ? gmmfr::kPrepTileBytes : gmmfr::kWTileBytes;
  lp.prepared2 = lp.prepared + p.gate.E * L.NT1 * L.KB1 * tile;
  lp.shared2 = lp.shared + L.NT1s * L.KB1 * tile;
  lp.hdr = reinterpret_cast<uint32_t*>(ws);
  lp.ximg = ws + L.ximg;
  lp.swimg = ws + L.swimg;
  lp.swimg_s = ws + L.swimg_s;
  lp.slots_up = reinterpret_cast<float*>(ws + L.slots_up);
  lp.slots_down = reinterpret_cast<float*>(ws + L.slots_down);
  lp.counters = reinterpret_cast<uint32_t*>(ws + L.counters);
  lp.up_done = lp.counters;
  lp.down_cnt = lp.counters + 1;
  lp.nan_rows = lp.down_cnt + L.NT2;
  lp.up_cnt = lp.nan_rows + p.gate.T;
  lp.n_counters = (int32_t)L.n_counters;
  lp.npad = (int32_t)L.npad;
  lp.NT1 = (int32_t)L.NT1;
  lp.KB1 = (int32_t)L.KB1;
  lp.NT2 = (int32_t)L.NT2;
  lp.KB2 = (int32_t)L.KB2;
  lp.NT1s = (int32_t)L.NT1s;
  lp.KB2s = (int32_t)L.KB2s;
  lp.timeout_ns = waits().limit_ns;
  lp.test_stall = waits().stall;
  cudaError_t e = gmmfr::launch_layer(lp, gmmfr::sm_count(), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "MoE layer launch");
  return GMMFR_OK;
}

gmmfr_status gmmfr_linear_workspace_size(const gmmfr_linear_problem* problem, size_t* bytes) {
  if (gmmfr_status st = validate_linear(problem)) return st;
  if (!bytes) return fail(GMMFR_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = linear_layout(problem).total;
  return GMMFR_OK;
}

gmmfr_status gmmfr_linear(const gmmfr_linear_problem* problem, const void* x, const void* weight, const void* bias,
                          const void* residual, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (gmmfr_status st = validate_linear(problem)) return st;
  return run_linear(problem, x, weight, bias, residual, out, workspace, workspace_bytes, stream, nullptr);
}

gmmfr_status gmmfr_lora_linear_workspace_size(const gmmfr_lora_problem* problem, size_t* bytes) {
  if (gmmfr_status st = validate_lora(problem)) return st;
  if (!bytes) return fail(GMMFR_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = lora_layout(problem, gmmfr::sm_count()).total;
  return GMMFR_OK;
}

gmmfr_status gmmfr_lora_linear(const gmmfr_lora_problem* problem, const void* x, const void* weight, const void* bias,
                               const void* residual, const void* lora_a, const void* lora_b, const float* lora_scale,
                               const int32_t* adapter_ids, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (gmmfr_status st = validate_lora(problem)) return st;
  const Adapters adapters{problem, lora_a, lora_b, lora_scale, adapter_ids};
  return run_linear(&problem->linear, x, weight, bias, residual, out, workspace, workspace_bytes, stream, &adapters);
}

gmmfr_status gmmfr_grouped_linear_workspace_size(const gmmfr_grouped_problem* problem, size_t* bytes) {
  if (gmmfr_status st = validate_grouped(problem)) return st;
  if (!bytes) return fail(GMMFR_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = grouped_layout(problem).total;
  return GMMFR_OK;
}

gmmfr_status gmmfr_grouped_linear(const gmmfr_grouped_problem* problem, const void* x, const void* weight,
                                  const int64_t* group_list, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (gmmfr_status st = validate_grouped(problem)) return st;
  const gmmfr_grouped_problem& p = *problem;
  if (p.accumulate) return fail(GMMFR_ERR_INVALID_ARG, "accumulate is the weights' gradient's");
  if (p.M == 0) return GMMFR_OK;
  if (!x || !weight || !group_list || !y)
    return fail(GMMFR_ERR_INVALID_ARG, "x, weight, group_list and y must be non-NULL when M > 0");
  if (!aligned(x, 16) || !aligned(weight, 16)) return fail(GMMFR_ERR_INVALID_ARG, "x and weight must be 16-byte aligned");
  const bool f32 = p.out_type == GMMFR_DT_F32;
  if (!aligned(group_list, 8) || !aligned(y, f32 ? 4 : 2))
    return fail(GMMFR_ERR_INVALID_ARG, "group_list or y is not aligned to its element size");
  if (gmmfr_status st = check_workspace(workspace, workspace_bytes, gmmfr::kHdrBytes)) return st;
  gmmfr::GroupedParams g{};
  g.group_list = group_list;
  g.out = y;
  g.hdr = static_cast<uint32_t*>(workspace);
  g.M = p.M;
  g.N = p.N;
  g.ldo = stride_or(p.ldy, p.N);
  g.timeout_ns = waits().limit_ns;
  g.test_stall = waits().stall;
  g.E = (int32_t)p.E;
  g.group_list_type = p.group_list_type;
  g.KB = (int32_t)cdiv(p.K, 64);
  g.out_f32 = f32;
  g.vec_out = aligned(y, 4) && g.ldo % 2 == 0;
  g.zero_rest = p.zero_rest;
  PFN_cuTensorMapEncodeTiled_v12000 encode = gmmfr::tensor_map_encoder();
  if (!encode) return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  gmmfr::GroupedMaps maps;
  bool ok = p.transposed ? encode_slices(encode, &maps.w, weight, false, p.E, p.K, p.N, 64, 64)
                         : encode_slices(encode, &maps.w, weight, false, p.E, p.N, p.K, 64, 128);
  for (int i = 0; i < 4; ++i) ok = ok && encode_rows(encode, &maps.x[i], x, p.M, p.K, stride_or(p.ldx, p.K), 16 << i);
  if (!ok) return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled failed (ldx=%lld)", (long long)p.ldx);
  cudaError_t e = gmmfr::launch_grouped(maps, g, p.transposed, gmmfr::sm_count(), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "grouped product launch");
  return GMMFR_OK;
}

gmmfr_status gmmfr_grouped_linear_grad_weight(const gmmfr_grouped_problem* problem, const void* dy, const void* x,
                                              const int64_t* group_list, void* dweight, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  if (gmmfr_status st = validate_grouped(problem)) return st;
  const gmmfr_grouped_problem& p = *problem;
  const bool f32 = p.out_type == GMMFR_DT_F32;
  if (p.zero_rest) return fail(GMMFR_ERR_INVALID_ARG, "zero_rest is the product's");
  if (p.accumulate && !f32) return fail(GMMFR_ERR_INVALID_ARG, "accumulate takes a gradient in FP32");
  if (p.ldy % 8) return fail(GMMFR_ERR_INVALID_ARG, "ldy=%lld is not a multiple of 8", (long long)p.ldy);
  if (p.M == 0 && p.accumulate) return GMMFR_OK;
  if (!dweight) return fail(GMMFR_ERR_INVALID_ARG, "dweight is NULL");
  if (p.M > 0 && (!dy || !x || !group_list)) return fail(GMMFR_ERR_INVALID_ARG, "dy, x and group_list must be non-NULL when M > 0");
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dweight, 16))
    return fail(GMMFR_ERR_INVALID_ARG, "dy, x and dweight must be 16-byte aligned");
  if (!aligned(group_list, 8)) return fail(GMMFR_ERR_INVALID_ARG, "group_list is not aligned to its element size");
  const GroupedLayout L = grouped_layout(problem);
  if (gmmfr_status st = check_workspace(workspace, workspace_bytes, L.total)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.M == 0) {
    cudaError_t e = cudaMemsetAsync(workspace, 0, 8, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dweight, 0, (size_t)p.E * p.N * p.K * (f32 ? 4 : 2), s);
    return e == cudaSuccess ? GMMFR_OK : cuda_fail(e, "zeros of the gradient");
  }
  gmmfr::GroupedGradParams g{};
  g.group_list = group_list;
  g.hdr = static_cast<uint32_t*>(workspace);
  g.ends = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + gmmfr::kHdrBytes);
  g.M = p.M;
  g.A = p.transposed ? p.K : p.N;  // the gradient's rows, then its columns
  g.B = p.transposed ? p.N : p.K;
  g.timeout_ns = waits().limit_ns;
  g.test_stall = waits().stall;
  g.E = (int32_t)p.E;
  g.group_list_type = p.group_list_type;
  g.out_f32 = f32;
  g.accumulate = p.accumulate;
  g.shares = L.shares;
  g.out = dweight;
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.parts);
  g.parts = parts;
  PFN_cuTensorMapEncodeTiled_v12000 encode = gmmfr::tensor_map_encoder();
  if (!encode) return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  gmmfr::GroupedGradMaps maps;
  if (!encode_rows(encode, p.transposed ? &maps.b : &maps.a, dy, p.M, p.N, stride_or(p.ldy, p.N), 64) ||
      !encode_rows(encode, p.transposed ? &maps.a : &maps.b, x, p.M, p.K, stride_or(p.ldx, p.K), 64) ||
      !(L.shares > 1 ? encode_slices(encode, &maps.out, parts, true, p.E * L.shares, g.A, g.B, 32, 32)
                     : encode_slices(encode, &maps.out, dweight, f32, p.E, g.A, g.B, f32 ? 32 : 64, 32)))
    return fail(GMMFR_ERR_CUDA, "cuTensorMapEncodeTiled failed (ldx=%lld ldy=%lld)", (long long)p.ldx, (long long)p.ldy);
  cudaError_t e = gmmfr::launch_grouped_grad(maps, g, gmmfr::sm_count(), s);
  if (e != cudaSuccess) return cuda_fail(e, "grouped gradient launch");
  return GMMFR_OK;
}

}  // extern "C"
