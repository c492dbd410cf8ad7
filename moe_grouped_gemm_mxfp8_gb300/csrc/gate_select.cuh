// The router's selection for one token by one warp: scores, eligible groups, top-k.
#pragma once
#include <cstdint>

#include "ops.cuh"

namespace gmmfr {

// A float's place in the selection order as an unsigned integer: larger floats map to larger
// integers, -0 and +0 to the same one, NaN to 1 (below -inf), so that 0 is free for "not eligible".
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {  // of a key above 1
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// One warp selects token `logits[0..E)`'s experts; lane k < topk returns the k-th expert and its
// weight.  Expert e sits in lane e % 32, register e / 32 (kPer registers: E <= 32 * kPer).
// All sums are FP32; the exponential's argument is at most 0 and its sum at least 1.  Maxima and minima over the
// warp are single redux instructions on order-preserving integers.
template <int kPer>
__device__ __forceinline__ void gate_select_warp(const GateRule& r, const float* logits, const float* select_bias,
                                                 int lane, int& id_out, float& w_out) {
  constexpr uint32_t kAll = 0xffffffffu;
  const float kNegInf = __int_as_float(0xff800000);
  float p[kPer], bias[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    p[i] = e < r.E ? logits[e] : kNegInf;
    bias[i] = select_bias != nullptr && e < r.E ? __ldg(select_bias + e) : 0.f;
  }
  if (r.sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = 1.0f / (1.0f + expf(-p[i]));
  } else {
    float mx = kNegInf;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mx = fmaxf(mx, p[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // logits that are all -inf leave nothing to weigh: p = 0 (a NaN among them stays one)
      p[i] = mx == kNegInf ? (p[i] != p[i] ? p[i] : 0.f) : expf(p[i] - mx);
      sum += p[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = mx == kNegInf && sum == 0.f ? 0.f : p[i] / sum;
  }
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < r.E ? order_key(p[i] + bias[i]) : 0u;
  if (r.n_group > 1) {
    const int per = r.E / r.n_group;
    uint32_t gkey[2] = {0u, 0u};  // of groups lane and lane + 32
    for (int g = 0; g < r.n_group; ++g) {
      const int first = g * per;
      uint32_t a = 0, b = 0;  // the lane's two highest keys of the group
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t k = (unsigned)(lane + 32 * i - first) < (unsigned)per ? key[i] : 0u;
        b = max(b, min(a, k));
        a = max(a, k);
      }
      const uint32_t top = __reduce_max_sync(kAll, a);
      float s = top > 1u ? key_value(top) : kNegInf;
      if (r.group_top == 2) {  // one lane that has the highest gives it up
        const bool holder = lane == __ffs(__ballot_sync(kAll, a == top)) - 1;
        const uint32_t second = __reduce_max_sync(kAll, holder ? b : a);
        s += second > 1u ? key_value(second) : kNegInf;
      }
      if (lane == (g & 31)) gkey[g >> 5] = order_key(s);
    }
    // eligible groups: fewer than topk_group groups are better, or equal and earlier
    int rank[2] = {0, 0};
    for (int g = 0; g < r.n_group; ++g) {
      const uint32_t o = __shfl_sync(kAll, g < 32 ? gkey[0] : gkey[1], g & 31);
      rank[0] += (o > gkey[0] || (o == gkey[0] && g < lane)) ? 1 : 0;
      rank[1] += (o > gkey[1] || (o == gkey[1] && g < lane + 32)) ? 1 : 0;
    }
    const uint32_t ok0 = __ballot_sync(kAll, lane < r.n_group && rank[0] < r.topk_group);
    const uint32_t ok1 = __ballot_sync(kAll, lane + 32 < r.n_group && rank[1] < r.topk_group);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = (lane + 32 * i) / per;
      if (!(((g < 32 ? ok0 : ok1) >> (g & 31)) & 1u)) key[i] = 0u;
    }
  }
  id_out = 0;
  w_out = 0.f;
  float total = 0.f;
  for (int k = 0; k < r.topk; ++k) {
    uint32_t best = 0;
    int at = 0;
    float pw = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (key[i] > best) {  // strictly: the lane's lowest index among equals
        best = key[i];
        at = i;
        pw = p[i];
      }
    }
    const uint32_t top = __reduce_max_sync(kAll, best);
    const uint32_t id = __reduce_min_sync(kAll, best == top ? (uint32_t)(lane + 32 * at) : kAll);
    const float w = __shfl_sync(kAll, pw, id & 31);
    total += w;
    if (lane == k) {
      id_out = (int)id;
      w_out = w;
    }
    if (lane == (int)(id & 31)) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == at) key[i] = 0u;
    }
  }
  if (r.renormalise) w_out = w_out / (total + 1e-20f);
  w_out *= r.scale;
}

}  // namespace gmmfr
