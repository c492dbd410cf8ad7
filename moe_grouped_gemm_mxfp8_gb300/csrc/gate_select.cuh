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

// One warp selects token `logits[0..E)`'s experts; lane k < topk returns the k-th expert and its
// weight.  Expert e sits in lane e % 32, register e / 32 (kPer registers: E <= 32 * kPer).
// `scratch`: E floats of shared memory of this warp, used when there are groups.
// All sums are FP32; the exponential's argument is at most 0 and its sum at least 1.
template <int kPer>
__device__ __forceinline__ void gate_select_warp(const GateRule& r, const float* logits, const float* select_bias,
                                                 float* scratch, int lane, int& id_out, float& w_out) {
  constexpr uint32_t kAll = 0xffffffffu;
  const float kNegInf = __int_as_float(0xff800000);
  float p[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    p[i] = e < r.E ? logits[e] : kNegInf;
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
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    float s = p[i];
    if (select_bias != nullptr && e < r.E) s += select_bias[e];
    key[i] = e < r.E ? order_key(s) : 0u;
    if (r.n_group > 1 && e < r.E) scratch[e] = s;
  }
  if (r.n_group > 1) {
    __syncwarp();
    const int per = r.E / r.n_group;
    uint32_t gkey[2] = {0u, 0u};  // groups lane and lane + 32
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = lane + 32 * h;
      if (g < r.n_group) {
        float a = kNegInf, b = kNegInf;  // the two highest scores of the group
        for (int i = 0; i < per; ++i) {
          // each lane starts at another place of its group: consecutive lanes read other banks
          const int k = (i + lane) % per;
          const float v = scratch[g * per + k];
          if (v > a) {
            b = a;
            a = v;
          } else if (v > b) {
            b = v;
          }
        }
        gkey[h] = order_key(r.group_top == 2 ? a + b : a);
      }
    }
    uint64_t ok = 0;  // eligible groups: fewer than topk_group groups are better, or equal and earlier
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int rank = 0;
      for (int g = 0; g < r.n_group; ++g) {
        const uint32_t lo = __shfl_sync(kAll, gkey[0], g & 31), hi = __shfl_sync(kAll, gkey[1], g & 31);
        const uint32_t o = g < 32 ? lo : hi;
        rank += (o > gkey[h] || (o == gkey[h] && g < lane + 32 * h)) ? 1 : 0;
      }
      const uint32_t m = __ballot_sync(kAll, lane + 32 * h < r.n_group && rank < r.topk_group);
      ok |= (uint64_t)m << (32 * h);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e < r.E && !((ok >> (e / per)) & 1)) key[i] = 0u;
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
