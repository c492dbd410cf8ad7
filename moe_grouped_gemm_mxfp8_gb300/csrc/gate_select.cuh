// The router's selection for one token by one warp: scores, eligible groups, top-k.
#pragma once
#include <cstdint>

#include "ops.cuh"
#include "ptx.cuh"

namespace gmmfr {

// A float's place in the selection order as an unsigned integer: larger floats map to larger
// integers, -0 and +0 to the same one, NaN to 1 (below -inf), so that 0 is free for "not eligible".
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// 1 / (1 + exp(-l)) with the approximate reciprocal (one more ulp; 0 for l = -inf)
__device__ __forceinline__ float gate_sigmoid(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }
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
  // the bias is asked for beside the logits (with many experts per lane it would cost too many registers)
  constexpr bool kBiasFirst = kPer <= 8;
  float p[kPer], bias[kBiasFirst ? kPer : 1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    p[i] = e < r.E ? logits[e] : kNegInf;
    if constexpr (kBiasFirst) bias[i] = select_bias != nullptr && e < r.E ? __ldg(select_bias + e) : 0.f;
  }
  if (r.sigmoid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = gate_sigmoid(p[i]);
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
    const float inv = mx == kNegInf && sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] *= inv;
  }
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    float b = 0.f;
    if constexpr (kBiasFirst) b = bias[i];
    else if (select_bias != nullptr && e < r.E) b = __ldg(select_bias + e);
    key[i] = e < r.E ? order_key(p[i] + b) : 0u;
  }
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
  for (int k = 0; k < r.topk; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    uint32_t mine = kAll;  // the lane's lowest index with that key
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) mine = key[i] == top ? (uint32_t)(lane + 32 * i) : mine;
    const uint32_t id = __reduce_min_sync(kAll, mine);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i == (int)id ? 0u : key[i];
    if (lane == k) id_out = (int)id;
  }
  w_out = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float v = __shfl_sync(kAll, p[i], id_out & 31);
    w_out = (id_out >> 5) == i ? v : w_out;
  }
  if (r.renormalise) {
    float total = lane < r.topk ? w_out : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    w_out = w_out / (total + 1e-20f);
  }
  w_out *= r.scale;
}

// ---------------------------------------------------------------- the router for a few tokens by one cluster
// A cluster of 8 CTAs takes 8 kTiles tokens: CTA c computes the logits of expert groups c, c + 8, ... (16 experts each,
// the 8 warps splitting groups and the K range), sends tokens c * kTiles ... to CTA c, which selects for them.  The
// weight rows are read straight into the operand registers of mma.sync: lane l holds 8 consecutive elements of rows
// l / 4 and l / 4 + 8, which serve as the lane's K slots of two products (the K slots of A and B are permuted alike,
// which leaves the sums alone), so each row is read in 16-byte pieces with no staging.
namespace gate {
constexpr int kCluster = 8;
constexpr int kThreads = 256;  // 128 registers each: half an SM, so that the kernel that follows fits beside it
constexpr int kWarps = kThreads / 32;
template <int kTiles>
struct Smem {
  float part[kWarps][16][8 * kTiles + 1];   // a warp's sums
  float logits[kTiles][kMaxExperts];        // of the tokens this CTA selects for
};
}  // namespace gate

template <int kTiles>
__device__ __forceinline__ void gate_cluster(const GateParams& p, int64_t t0, gate::Smem<kTiles>& sm, uint32_t rank) {
  constexpr int kTok = 8 * kTiles;
  ptx::cluster_arrive_relaxed();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.rule.E, groups = (E + 15) / 16;
  const int per_cta = (groups + gate::kCluster - 1) / gate::kCluster;  // 1..8
  const int splits = gate::kWarps / per_cta;
  const int gi = warp % per_cta, split = warp / per_cta;
  const int grp = (int)rank + gate::kCluster * gi;
  if (split < splits && grp < groups) {
    // rows past the end repeat the last one; what they give is not read
    const int ea = min(grp * 16 + (lane >> 2), E - 1), eb = min(grp * 16 + 8 + (lane >> 2), E - 1);
    const __nv_bfloat16* wa = p.weight + (int64_t)ea * p.H;
    const __nv_bfloat16* wb = p.weight + (int64_t)eb * p.H;
    const __nv_bfloat16* xr[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int64_t t = t0 + 8 * i + (lane >> 2);
      xr[i] = p.x + (t < p.T ? t : p.T - 1) * p.ldx;
    }
    float acc[kTiles][4] = {};
    const int blocks = (int)((p.H + 31) / 32);
    constexpr int kU = kTiles == 1 ? 6 : (kTiles == 2 ? 4 : 2);  // blocks of 32 K in flight
    for (int b0 = split; b0 < blocks; b0 += splits * kU) {
      uint4 a[kU], b[kU], x[kU][kTiles];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = (int64_t)(b0 + u * splits) * 32 + (lane & 3) * 8;
        a[u] = b[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) x[u][i] = make_uint4(0, 0, 0, 0);
        if (k < p.H) {
          a[u] = __ldg(reinterpret_cast<const uint4*>(wa + k));
          b[u] = __ldg(reinterpret_cast<const uint4*>(wb + k));
#pragma unroll
          for (int i = 0; i < kTiles; ++i) x[u][i] = __ldg(reinterpret_cast<const uint4*>(xr[i] + k));
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          ptx::mma_16816(acc[i], a[u].x, b[u].x, a[u].y, b[u].y, x[u][i].x, x[u][i].y);
          ptx::mma_16816(acc[i], a[u].z, b[u].z, a[u].w, b[u].w, x[u][i].z, x[u][i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      float* d = &sm.part[warp][lane >> 2][8 * i + (lane & 3) * 2];
      d[0] = acc[i][0];
      d[1] = acc[i][1];
      d[8 * (kTok + 1)] = acc[i][2];
      d[8 * (kTok + 1) + 1] = acc[i][3];
    }
  }
  ptx::cluster_wait();  // the other CTAs have started: their shared memory may be written
  __syncthreads();
  for (int i = tid; i < per_cta * 16 * kTok; i += gate::kThreads) {
    const int g = i / (16 * kTok), tok = i / 16 % kTok, r = i & 15;
    const int e = ((int)rank + gate::kCluster * g) * 16 + r;
    if (e < E && t0 + tok < p.T) {
      float s = 0.f;
#pragma unroll 4
      for (int k = 0; k < splits; ++k) s += sm.part[k * per_cta + g][r][tok];
      ptx::st_cluster_f32(ptx::map_to_rank(ptx::smem_u32(&sm.logits[tok % kTiles][e]), (uint32_t)(tok / kTiles)), s);
    }
  }
  ptx::cluster_sync();
  const int64_t t = t0 + rank * kTiles;
  if (p.logits) {
    for (int i = 0; i < kTiles; ++i)
      if (t + i < p.T)
        for (int e = tid; e < E; e += gate::kThreads) p.logits[(t + i) * E + e] = sm.logits[i][e];
  }
  if (warp < kTiles && t + warp < p.T) {
    const float* l = sm.logits[warp];
    int id;
    float w;
    if (E <= 64) gate_select_warp<2>(p.rule, l, p.select_bias, lane, id, w);
    else if (E <= 256) gate_select_warp<8>(p.rule, l, p.select_bias, lane, id, w);
    else gate_select_warp<32>(p.rule, l, p.select_bias, lane, id, w);
    if (lane < p.rule.topk) {
      const int64_t o = (t + warp) * p.rule.topk + lane;
      if (p.ids_i64) static_cast<int64_t*>(p.ids)[o] = id;
      else static_cast<int32_t*>(p.ids)[o] = id;
      p.weights[o] = w;
    }
  }
}

}  // namespace gmmfr
