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

// One warp selects token `logits[0..E)`'s experts (long choices of many experts); lane k < topk returns the k-th expert and
// its weight.  Expert e sits in lane e % 32, register e / 32; select_bias may be in shared memory.
// All sums are FP32; the exponential's argument is at most 0 and its sum at least 1.  Maxima and minima over the
// warp are single redux instructions on order-preserving integers.
__device__ __forceinline__ void gate_select_warp(const GateRule& r, const float* logits, const float* select_bias,
                                                 int lane, int& id_out, float& w_out) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int kPer = kMaxExperts / 32;
  const float kNegInf = __int_as_float(0xff800000);
  float p[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    p[i] = e < r.E ? logits[e] : kNegInf;
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
    key[i] = e < r.E ? order_key(select_bias ? p[i] + select_bias[e] : p[i]) : 0u;
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
// A cluster of 8 CTAs takes 8 kTiles tokens.  Its warps (64 or 128) share the products: a warp takes one or two groups of 16
// experts and one of the splits of K (blocks of 32, taken in turn) against all the tokens, and sends its sums straight to
// the CTAs that select for those tokens (CTA c: tokens c * kTiles ...), which add the splits in order.  The weight rows
// are read straight into the operand registers of mma.sync: lane l holds 8 consecutive elements of rows l / 4 and
// l / 4 + 8, which serve as the lane's K slots of two products (the K slots of A and B are permuted alike, which leaves
// the sums alone), so each row is read in 16-byte pieces with no staging.
// One token of H = 2048 and 256 experts takes 5.9 us: about 2 until the weights are there (they come through 8 SMs),
// 0.6 for the sums, 2.9 for the selection, all of it latency.
namespace gate {
constexpr int kCluster = 8;
// Threads of a CTA: of 256 two CTAs share an SM; 512 ask for the weights in fewer rounds, when there are more than the
// six blocks that a warp of the 64 asks for at once, and the clusters are few (15 with a CTA per SM).  One token,
// H = 2048, 256 experts: 5.9 us with 512, 6.6 with 256; H = 7168, 16 experts: 5.8 and 5.0.
constexpr int kSmall = 512, kLarge = 256;
// Groups of 16 experts that a warp takes: with 16 or 32 tokens two share its tokens' loads, since what reaches an SM is what
// bounds it then, unless that leaves too few pairs of groups for the warps.  1024 tokens of 7168, 512 experts: 71.5 us
// with one, 52.5 with two; 333 of 5120, 160 experts: 14.0 and 13.2; 300 of 4096, 64 experts: 7.8 and 8.7.
inline int cluster_groups(int64_t T, int E) { return T > 32 * 8 && E > 64 ? 2 : 1; }
inline int cluster_threads(int64_t T, int64_t H, int E) {
  return T <= 15 * 8 && (int64_t)((E + 15) / 16) * ((H + 31) / 32) > 64 * 6 ? kSmall : kLarge;
}
constexpr int kMaxCand = 256;
// What a team of threads needs to select for one token.
struct TeamScratch {
  uint32_t cand_key[kMaxCand];
  uint16_t cand_e[kMaxCand];
  uint32_t group_key[kMaxGroups];
  uint32_t eligible[2];
  float stat[16];
  uint32_t out_e[kMaxTopk];
  float out_p[kMaxTopk];
};
template <int kTiles, int kThr>
struct Smem {
  // of the tokens this CTA selects for: the splits' sums; then the logits, the probabilities, and the selection's keys
  // behind them
  float logits[kTiles][2 * kMaxExperts];
  TeamScratch team[kTiles];
  float bias[kMaxExperts];
};
}  // namespace gate

// Selects for one token with kTeam threads (`tid` 0 .. kTeam - 1, named barrier `bar`), in steps that are short even
// when no instruction of them is in the cache yet (3.8 us by one warp, 2.9 by eight: 256 experts, sigmoid, groups):
//   scores and keys, a thread per expert;  groups, a warp per group
//   per 32 consecutive experts their topk best, by counting for each lane the keys that precede it (equal keys: the lower
//   index precedes)
//   of those candidates the topk best, again by counting
// p holds the logits and then the probabilities.  At most kMaxCand candidates (topk per 32 experts).
template <int kTeam>
__device__ __forceinline__ void gate_select_team(const GateRule& r, const float* select_bias, float* p, uint32_t* key,
                                                 gate::TeamScratch& sc, int tid, int bar, void* ids, int ids_i64,
                                                 float* weights, int64_t out_at) {
  constexpr uint32_t kAll = 0xffffffffu;
  constexpr int kTeamWarps = kTeam / 32;
  const float kNegInf = __int_as_float(0xff800000);
  const int lane = tid & 31, warp = tid >> 5, E = r.E, topk = r.topk;
  auto sync = [&]() { ptx::bar_sync(bar, kTeam); };
  float inv = 1.f, mx = kNegInf;
  if (!r.sigmoid) {
    for (int e = tid; e < E; e += kTeam) mx = fmaxf(mx, p[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
    if (lane == 0) sc.stat[warp] = mx;
    sync();
#pragma unroll
    for (int w = 0; w < kTeamWarps; ++w) mx = fmaxf(mx, sc.stat[w]);
    float sum = 0.f;
    for (int e = tid; e < E; e += kTeam) {
      // logits that are all -inf leave nothing to weigh: p = 0 (a NaN among them stays one)
      const float l = p[e], v = mx == kNegInf ? (l != l ? l : 0.f) : expf(l - mx);
      p[e] = v;
      sum += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (lane == 0) sc.stat[8 + warp] = sum;
    sync();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kTeamWarps; ++w) sum += sc.stat[8 + w];
    inv = mx == kNegInf && sum == 0.f ? 0.f : 1.0f / sum;
  }
  for (int e = tid; e < E; e += kTeam) {
    const float v = r.sigmoid ? gate_sigmoid(p[e]) : p[e] * inv;
    p[e] = v;
    key[e] = order_key(select_bias ? v + select_bias[e] : v);
  }
  sync();
  const int per = E / r.n_group;
  if (r.n_group > 1) {
    for (int g = warp; g < r.n_group; g += kTeamWarps) {
      uint32_t a = 0, b = 0;  // the lane's two highest keys of the group
      for (int i = lane; i < per; i += 32) {
        const uint32_t k = key[g * per + i];
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
      if (lane == 0) sc.group_key[g] = order_key(s);
    }
    sync();
    if (tid < 64) {  // fewer than topk_group groups are better, or equal and earlier
      bool in = false;
      if (tid < r.n_group) {
        const uint32_t mine = sc.group_key[tid];
        int better = 0;
        for (int h = 0; h < r.n_group; ++h) {
          const uint32_t o = sc.group_key[h];
          better += (o > mine || (o == mine && h < tid)) ? 1 : 0;
        }
        in = better < r.topk_group;
      }
      const uint32_t m = __ballot_sync(kAll, in);
      if (lane == 0) sc.eligible[warp] = m;
    }
    sync();
  }
  const int segs = (E + 31) / 32;
  const float per_inv = 1.0f / (float)per;
  for (int s = warp; s < segs; s += kTeamWarps) {
    const int e = s * 32 + lane;
    uint32_t k = e < E ? key[e] : 0u;
    if (r.n_group > 1 && e < E) {
      const int g = (int)(((float)e + 0.5f) * per_inv);  // e / per: the half keeps it clear of rounding (e < 1024)
      if (!((sc.eligible[g >> 5] >> (g & 31)) & 1)) k = 0u;
    }
    const uint32_t k_1 = k - 1;  // o >= k of an earlier lane: o > k - 1
    if (lane < topk) sc.cand_key[s * topk + lane] = 0u;  // places that stay free
    __syncwarp();
    int place = 0;
#pragma unroll 4
    for (int l = 0; l < 32; ++l) {
      const uint32_t o = __shfl_sync(kAll, k, l);
      place += o > (l < lane ? k_1 : k) ? 1 : 0;
    }
    if (k != 0 && place < topk) {
      sc.cand_key[s * topk + place] = k;
      sc.cand_e[s * topk + place] = (uint16_t)e;
    }
  }
  sync();
  // several lanes share a candidate when there are threads enough
  const int n = segs * topk;
  int sh = 0;
  while (sh < 4 && (2 << sh) * n <= kTeam) ++sh;
  const int share = 1 << sh, part = tid & (share - 1);
  for (int c0 = 0; c0 < n; c0 += kTeam >> sh) {
    const int c = c0 + (tid >> sh);
    const uint32_t k = c < n ? sc.cand_key[c] : 0u;
    int place = 0;  // equal candidates stand in the order of their indices
#pragma unroll 4
    for (int o = part; o < n; o += share) {
      const uint32_t v = sc.cand_key[o];
      place += (v > k || (v == k && o < c)) ? 1 : 0;
    }
    for (int o = share / 2; o > 0; o >>= 1) place += __shfl_xor_sync(kAll, place, o);
    if (k != 0 && place < topk && part == 0) {
      sc.out_e[place] = sc.cand_e[c];
      sc.out_p[place] = p[sc.cand_e[c]];
    }
  }
  sync();
  if (warp == 0) {
    float w = lane < topk ? sc.out_p[lane] : 0.f;
    if (r.renormalise) {
      float total = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
      w = w / (total + 1e-20f);
    }
    if (lane < topk) {
      if (ids_i64) static_cast<int64_t*>(ids)[out_at + lane] = sc.out_e[lane];
      else static_cast<int32_t*>(ids)[out_at + lane] = (int32_t)sc.out_e[lane];
      weights[out_at + lane] = w * r.scale;
    }
  }
}

template <int kTiles, int kThr, int kG>
__device__ __forceinline__ void gate_cluster_logits(const GateParams& p, int64_t t0, gate::Smem<kTiles, kThr>& sm, uint32_t rank,
                                                    int warp, int lane) {
  // blocks of 32 K in flight
  constexpr int kU = kThr == gate::kSmall ? 8 : (kTiles == 1 ? 6 : (kTiles == 2 ? (kG == 1 ? 4 : 3) : (kG == 1 ? 3 : 2)));
  const int tid = threadIdx.x, E = p.rule.E, groups = ((E + 15) / 16 + kG - 1) / kG;  // of kG x 16 experts
  const int blocks = (int)((p.H + 31) / 32);
  const int w = (int)rank * (kThr / 32) + warp;
  const int splits = min(gate::kCluster * (kThr / 32) / groups, (blocks + kU - 1) / kU);
  const int split = w / groups, grp = w - split * groups, row = groups * kG * 16;
  ptx::cluster_wait();  // the other CTAs have started: their shared memory may be written
  if (split < splits) {
    // rows past the end repeat the last one; what they give is not read
    const __nv_bfloat16* wr[2 * kG];
#pragma unroll
    for (int i = 0; i < 2 * kG; ++i) wr[i] = p.weight + (int64_t)min((grp * 2 * kG + i) * 8 + (lane >> 2), E - 1) * p.H;
    const __nv_bfloat16* xr[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int64_t t = t0 + 8 * i + (lane >> 2);
      xr[i] = p.x + (t < p.T ? t : p.T - 1) * p.ldx;
    }
    float acc[kG][kTiles][4] = {};
    for (int b0 = split; b0 < blocks; b0 += splits * kU) {
      uint4 a[kU][2 * kG], x[kU][kTiles];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = (int64_t)(b0 + u * splits) * 32 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 2 * kG; ++i) a[u][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) x[u][i] = make_uint4(0, 0, 0, 0);
        if (k < p.H) {
#pragma unroll
          for (int i = 0; i < 2 * kG; ++i) a[u][i] = __ldg(reinterpret_cast<const uint4*>(wr[i] + k));
#pragma unroll
          for (int i = 0; i < kTiles; ++i) x[u][i] = __ldg(reinterpret_cast<const uint4*>(xr[i] + k));
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int g = 0; g < kG; ++g)
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const uint4 &lo = a[u][2 * g], &hi = a[u][2 * g + 1];
            ptx::mma_16816(acc[g][i], lo.x, hi.x, lo.y, hi.y, x[u][i].x, x[u][i].y);
            ptx::mma_16816(acc[g][i], lo.z, hi.z, lo.w, hi.w, x[u][i].z, x[u][i].w);
          }
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int at = split * row + (grp * kG + g) * 16 + (lane >> 2);  // at most the cluster's warps x kG x 16: 2 kMaxExperts
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int tok = 8 * i + (lane & 3) * 2 + c;
          const uint32_t dst = ptx::map_to_rank(ptx::smem_u32(&sm.logits[tok % kTiles][at]), (uint32_t)(tok / kTiles));
          ptx::st_cluster_f32(dst, acc[g][i][c]);
          ptx::st_cluster_f32(dst + 32, acc[g][i][2 + c]);
        }
    }
  }
  ptx::cluster_sync();
  if (splits > 1) {  // the splits' sums, in order
    constexpr int kTeam = kThr / kTiles;
    float* l = sm.logits[tid / kTeam];
    for (int e = tid % kTeam; e < E; e += kTeam) {
      float s = 0.f;
#pragma unroll 4
      for (int k = 0; k < splits; ++k) s += l[k * row + e];
      l[e] = s;
    }
    __syncthreads();
  }
}

template <int kTiles, int kThr, int kG>
__device__ __forceinline__ void gate_cluster(const GateParams& p, int64_t t0, gate::Smem<kTiles, kThr>& sm, uint32_t rank) {
  constexpr int kTeam = (kThr < 256 ? kThr : 256) / kTiles;  // more threads than that would wait on one another for longer
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int E = p.rule.E;
  const int64_t t = t0 + rank * kTiles;
  const bool by_team = (E + 31) / 32 * p.rule.topk <= gate::kMaxCand;
  ptx::cluster_arrive_relaxed();
  if (p.select_bias)
    for (int e = tid; e < E; e += kThr) sm.bias[e] = p.select_bias[e];
  gate_cluster_logits<kTiles, kThr, kG>(p, t0, sm, rank, warp, lane);
  if (p.logits) {
    for (int i = 0; i < kTiles; ++i)
      if (t + i < p.T)
        for (int e = tid; e < E; e += kThr) p.logits[(t + i) * E + e] = sm.logits[i][e];
    __syncthreads();  // the probabilities take the logits' place
  }
  const float* bias = p.select_bias ? sm.bias : nullptr;
  if (by_team) {
    const int i = tid / kTeam;  // the team's token
    if (i < kTiles && t + i < p.T)
      gate_select_team<kTeam>(p.rule, bias, sm.logits[i], reinterpret_cast<uint32_t*>(sm.logits[i] + kMaxExperts),
                              sm.team[i], tid % kTeam, 1 + i, p.ids, p.ids_i64,
                              p.weights, (t + i) * p.rule.topk);
  } else if (warp < kTiles && t + warp < p.T) {
    const float* l = sm.logits[warp];
    int id;
    float w;
    gate_select_warp(p.rule, l, bias, lane, id, w);
    if (lane < p.rule.topk) {
      const int64_t o = (t + warp) * p.rule.topk + lane;
      if (p.ids_i64) static_cast<int64_t*>(p.ids)[o] = id;
      else static_cast<int32_t*>(p.ids)[o] = id;
      p.weights[o] = w;
    }
  }
}

}  // namespace gmmfr
