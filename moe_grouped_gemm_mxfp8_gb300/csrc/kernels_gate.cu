// The router: logits = x W^T (FP32 sums of BF16 products), then the selection of each token.
//   cluster  few tokens: clusters of 8 CTAs for 8, 16 or 32 tokens each (gate_select.cuh)
//   pair     many tokens: CTA pairs take 256 tokens against all experts (tcgen05, cta_group::2), and the selection
//            reads the logits where they are, in TMEM: a token is a TMEM lane, so a thread walks its token's
//            columns.  Four threads share a token, a quarter of the columns each.  16384 tokens of 2048, 256 experts,
//            sigmoid and groups: 35.5 us (69 MB, 1.9 TB/s), one tile per pair.  24 of them remain with H = 64: the
//            selection is what bounds it, a thread's chain of exponentials, keys and compares over 64 columns (tiles
//            of fewer tokens, on fewer warps, take as long), and a CTA with one tile has nothing to run beside it.
#include "gate_select.cuh"
#include "ops.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace gmmfr {

namespace gate {
constexpr int kPairThreads = 64 + 512;  // warp 0 TMA, warp 1 MMA, 16 epilogue warps
// The ring; the selection's exchange areas, which the ring has too when no tile follows; barriers, biases
constexpr int kArena = 128 * 1024;
constexpr int kMaxStages = 8;
constexpr int kTop = 8;  // the pair form's longest choice
constexpr int kStatOff = kArena;                         // float [2][4][128]: maxima and sums; eligible groups
constexpr int kListOff = kStatOff + 2 * 4 * 128 * 4;     // uint32 [4][8][128]: each quarter's best keys
constexpr int kCap = 16;                                 // candidates a quarter has room for
constexpr int kCandOff = kListOff + 4 * kTop * 128 * 4;  // group keys [64][128], then candidates [4][kCap][2][128]
constexpr int kSelOff = kCandOff + 4 * kCap * 2 * 128 * 4;  // the choice [8][2][128]
constexpr int kBars = 2 * kMaxStages + 3;
constexpr int kBarOff = kSelOff + kTop * 2 * 128 * 4;
constexpr int kMiscOff = kBarOff + kBars * 8 + 8;
constexpr int kBiasOff = kMiscOff + 32;                  // float bias[512]
constexpr int kPairSmem = kBiasOff + 512 * 4 + 1024;
static_assert(kMaxGroups <= 4 * kCap * 2 && kPairSmem <= 232448, "shared memory");
constexpr int kPairExperts = 512;  // the pair form's most: their logits fill TMEM
}  // namespace gate

// ============================================================================ cluster form
template <int kTiles, int kThr, int kG = 1>
__global__ void __launch_bounds__(kThr) gate_cluster_kernel(const __grid_constant__ GateParams p) {
  __shared__ gate::Smem<kTiles, kThr> sm;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) {  // no wait here can give up
    p.hdr[0] = 1;
    p.hdr[1] = 0;
  }
  gate_cluster<kTiles, kThr, kG>(p, (int64_t)(blockIdx.x / gate::kCluster) * 8 * kTiles, sm, ptx::cluster_rank());
}

// ============================================================================ pair form
// kBlocks: experts in blocks of 256 (1 or 2).  TMEM: the logits, which the probabilities replace; with one block the
// selection keys in columns 256 .. 511 (with two they are made anew whenever the columns are walked).
template <int kBlocks>
__global__ void __launch_bounds__(gate::kPairThreads, 1)
    gate_pair_kernel(const __grid_constant__ GateMaps maps, const __grid_constant__ GateParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + gate::kBarOff);  // used in rank 0: both CTAs' loads
  uint64_t* empty = full + gate::kMaxStages;
  uint64_t* accf = empty + gate::kMaxStages;
  uint64_t* acce = accf + 1;  // used in rank 0: both CTAs' epilogue warps
  uint64_t* drain = acce + 1;
  int32_t* misc = reinterpret_cast<int32_t*>(smem + gate::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&misc[0]);
  int* abort_flag = &misc[1];
  uint32_t* s_err = reinterpret_cast<uint32_t*>(&misc[2]);
  float* s_bias = reinterpret_cast<float*>(smem + gate::kBiasOff);
  float* s_stat = reinterpret_cast<float*>(smem + gate::kStatOff);
  uint32_t* s_list = reinterpret_cast<uint32_t*>(smem + gate::kListOff);
  uint32_t* s_cand = reinterpret_cast<uint32_t*>(smem + gate::kCandOff);
  uint32_t* s_sel = reinterpret_cast<uint32_t*>(smem + gate::kSelOff);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const uint32_t rank = ptx::cluster_rank();
  const GateRule& r = p.rule;
  const int E = r.E, BN = p.bn;
  constexpr int kXBytes = 128 * 128;
  constexpr bool kKeys = kBlocks == 1;
  const int block_bytes = BN * 64, stage_bytes = kXBytes + kBlocks * block_bytes, n_stages = p.n_stages, KB = p.KB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(accf), 1 + p.test_stall);
    ptx::mbar_init(ptx::smem_u32(acce), 32);
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    *abort_flag = 0;
    *s_err = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane < 2) ptx::prefetch_tensormap(lane ? &maps.w : &maps.x);
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::griddep_wait();
  for (int e = threadIdx.x; e < 512; e += gate::kPairThreads) s_bias[e] = p.select_bias && e < E ? p.select_bias[e] : 0.f;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  ptx::griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  const Ctl ctl{abort_flag, s_err, p.timeout_ns};
  const uint32_t smem_base = ptx::smem_u32(smem);
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
  const int tiles = (int)((p.T + 255) / 256);

  if (warp == 0) {
    const uint64_t pol_x = ptx::l2_evict_first_policy(), pol_w = ptx::l2_evict_last_policy();
    const uint32_t full_own = ptx::smem_u32(full), full0 = ptx::map_to_rank(full_own, 0), empty0 = ptx::smem_u32(empty);
    int stage = 0;
    uint32_t phase = 0, sb = smem_base;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += pairs) {
      const int ym = t * 256 + (int)rank * 128, yn = (int)rank * (BN / 2);
      for (int kb = 0, x = 0; kb < KB; ++kb, x += 64) {
        if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
          ok = false;
          break;
        }
        if (ptx::elect_one()) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(full_own + 8 * stage, 2 * stage_bytes);
          ptx::tma_load_2d_pair(sb, &maps.x, x, ym, full0 + 8 * stage, pol_x);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            ptx::tma_load_2d_pair(sb + kXBytes + b * block_bytes, &maps.w, x, yn + b * 256, full0 + 8 * stage, pol_w);
        }
        sb += stage_bytes;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
          sb = smem_base;
        }
      }
    }
    for (int s = 0; ok && s < n_stages; ++s) {  // no load is in flight at exit
      ok = warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl);
      if (++stage == n_stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok && rank == 0) {  // aborted: let what is in flight land (both CTAs' loads count on rank 0's barriers)
      for (int s = 0; s < n_stages; ++s)
        if (!wait_bar_drain(ptx::smem_u32(&full[s]), s < stage ? phase : phase ^ 1)) break;  // rank 1 gave up before its load
    } else if (!ok) {
      let_loads_land();  // of a stage that rank 0 may not wait for: it may have given up before its own load
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
      const uint64_t da0 = ptx::smem_desc(smem_base, 16, 1024, ptx::kSwizzle128B);
      const uint32_t lo0 = (uint32_t)da0, desc_hi = (uint32_t)(da0 >> 32);
      const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
      const uint32_t lo_step = (uint32_t)stage_bytes >> 4, lo_block = (uint32_t)block_bytes >> 4;
      int stage = 0;
      uint32_t phase = 0, aph = 0, lo = lo0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += pairs) {
        if (!__all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(acce), aph ^ 1, ctl))) break;
        ptx::tc_fence_after();
        uint32_t accumulate = 0;
        for (int kb = 0; kb < KB; ++kb) {
          if (!warp_wait_quick(full0 + 8 * stage, phase, ctl)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::tc_mma_f16_pair_lo(tmem_base + b * 256, lo + 2 * q, lo + (kXBytes >> 4) + b * lo_block + 2 * q, desc_hi, idesc,
                                        q > 0 ? 1u : accumulate);
            ptx::tc_commit_pair(empty0 + 8 * stage);
            if (kb == KB - 1) ptx::tc_commit_pair(ptx::smem_u32(accf));
          }
          accumulate = 1;
          lo += lo_step;
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
            lo = lo0;
          }
        }
        aph ^= 1;
      }
      if (ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(drain));
      wait_bar_drain(ptx::smem_u32(drain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ selection
    const int q = warp & 3, part = (warp - 2) >> 2;  // TMEM lane quadrant; quarter of the columns
    const int tok = q * 32 + lane;                   // token of this CTA's half of the tile, and exchange column
    const int chunks = (E + 15) / 16, c_lo = chunks * part / 4, c_hi = chunks * (part + 1) / 4;
    const float kNegInf = __int_as_float(0xff800000);
    const bool softmax = !r.sigmoid, grouped = r.n_group > 1;
    const int per = E / r.n_group;
    auto quadrant_sync = [&]() { ptx::bar_sync(1 + q, 128); };  // the four warps that share this quadrant's tokens
    uint32_t ph = 0;
    for (int t = first; t < tiles; t += pairs, ph ^= 1) {
      const bool ok = wait_quick(ptx::smem_u32(accf), ph, ctl);
      if (!ptx::bar_all(1 + q, 128, ok)) break;  // the four leave together
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
      const int64_t token = (int64_t)t * 256 + rank * 128 + tok;
      // chunk c's columns that are experts (past E the rows of W are zeros that do not exist)
      auto valid = [&](int c) { return c * 16 + 16 <= E ? 0xffffu : (1u << (E - c * 16)) - 1; };
      float mx = kNegInf, inv = 1.f;
      if (softmax || p.logits) {
        for (int c = c_lo; c < c_hi; ++c) {
          uint32_t v[16];
          ptx::tmem_ld_32x32b_x16(taddr + c * 16, v);
          const uint32_t in = valid(c);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((in >> j) & 1) mx = fmaxf(mx, __uint_as_float(v[j]));
          if (p.logits && token < p.T) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if ((in >> j) & 1) p.logits[token * E + c * 16 + j] = __uint_as_float(v[j]);
          }
        }
      }
      if (softmax) {
        s_stat[part * 128 + tok] = mx;
        quadrant_sync();
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = fmaxf(mx, s_stat[k * 128 + tok]);
        float sum = 0.f;
        for (int c = c_lo; c < c_hi; ++c) {
          uint32_t v[16];
          ptx::tmem_ld_32x32b_x16(taddr + c * 16, v);
          const uint32_t in = valid(c);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float l = __uint_as_float(v[j]);
            const float e = mx == kNegInf ? (l != l ? l : 0.f) : expf(l - mx);
            if ((in >> j) & 1) sum += e;
            v[j] = __float_as_uint(e);
          }
          ptx::tmem_st_32x32b_x16(taddr + c * 16, v);
        }
        s_stat[(4 + part) * 128 + tok] = sum;
        ptx::tmem_wait_st();
        quadrant_sync();
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += s_stat[(4 + k) * 128 + tok];
        // logits that are all -inf leave nothing to weigh
        inv = mx == kNegInf && sum == 0.f ? 0.f : 1.0f / sum;
      }
      auto probability = [&](uint32_t v) { return __uint_as_float(v) * inv; };
      // chunk c's keys, from TMEM
      auto load_keys = [&](int c, uint32_t (&k)[16]) {
        if constexpr (kKeys) {
          ptx::tmem_ld_32x32b_x16(taddr + 256 + c * 16, k);
          ptx::tmem_wait_ld();
        } else {
          ptx::tmem_ld_32x32b_x16(taddr + c * 16, k);
          const uint32_t in = valid(c);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) k[j] = (in >> j) & 1 ? order_key(__uint_as_float(k[j]) + s_bias[c * 16 + j]) : 0u;
        }
      };
      // probabilities and selection keys, and the highest key of each run of 8 columns (16 when there are more than
      // four chunks: at most 8 runs)
      uint32_t* runs = s_list + part * gate::kTop * 128 + tok;
      const bool halves = c_hi - c_lo <= 4;
      for (int c = c_lo; c < c_hi; ++c) {
        uint32_t v[16], k[16];
        ptx::tmem_ld_32x32b_x16(taddr + c * 16, v);
        float b[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(b + 4 * j) = *reinterpret_cast<const float4*>(s_bias + c * 16 + 4 * j);
        const uint32_t in = valid(c);
        ptx::tmem_wait_ld();
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float pv = softmax ? probability(v[j]) : gate_sigmoid(__uint_as_float(v[j]));
          v[j] = __float_as_uint(pv);
          k[j] = (in >> j) & 1 ? order_key(pv + b[j]) : 0u;
          if (j < 8) lo = max(lo, k[j]);
          else hi = max(hi, k[j]);
        }
        ptx::tmem_st_32x32b_x16(taddr + c * 16, v);
        if constexpr (kKeys) ptx::tmem_st_32x32b_x16(taddr + 256 + c * 16, k);
        if (halves) {
          runs[2 * (c - c_lo) * 128] = lo;
          runs[(2 * (c - c_lo) + 1) * 128] = hi;
        } else {
          runs[(c - c_lo) * 128] = max(lo, hi);
        }
      }
      for (int k = halves ? 2 * (c_hi - c_lo) : c_hi - c_lo; k < gate::kTop; ++k) runs[k * 128] = 0;
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      quadrant_sync();
      ptx::tc_fence_after();
      uint64_t eligible = ~0ull;
      if (grouped) {
        for (int g = part; g < r.n_group; g += 4) {  // this quarter's share of the groups
          uint32_t a = 0, b = 0;                     // the two highest keys
          const int lo = g * per, hi = lo + per;
          for (int c = lo >> 4; c * 16 < hi; ++c) {
            uint32_t k[16];
            load_keys(c, k);
            uint32_t in = 0xffffu;  // the chunk's columns of this group
            if (c * 16 < lo) in &= 0xffffu << (lo - c * 16);
            if (c * 16 + 16 > hi) in &= (1u << (hi - c * 16)) - 1;
            if (in == 0xffffu) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                b = max(b, min(a, k[j]));
                a = max(a, k[j]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t x = (in >> j) & 1 ? k[j] : 0u;
                b = max(b, min(a, x));
                a = max(a, x);
              }
            }
          }
          float s = a > 1u ? key_value(a) : kNegInf;
          if (r.group_top == 2) s += b > 1u ? key_value(b) : kNegInf;
          s_cand[g * 128 + tok] = order_key(s);
        }
        quadrant_sync();
        uint64_t mine = 0;
        for (int g = part; g < r.n_group; g += 4) {  // fewer than topk_group groups better, or equal and earlier
          const uint32_t k = s_cand[g * 128 + tok];
          int better = 0;
          for (int h = 0; h < r.n_group; ++h) {
            const uint32_t o = s_cand[h * 128 + tok];
            better += (o > k || (o == k && h < g)) ? 1 : 0;
          }
          if (better < r.topk_group) mine |= 1ull << g;
        }
        uint32_t* m = reinterpret_cast<uint32_t*>(s_stat);  // [2][4][128]: low and high words
        m[part * 128 + tok] = (uint32_t)mine;
        m[(4 + part) * 128 + tok] = (uint32_t)(mine >> 32);
        quadrant_sync();
        eligible = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) eligible |= (uint64_t)m[(4 + k) * 128 + tok] << 32 | m[k * 128 + tok];
      }
      // chunk c's columns in eligible groups
      auto in_groups = [&](int c) {
        if (!grouped) return 0xffffu;
        if (per % 16 == 0) return (eligible >> (c * 16 / per)) & 1 ? 0xffffu : 0u;
        uint32_t in = 0;
        for (int j = 0; j < 16 && c * 16 + j < E; ++j) in |= (uint32_t)((eligible >> ((c * 16 + j) / per)) & 1) << j;
        return in;
      };
      // Walks this quarter's columns, 16 at a time, with their keys (0 outside the eligible groups).
      auto columns = [&](auto&& visit) {
        for (int c = c_lo; c < c_hi; ++c) {
          uint32_t k[16];
          load_keys(c, k);
          if (grouped) {
            const uint32_t in = in_groups(c);
#pragma unroll
            for (int j = 0; j < 16; ++j) k[j] = (in >> j) & 1 ? k[j] : 0u;
          }
          visit(c, k);
        }
      };
      uint32_t key[gate::kTop];  // in descending order
      auto put = [&](uint32_t x) {
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) {
          const uint32_t hi = max(key[k], x);
          x = min(key[k], x);
          key[k] = hi;
        }
      };
      // Takes the best of the four quarters' lists (in shared memory) into this thread's: the best 8 of two descending
      // lists are max(a[i], b[7 - i]), put in order by the halving steps of a bitonic sort.
      auto merge = [&]() {
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) s_list[(part * gate::kTop + k) * 128 + tok] = key[k];
        quadrant_sync();
#pragma unroll
        for (int h = 1; h < 4; ++h) {
          const uint32_t* o = s_list + ((part + h) & 3) * gate::kTop * 128 + tok;
#pragma unroll
          for (int k = 0; k < gate::kTop; ++k) key[k] = max(key[k], o[(gate::kTop - 1 - k) * 128]);
#pragma unroll
          for (int d = gate::kTop / 2; d > 0; d >>= 1)
#pragma unroll
            for (int k = 0; k < gate::kTop; ++k)
              if (!(k & d)) {
                const uint32_t a = max(key[k], key[k + d]), b = min(key[k], key[k + d]);
                key[k] = a;
                key[k + d] = b;
              }
        }
      };
      auto topk_th = [&]() {
        uint32_t last = key[0];
#pragma unroll
        for (int k = 1; k < gate::kTop; ++k) last = k < r.topk ? key[k] : last;
        return last;
      };
      // Keeping the best 8 of all columns in order (8 maxima and 8 minima per column) is what a token would mostly spend
      // its time on.  Instead:
      // 1. a bound from below on the topk-th key: the topk-th of the runs' maxima
#pragma unroll
      for (int k = 0; k < gate::kTop; ++k) key[k] = 0;
      if (grouped) {
        columns([&](int c, const uint32_t (&k)[16]) {
          uint32_t a = 0, b = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a = max(a, k[j]);
            b = max(b, k[8 + j]);
          }
          if (halves) {
            put(a);
            put(b);
          } else {
            put(max(a, b));
          }
        });
      } else {
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) put(runs[k * 128]);
      }
      merge();
      uint32_t last = topk_th();
      last = token < p.T ? (last > 0 ? last : 1u) : 0xffffffffu;  // past the tokens all scores are equal: none is taken
      // 2. the columns that reach it: few, unless many scores are equal (or one run holds them all)
      int n = 0;
      uint32_t* cand = s_cand + part * gate::kCap * 2 * 128 + tok;  // column and probability
      auto cand_key = [&](int i) { return order_key(__uint_as_float(cand[(2 * i + 1) * 128]) + s_bias[cand[2 * i * 128]]); };
      columns([&](int c, const uint32_t (&k)[16]) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(taddr + c * 16, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (k[j] >= last) {
            uint32_t* o = cand + (n & (gate::kCap - 1)) * 2 * 128;
            o[0] = (uint32_t)(c * 16 + j);
            o[128] = v[j];
            ++n;
          }
        }
      });
      // 3. the topk-th key: from the candidates, or, when they did not fit, from all columns
      const bool fits = ptx::bar_all(1 + q, 128, n <= gate::kCap);
#pragma unroll
      for (int k = 0; k < gate::kTop; ++k) key[k] = 0;
      if (fits) {
        for (int i = 0; i < n; ++i) put(cand_key(i));
      } else {
        columns([&](int, const uint32_t (&k)[16]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) put(k[j]);
        });
      }
      merge();
      last = topk_th();
      if (!fits) {  // the columns above it, and of its equals the first that fill the choice: at most topk per quarter
        int need = r.topk;
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) need -= key[k] > last ? 1 : 0;
        n = 0;
        columns([&](int c, const uint32_t (&k)[16]) {
          uint32_t v[16];
          ptx::tmem_ld_32x32b_x16(taddr + c * 16, v);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (k[j] > last || (k[j] == last && need > 0)) {
              need -= k[j] == last ? 1 : 0;
              cand[2 * n * 128] = (uint32_t)(c * 16 + j);
              cand[(2 * n + 1) * 128] = v[j];
              ++n;
            }
          }
        });
      }
      // TMEM is read: the next tile's products may overwrite it
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(acce), 0));
      // 4. each candidate's place: the keys above it, and its equals in earlier columns
      for (int i = 0; i < n; ++i) {
        const uint32_t x = cand_key(i);
        int place = 0, equal = 0;
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) {
          place += key[k] > x ? 1 : 0;
          equal += key[k] == x ? 1 : 0;
        }
        if (equal > 1 || x == last) {  // equals of the last may lie beyond the list
          for (int k = 0; k < i; ++k) place += cand_key(k) == x ? 1 : 0;
          for (int k = 0; k < part * gate::kTop; ++k) place += s_list[k * 128 + tok] == x ? 1 : 0;
        }
        if (place < r.topk) {
          s_sel[2 * place * 128 + tok] = cand[2 * i * 128];
          s_sel[(2 * place + 1) * 128 + tok] = cand[(2 * i + 1) * 128];
        }
      }
      quadrant_sync();
      if (part == 0 && token < p.T) {
        float w[gate::kTop], total = 0.f;
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) {
          w[k] = k < r.topk ? __uint_as_float(s_sel[(2 * k + 1) * 128 + tok]) : 0.f;
          total += w[k];
        }
#pragma unroll
        for (int k = 0; k < gate::kTop; ++k) {
          if (k < r.topk) {
            const int64_t o = token * r.topk + k;
            const uint32_t e = s_sel[2 * k * 128 + tok];
            if (p.ids_i64) static_cast<int64_t*>(p.ids)[o] = e;
            else static_cast<int32_t*>(p.ids)[o] = (int32_t)e;
            p.weights[o] = (r.renormalise ? w[k] / (total + 1e-20f) : w[k]) * r.scale;
          }
        }
      }
      quadrant_sync();  // the exchange areas are written again
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (rank == 1 && threadIdx.x == 0) wait_bar_drain(ptx::smem_u32(drain), 0);  // rank 0's last arrival here
  __syncthreads();
  ptx::cluster_sync();  // the other CTA's products read this one's shared memory, its epilogue arrives here
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, 512);
  }
  if (threadIdx.x == 0) {
    p.hdr[1 + blockIdx.x] = *s_err;
    if (blockIdx.x == 0) p.hdr[0] = gridDim.x;
  }
}

// ============================================================================ plan and launch
bool plan_gate(GateParams& p, int sms) {
  p.pair = p.T > kGateClusterTokens && p.rule.E <= gate::kPairExperts && p.rule.topk <= gate::kTop;
  if (!p.pair) return false;
  p.bn = p.rule.E <= 256 ? (p.rule.E + 31) / 32 * 32 : 256;
  p.KB = (int32_t)((p.H + 63) / 64);
  const int stage = 128 * 128 + (p.rule.E <= 256 ? 1 : 2) * p.bn * 64;
  const int64_t tiles = (p.T + 255) / 256;
  // more stages where the selection's areas are free until the only tile's products are done (2048 tokens of 7168, 512
  // experts: two stages 117 us, four 95.6; 16384 of 2048, 256 experts: four 36.7, six 35.5)
  const int room = tiles <= sms / 2 ? gate::kBarOff : gate::kArena;
  p.n_stages = room / stage < gate::kMaxStages ? room / stage : gate::kMaxStages;
  p.grid = (int32_t)(2 * (tiles < sms / 2 ? tiles : sms / 2));
  return true;
}

cudaError_t launch_gate(const GateMaps& maps, const GateParams& p, cudaStream_t s) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.pair ? 2 : gate::kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  lc.stream = s;
  if (!p.pair) {
    // tokens per cluster: the fewest whose clusters all run at once (32 of 8 CTAs, two CTAs per SM).  H = 2048, 256
    // experts: 256 tokens 9.5 us in clusters of 8, 11.8 of 16; 512 tokens 12.4 of 16, 18.0 of 32 and of 8
    const int tiles = p.T <= 32 * 8 ? 1 : (p.T <= 32 * 16 ? 2 : 4);
    lc.gridDim = dim3((unsigned)((p.T + 8 * tiles - 1) / (8 * tiles) * gate::kCluster));
    const int threads = gate::cluster_threads(p.T, p.H, p.rule.E);
    lc.blockDim = dim3((unsigned)threads);
    auto kernel = threads == gate::kSmall ? gate_cluster_kernel<1, gate::kSmall> : gate_cluster_kernel<1, gate::kLarge>;
    const bool two = gate::cluster_groups(p.T, p.rule.E) == 2;
    if (tiles == 2) kernel = two ? gate_cluster_kernel<2, gate::kLarge, 2> : gate_cluster_kernel<2, gate::kLarge>;
    if (tiles == 4) kernel = two ? gate_cluster_kernel<4, gate::kLarge, 2> : gate_cluster_kernel<4, gate::kLarge>;
    return cudaLaunchKernelEx(&lc, kernel, p);
  }
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    for (auto k : {gate_pair_kernel<1>, gate_pair_kernel<2>})
      if (cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, gate::kPairSmem)) return e;
    configured_device = dev;
  }
  lc.gridDim = dim3((unsigned)p.grid);
  lc.blockDim = dim3(gate::kPairThreads);
  lc.dynamicSmemBytes = gate::kPairSmem;
  return cudaLaunchKernelEx(&lc, p.rule.E <= 256 ? gate_pair_kernel<1> : gate_pair_kernel<2>, maps, p);
}

}  // namespace gmmfr
