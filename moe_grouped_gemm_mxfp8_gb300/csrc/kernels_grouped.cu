// Products grouped by expert and the gradient of their weights (BF16 operands, FP32 sums).
//
//   rows of expert e, [start_e, end_e):  y[t] = W_e x[t]     (the gradient of the rows is the same product with W_e^T)
//                                        dW_e = sum over t of dy[t] x[t]^T
//
// Both are persistent over pairs of CTAs (tcgen05 cta_group::2, operands by TMA, accumulators double-buffered in TMEM).
// Neither wants its operands laid out first: tcgen05 takes a matrix whose rows run along K or along its other index, so
// W_e serves as it lies, [N, K] or [K, N], and the weights' gradient takes both of its operands "transposed".
//
//   rows     The weights are the 256-row operand, the expert's rows the other, 32 to 256 wide: an expert with few rows
//            streams its weights once and multiplies little beside them, one with many takes full tiles.
//   weights  A tile is 256 x 256 of dW_e, the sum runs over the expert's rows.  The last 64 rows of an expert are
//            loaded with what follows them: rows of the next expert, which may be infinite or NaN, so both operands'
//            rows past the end are overwritten with zeros in shared memory before the products.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "ops.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"
#include "row_tiles.h"

namespace gmmfr {
namespace grp {

constexpr int kAddThreads = 256;
constexpr int kThreads = 320;  // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue
constexpr int kBK = 64;        // K (or rows) per stage
constexpr int kTileBytes = 128 * 128;
constexpr int kChunk = 16;  // FP32 results: blocks of 64 to an accumulator, whose truncating sums are added in registers

// ---- rows
constexpr int kArena = 6 * 32768;
constexpr int kMaxStages = 10;
constexpr int kBarOff = kArena;                          // full, empty, accf[2], acce[2], drain
constexpr int kEndOff = kBarOff + (2 * kMaxStages + 5) * 8;
constexpr int kGbaseOff = kEndOff + 4 * kMaxExperts;     // int32 [1025]
constexpr int kScanOff = (kGbaseOff + 4 * (kMaxExperts + 1) + 7) / 8 * 8;
constexpr int kMiscOff = kScanOff + 8 * (kThreads / 32);
constexpr int kSmem = kMiscOff + 32 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

// ---- weights
constexpr int kGradStages = 6;
constexpr int kGradStage = 2 * kTileBytes;               // 64 rows of 128 columns of either operand
constexpr int kGradTurnOff = kGradStages * kGradStage;   // 4 KB for each of 8 epilogue warps
constexpr int kGradBarOff = kGradTurnOff + 8 * 4096;     // full, empty, landed, peer, accf[2], acce[2], drain
constexpr int kGradScanOff = kGradBarOff + (4 * kGradStages + 5) * 8;
constexpr int kGradMiscOff = kGradScanOff + 8 * (kThreads / 32);
constexpr int kGradSmem = kGradMiscOff + 32 + 1024;
static_assert(kGradSmem <= 232448 && kGradScanOff % 8 == 0, "shared memory budget, alignment");
// blocks of 64 rows to an accumulator where the result is BF16: what truncation takes off, 7.6e-6 of 8192 products, is a
// five-hundredth of its rounding
constexpr int kGradChunk = 128;

}  // namespace grp

namespace {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// end[e]: where expert e's rows end (they start where the expert before ends, the first one's at 0).  A list that
// decreases, is negative or leaves [0, M] sets kErrBadGroupList and is clamped.  Every thread calls it.
__device__ void grouped_ends(const int64_t* list, int type, int E, int64_t M, int32_t* end, int64_t* scratch, uint32_t* s_err) {
  int64_t carry = 0;
  for (int base = 0; base < E; base += grp::kThreads) {
    const int e = base + (int)threadIdx.x;
    const int64_t g = e < E ? list[e] : 0;
    int64_t v, tot;
    if (type == 1) {
      if (g < 0) atomicOr(s_err, kErrBadGroupList);
      v = cta_scan<false, grp::kThreads>(g < 0 ? 0 : (g > M ? M + 1 : g), scratch, tot) + carry;
      carry += tot;
    } else {
      const int64_t prev = e > 0 && e < E ? list[e - 1] : 0;
      if (e < E && (g < prev || g > M)) atomicOr(s_err, kErrBadGroupList);
      v = cta_scan<true, grp::kThreads>(g < 0 ? 0 : (g > M ? M : g), scratch, tot);
      v = v > carry ? v : carry;
      carry = tot > carry ? tot : carry;
    }
    if (e < E) end[e] = (int32_t)(v < M ? v : M);
  }
  if (type == 1 && threadIdx.x == 0 && carry > M) atomicOr(s_err, kErrBadGroupList);
  __syncthreads();
}

// The tiles of rows: expert e has ceil(rows / bn) of them, shared out by row_tile.
struct RowTiles {
  const int32_t *end, *gbase;
  int E, bn;
  // e is also a hint: the expert of an earlier tile, or 0
  __device__ void info(int g, int& e, int& t0, int& T) const {
    if (gbase[e + 1] <= g) {
      int lo = e + 1, hi = E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (gbase[mid] <= g) lo = mid;
        else hi = mid - 1;
      }
      e = lo;
    }
    const int start = e ? end[e - 1] : 0, rows = end[e] - start, n = gbase[e + 1] - gbase[e];
    row_tile(rows, n, g - gbase[e], t0, T);
    t0 += start;
  }
};

// The first tile of every expert, and bn, the width of the tiles, from the largest: 32, 64, 128 or 256.
__device__ int row_tiles(int E, const int32_t* s_end, int32_t* s_gbase, int64_t* scratch, int& bn) {
  int64_t most = 0, all;
  for (int e = threadIdx.x; e < E; e += grp::kThreads) most = max(most, (int64_t)s_end[e] - (e ? s_end[e - 1] : 0));
  cta_scan<true, grp::kThreads>(most, scratch, all);
  bn = all <= 32 ? 32 : (all <= 64 ? 64 : (all <= 128 ? 128 : 256));
  int64_t carry = 0;
  for (int base = 0; base < E; base += grp::kThreads) {
    const int e = base + (int)threadIdx.x;
    const int64_t rows = e < E ? s_end[e] - (e ? s_end[e - 1] : 0) : 0, n = (rows + bn - 1) / bn;
    int64_t tot;
    const int64_t incl = cta_scan<false, grp::kThreads>(n, scratch, tot) + carry;
    if (e < E) s_gbase[e] = (int32_t)(incl - n);
    carry += tot;
  }
  if (threadIdx.x == 0) s_gbase[E] = (int32_t)carry;
  __syncthreads();
  return (int)carry;
}

// A warp's 32 columns n.. of y by `count` rows m0.., lane l holding column n + l.
template <bool kF32>
__device__ __forceinline__ void store_columns(const GroupedParams& p, int64_t m0, int count, int64_t n, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  if constexpr (kF32) {
    if (n + lane >= p.N) return;
    float* o = static_cast<float*>(p.out) + m0 * p.ldo + n + lane;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < count) o[j * p.ldo] = v[j];
  } else if (p.vec_out) {
    // two lanes exchange, so that each has two columns of every other row
    const int odd = lane & 1;
    const bool mine = n + lane < p.N;  // N is even: both of a pair, or none
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (m0 + odd) * p.ldo + n + (lane & ~1);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
      const uint32_t two = odd ? pack_bf16(got, v[j + 1]) : pack_bf16(v[j], got);
      if (mine && j + odd < count) *reinterpret_cast<uint32_t*>(o + j * p.ldo) = two;
    }
  } else {
    if (n + lane >= p.N) return;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + m0 * p.ldo + n + lane;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < count) o[j * p.ldo] = __float2bfloat16_rn(v[j]);
  }
}

}  // namespace

// ============================================================================ rows
// Unit u is tile u / NT of the rows and tile u % NT of the columns; pair c takes the units c, c + pairs, ...
template <bool kTransW, bool kF32>
__global__ void __launch_bounds__(grp::kThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps maps, const __grid_constant__ GroupedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + grp::kBarOff);  // used in rank 0: both CTAs' loads
  uint64_t* empty = full + grp::kMaxStages;
  uint64_t* accf = empty + grp::kMaxStages;
  uint64_t* acce = accf + 2;  // used in rank 0: both CTAs' epilogue warps
  uint64_t* drain = acce + 2;
  int32_t* s_end = reinterpret_cast<int32_t*>(smem + grp::kEndOff);
  int32_t* s_gbase = reinterpret_cast<int32_t*>(smem + grp::kGbaseOff);
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + grp::kScanOff);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + grp::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&misc[0]);
  int* abort_flag = &misc[1];
  uint32_t* s_err = reinterpret_cast<uint32_t*>(&misc[2]);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const uint32_t rank = ptx::cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < grp::kMaxStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&accf[b]), 1 + p.test_stall);
      ptx::mbar_init(ptx::smem_u32(&acce[b]), 16);
    }
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    *abort_flag = 0;
    *s_err = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane < 5) ptx::prefetch_tensormap(lane == 4 ? &maps.w : &maps.x[lane]);
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  grouped_ends(p.group_list, p.group_list_type, p.E, p.M, s_end, s_scan, s_err);
  int bn;
  const int n_tiles = row_tiles(p.E, s_end, s_gbase, s_scan, bn);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Ctl ctl{abort_flag, s_err, p.timeout_ns};
  const uint32_t smem_base = ptx::smem_u32(smem);
  // a stage: 128 rows (columns of y) of the weights, then up to bn / 2 rows of x
  const int stage_bytes = grp::kTileBytes + bn * 64, n_stages = min(grp::kMaxStages, grp::kArena / stage_bytes);
  const int KB = p.KB, per = kF32 ? grp::kChunk : KB;  // blocks to an accumulator
  const int NT = (int)((p.N + 255) / 256);
  const RowTiles tiles{s_end, s_gbase, p.E, bn};
  const int64_t units = (int64_t)n_tiles * NT;
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;

  if (warp == 0) {
    const uint64_t pol_once = ptx::l2_evict_first_policy(), pol_keep = ptx::l2_evict_last_policy();
    const uint32_t full_own = ptx::smem_u32(full), full0 = ptx::map_to_rank(full_own, 0), empty0 = ptx::smem_u32(empty);
    int stage = 0, e = 0;
    uint32_t phase = 0, sb = smem_base;
    bool ok = true;
    for (int64_t u = first; ok && u < units; u += pairs) {
      const int g = (int)(u / NT), n0 = (int)(u - (int64_t)g * NT) * 256 + (int)rank * 128;
      int t0, T;
      tiles.info(g, e, t0, T);
      const int half = (T + 31) / 32 * 16, box = half <= 16 ? 0 : (half <= 32 ? 1 : (half <= 64 ? 2 : 3));
      const uint32_t tx = 2 * (grp::kTileBytes + (2048 << box));
      const uint64_t pol_w = s_gbase[e + 1] - s_gbase[e] > 1 ? pol_keep : pol_once;
      const int y = t0 + (int)rank * half;
      for (int kb = 0, x = 0; kb < KB; ++kb, x += grp::kBK) {
        if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
          ok = false;
          break;
        }
        if (ptx::elect_one()) {
          const uint32_t fb = full0 + 8 * stage;
          if (rank == 0) ptx::mbar_arrive_expect_tx(full_own + 8 * stage, tx);
          if constexpr (kTransW) {
            ptx::tma_load_3d_pair(sb, &maps.w, n0, x, e, fb, pol_w);
            ptx::tma_load_3d_pair(sb + 8192, &maps.w, n0 + 64, x, e, fb, pol_w);
          } else {
            ptx::tma_load_3d_pair(sb, &maps.w, x, n0, e, fb, pol_w);
          }
          ptx::tma_load_2d_pair(sb + grp::kTileBytes, &maps.x[box], x, y, fb, pol_keep);
        }
        sb += stage_bytes;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
          sb = smem_base;
        }
      }
    }
    // the last stages: released once their products are done, so that no load is in flight at exit
    for (int s = 0; ok && s < n_stages; ++s) {
      ok = warp_wait_quick(ptx::smem_u32(&empty[stage]), phase ^ 1, ctl);
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
      // kind::f16: FP32 accumulator, A and B BF16, M = 256; bit 15: A runs along M
      const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | (kTransW ? 1u << 15 : 0u) | ((256u >> 4) << 24);
      // A along M: 64 of its rows are a 128-byte row of a box (8 KB to the next 64), 16 K are 16 such rows
      const uint64_t da0 = ptx::smem_desc(smem_base, kTransW ? 8192 : 16, 1024, ptx::kSwizzle128B);
      const uint64_t db0 = ptx::smem_desc(smem_base + grp::kTileBytes, 16, 1024, ptx::kSwizzle128B);
      const uint32_t desc_hi = (uint32_t)(da0 >> 32), lo_step = (uint32_t)stage_bytes >> 4;
      constexpr uint32_t kStepA = kTransW ? 2048 >> 4 : 2;
      const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
      int stage = 0, e = 0, acc_i = 0;
      uint32_t phase = 0, la = (uint32_t)da0, lb = (uint32_t)db0;
      bool ok = true;
      for (int64_t u = first; ok && u < units; u += pairs) {
        int t0, T;
        tiles.info((int)(u / NT), e, t0, T);
        const uint32_t idesc = idesc0 | ((uint32_t)((T + 31) / 32 * 4) << 17);
        for (int k0 = 0; ok && k0 < KB; k0 += per) {
          const int n = min(per, KB - k0), buf = acc_i & 1;
          if (!__all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(&acce[buf]), ((acc_i >> 1) & 1) ^ 1, ctl))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d = tmem_base + buf * 256;
          for (int kb = 0; kb < n; ++kb) {
            if (!warp_wait_quick(full0 + 8 * stage, phase, ctl)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::tc_mma_f16_pair_lo(d, la + q * kStepA, lb + 2 * q, desc_hi, idesc, kb + q > 0 ? 1u : 0u);
              ptx::tc_commit_pair(empty0 + 8 * stage);
              if (kb == n - 1) ptx::tc_commit_pair(ptx::smem_u32(&accf[buf]));
            }
            la += lo_step;
            lb += lo_step;
            if (++stage == n_stages) {
              stage = 0;
              phase ^= 1;
              la = (uint32_t)da0;
              lb = (uint32_t)db0;
            }
          }
          ++acc_i;
        }
      }
      if (ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(drain));
      wait_bar_drain(ptx::smem_u32(drain), 0);
    }
    __syncwarp();
  } else {
    // two warps per TMEM lane quadrant, taking its 32-row chunks in turn
    const int q = warp & 3, half = (warp - 2) >> 2;
    if (p.zero_rest)
      for (int64_t r = (int64_t)s_end[p.E - 1] + blockIdx.x; r < p.M; r += gridDim.x)
        for (int64_t c = threadIdx.x - 64; c < p.N; c += 256) {
          if constexpr (kF32) static_cast<float*>(p.out)[r * p.ldo + c] = 0.f;
          else static_cast<__nv_bfloat16*>(p.out)[r * p.ldo + c] = __nv_bfloat16(0.f);
        }
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    int acc_i = 0, e = 0;
    auto wait_full = [&]() {
      const bool ok = warp_wait_quick(ptx::smem_u32(&accf[acc_i & 1]), (acc_i >> 1) & 1, ctl);
      ptx::tc_fence_after();
      return ok;
    };
    auto release = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote(ptx::map_to_rank(ptx::smem_u32(&acce[acc_i & 1]), 0));
      ++acc_i;
    };
    for (int64_t u = first; u < units; u += pairs) {
      const int g = (int)(u / NT);
      const int64_t n = (u - (int64_t)g * NT) * 256 + rank * 128 + q * 32;  // this warp's columns
      int t0, T;
      tiles.info(g, e, t0, T);
      if constexpr (!kF32) {
        if (!wait_full()) break;
        const uint32_t at = taddr + (acc_i & 1) * 256;
        int c0 = 32 * half;
        if (c0 >= T) release();
        for (; c0 < T; c0 += 64) {
          uint32_t r[32];
          float v[32];
          ptx::tmem_ld_32x32b_x32(at + c0, r);
          ptx::tmem_wait_ld();
          if (c0 + 64 >= T) release();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          store_columns<false>(p, t0 + c0, min(T - c0, 32), n, v);
        }
      } else {
        float sum[4][32] = {};
        bool ok = true;
        for (int kb = 0; kb < KB; kb += per) {
          ok = wait_full();
          if (!ok) break;
          const uint32_t at = taddr + (acc_i & 1) * 256;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c0 = 32 * half + 64 * i;
            if (c0 < T) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {  // 32 at a time would not fit in registers beside the sums
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(at + c0 + h, r);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[i][h + j] += __uint_as_float(r[j]);
              }
            }
          }
          release();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c0 = 32 * half + 64 * i;
          if (c0 < T) store_columns<true>(p, t0 + c0, min(T - c0, 32), n, sum[i]);
        }
      }
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

// ============================================================================ weights
// Unit u is tile u % (TA TB) of slice u / (TA TB): share s of expert e's rows is slice s E + e.  Pair c takes the units c,
// c + pairs, ...  Both CTAs' loads count on rank 0's barrier, but for an expert's last rows where their number is not a
// multiple of 16 (a product's K): these count on each CTA's own, its warp 1 puts zeros in place of the rows that follow, and
// rank 1's tells rank 0's.  (With that way for all rows, which takes some 500 cycles longer, 65536 rows of 64 experts,
// 2048 x 1024: 200 us.)
template <bool kF32>
__global__ void __launch_bounds__(grp::kThreads, 1)
    grouped_grad_kernel(const __grid_constant__ GroupedGradMaps maps, const __grid_constant__ GroupedGradParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + grp::kGradBarOff);  // used in rank 0: both CTAs' loads
  uint64_t* empty = full + grp::kGradStages;
  uint64_t* landed = empty + grp::kGradStages;  // last rows
  uint64_t* peer = landed + grp::kGradStages;   // used in rank 0: rank 1's last rows are ready
  uint64_t* accf = peer + grp::kGradStages;
  uint64_t* acce = accf + 2;  // used in rank 0: both CTAs' epilogue warps
  uint64_t* drain = acce + 2;
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + grp::kGradScanOff);
  int32_t* misc = reinterpret_cast<int32_t*>(smem + grp::kGradMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&misc[0]);
  int* abort_flag = &misc[1];
  uint32_t* s_err = reinterpret_cast<uint32_t*>(&misc[2]);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const uint32_t rank = ptx::cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < grp::kGradStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&landed[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&peer[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&accf[b]), 1 + p.test_stall);
      ptx::mbar_init(ptx::smem_u32(&acce[b]), 16);
    }
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    *abort_flag = 0;
    *s_err = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane < 3) ptx::prefetch_tensormap(lane == 0 ? &maps.a : (lane == 1 ? &maps.b : &maps.out));
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __syncthreads();
  // Where the experts' rows end, in global memory, each CTA's copy by itself: the sixth stage takes the room for 1024 of them
  // (65536 rows of 64 experts, 2048 x 1024: 178 us with five stages, 169 with six).
  int32_t* ends = p.ends + (int64_t)blockIdx.x * p.E;
  grouped_ends(p.group_list, p.group_list_type, p.E, p.M, ends, s_scan, s_err);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Ctl ctl{abort_flag, s_err, p.timeout_ns};
  const uint32_t smem_base = ptx::smem_u32(smem);
  const int TA = (int)((p.A + 255) / 256), TB = (int)((p.B + 255) / 256), TT = TA * TB;
  const int64_t units = (int64_t)p.E * p.shares * TT;
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
  constexpr int kPer = kF32 ? grp::kChunk : grp::kGradChunk;  // blocks to an accumulator
  auto unit_at = [&](int64_t u, int& e, int& ta, int& tb) {
    e = (int)(u / TT);
    const int r = (int)(u - (int64_t)e * TT);
    ta = r / TB;
    tb = r - ta * TB;
  };
  auto rows_of = [&](int slice, int& start) {
    const int share = p.shares > 1 ? slice / p.E : 0, e = slice - share * p.E;
    start = e ? ends[e - 1] : 0;
    const int rows = ends[e] - start;
    if (p.shares == 1) return rows;
    const int64_t blocks = (rows + grp::kBK - 1) / grp::kBK;
    const int r0 = (int)(blocks * share / p.shares * grp::kBK);
    start += r0;
    return (int)min((int64_t)rows, blocks * (share + 1) / p.shares * grp::kBK) - r0;
  };

  if (warp == 0) {
    const uint64_t pol = ptx::l2_evict_last_policy();
    const uint32_t full_own = ptx::smem_u32(full), full0 = ptx::map_to_rank(full_own, 0), landed0 = ptx::smem_u32(landed),
                   empty0 = ptx::smem_u32(empty);
    int stage = 0;
    uint32_t phase = 0, sb = smem_base;
    bool ok = true;
    for (int64_t u = first; ok && u < units; u += pairs) {
      int e, ta, tb, start;
      unit_at(u, e, ta, tb);
      const int rows = rows_of(e, start);
      const int xa = ta * 256 + (int)rank * 128, xb = tb * 256 + (int)rank * 128;
      for (int r = 0; r < rows; r += grp::kBK) {
        if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
          ok = false;
          break;
        }
        if (ptx::elect_one()) {
          const bool last = rows - r < grp::kBK && rows % 16;
          auto load = [&](auto copy, uint32_t bar) {
            copy(sb, &maps.a, xa, start + r, bar, pol);
            copy(sb + 8192, &maps.a, xa + 64, start + r, bar, pol);
            copy(sb + grp::kTileBytes, &maps.b, xb, start + r, bar, pol);
            copy(sb + grp::kTileBytes + 8192, &maps.b, xb + 64, start + r, bar, pol);
          };
          if (last) {
            ptx::mbar_arrive_expect_tx(landed0 + 8 * stage, grp::kGradStage);
            load([](auto... a) { ptx::tma_load_2d(a...); }, landed0 + 8 * stage);
          } else {
            if (rank == 0) ptx::mbar_arrive_expect_tx(full_own + 8 * stage, 2 * grp::kGradStage);
            load([](auto... a) { ptx::tma_load_2d_pair(a...); }, full0 + 8 * stage);
          }
        }
        sb += grp::kGradStage;
        if (++stage == grp::kGradStages) {
          stage = 0;
          phase ^= 1;
          sb = smem_base;
        }
      }
    }
    for (int s = 0; ok && s < grp::kGradStages; ++s) {  // no load is in flight at exit
      ok = warp_wait_quick(ptx::smem_u32(&empty[stage]), phase ^ 1, ctl);
      if (++stage == grp::kGradStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) let_loads_land();  // aborted
    __syncwarp();
  } else if (warp == 1) {
    // kind::f16: FP32 accumulator, A and B BF16, M = N = 256; bits 15, 16: A and B run along M and N
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (3u << 15) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
    const uint64_t da0 = ptx::smem_desc(smem_base, 8192, 1024, ptx::kSwizzle128B);
    const uint32_t desc_hi = (uint32_t)(da0 >> 32);
    const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty), landed0 = ptx::smem_u32(landed),
                   peer0 = ptx::smem_u32(peer);
    int stage = 0, acc_i = 0;
    uint32_t full_bits = 0, landed_bits = 0, peer_bits = 0;  // a barrier's phase by its own uses
    bool ok = true;
    // an expert's last rows, when they have landed: zeros up to the next 16 in each box of 64 columns
    auto end_rows = [&](int valid) {
      if (!warp_wait_quick(landed0 + 8 * stage, landed_bits >> stage & 1, ctl)) return false;
      landed_bits ^= 1u << stage;
      uint8_t* at = smem + stage * grp::kGradStage + (lane >> 3) * 8192 + (lane & 7) * 16;
      for (int r = valid; r & 15; ++r) *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0, 0, 0, 0);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      return true;
    };
    for (int64_t u = first; ok && u < units; u += pairs) {
      int e, ta, tb, start;
      unit_at(u, e, ta, tb);
      const int rows = rows_of(e, start), blocks = (rows + grp::kBK - 1) / grp::kBK;
      if (rank == 1) {
        if (rows % 16) {
          stage = (stage + blocks - 1) % grp::kGradStages;
          if (!(ok = end_rows(rows - (blocks - 1) * grp::kBK))) break;
          if (lane == 0) ptx::mbar_arrive_remote(ptx::map_to_rank(peer0 + 8 * stage, 0));
          stage = (stage + 1) % grp::kGradStages;
        } else {
          stage = (stage + blocks) % grp::kGradStages;
        }
        continue;
      }
      for (int k0 = 0; ok && k0 < blocks; k0 += kPer) {
        const int n = min(kPer, blocks - k0), buf = acc_i & 1;
        if (!__all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(&acce[buf]), ((acc_i >> 1) & 1) ^ 1, ctl))) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + buf * 256;
        for (int kb = 0; kb < n; ++kb) {
          const int valid = min(grp::kBK, rows - (k0 + kb) * grp::kBK);
          if (valid & 15) {
            ok = end_rows(valid) && __all_sync(0xffffffffu, wait_bar_cluster(peer0 + 8 * stage, peer_bits >> stage & 1, ctl));
            peer_bits ^= 1u << stage;
          } else {
            ok = warp_wait_quick(full0 + 8 * stage, full_bits >> stage & 1, ctl);
            full_bits ^= 1u << stage;
          }
          if (!ok) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint32_t la = (uint32_t)da0 + stage * (grp::kGradStage >> 4), lb = la + (grp::kTileBytes >> 4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (16 * q < valid)
                ptx::tc_mma_f16_pair_lo(d, la + q * (2048 >> 4), lb + q * (2048 >> 4), desc_hi, idesc, kb + q > 0 ? 1u : 0u);
            ptx::tc_commit_pair(empty0 + 8 * stage);
            if (kb == n - 1) ptx::tc_commit_pair(ptx::smem_u32(&accf[buf]));
          }
          if (++stage == grp::kGradStages) stage = 0;
        }
        ++acc_i;
      }
    }
    if (rank == 0) {
      if (ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(drain));
      wait_bar_drain(ptx::smem_u32(drain), 0);
    }
    __syncwarp();
  } else {
    // two warps per TMEM lane quadrant, 128 columns each
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + half * 128;
    uint8_t* turn = smem + grp::kGradTurnOff + (warp - 2) * 4096;
    const uint32_t turn_at = ptx::smem_u32(turn);
    int acc_i = 0;
    for (int64_t u = first; u < units; u += pairs) {
      int e, ta, tb, start;
      unit_at(u, e, ta, tb);
      const int rows = rows_of(e, start), blocks = (rows + grp::kBK - 1) / grp::kBK;
      float sum[4][32];
      // One accumulator's sums are the tile's, read in whole: 413 rows to each of 24 experts of 5120 x 1288 137 -> 130 us.  With one
      // or two blocks the writes bound it, and go better as the chunks come (16 rows to each of 256, 2048 x 1024: 180, 192).
      const bool alone = blocks > 2 && blocks <= kPer;
      if (!alone) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.f;
      }
      bool ok = true;
      for (int k0 = 0; k0 < blocks; k0 += kPer) {
        ok = warp_wait_quick(ptx::smem_u32(&accf[acc_i & 1]), (acc_i >> 1) & 1, ctl);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t at = taddr + (acc_i & 1) * 256;
        if (alone) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ptx::tmem_ld_32x32b_x32(at + 32 * i, reinterpret_cast<uint32_t(&)[32]>(sum[i]));
          ptx::tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 32; h += 16) {  // 32 at a time would not fit in registers beside the sums
              uint32_t r[16];
              ptx::tmem_ld_32x32b_x16(at + 32 * i + h, r);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[i][h + j] += __uint_as_float(r[j]);
            }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(ptx::map_to_rank(ptx::smem_u32(&acce[acc_i & 1]), 0));
        ++acc_i;
      }
      if (!ok) break;
      if (p.accumulate && rows == 0) continue;
      const int ya = ta * 256 + (int)rank * 128 + q * 32;
      if (ya >= p.A) continue;
      // boxes of 32 rows of 128 bytes, their 16-byte pieces in the map's order (piece c of row r at c ^ (r & 7))
      constexpr int kBoxes = kF32 ? 4 : 2, kBoxCols = 128 / kBoxes;
#pragma unroll
      for (int b = 0; b < kBoxes; ++b) {
        const int xb = tb * 256 + half * 128 + b * kBoxCols;
        if (xb >= p.B) break;
        if (ptx::elect_one()) ptx::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint4 v;
          if constexpr (kF32) {
            const float* s = &sum[b][4 * c];
            v = make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]), __float_as_uint(s[3]));
          } else {
            const float* s = &sum[2 * b + c / 4][8 * (c & 3)];
            v = make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7]));
          }
          *reinterpret_cast<uint4*>(turn + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (ptx::elect_one()) {
          if (kF32 && p.accumulate) ptx::tma_add_3d(&maps.out, xb, ya, e, turn_at);
          else ptx::tma_store_3d(&maps.out, xb, ya, e, turn_at);
          ptx::bulk_commit();
        }
      }
    }
    if (ptx::elect_one()) ptx::bulk_wait();
    __syncwarp();
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

// The shares' sums of the weights' gradient, added in their order
__global__ void __launch_bounds__(grp::kAddThreads) add_shares_kernel(const __grid_constant__ GroupedGradParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int64_t pieces = p.E * p.A * p.B / 8;  // of 8 numbers: rows are multiples of 8
  for (int64_t i = (int64_t)blockIdx.x * grp::kAddThreads + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * grp::kAddThreads) {
    const float4* at = reinterpret_cast<const float4*>(p.parts) + 2 * i;
    float4 v[2] = {};
#pragma unroll 4
    for (int s = 0; s < p.shares; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = at[2 * pieces * s + h];
        v[h] = make_float4(v[h].x + w.x, v[h].y + w.y, v[h].z + w.z, v[h].w + w.w);
      }
    }
    if (p.out_f32) {
      float4* to = static_cast<float4*>(p.out) + 2 * i;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (p.accumulate) {
          const float4 w = to[h];
          v[h] = make_float4(w.x + v[h].x, w.y + v[h].y, w.z + v[h].z, w.w + v[h].w);
        }
        to[h] = v[h];
      }
    } else {
      static_cast<uint4*>(p.out)[i] = make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[0].z, v[0].w), pack_bf16(v[1].x, v[1].y),
                                                 pack_bf16(v[1].z, v[1].w));
    }
  }
}

// ============================================================================ launch
template <auto kKernel, int kSmem, typename Maps, typename Params>
static cudaError_t launch_pairs(const Maps& maps, const Params& p, int64_t units, int sms, cudaStream_t s) {
  static std::atomic<int> configured_device{-1};
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device.load(std::memory_order_relaxed) != dev) {
    cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured_device.store(dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(2 * std::max<int64_t>(1, std::min<int64_t>(sms / 2, units))));
  lc.blockDim = dim3(grp::kThreads);
  lc.dynamicSmemBytes = kSmem;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 2;
  return cudaLaunchKernelEx(&lc, kKernel, maps, p);
}

cudaError_t launch_grouped(const GroupedMaps& maps, const GroupedParams& p, bool transposed, int sms, cudaStream_t s) {
  // the experts' sizes are on the device: at most this many tiles
  const int64_t units = (std::min<int64_t>(p.E, p.M) + p.M / 32) * ((p.N + 255) / 256);
  if (transposed) {
    if (p.out_f32) return launch_pairs<grouped_kernel<true, true>, grp::kSmem>(maps, p, units, sms, s);
    return launch_pairs<grouped_kernel<true, false>, grp::kSmem>(maps, p, units, sms, s);
  }
  if (p.out_f32) return launch_pairs<grouped_kernel<false, true>, grp::kSmem>(maps, p, units, sms, s);
  return launch_pairs<grouped_kernel<false, false>, grp::kSmem>(maps, p, units, sms, s);
}

// Where the experts' tiles leave half of the pairs idle or more, shares of their rows take these, of 512 on average if there are
// three of them.  One expert of 136 x 200 and 16384 rows 94 us, in shares 15.4; of 392 x 648 and 22395 rows 127, 26.4; eight of
// 512 x 512 and 65536 rows 40.7, 35.7, with all rows in one 274, 148.  The second launch and the parts' way cost 1 to 2 us: 1024
// rows of 256 x 256 9.6, in two shares 10.6; 2048 rows 13.7, in four 10.6.  Shares of 256: 18.8 for the first.
int grouped_grad_shares(int64_t M, int64_t A, int64_t B, int64_t E, int sms) {
  const int64_t tiles = E * ((A + 255) / 256) * ((B + 255) / 256), wanted = M / E / 512;
  return wanted < 3 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(sms / 2 / tiles, wanted));
}

int grouped_grad_ctas(int64_t A, int64_t B, int64_t slices, int sms) {
  return (int)(2 * std::min<int64_t>(sms / 2, slices * ((A + 255) / 256) * ((B + 255) / 256)));
}

cudaError_t launch_grouped_grad(const GroupedGradMaps& maps, const GroupedGradParams& p, int sms, cudaStream_t s) {
  const int64_t units = grouped_grad_ctas(p.A, p.B, (int64_t)p.E * p.shares, sms) / 2;
  if (p.shares > 1) {
    GroupedGradParams q = p;
    q.accumulate = 0;
    cudaError_t e = launch_pairs<grouped_grad_kernel<true>, grp::kGradSmem>(maps, q, units, sms, s);
    if (e != cudaSuccess) return e;
    const int64_t pieces = p.E * p.A * p.B / 8;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)std::min<int64_t>((pieces + grp::kAddThreads - 1) / grp::kAddThreads, 4 * sms));
    lc.blockDim = dim3(grp::kAddThreads);
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, add_shares_kernel, p);
  }
  if (p.out_f32) return launch_pairs<grouped_grad_kernel<true>, grp::kGradSmem>(maps, p, units, sms, s);
  return launch_pairs<grouped_grad_kernel<false>, grp::kGradSmem>(maps, p, units, sms, s);
}

}  // namespace gmmfr
