// The dense product with low-rank adapters of many requests (forms: linear_forms.cuh, with kLora), and the sums that it
// starts from: s[t] = scale_a (A_a x[t]) for the adapter a of row t.
//
// The sums read r (16, say) rows of K for every adapter in use, and the rows of x.
//   few   up to 128 rows: each adapter's rows gathered, so that every factor is read once and all of them are on their way at
//         once.  Products by mma.sync, 16 bytes of a row at a time from global memory straight into a lane's operand
//         registers: they wait for memory, and an adapter has a few rows.
//   many  128 rows of x at a time, by TMA and tcgen05: the rows are one operand, 16 ranks of up to 8 of their adapters'
//         factors the other; of what comes out a row keeps its own adapter's columns.
// Several CTAs share a K range.  CTAs also list the adapters of each 256 rows.  The product's launch follows
// at once and begins with its weights; only its adapters wait.
#include "linear_forms.cuh"

namespace gmmfr {
namespace lora {
constexpr int kFewThreads = 512;
constexpr int kTileThreads = 448, kTileStages = 10, kTileArena = 10 * (lin::kTileBytes + 2048);
constexpr int kPass = 8;  // units of a pass
constexpr int kChunk = 16;  // FP32 results: blocks of 64 to an accumulator, as the dense product's
}  // namespace lora

namespace {

// Lane l's 16 bytes at k of rows l / 4 + 8 i of x, and of kRt times 16 rows of a factor (rows from `left` on repeat the last
// one; what they give is not stored).  in: whether k is in the warp's share; zeros otherwise.  All loads are made, at 0 where
// k is not, so that they are in flight together.
template <int kTiles, int kRt>
struct SumOperands {
  uint4 w[kRt][2], x[kTiles];
  __device__ __forceinline__ void load(const __nv_bfloat16* a, int left, int64_t K, const __nv_bfloat16* const (&xr)[kTiles], int64_t k,
                                       bool in) {
    const int row = (threadIdx.x & 31) >> 2;
    const int64_t at = in ? k : 0;
#pragma unroll
    for (int i = 0; i < kRt; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[i][h] = ptx::ld_nc_v4(a + min(16 * i + 8 * h + row, left - 1) * K + at);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) x[i] = ptx::ld_nc_v4(xr[i] + at);
  }
  __device__ __forceinline__ void keep(bool in) {
    auto zero = [&](uint4& v) {
      if (!in) v = make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < kRt; ++i) zero(w[i][0]), zero(w[i][1]);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) zero(x[i]);
  }
  __device__ __forceinline__ void multiply(float (&acc)[kTiles][kRt][4]) const {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < kRt; ++j) {
        ptx::mma_16816(acc[i][j], w[j][0].x, w[j][1].x, w[j][0].y, w[j][1].y, x[i].x, x[i].y);
        ptx::mma_16816(acc[i][j], w[j][0].z, w[j][1].z, w[j][0].w, w[j][1].w, x[i].z, x[i].w);
      }
  }
};

// Whether this thread's row is the first with its adapter among `rows` rows (of which it has number tid; id -1: none)
__device__ __forceinline__ bool first_of(const int* s_id, int tid, int id) {
  bool first = id >= 0;
  for (int j = 0; j < tid && first; j += 4) {
    const int4 v = *reinterpret_cast<const int4*>(&s_id[j]);
    first &= v.x != id && (v.y != id || j + 1 >= tid) && (v.z != id || j + 2 >= tid) && (v.w != id || j + 3 >= tid);
  }
  return first;
}

__device__ __forceinline__ int adapter_at(const LoraParams& p, int64_t m) {
  const int id = m < p.M ? p.ids[m] : -1;
  return (uint32_t)id < (uint32_t)p.count ? id : -1;
}

// The list of rows 256 block and up, by kT threads (of which this one is `t`) that share barrier 1.
template <int kT>
__device__ void list_adapters(const LoraParams& p, int64_t block, int t) {
  constexpr int kPer = kT < 256 ? 256 / kT : 1;  // rows of the list for each thread
  __shared__ __align__(16) int l_id[256];
  __shared__ uint32_t l_first[8];
  const int lane = t & 31;
  int id[kPer];
  uint32_t firsts[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    id[k] = t < 256 ? adapter_at(p, block * 256 + k * kT + t) : -1;
    if (t < 256) l_id[k * kT + t] = id[k];
  }
  ptx::bar_sync(1, kT);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    firsts[k] = __ballot_sync(0xffffffffu, first_of(l_id, k * kT + t, id[k]));  // (nothing past 256: id -1)
    if (lane == 0 && t < 256) l_first[(k * kT + t) >> 5] = firsts[k];
  }
  ptx::bar_sync(1, kT);
  int32_t* list = p.lists + block * kLoraListInts;
  int n = 0;
  for (int w = 0; w < 8; ++w) n += __popc(l_first[w]);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    int at = __popc(firsts[k] & ((1u << lane) - 1));
    for (int w = 0; w < min((k * kT + t) >> 5, 8); ++w) at += __popc(l_first[w]);
    if (firsts[k] >> lane & 1) list[4 + at] = id[k];
  }
  if (t == 0) list[0] = n;
}

}  // namespace

// ============================================================================ few rows
// CTA (d, r, c): the d-th adapter in the order of the rows, ranks 16 r and up, share c of the K range (more than one where a
// warp's loads would not all be on their way at once); where there are fewer adapters than places for them, several places
// share an adapter's rows.  The last CTA lists.
__global__ void __launch_bounds__(lora::kFewThreads, 1) lora_sums_few_kernel(const __grid_constant__ LoraParams p) {
  constexpr int kU = 8, kWarps = lora::kFewThreads / 32;
  __shared__ __align__(16) int s_id[kLoraFewRows];
  __shared__ uint32_t s_first[4];
  __shared__ int s_row[kLoraFewRows];
  __shared__ __align__(16) float part[8 * kWarps][16];
  static_assert(8 * kWarps >= kLoraFewRows, "a slot for each row");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rc = (p.rank + 15) / 16, places = (int)min(p.M, (int64_t)p.count), items = places * rc * p.split;
  // the launch after this one reads x and its weights without waiting for this one: it may start when all before has ended
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (blockIdx.x >= items) {
    list_adapters<lora::kFewThreads>(p, 0, tid);
    return;
  }
  int id = -1;
  if (tid < kLoraFewRows) s_id[tid] = id = adapter_at(p, tid);
  __syncthreads();
  if (tid < kLoraFewRows) {
    const uint32_t b = __ballot_sync(0xffffffffu, first_of(s_id, tid, id));
    if (lane == 0) s_first[warp] = b;
  }
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) n += __popc(s_first[w]);
  const int c = blockIdx.x % p.split, place = blockIdx.x / p.split / rc, r0 = blockIdx.x / p.split % rc * 16;
  const int shares = n ? places / n : 0;  // of an adapter's rows
  if (place >= n * shares) return;
  const int share = place / n;
  int a = -1;
  {
    int skip = place % n;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t b = s_first[w];
      const int here = __popc(b);
      if (a < 0 && skip < here) {
        for (int i = 0; i < skip; ++i) b &= b - 1;
        a = s_id[32 * w + __ffs(b) - 1];
      }
      skip -= here;
    }
  }
  int rows = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t mine = __ballot_sync(0xffffffffu, s_id[32 * w + lane] == a);
    if (w == warp && mine >> lane & 1) s_row[rows + __popc(mine & ((1u << lane) - 1))] = tid;
    rows += __popc(mine);
  }
  __syncthreads();
  // the warps share the tiles of 8 rows, and the K range where the tiles are fewer
  const int all = (rows + 7) / 8, tile0 = all * share / shares, tiles = all * (share + 1) / shares - tile0;
  int sharing = 1;
  while (sharing < tiles) sharing *= 2;
  const int splits = kWarps / sharing, split = warp % splits, t = warp / splits;
  const int blocks = (int)((p.K + 31) / 32), b_begin = blocks * c / p.split, b_end = blocks * (c + 1) / p.split;
  if (t < tiles) {
    const __nv_bfloat16* ar = p.a + ((int64_t)a * p.rank + r0) * p.K;
    const __nv_bfloat16* const xr[1] = {p.x + (int64_t)s_row[min((tile0 + t) * 8 + (lane >> 2), rows - 1)] * p.ldx};
    float acc[1][1][4] = {}, sum[4] = {};
    for (int b0 = b_begin + split; b0 < b_end; b0 += splits * kU) {
      SumOperands<1, 1> o[kU];
#pragma unroll
      for (int v = 0; v < kU; ++v) {
        const int64_t k = (int64_t)(b0 + splits * v) * 32 + (lane & 3) * 8;
        o[v].load(ar, p.rank - r0, p.K, xr, k, b0 + splits * v < b_end && k < p.K);
      }
#pragma unroll
      for (int v = 0; v < kU; ++v) {
        o[v].keep(b0 + splits * v < b_end && (int64_t)(b0 + splits * v) * 32 + (lane & 3) * 8 < p.K);
        o[v].multiply(acc);
      }
      if (p.precise) {  // the tensor core adds 256 products, truncating; those sums are added to nearest
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i] += acc[0][0][i];
          acc[0][0][i] = 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      part[(split * tiles + t) * 8 + (lane & 3) * 2 + (i & 1)][8 * (i >> 1) + (lane >> 2)] = p.precise ? sum[i] : acc[0][0][i];
  }
  __syncthreads();
  // the splits' parts in order
  const float scale = p.scale ? p.scale[a] : 1.f;
  const float4* sums = reinterpret_cast<const float4*>(&part[0][0]);
  for (int i = tid; i < tiles * 32; i += lora::kFewThreads) {
    const int row = tile0 * 8 + i / 4, r = r0 + i % 4 * 4;
    if (row >= rows || r >= p.rank) continue;
    float4 v = sums[i];
    for (int s = 1; s < splits; ++s) {
      const float4 z = sums[s * tiles * 32 + i];
      v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
    }
    *reinterpret_cast<float4*>(p.s + (c * p.M + s_row[row]) * p.rank + r) = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
  }
}

// ============================================================================ many rows
// A tile is 128 rows; its items are passes over up to 8 units (16 ranks of an adapter) in shares of K, which its CTAs take in
// turn: how many adapters a tile has is known here only.  Who reads the sums adds the shares' parts.  (Clusters that join them
// on the chip wait for SMs that lie together: 16 us more with clusters of 8.)  With passes given out by what all adapters
// would need, 2048 rows of 4096 x 4096 and one, 16, 32 of 64 adapters took 51.6, 88.9, 101 us with the product; so 47.9, 67.0,
// 89.1.  Passes of 16: 47.9, 73.3, 87.1; 300 rows of 16 adapters of rank 64: 50.6, of 8: 43.7.  Up to 8 shares: 27.9 for one of
// them, 4: 22.8 (their reader adds the parts).
// Warp 0 TMA, warp 1 MMA, warps 2..5 epilogue, warps 6..13 lists.
template <bool kPrecise>
__global__ void __launch_bounds__(lora::kTileThreads, 1)
    lora_sums_many_kernel(const __grid_constant__ LoraMaps maps, const __grid_constant__ LoraParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[lora::kTileStages], empty[lora::kTileStages], accf[2], acce[2], drain;
  __shared__ __align__(16) int s_id[128];
  __shared__ int s_list[128];
  __shared__ uint32_t s_first[4], tmem_slot, s_err;
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // warp: uniform
  const int C = p.split, first = blockIdx.x % p.tile_ctas;
  const int64_t row0 = (int64_t)(blockIdx.x / p.tile_ctas) * 128;
  if (tid == 0) {
    for (int s = 0; s < lora::kTileStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&accf[b]), 1 + p.test_stall);
      ptx::mbar_init(ptx::smem_u32(&acce[b]), 4);
    }
    ptx::mbar_init(ptx::smem_u32(&drain), 1);
    abort_flag = 0;
    s_err = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane < 2) ptx::prefetch_tensormap(lane ? &maps.a : &maps.x);
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int id = -1;
  if (tid < 128) s_id[tid] = id = adapter_at(p, row0 + tid);
  __syncthreads();
  if (tid < 128) {
    const uint32_t b = __ballot_sync(0xffffffffu, first_of(s_id, tid, id));
    if (lane == 0) s_first[warp] = b;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  int n = 0;
  for (int w = 0; w < 4; ++w) {
    if (tid >> 5 == w && s_first[w] >> lane & 1) s_list[n + __popc(s_first[w] & ((1u << lane) - 1))] = id;
    n += __popc(s_first[w]);
  }
  __syncthreads();
  const uint32_t tmem_base = tmem_slot, smem_base = ptx::smem_u32(smem);
  const Ctl ctl{&abort_flag, &s_err, p.timeout_ns};
  const int rc = (p.rank + 15) / 16, units = n * rc;  // unit u: adapter u / rc, ranks 16 (u % rc) and up
  const int stage_bytes = lin::kTileBytes + min(units, lora::kPass) * 2048, n_stages = min(lora::kTileStages, lora::kTileArena / stage_bytes);
  // item i: the units from kPass (i / C) on, share i % C of the K blocks
  const int KB = (int)((p.K + 63) / 64), items = (units + lora::kPass - 1) / lora::kPass * C;
  auto item = [&](int i, int& u0, int& kb0, int& kb1) {
    u0 = i / C * lora::kPass;
    kb0 = (int)((int64_t)KB * (i % C) / C);
    kb1 = (int)((int64_t)KB * (i % C + 1) / C);
  };
  // where the accumulator of blocks kb and up ends; FP32 results: who reads them adds those of a longer share up, to nearest
  auto end_of = [&](int kb, int kb1) { return kPrecise ? min(kb + lora::kChunk, kb1) : kb1; };

  if (warp == 0) {
    const uint64_t pol = ptx::l2_evict_last_policy();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = first; ok && i < items; i += p.tile_ctas) {
      int u0, kb0, kb1;
      item(i, u0, kb0, kb1);
      const int m = min(lora::kPass, units - u0);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait_quick(ptx::smem_u32(&empty[stage]), phase ^ 1, ctl)) {
          ok = false;
          break;
        }
        if (ptx::elect_one()) {
          const uint32_t fb = ptx::smem_u32(&full[stage]), sb = smem_base + stage * stage_bytes;
          ptx::mbar_arrive_expect_tx(fb, lin::kTileBytes + m * 2048);
          ptx::tma_load_2d(sb, &maps.x, kb * 64, (int)row0, fb, pol);
          for (int u = 0; u < m; ++u)
            ptx::tma_load_3d(sb + lin::kTileBytes + u * 2048, &maps.a, kb * 64, (u0 + u) % rc * 16, s_list[(u0 + u) / rc], fb, pol);
        }
        __syncwarp();
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    for (int s = 0; ok && s < n_stages; ++s) {  // no load is in flight at exit
      ok = warp_wait_quick(ptx::smem_u32(&empty[stage]), phase ^ 1, ctl);
      if (++stage == n_stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok)  // aborted: let what is in flight land
      for (int s = 0; s < n_stages; ++s) wait_bar_drain(ptx::smem_u32(&full[s]), s < stage ? phase : phase ^ 1);
    __syncwarp();
  } else if (warp == 1) {
    const uint64_t da0 = ptx::smem_desc(smem_base, 16, 1024, ptx::kSwizzle128B);
    const uint32_t desc_hi = (uint32_t)(da0 >> 32);
    int stage = 0, acc_i = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = first; ok && i < items; i += p.tile_ctas) {
      int u0, kb0, kb1;
      item(i, u0, kb0, kb1);
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)min(lora::kPass, units - u0) << 18) | ((128u >> 4) << 24);
      for (int c0 = kb0, c1; ok && c0 < kb1; c0 = c1, ++acc_i) {
        const int buf = acc_i & 1;
        c1 = end_of(c0, kb1);
        if (!(ok = warp_wait_quick(ptx::smem_u32(&acce[buf]), ((acc_i >> 1) & 1) ^ 1, ctl))) break;
        ptx::tc_fence_after();
        for (int kb = c0; kb < c1; ++kb) {
          if (!(ok = warp_wait_quick(ptx::smem_u32(&full[stage]), phase, ctl))) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint32_t la = (uint32_t)da0 + stage * (stage_bytes >> 4), lb = la + (lin::kTileBytes >> 4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              ptx::tc_mma_f16_lo(tmem_base + buf * 256, la + 2 * q, lb + 2 * q, desc_hi, idesc, kb > c0 || q > 0 ? 1u : 0u);
            ptx::tc_commit(ptx::smem_u32(&empty[stage]));
            if (kb == c1 - 1) ptx::tc_commit(ptx::smem_u32(&accf[buf]));
          }
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (ptx::elect_one()) ptx::tc_commit(ptx::smem_u32(&drain));
    wait_bar_drain(ptx::smem_u32(&drain), 0);
    __syncwarp();
  } else if (warp >= 6) {
    if (blockIdx.x < (p.M + 255) / 256) list_adapters<256>(p, blockIdx.x, tid - 192);
  } else {
    const int q = warp & 3, row = q * 32 + lane, mine = s_id[row];
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    const float scale = mine >= 0 && p.scale ? p.scale[mine] : 1.f;
    int acc_i = 0;
    bool ok = true;
    for (int i = first; ok && i < items; i += p.tile_ctas) {
      int u0, kb0, kb1;
      item(i, u0, kb0, kb1);
      float* to = p.s + (i % C * p.M + row0 + row) * p.rank;
      for (int c0 = kb0; c0 < kb1; c0 = end_of(c0, kb1), ++acc_i) {
        const int buf = acc_i & 1;
        if (!(ok = warp_wait_quick(ptx::smem_u32(&accf[buf]), (acc_i >> 1) & 1, ctl))) break;
        ptx::tc_fence_after();
        // (the addition in a copy of its own, not beside the plain store: 777 rows of 32 adapters 48.0 -> 46.6 us)
        auto store = [&](auto more) {
          for (int u = u0; u < min(u0 + lora::kPass, units); ++u) {
            const bool own = mine == s_list[u / rc];
            if (!__any_sync(0xffffffffu, own)) continue;
            uint32_t v[16];
            ptx::tmem_ld_32x32b_x16(taddr + buf * 256 + (u - u0) * 16, v);
            ptx::tmem_wait_ld();
            const int r0 = u % rc * 16;
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              if (own && r0 + j < p.rank) {
                float4 s = make_float4(__uint_as_float(v[j]) * scale, __uint_as_float(v[j + 1]) * scale,
                                       __uint_as_float(v[j + 2]) * scale, __uint_as_float(v[j + 3]) * scale);
                float4* at = reinterpret_cast<float4*>(to + r0 + j);
                if constexpr (decltype(more)::value) {  // to what this thread wrote there
                  const float4 w = *at;
                  s = make_float4(w.x + s.x, w.y + s.y, w.z + s.z, w.w + s.w);
                }
                *at = s;
              }
          }
        };
        if (!kPrecise || c0 == kb0) store(std::false_type{});
        else store(std::true_type{});
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&acce[buf]));
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
  if (tid == 0) p.errs[blockIdx.x] = s_err;
}

// ============================================================================ plan and launch
void plan_lora_sums(LoraParams& p, int sms) {
  const int64_t ranks = (p.rank + 15) / 16;
  p.split = p.tile_ctas = p.parts = 1;
  if (p.M <= kLoraFewRows) {
    int64_t items = std::min<int64_t>(p.M, p.count) * ranks;
    if (p.K > 2048 && 2 * items + 64 <= sms) p.split = p.parts = 2;
    items *= p.split;
    p.grid = (int32_t)(items + p.listed);
    return;
  }
  // as many CTAs as SMs, which share out a tile's items: passes over its adapters in shares of K, of two blocks and more
  const int64_t tiles = (p.M + 127) / 128, most = (std::min<int64_t>(128, p.count) * ranks + lora::kPass - 1) / lora::kPass;
  const int64_t ctas = std::max<int64_t>(sms / tiles, 1);
  while (p.split < 4 && p.split * 2 <= ctas && 2 * p.split * 128 <= p.K) p.split *= 2;
  // FP32 results: shares of 1024 products, which is what an accumulator, whose additions truncate, takes (of K above 16384 longer
  // ones, of several accumulators)
  if (p.precise) p.split = (int32_t)std::max<int64_t>(p.split, std::min<int64_t>((p.K + 1023) / 1024, 16));
  p.parts = p.split;
  p.tile_ctas = (int32_t)std::min(ctas, most * p.split);
  p.grid = (int32_t)(tiles * p.tile_ctas);
}

cudaError_t launch_lora_sums(const LoraMaps& maps, const LoraParams& p, cudaStream_t s) {
  const bool few = p.M <= kLoraFewRows;
  const auto many = p.precise ? lora_sums_many_kernel<true> : lora_sums_many_kernel<false>;
  if (!few) {
    static std::atomic<int> configured_device{-1};
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device.load(std::memory_order_relaxed) != dev) {
      for (auto kernel : {lora_sums_many_kernel<true>, lora_sums_many_kernel<false>}) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lora::kTileArena + 1024);
        if (e != cudaSuccess) return e;
      }
      configured_device.store(dev, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)p.grid);
  lc.blockDim = dim3(few ? lora::kFewThreads : lora::kTileThreads);
  lc.dynamicSmemBytes = few ? 0 : lora::kTileArena + 1024;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&lc, lora_sums_few_kernel, p) : cudaLaunchKernelEx(&lc, many, maps, p);
}

cudaError_t launch_lora_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  return p.out_f32 ? launch_form<true, true>(maps, p, s) : launch_form<false, true>(maps, p, s);
}

}  // namespace gmmfr
