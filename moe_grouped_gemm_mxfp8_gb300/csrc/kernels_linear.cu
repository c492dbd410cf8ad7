// The dense product with its epilogue: y = act(x W^T + bias) + residual.
//
// Three forms, all on the tensor cores with FP32 sums:
//   direct  up to 32 rows of x and small weights.  Weights from global memory straight into the operand registers of mma.sync: no
//           staging, no accumulator to set up; what counts here is the time to the first byte and the last.
//   stream  up to 128 rows (tcgen05 kind::f16, accumulators in TMEM, operands by TMA).  The weights are the 128-row
//           operand, the rows of x the N-wide one, so every weight byte crosses HBM once; the K range of a tile is
//           split over the CTAs of a cluster, whose partial sums meet in shared memory (in rank order: deterministic).
//           W of 4096 x 14336 takes 22.9 us with 64 rows (5.2 TB/s; 6.8 in the loop, about 5 us are launch, ramp and
//           join), the gated 2 x 2048 x 7168 with 48 rows 14.6 us.
//   pair    many rows.  A pair of CTAs holds a 256 x BN tile of y (cta_group::2: each CTA loads 128 rows of x
//           and half of the BN rows of W), accumulators double-buffered in TMEM, so that a tile's epilogue
//           runs beside the next tile's products.  8192 rows of 7168 x 4096: 261 us, 1.84 PFLOP/s (97% of the
//           library's burst rate; the tensor pipe is active 88% of the time), bound by the products and, called for
//           long, by the power limit.  Products of some hundred rows are bound by what reaches an SM from L2, about
//           64 bytes a cycle: 300 rows of 4096 x 4096 take 16.7 us.
// Rows of x or W that do not start on 16-byte boundaries (a TMA rule) are first copied to a pitch that does.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "epilogue.cuh"
#include "ops.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace gmmfr {
namespace lin {

constexpr int kThreads = 320;      // stream: warp 0 TMA, warp 1 MMA, warps 2..9 epilogue
constexpr int kPairThreads = 320;  // pair: warps 2..9 epilogue
constexpr int kBK = 64;        // K per stage: 128-byte rows
constexpr int kTileBytes = 128 * 128;
// FP32 results: K blocks of 64 that are added up in one accumulator; sums of so many are added in registers, to nearest.  The
// tensor core's additions truncate, which takes 9.4e-7 off a sum of 1024 products, in proportion to their number, and twice
// that off a gated value (K = 7168 in one accumulator: 7.9e-6 and 1.6e-5).  To go on in the other accumulator costs the
// tensor pipe about 0.5 us: 8192 rows of 7168 x 4096 262 us in one, 287 with 16 blocks, 309 with 8, 393 with 4; gated, 2000 rows
// of 4096 x 7168 138, 143, 149, 198.
template <bool kGated>
constexpr int kChunk = kGated ? 8 : 16;

// ---- pair form
constexpr int kPairArena = 6 * 32768;
constexpr int kPairMaxStages = 10;
constexpr int kPairBars = 2 * kPairMaxStages + 5;
constexpr int kPairTurnOff = (kPairArena + kPairBars * 8 + 32 + 15) / 16 * 16;  // float [8][32][33]: an epilogue warp's 32 x 32 outputs
constexpr int kPairSmem = kPairTurnOff + 8 * 32 * 33 * 4 + 1024;
static_assert(kPairSmem <= 232448 && 32 * 33 * 4 % 16 == 0, "shared memory budget; 16-byte reads of the turn buffers");

// ---- stream form
constexpr int kStreamMaxStages = 6;
constexpr int kStreamBars = 2 * kStreamMaxStages + 8;
constexpr int kStreamKps = 2;  // K blocks per stage: 0.33 us per stage where a CTA has the memory to itself, 0.25 with one
constexpr int kStreamArena = 220 * 1024;  // the ring, and the partial sums unless they take its place
constexpr int kStreamSmem = kStreamArena + kStreamBars * 8 + 32 + 1024;
static_assert(kStreamSmem <= 232448, "shared memory budget");

}  // namespace lin

namespace {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store_out(const LinearParams& p, int64_t m, int64_t n, float v) {
  if (p.residual) v += __bfloat162float(p.residual[m * p.ldr + n]);
  if (p.out_f32) static_cast<float*>(p.out)[m * p.ldo + n] = v;
  else static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
}

// A warp's 32 rows m0.. by 32 columns n.., activated values in v (bias included), lane l holding row m0 + l.
template <bool kF32>
__device__ __forceinline__ void store_tile32(const LinearParams& p, int64_t m0, int64_t n, float (&v)[32], float* turn) {
  const int lane = threadIdx.x & 31;
  const int64_t m = m0 + lane;
  if (p.vec_out && n + 32 <= p.N) {
    if (m >= p.M) return;
    if (p.residual) {
      const uint4* r = reinterpret_cast<const uint4*>(p.residual + m * p.ldr + n);
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = r[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] += bf16_lo(u[j]);
          v[8 * i + 2 * j + 1] += bf16_hi(u[j]);
        }
      }
    }
    if constexpr (kF32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + m * p.ldo + n);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + m * p.ldo + n);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                          pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
    }
  } else {
    // rows off 16-byte boundaries, or the ragged last columns: turned around in shared memory, so that the warp
    // writes one row after the other in consecutive elements, eight rows in flight
#pragma unroll
    for (int j = 0; j < 32; ++j) turn[lane * 33 + j] = v[j];
    __syncwarp();
    const int rows = p.M - m0 < 32 ? (int)(p.M - m0) : 32;
    if (n + lane < p.N) {
      const __nv_bfloat16* res = p.residual ? p.residual + m0 * p.ldr + n + lane : nullptr;
      __nv_bfloat16* o16 = static_cast<__nv_bfloat16*>(p.out) + m0 * p.ldo + n + lane;
      float* o32 = static_cast<float*>(p.out) + m0 * p.ldo + n + lane;
      for (int r0 = 0; r0 < rows; r0 += 8) {
        float f[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) f[r] = turn[(r0 + r) * 33 + lane];
        if (res) {
          __nv_bfloat16 w[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) w[r] = r0 + r < rows ? res[r * p.ldr] : __nv_bfloat16(0.f);
#pragma unroll
          for (int r = 0; r < 8; ++r) f[r] += __bfloat162float(w[r]);
          res += 8 * p.ldr;
        }
        if constexpr (kF32) {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r0 + r < rows) o32[r * p.ldo] = f[r];
          o32 += 8 * p.ldo;
        } else {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r0 + r < rows) o16[r * p.ldo] = __float2bfloat16_rn(f[r]);
          o16 += 8 * p.ldo;
        }
      }
    }
    __syncwarp();
  }
}

// The first n (below 8) elements at p, and zeros.
__device__ __forceinline__ uint4 load_part(const __nv_bfloat16* p, int n) {
  const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
  uint32_t v[4] = {};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) v[i >> 1] |= (uint32_t)__ldg(e + i) << (16 * (i & 1));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Lane j's bias, of column j of 32, onto a thread's 32 columns, by way of 128 bytes of the warp's.
__device__ __forceinline__ void add_bias32(float bias, float (&v)[32], float* room) {
  room[threadIdx.x & 31] = bias;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 b = *reinterpret_cast<const float4*>(room + j);
    v[j] += b.x;
    v[j + 1] += b.y;
    v[j + 2] += b.z;
    v[j + 3] += b.w;
  }
  __syncwarp();
}

}  // namespace

// ============================================================================ direct form
// A warp multiplies 16 rows of W (with the gated activation 8 gate rows and the 8 up rows of the same columns) by the
// rows of x over its share of the K range, both read straight into the operand registers of mma.sync: lane l holds
// 8 consecutive elements of rows l / 4 and l / 4 + 8, its K slots of two products (A and B permute K alike).  The 16
// warps of a CTA are `groups` row groups times 16 / groups shares of K, interleaved in blocks of 32, so that the CTA
// reads each row in long pieces; their sums meet in shared memory in the order of the shares.
template <bool kGated, int kTiles, bool kF32>
__global__ void __launch_bounds__(512, 1) linear_direct_kernel(const __grid_constant__ LinearParams p) {
  constexpr int kTok = 8 * kTiles;
  constexpr int kU = kTiles == 1 ? 4 : (kTiles == 2 ? 2 : 1);  // blocks of 32 K of an operand set
  __shared__ float part[16][16][kTok + 1];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) {  // no wait here can give up
    p.hdr[0] = 1;
    p.hdr[1] = 0;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = p.group_m, splits = 16 / groups, grp = warp % groups, split = warp / groups;
  constexpr int kCols = kGated ? 8 : 16;  // columns of y per group
  const int64_t n0 = ((int64_t)blockIdx.x * groups + grp) * kCols;
  const int M = (int)p.M;
  if (split < splits && n0 < p.N) {
    // rows past the end repeat the last one; what they give is not stored
    const int64_t ra = min(n0 + (lane >> 2), p.N - 1);
    const int64_t rb = kGated ? p.N + ra : min(n0 + 8 + (lane >> 2), p.N - 1);
    const __nv_bfloat16* wa = p.w + ra * p.ldw;
    const __nv_bfloat16* wb = p.w + rb * p.ldw;
    const __nv_bfloat16* xr[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) xr[i] = p.x + (int64_t)min(8 * i + (lane >> 2), M - 1) * p.ldx;
    float acc[kTiles][4] = {};
    const int64_t blocks = (p.K + 31) / 32, whole = p.K & ~int64_t(7);  // K in 16-byte pieces
    struct Operands {
      uint4 a[kU], b[kU], x[kU][kTiles];
    };
    auto load = [&](Operands& o, int64_t b0) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = (b0 + u * splits) * 32 + (lane & 3) * 8;
        o.a[u] = o.b[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o.x[u][i] = make_uint4(0, 0, 0, 0);
        if (k < whole) {
          o.a[u] = __ldg(reinterpret_cast<const uint4*>(wa + k));
          o.b[u] = __ldg(reinterpret_cast<const uint4*>(wb + k));
#pragma unroll
          for (int i = 0; i < kTiles; ++i) o.x[u][i] = __ldg(reinterpret_cast<const uint4*>(xr[i] + k));
        }
      }
    };
    auto add_products = [&](const Operands& o, float (&sums)[kTiles][4]) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          ptx::mma_16816(sums[i], o.a[u].x, o.b[u].x, o.a[u].y, o.b[u].y, o.x[u][i].x, o.x[u][i].y);
          ptx::mma_16816(sums[i], o.a[u].z, o.b[u].z, o.a[u].w, o.b[u].w, o.x[u][i].z, o.x[u][i].w);
        }
    };
    auto multiply = [&](const Operands& o) {
      if constexpr (!kF32) {
        add_products(o, acc);
      } else {  // the tensor core adds 32 to 128 products, truncating; those sums are added to nearest
        float some[kTiles][4] = {};
        add_products(o, some);
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[i][c] += some[i][c];
      }
    };
    // two sets of operands: one is on its way while the other is multiplied
    Operands even, odd;
    const int64_t step = (int64_t)splits * kU;
    load(even, split);
    for (int64_t b0 = split; b0 < blocks; b0 += 2 * step) {
      const bool more = b0 + step < blocks;
      if (more) load(odd, b0 + step);
      multiply(even);
      if (!more) break;
      if (b0 + 2 * step < blocks) load(even, b0 + 2 * step);
      multiply(odd);
    }
    // The elements past the last whole piece, one by one: what lies behind a row is another's, or nobody's, and a zero on
    // one side would not do (0 x NaN).
    if (whole < p.K && split == (int)(whole / 32 % splits)) {
      const bool mine = (lane & 3) == (int)(whole % 32 / 8);
      const int n = mine ? (int)(p.K - whole) : 0;
      const uint4 a = load_part(wa + whole, n), b = load_part(wb + whole, n);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const uint4 x = load_part(xr[i] + whole, n);
        ptx::mma_16816(acc[i], a.x, b.x, a.y, b.y, x.x, x.y);
        ptx::mma_16816(acc[i], a.z, b.z, a.w, b.w, x.z, x.w);
      }
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      float* d = &part[warp][lane >> 2][8 * i + (lane & 3) * 2];
      d[0] = acc[i][0];
      d[1] = acc[i][1];
      d[8 * (kTok + 1)] = acc[i][2];
      d[8 * (kTok + 1) + 1] = acc[i][3];
    }
  }
  __syncthreads();
  for (int i = tid; i < groups * kCols * M; i += 512) {  // columns fastest
    const int c = i % (groups * kCols), t = i / (groups * kCols), g = c / kCols, r = c - g * kCols;
    const int64_t n = ((int64_t)blockIdx.x * groups + g) * kCols + r;
    if (n >= p.N) continue;
    float v = 0.f, u = 0.f;
    for (int k = 0; k < splits; ++k) {
      v += part[k * groups + g][r][t];
      if constexpr (kGated) u += part[k * groups + g][8 + r][t];
    }
    if (p.bias) v += __bfloat162float(p.bias[n]);
    if constexpr (kGated) {
      if (p.bias) u += __bfloat162float(p.bias[p.N + n]);
      v = silu(v) * u;
    } else {
      v = activate(p.act, v);
    }
    store_out(p, t, n, v);
  }
}

// ============================================================================ pair form
// Tiles of 256 x BN in groups of kGroupM row tiles, column tiles outermost within a group, so that the
// tiles in flight share rows of x and of W in L2.
template <int kAct, int kKps, bool kF32>
__global__ void __launch_bounds__(lin::kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearParams p) {
  constexpr bool kGated = kAct == GMMFR_ACT_SWIGLU;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lin::kPairArena);  // used in rank 0: both CTAs' loads
  uint64_t* empty = full + lin::kPairMaxStages;
  uint64_t* accf = empty + lin::kPairMaxStages;
  uint64_t* acce = accf + 2;  // used in rank 0: both CTAs' epilogue warps
  uint64_t* drain = acce + 2;
  int32_t* misc = reinterpret_cast<int32_t*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&misc[0]);
  int* abort_flag = &misc[1];
  uint32_t* s_err = reinterpret_cast<uint32_t*>(&misc[2]);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const uint32_t rank = ptx::cluster_rank();
  const int BN = p.bn;
  // a stage: kKps K blocks of 64, each 128 rows of x and then BN / 2 rows of W
  const int block_bytes = lin::kTileBytes + BN * 64, stage_bytes = kKps * block_bytes, n_stages = p.n_stages;
  const int KB = (p.KB + kKps - 1) / kKps;
  const int per = kF32 ? lin::kChunk<kGated> / kKps : KB;  // stages to an accumulator

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
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
  if (warp == 0 && lane < 2) ptx::prefetch_tensormap(lane ? &maps.w : &maps.x);
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Ctl ctl{abort_flag, s_err, p.timeout_ns};
  const uint32_t smem_base = ptx::smem_u32(smem);
  const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
  const int tiles = p.tiles_m * p.tiles_n;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  auto tile_at = [&](int t, int& mt, int& nt) {
    const int per = p.group_m * p.tiles_n, g = t / per, r = t - g * per;
    const int rows = min(p.group_m, p.tiles_m - g * p.group_m);
    nt = r / rows;
    mt = g * p.group_m + (r - nt * rows);
  };

  if (warp == 0) {
    const uint64_t pol = ptx::l2_evict_last_policy();
    const uint32_t full_own = ptx::smem_u32(full), full0 = ptx::map_to_rank(full_own, 0), empty0 = ptx::smem_u32(empty);
    int stage = 0;
    uint32_t phase = 0, sb = smem_base;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += pairs) {
      int mt, nt;
      tile_at(t, mt, nt);
      const int ym = mt * 256 + (int)rank * 128;
      const int yn = kGated ? nt * (BN / 2) + (rank ? (int)p.N : 0) : nt * BN + (int)rank * (BN / 2);
      for (int kb = 0, x = 0; kb < KB; ++kb, x += kKps * lin::kBK) {
        if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
          ok = false;
          break;
        }
        if (ptx::elect_one()) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(full_own + 8 * stage, 2 * stage_bytes);
#pragma unroll
          for (int i = 0; i < kKps; ++i) {  // past K the loads fill zeros
            ptx::tma_load_2d_pair(sb + i * block_bytes, &maps.x, x + i * lin::kBK, ym, full0 + 8 * stage, pol);
            ptx::tma_load_2d_pair(sb + i * block_bytes + lin::kTileBytes, &maps.w, x + i * lin::kBK, yn, full0 + 8 * stage, pol);
          }
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
      // kind::f16: FP32 accumulator, A and B BF16, M = 256
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
      // the start address is a field of 16-byte units in the low word: stages stay below 2^18 bytes
      const uint64_t da0 = ptx::smem_desc(smem_base, 16, 1024, ptx::kSwizzle128B);
      const uint32_t lo0 = (uint32_t)da0, desc_hi = (uint32_t)(da0 >> 32);
      const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
      const uint32_t lo_step = (uint32_t)stage_bytes >> 4, lo_block = (uint32_t)block_bytes >> 4;
      int stage = 0;
      uint32_t phase = 0, lo = lo0;
      int acc_i = 0;
      bool ok = true;
      for (int t = first, left = KB; ok && t < tiles; t += left == KB ? pairs : 0) {  // left: stages left of the tile
        const int buf = acc_i & 1, n = kF32 ? min(per, left) : KB;
        if (!__all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(&acce[buf]), ((acc_i >> 1) & 1) ^ 1, ctl))) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + buf * 256;
        uint32_t accumulate = 0;
        for (int kb = 0; kb < n; ++kb) {
          if (!warp_wait_quick(full0 + 8 * stage, phase, ctl)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int i = 0; i < kKps; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::tc_mma_f16_pair_lo(d, lo + i * lo_block + 2 * q, lo + i * lo_block + (lin::kTileBytes >> 4) + 2 * q, desc_hi,
                                        idesc, i + q > 0 ? 1u : accumulate);
            ptx::tc_commit_pair(empty0 + 8 * stage);
            if (kb == n - 1) ptx::tc_commit_pair(ptx::smem_u32(&accf[buf]));
          }
          accumulate = 1;
          lo += lo_step;
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
            lo = lo0;
          }
        }
        ++acc_i;
        if (kF32) left = left > n ? left - n : KB;
      }
      if (ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(drain));
      wait_bar_drain(ptx::smem_u32(drain), 0);
    }
    __syncwarp();
  } else {
    // two warps per TMEM lane quadrant, taking its 32-column chunks in turn
    const int q = warp & 3, half = (warp - 2) >> 2;
    float* turn = reinterpret_cast<float*>(smem + lin::kPairTurnOff) + (warp - 2) * 32 * 33;
    int acc_i = 0;
    for (int t = first; t < tiles; t += pairs) {
      int mt, nt;
      tile_at(t, mt, nt);
      const int cols = kGated ? BN / 2 : BN;
      const int64_t n0 = (int64_t)nt * cols;
      // the tile's biases, a column per lane, before the wait for its products
      constexpr int kChunks = kGated ? 2 : 4;
      float bias[kChunks] = {}, bias_up[kChunks] = {};
      auto load_bias = [&](int i) {
        const int64_t n = n0 + 32 * half + 64 * i + lane;
        if (p.bias && n < p.N) {
          bias[i] = __bfloat162float(p.bias[n]);
          if constexpr (kGated) bias_up[i] = __bfloat162float(p.bias[p.N + n]);
        }
      };
      if constexpr (!kF32) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) load_bias(i);
      }
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
      const int64_t m0 = (int64_t)mt * 256 + rank * 128 + q * 32;  // this warp's rows
      auto wait_full = [&]() {
        const bool ok = warp_wait_quick(ptx::smem_u32(&accf[acc_i & 1]), (acc_i >> 1) & 1, ctl);
        ptx::tc_fence_after();
        return ok;
      };
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(&acce[acc_i & 1]), 0));
        ++acc_i;
      };
      // chunk i's values v (gated: and up values u), biased, activated, with the residual, to memory
      auto finish = [&](int i, float (&v)[32], float (&u)[32]) {
        if (p.bias) add_bias32(bias[i], v, turn);
        if constexpr (kGated) {
          if (p.bias) add_bias32(bias_up[i], u, turn);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = silu<!kF32>(v[j]) * u[j];
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = activate<!kF32>(kAct, v[j]);
        }
        store_tile32<kF32>(p, m0, n0 + 32 * half + 64 * i, v, turn);
      };
      if constexpr (!kF32) {
        if (!wait_full()) break;
        const uint32_t at = taddr + (acc_i & 1) * 256;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c0 = 32 * half + 64 * i;
          if (c0 >= cols) break;
          uint32_t r[32];
          float v[32], u[32];
          ptx::tmem_ld_32x32b_x32(at + c0, r);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          if constexpr (kGated) {
            ptx::tmem_ld_32x32b_x32(at + BN / 2 + c0, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __uint_as_float(r[j]);
          }
          finish(i, v, u);
        }
        release();
      } else {
        float sum[4][32] = {};  // gated: two chunks of gate values, then their up values
        bool ok = true;
        for (int kb = 0; kb < KB; kb += per) {
          ok = wait_full();
          if (!ok) break;
          const uint32_t at = taddr + (acc_i & 1) * 256;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c0 = 32 * half + 64 * (i % kChunks);
            if (c0 < cols) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {  // 32 at a time would not fit in registers beside the sums
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(at + c0 + h + i / kChunks * (BN / 2), r);
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
        for (int i = 0; i < kChunks; ++i) {
          if (32 * half + 64 * i >= cols) break;
          load_bias(i);  // (not before: the sums have the registers)
          finish(i, sum[i], sum[i + 4 - kChunks]);
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
    p.hdr[1 + p.slot_base + blockIdx.x] = *s_err;
    if (p.slot_base + blockIdx.x == 0) p.hdr[0] = p.slots;
  }
}

// ============================================================================ stream form
// Cluster c takes the tiles c, c + clusters, ...; its CTA of rank r the K blocks [KB r / S, KB (r + 1) / S).
// A tile is 128 rows of W; with the gated activation 64 gate rows and the 64 up rows of the same columns.
template <int kAct, bool kF32>
__global__ void __launch_bounds__(lin::kThreads, 1)
    linear_stream_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearParams p) {
  constexpr bool kGated = kAct == GMMFR_ACT_SWIGLU;
  constexpr int kCols = kGated ? 64 : 128;  // columns of y per tile
  constexpr int kEpi = lin::kThreads - 64, kKps = lin::kStreamKps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lin::kStreamArena);
  uint64_t* empty = full + lin::kStreamMaxStages;
  uint64_t* accf = empty + lin::kStreamMaxStages;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint64_t* pready = drain + 1;  // every CTA's partial sums are in its shared memory
  uint64_t* pfree = pready + 1;  // every CTA has read this one's
  int32_t* misc = reinterpret_cast<int32_t*>(pfree + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&misc[0]);
  int* abort_flag = &misc[1];
  uint32_t* s_err = reinterpret_cast<uint32_t*>(&misc[2]);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const int S = p.split;
  const uint32_t rank = S > 1 ? ptx::cluster_rank() : 0u;
  const int T = (int)p.M, npad = p.bn;
  const int block_bytes = lin::kTileBytes + npad * 128, stage_bytes = kKps * block_bytes, n_stages = p.n_stages;
  const int clusters = gridDim.x / S, first = blockIdx.x / S, tiles = p.tiles_n;
  // [T][128]: in the ring's place when no tile follows, whose loads would write there
  float* part = reinterpret_cast<float*>(smem + (tiles <= clusters ? 0 : n_stages * stage_bytes));
  // one accumulator, or two in turn for the chunks of FP32 results
  const uint32_t acc_cols = npad <= 32 ? 32 : (npad <= 64 ? 64 : 128), tmem_cols = kF32 ? 2 * acc_cols : acc_cols;
  auto acc_of = [&](uint32_t i) { return kF32 ? i & 1 : 0; };
  auto phase_of = [&](uint32_t i) { return kF32 ? (i >> 1) & 1 : i & 1; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&accf[b]), 1 + p.test_stall);
      ptx::mbar_init(ptx::smem_u32(&acce[b]), 8);
    }
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    ptx::mbar_init(ptx::smem_u32(pready), S);
    ptx::mbar_init(ptx::smem_u32(pfree), S);
    *abort_flag = 0;
    *s_err = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane < 2) ptx::prefetch_tensormap(lane ? &maps.w : &maps.x);
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (S > 1) ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Ctl ctl{abort_flag, s_err, p.timeout_ns};
  const uint32_t smem_base = ptx::smem_u32(smem);
  const int units = (p.KB + kKps - 1) / kKps;  // what lies past K is loaded as zeros
  const int kb0 = (int)((int64_t)units * rank / S), kb1 = (int)((int64_t)units * (rank + 1) / S);
  const int per = kF32 ? lin::kChunk<kGated> / kKps : kb1 - kb0;  // stages to an accumulator
  // Beside the pair form: this kernel starts when every CTA of that one has seen its predecessors end, and may not end
  // before it does.
  if (!p.beside) ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  if (warp == 0) {
    const uint64_t pol_w = ptx::l2_evict_first_policy(), pol_x = ptx::l2_evict_last_policy();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
    uint32_t sb = smem_base;
    for (int t = first; ok && t < tiles; t += clusters) {
      const int y = t * (kGated ? 64 : 128), y_up = (int)p.N + t * 64;
      for (int kb = kb0, x = kb0 * kKps * lin::kBK; kb < kb1; ++kb, x += kKps * lin::kBK) {
        if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
          ok = false;
          break;
        }
        if (ptx::elect_one()) {
          const uint32_t fb = full0 + 8 * stage;
          ptx::mbar_arrive_expect_tx(fb, stage_bytes);
#pragma unroll
          for (int h = 0; h < kKps; ++h) {
            const uint32_t d = sb + h * block_bytes;
            ptx::tma_load_2d(d, &maps.w, x + h * lin::kBK, y, fb, pol_w);
            if constexpr (kGated) ptx::tma_load_2d(d + 64 * 128, &maps.w, x + h * lin::kBK, y_up, fb, pol_w);
            ptx::tma_load_2d(d + lin::kTileBytes, &maps.x, x + h * lin::kBK, 0, fb, pol_x);
          }
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
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(npad >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t da0 = ptx::smem_desc(smem_base, 16, 1024, ptx::kSwizzle128B);
    const uint32_t lo0 = (uint32_t)da0, desc_hi = (uint32_t)(da0 >> 32), lo_step = (uint32_t)stage_bytes >> 4,
                   lo_block = (uint32_t)block_bytes >> 4;
    const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
    int stage = 0;
    uint32_t phase = 0, acc_i = 0, lo = lo0;
    bool ok = true;
    for (int t = first, k0 = kb0; ok && t < tiles; t += k0 == kb0 ? clusters : 0) {
      const int k1 = kF32 ? min(k0 + per, kb1) : kb1;
      if (!warp_wait_quick(ptx::smem_u32(&acce[acc_of(acc_i)]), phase_of(acc_i) ^ 1, ctl)) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem_base + acc_of(acc_i) * acc_cols;
      uint32_t accumulate = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!warp_wait_quick(full0 + 8 * stage, phase, ctl)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll
          for (int h = 0; h < kKps; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              ptx::tc_mma_f16_lo(d, lo + h * lo_block + 2 * q, lo + h * lo_block + (lin::kTileBytes >> 4) + 2 * q, desc_hi, idesc,
                                 h + q > 0 ? 1u : accumulate);
          ptx::tc_commit(empty0 + 8 * stage);
          if (kb == k1 - 1) ptx::tc_commit(ptx::smem_u32(&accf[acc_of(acc_i)]));
        }
        accumulate = 1;
        lo += lo_step;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
          lo = lo0;
        }
      }
      ++acc_i;
      if (kF32) k0 = k1 == kb1 ? kb0 : k1;
    }
    if (ptx::elect_one()) ptx::tc_commit(ptx::smem_u32(drain));
    wait_bar_drain(ptx::smem_u32(drain), 0);
    __syncwarp();
  } else {
    const int q = warp & 3, ep = threadIdx.x - 64;
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    const int c_first = (warp - 2) / 4 * 16;  // every other 16 rows of x from there
    uint32_t ph = 0, acc_i = 0;
    auto wait_full = [&]() {
      const bool ok = warp_wait_quick(ptx::smem_u32(&accf[acc_of(acc_i)]), phase_of(acc_i), ctl);
      ptx::tc_fence_after();
      return ok;
    };
    auto release = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&acce[acc_of(acc_i)]));
      ++acc_i;
    };
    for (int t = first; t < tiles; t += clusters, ph ^= 1) {
      [[maybe_unused]] float sum[4][16] = {};
      bool ok = true;
      if constexpr (kF32) {
        for (int kb = kb0; ok && kb < kb1; kb += per) {
          ok = wait_full();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (c_first + 32 * i < T) {
              uint32_t r[16];
              ptx::tmem_ld_32x32b_x16(taddr + acc_of(acc_i) * acc_cols + c_first + 32 * i, r);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[i][j] += __uint_as_float(r[j]);
            }
          }
          release();
        }
      } else {
        ok = wait_full();
      }
      // the partial sums of the tile before have been read by every CTA of the cluster
      if (ok && S > 1) ok = wait_bar_cluster(ptx::smem_u32(pfree), ph ^ 1, ctl);
      if (!ptx::bar_all(1, kEpi, ok)) break;  // the warps leave together: they share named barriers
      ptx::tc_fence_after();
      if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c_first + 32 * i + j < T) part[(c_first + 32 * i + j) * 128 + q * 32 + lane] = sum[i][j];
      } else {
        for (int c0 = c_first; c0 < T; c0 += 32) {
          uint32_t r[16];
          ptx::tmem_ld_32x32b_x16(taddr + c0, r);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c0 + j < T) part[(c0 + j) * 128 + q * 32 + lane] = __uint_as_float(r[j]);
        }
        release();
      }
      ptx::bar_sync(1, kEpi);
      if (S > 1) {
        if (ep < S) ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(pready), ep));
        if (!ptx::bar_all(1, kEpi, wait_bar_cluster(ptx::smem_u32(pready), ph, ctl))) break;
      }
      // this CTA's share of the tile's T x kCols outputs, four columns at a time, columns fastest; a thread has kTwo in
      // flight.  kEpi is a multiple of the column groups: a thread's columns, and with them its bias, stay the same.
      const int total = T * (kCols / 4), lo = (int)((int64_t)total * rank / S), hi = (int)((int64_t)total * (rank + 1) / S);
      const int c = (lo + ep) % (kCols / 4) * 4;
      const int64_t n = (int64_t)t * kCols + c;
      const int cols = p.N - n < 4 ? (int)(p.N - n) : 4;
      float bias[4] = {}, bias_up[4] = {};
      if (p.bias) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < cols) {
            bias[k] = __bfloat162float(p.bias[n + k]);
            if constexpr (kGated) bias_up[k] = __bfloat162float(p.bias[p.N + n + k]);
          }
      }
      constexpr int kTwo = 2;
      for (int i0 = lo + ep; i0 < hi && cols > 0; i0 += kTwo * kEpi) {
        float4 v[kTwo], u[kTwo];
        uint2 res[kTwo];
        uint32_t at[kTwo];
#pragma unroll
        for (int w = 0; w < kTwo; ++w) {
          const int tok = min(i0 + w * kEpi, hi - 1) / (kCols / 4);  // past the end: not stored
          v[w] = u[w] = make_float4(0.f, 0.f, 0.f, 0.f);
          at[w] = ptx::smem_u32(part + tok * 128 + c);
          res[w] = make_uint2(0, 0);
          if (p.residual && p.vec_out && cols == 4) res[w] = *reinterpret_cast<const uint2*>(p.residual + tok * p.ldr + n);
        }
#pragma unroll 4
        for (int s = 0; s < S; ++s) {
#pragma unroll
          for (int w = 0; w < kTwo; ++w) {
            const uint32_t b = S > 1 ? ptx::map_to_rank(at[w], s) : at[w];
            const float4 x = ptx::ld_cluster_v4(b);
            v[w] = make_float4(v[w].x + x.x, v[w].y + x.y, v[w].z + x.z, v[w].w + x.w);
            if constexpr (kGated) {
              const float4 z = ptx::ld_cluster_v4(b + 64 * 4);
              u[w] = make_float4(u[w].x + z.x, u[w].y + z.y, u[w].z + z.z, u[w].w + z.w);
            }
          }
        }
#pragma unroll
        for (int w = 0; w < kTwo; ++w) {
          if (i0 + w * kEpi >= hi) continue;
          const int tok = (i0 + w * kEpi) / (kCols / 4);
          float f[4] = {v[w].x + bias[0], v[w].y + bias[1], v[w].z + bias[2], v[w].w + bias[3]};
          const float g[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kGated) f[k] = silu(f[k]) * (g[k] + bias_up[k]);
            else f[k] = activate(kAct, f[k]);
          }
          if (p.vec_out && cols == 4) {
            f[0] += bf16_lo(res[w].x);
            f[1] += bf16_hi(res[w].x);
            f[2] += bf16_lo(res[w].y);
            f[3] += bf16_hi(res[w].y);
            if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + tok * p.ldo + n) = make_float4(f[0], f[1], f[2], f[3]);
            else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + tok * p.ldo + n) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < cols) store_out(p, tok, n + k, f[k]);
          }
        }
      }
      ptx::bar_sync(1, kEpi);
      if (S > 1 && ep < S) ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(pfree), ep));
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (S > 1) ptx::cluster_sync();  // other CTAs read this one's partial sums and arrive on its barriers
  if (p.beside) ptx::griddep_wait();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, tmem_cols);
  }
  if (threadIdx.x == 0) {
    p.hdr[1 + p.slot_base + blockIdx.x] = *s_err;
    if (p.slot_base + blockIdx.x == 0) p.hdr[0] = p.slots;
  }
}

// ============================================================================ rows off 16-byte boundaries
// dst [rows, Kp] = src [rows, K] (row stride ld), zero past K; Kp = K rounded up to 8.
__global__ void __launch_bounds__(256) linear_repitch_kernel(const uint16_t* src, uint16_t* dst, int64_t rows, int64_t K,
                                                             int64_t Kp, int64_t ld) {
  ptx::griddep_wait();
  const int64_t per = Kp / 8, n = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per, k = (i - r * per) * 8;
    const uint16_t* s = src + r * ld + k;
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k + j < K ? s[j] : (uint16_t)0;
    *reinterpret_cast<uint4*>(dst + r * Kp + k) = *reinterpret_cast<const uint4*>(v);
  }
}

cudaError_t launch_linear_repitch(const __nv_bfloat16* src, __nv_bfloat16* dst, int64_t rows, int64_t K, int64_t Kp,
                                  int64_t ld, int sms, cudaStream_t s) {
  const int64_t n = rows * (Kp / 8), blocks = (n + 255) / 256;
  linear_repitch_kernel<<<(unsigned)std::min<int64_t>(blocks, (int64_t)sms * 16), 256, 0, s>>>(
      reinterpret_cast<const uint16_t*>(src), reinterpret_cast<uint16_t*>(dst), rows, K, Kp, ld);
  return cudaGetLastError();
}

// ============================================================================ plan and launch
// Clusters of S CTAs of the stream form that run at once: what the driver says of this device, whose SMs are not all in
// groups of 8 (152 SMs: 15 clusters of 8); without an answer, as many as the SMs hold.  One CTA each: `sms`.
static int64_t stream_slots(int S, int sms) {
  if (S == 1) return std::max(1, sms);
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][3];  // S = 2, 4, 8
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return std::max(1, sms / S);
  std::atomic<int>& kept = known[dev][S == 2 ? 0 : (S == 4 ? 1 : 2)];
  int n = kept.load(std::memory_order_relaxed);
  if (n == 0) {
    auto kernel = linear_stream_kernel<GMMFR_ACT_NONE, false>;
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)S;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    lc.gridDim = dim3((unsigned)S);
    lc.blockDim = dim3(lin::kThreads);
    lc.dynamicSmemBytes = lin::kStreamSmem;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lin::kStreamSmem) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, kernel, &lc) == cudaSuccess && clusters > 0) {
      n = clusters;
    } else {
      cudaGetLastError();
      n = std::max(1, sms / S);
    }
    kept.store(n, std::memory_order_relaxed);
  }
  return n;
}

// The stream form's plan on `sms` SMs; microseconds that it takes.  Beside another kernel a tile is one CTA's.
static double plan_stream(LinearParams& p, int sms, bool beside) {
  p.form = kLinearStream;
  p.bn = (int32_t)((p.M + 15) / 16 * 16);
  p.tiles_m = 1;
  p.tiles_n = (int32_t)(p.act == GMMFR_ACT_SWIGLU ? (p.N + 63) / 64 : (p.N + 127) / 128);
  // The cluster size that ends soonest, with what was measured: a stage takes a CTA 0.33 us and more with more rows,
  // or its share of HBM; a wave ends with the epilogue, and with the join in a cluster.  W of 7168 x 4096, 32 rows:
  // clusters of 1, 2, 4, 8 take 14.9, 14.0, 15.1, 20.8 us; of 512 x 8192: 24.9, 15.3, 10.5, 8.3.
  const int stage = lin::kStreamKps * (lin::kTileBytes + p.bn * 128), units = (p.KB + lin::kStreamKps - 1) / lin::kStreamKps;
  double best = 1e30;
  for (int S = 1; S <= (beside ? 1 : 8) && S <= units; S *= 2) {
    const int64_t slots = stream_slots(S, sms);
    const int64_t waves = (p.tiles_n + slots - 1) / slots, ctas = std::min<int64_t>(p.tiles_n, slots) * S;
    const double t_stage = std::max(0.33 + 0.0009 * p.bn, lin::kStreamKps * lin::kTileBytes * (double)ctas / 6.7e6);
    const double join = S > 1 ? 1.2 + 0.15 * S : 0.0;
    const double t = waves * ((double)((units + S - 1) / S) * t_stage + 1.0 + 0.02 * p.bn / S + join) + 3.0;
    if (t < best) {
      best = t;
      p.split = S;
      p.n_stages = std::min<int>(lin::kStreamMaxStages, (lin::kStreamArena - (waves > 1 ? (int)p.M * 512 : 0)) / stage);
      p.grid = (int32_t)ctas;
    }
  }
  return best;
}

// The pair form's time in microseconds with tiles of bn columns: the products take 2.1 BN cycles per K block, the loads
// of a CTA's operands (128 + BN / 2 rows of 128 bytes) about a byte per 1/50 cycle; waves of tiles over the pairs.
static double pair_time(const LinearParams& p, int64_t M, int64_t rows_w, int bn, int pairs, int64_t* tiles) {
  *tiles = (rows_w + bn - 1) / bn * ((M + 255) / 256);
  const double waves = (double)((*tiles + pairs - 1) / pairs);
  return (waves * (p.KB * std::max(2.1 * bn, (16384.0 + 64.0 * bn) / 50.0) + 300.0) + 12.0 * bn) / 1900.0 + 4.0;
}

void plan_linear(LinearParams& p, LinearParams& tail, int sms) {
  tail.M = 0;
  if (p.M <= kLinearDirectRows) {
    // one CTA per SM: as many row groups each as that takes (up to 8; then in waves)
    const int cols = p.act == GMMFR_ACT_SWIGLU ? 8 : 16;
    const int64_t row_groups = (p.N + cols - 1) / cols;
    p.group_m = 1;
    while (p.group_m < 8 && (row_groups + p.group_m - 1) / p.group_m > sms) ++p.group_m;
    // Its products come out of the registers that the loads need, so it falls behind with rows x weights per CTA: W of
    // 2048 x 2048 and 32 rows (1.0 M) 6.0 us, the stream form 6.7; 5125 x 1288 and 32 (2.0 M) 8.7 and 7.9;
    // 7168 x 4096: 8 rows (1.6 M) 12.5 and 13.8, 16 (3.1 M) 13.6 and 13.9, 32 (6.3 M) 17.7 and 14.0.
    if (p.M == 1 || p.M * p.group_m * 16 * p.K <= 1900000) {
      p.form = kLinearDirect;
      p.grid = (int32_t)((row_groups + p.group_m - 1) / p.group_m);
      return;
    }
  }
  const int64_t rows_w = p.act == GMMFR_ACT_SWIGLU ? 2 * p.N : p.N;
  p.KB = (int32_t)((p.K + lin::kBK - 1) / lin::kBK);
  if (p.M <= kLinearStreamRows) {
    plan_stream(p, sms, false);
    p.slots = p.grid;
    return;
  }
  p.form = kLinearPair;
  const int pairs = sms / 2;
  int64_t tiles;
  double best = 1e30;
  for (int bn = 256; bn >= 64; bn -= 32) {
    if (p.act == GMMFR_ACT_SWIGLU && bn % 64) continue;
    const double t = pair_time(p, p.M, rows_w, bn, pairs, &tiles);
    if (t < best) {
      best = t;
      p.bn = bn;
    }
  }
  // The rows past the last full 256 cost as much as 256.  When the tiles of the others leave SMs idle, the stream form
  // takes those rows there at the same time.  W of 5120 x 1288: 777 rows 17.8 us, in the pair form alone 20.8; of
  // 4096 x 4096: 1030 rows 27.4 and 32.8.
  const int64_t rest = p.M % 256;
  if (p.M > 256 && rest > 0 && rest <= kLinearStreamRows) {
    double least = 0.9 * best;
    for (int bn = 256; bn >= 64; bn -= 32) {
      if (p.act == GMMFR_ACT_SWIGLU && bn % 64) continue;
      const double t = pair_time(p, p.M - rest, rows_w, bn, pairs, &tiles);
      const int left = sms - 2 * (int)std::min<int64_t>(tiles, pairs);
      if (left < 8 || t >= least) continue;
      LinearParams q = p;
      q.M = rest;
      const double both = std::max(t, plan_stream(q, left, true) + 2.0);
      if (both < least) {
        least = both;
        p.bn = bn;
        tail = q;
      }
    }
  }
  if (tail.M) {
    p.M -= rest;
    const int64_t at = p.M;
    tail.x += at * p.ldx;
    if (tail.residual) tail.residual += at * p.ldr;
    tail.out = static_cast<char*>(p.out) + at * p.ldo * (p.out_f32 ? 4 : 2);
    tail.beside = 1;
  }
  p.tiles_m = (int32_t)((p.M + 255) / 256);
  p.tiles_n = (int32_t)(p.act == GMMFR_ACT_SWIGLU ? (p.N + p.bn / 2 - 1) / (p.bn / 2) : (rows_w + p.bn - 1) / p.bn);
  p.kps = p.bn <= 128 && p.KB > 1 ? 2 : 1;
  p.n_stages = std::min<int>(lin::kPairMaxStages, lin::kPairArena / (p.kps * (lin::kTileBytes + p.bn * 64)));
  p.group_m = 8;
  p.grid = (int32_t)(2 * std::min<int64_t>(pairs, (int64_t)p.tiles_m * p.tiles_n));
  p.split = 2;
  p.slots = p.grid + (tail.M ? tail.grid : 0);
  tail.slot_base = p.grid;
}

template <int kAct, bool kF32>
static cudaError_t launch_one(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  auto kernel = p.form == kLinearStream ? linear_stream_kernel<kAct, kF32>
                                        : (p.kps == 1 ? linear_pair_kernel<kAct, 1, kF32> : linear_pair_kernel<kAct, 2, kF32>);
  const int smem = p.form == kLinearStream ? lin::kStreamSmem : lin::kPairSmem;
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(linear_stream_kernel<kAct, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         lin::kStreamSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(linear_pair_kernel<kAct, 1, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, lin::kPairSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(linear_pair_kernel<kAct, 2, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, lin::kPairSmem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)p.grid);
  lc.blockDim = dim3(p.form == kLinearStream ? lin::kThreads : lin::kPairThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, maps, p);
}

template <bool kF32>
static cudaError_t launch_form(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  if (p.form == kLinearDirect) {
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.grid);
    lc.blockDim = dim3(512);
    lc.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const int tiles = p.M <= 8 ? 0 : (p.M <= 16 ? 1 : 2);
    constexpr decltype(&linear_direct_kernel<true, 1, kF32>) kernels[2][3] = {
        {linear_direct_kernel<false, 1, kF32>, linear_direct_kernel<false, 2, kF32>, linear_direct_kernel<false, 4, kF32>},
        {linear_direct_kernel<true, 1, kF32>, linear_direct_kernel<true, 2, kF32>, linear_direct_kernel<true, 4, kF32>}};
    return cudaLaunchKernelEx(&lc, kernels[p.act == GMMFR_ACT_SWIGLU][tiles], p);
  }
  switch (p.act) {
    case GMMFR_ACT_RELU: return launch_one<GMMFR_ACT_RELU, kF32>(maps, p, s);
    case GMMFR_ACT_GELU: return launch_one<GMMFR_ACT_GELU, kF32>(maps, p, s);
    case GMMFR_ACT_GELU_TANH: return launch_one<GMMFR_ACT_GELU_TANH, kF32>(maps, p, s);
    case GMMFR_ACT_SILU: return launch_one<GMMFR_ACT_SILU, kF32>(maps, p, s);
    case GMMFR_ACT_SWIGLU: return launch_one<GMMFR_ACT_SWIGLU, kF32>(maps, p, s);
    default: return launch_one<GMMFR_ACT_NONE, kF32>(maps, p, s);
  }
}

cudaError_t launch_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  return p.out_f32 ? launch_form<true>(maps, p, s) : launch_form<false>(maps, p, s);
}

}  // namespace gmmfr
