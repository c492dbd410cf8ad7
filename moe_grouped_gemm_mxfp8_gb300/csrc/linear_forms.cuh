// The dense product with its epilogue: y = act(x W^T + bias) + residual; with kLora the rows' adapters are added before act.
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
#pragma once
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

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

// ---- adapters
constexpr int kLoraWarp = kThreads / 32;
template <bool kF32>
constexpr int kLoraWarps = kF32 ? 2 : 4;  // more: four, or two where the registers do not allow it

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

// kLora: the activation is a choice at run time (a third of the kernels; the plain product's are compiled for each)
template <bool kBf16, int kN>
__device__ __forceinline__ void activate_all(int act, float (&v)[kN]) {
  auto all = [&](auto a) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = activate<kBf16>(decltype(a)::value, v[j]);
  };
  switch (act) {
    case GMMFR_ACT_RELU: return all(std::integral_constant<int, GMMFR_ACT_RELU>{});
    case GMMFR_ACT_GELU: return all(std::integral_constant<int, GMMFR_ACT_GELU>{});
    case GMMFR_ACT_GELU_TANH: return all(std::integral_constant<int, GMMFR_ACT_GELU_TANH>{});
    case GMMFR_ACT_SILU: return all(std::integral_constant<int, GMMFR_ACT_SILU>{});
    default: return;
  }
}

// What a row's adapter adds to columns n.. (rows n.. of the second factors) of y before the activation: the FP32
// products of the row's first-factor sums, scaled already, with `cols` rows of the adapter's second factor.  at: the sums'
// first part, `part` elements before the next of `parts`.  kNotFinite: of those of its elements alone that are infinite or NaN.
template <int kCols, bool kNotFinite = false>
__device__ __forceinline__ void add_adapter(const LinearParams& p, int adapter, const float* at, int parts, int64_t part, int64_t n, int cols,
                                            float (&f)[kCols]) {
  if ((uint32_t)adapter >= (uint32_t)p.lora_count) return;
  const __nv_bfloat16* b = p.lora_b + ((int64_t)adapter * p.lora_rows + n) * p.lora_rank;
  auto add = [](float& f, float s, float b) {
    if (!kNotFinite || !isfinite(b)) f += s * b;
  };
  if constexpr (kCols == 1 && !kNotFinite) {  // four pieces of the factor's row, and of the sums, on their way at once
    // A sum's parts (two at most, of up to 32 rows) before its products: an infinite part beside a finite one of the other sign, and
    // an infinite factor, come to an infinity, not to NaN.
    const float4* s = reinterpret_cast<const float4*>(at);
    const float4* more = reinterpret_cast<const float4*>(at + part);
#pragma unroll 4
    for (int j = 0; j < p.lora_rank; j += 8) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(b + j));
      float4 lo = s[j / 4], hi = s[j / 4 + 1];
      if (parts > 1) {
        const float4 l = more[j / 4], h = more[j / 4 + 1];
        lo = make_float4(lo.x + l.x, lo.y + l.y, lo.z + l.z, lo.w + l.w);
        hi = make_float4(hi.x + h.x, hi.y + h.y, hi.z + h.z, hi.w + h.w);
      }
      add(f[0], lo.x, bf16_lo(w.x)), add(f[0], lo.y, bf16_hi(w.x)), add(f[0], lo.z, bf16_lo(w.y)), add(f[0], lo.w, bf16_hi(w.y));
      add(f[0], hi.x, bf16_lo(w.z)), add(f[0], hi.y, bf16_hi(w.z)), add(f[0], hi.z, bf16_lo(w.w)), add(f[0], hi.w, bf16_hi(w.w));
    }
  } else {
    for (int j = 0; j < p.lora_rank; j += 8) {
      float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
      for (int c = 0; c < parts; ++c) {
        const float4* s = reinterpret_cast<const float4*>(at + c * part + j);
        lo = make_float4(lo.x + s[0].x, lo.y + s[0].y, lo.z + s[0].z, lo.w + s[0].w);
        hi = make_float4(hi.x + s[1].x, hi.y + s[1].y, hi.z + s[1].z, hi.w + s[1].w);
      }
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        if (k < cols) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(b + (int64_t)k * p.lora_rank + j));
          add(f[k], lo.x, bf16_lo(w.x)), add(f[k], lo.y, bf16_hi(w.x)), add(f[k], lo.z, bf16_lo(w.y)), add(f[k], lo.w, bf16_hi(w.y));
          add(f[k], hi.x, bf16_lo(w.z)), add(f[k], hi.y, bf16_hi(w.z)), add(f[k], hi.z, bf16_lo(w.w)), add(f[k], hi.w, bf16_hi(w.w));
        }
      }
    }
  }
}

// The adapter of row m; one that there is not sets kErrBadAdapterId, and counts as none.
__device__ __forceinline__ int adapter_of(const LinearParams& p, int64_t m, uint32_t* err) {
  const int a = p.lora_ids[m];
  if (a < -1 || a >= p.lora_count) atomicOr(err, kErrBadAdapterId);
  return a;
}

// ---------------------------------------------------------------- adapters in the stream and pair form
// The second factors join a tile's sum as further K blocks: for each adapter that any of the tile's rows has, and each 32 of
// its ranks, a block whose W rows are the second factor's (by TMA) and whose x rows are the rows' sums, zeros in the rows of
// other adapters.  Warps of their own write those x rows and hand the stage over.  A sum enters as two BF16 numbers, the
// first truncated, so that it is off by 2^-17 at most; they take the halves of a 128-byte row, both against the same 32
// ranks.  For FP32 results it is three numbers, which leave nothing out, of 16 ranks.  The lists of the adapters of 256 rows
// come with the sums.
// A zero does not keep an infinity or NaN of another adapter's factor out of a row.  The warps look at each factor where it has
// landed and put the smallest normal number, of the same sign, in the place of any; from then on the cluster's epilogues add, row by
// row, what those elements give the rows whose adapter has them.  (A zero in their place would do for a finite sum, but make NaN of
// an infinite one, whose product with an infinity is an infinity.  What the small number adds to a finite sum is lost in what the
// element itself adds.)
template <bool kF32>
struct SumTerms {
  static constexpr int kTerms = kF32 ? 3 : 2, kRanks = kF32 ? 16 : 32;  // of a block: BF16 numbers of a sum, ranks
  static constexpr int kPieces = kRanks / 8;                            // 16-byte pieces of a row that a term takes
  __device__ static int blocks(int rank) { return (rank + kRanks - 1) / kRanks; }
  // FP32 results: what the adapters add has an accumulator of its own.  Each of its 3 rank / 16 truncating additions is of a running
  // sum that holds the dense one already: 300 rows, K = 256, rank 256, of one sign: 5.5e-6 off in one accumulator, 1.4e-6
  // in two.  Up to rank 16 (3 additions) they share the last: 8192 rows of 7168 x 4096 353 us, apart 364.
  __device__ static bool apart(int rank) { return kF32 && rank > 16; }
  // products of 16 ranks in the block from r0 on
  __device__ static int steps(int rank, int r0) { return kRanks == 32 && rank - r0 > 16 ? 2 : 1; }
};
struct AdapterShared {
  uint64_t loaded[lin::kPairMaxStages];  // a stage's second factors have landed in this CTA
  uint64_t built[lin::kPairMaxStages];   // in the CTA that issues the products: a stage is ready
  int32_t not_finite;                    // a factor of this cluster's tiles was not finite
};

// built_by: warps
__device__ __forceinline__ void init_adapters(AdapterShared& a, int n_stages, int built_by) {
  for (int s = 0; s < n_stages; ++s) {
    ptx::mbar_init(ptx::smem_u32(&a.loaded[s]), 1);
    ptx::mbar_init(ptx::smem_u32(&a.built[s]), built_by);
  }
  a.not_finite = 0;
}

__device__ __forceinline__ int adapters_of(const int32_t* list) { return (int)min((uint32_t)list[0], 256u); }

// A list in a warp's registers: entry 32 k + lane in e[k] (past the last: whatever lies there).
struct AdapterList {
  int n, e[8];
  __device__ __forceinline__ void load(const LinearParams& p, int64_t block) {
    const int32_t* list = p.lora_lists + block * kLoraListInts;
    n = adapters_of(list);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = list[4 + 32 * k + (threadIdx.x & 31)];
  }
  __device__ __forceinline__ int row_of(int k) const {
    int v = e[0];
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (k == i) v = e[i];
    return v;
  }
};

// The adapters of a tile's blocks one after the other: all of a list for the first ranks, then for the next, ...
struct AdapterBlocks {
  const AdapterList& list;
  int c, d, held;  // the c-th ranks of entry d; the 32 entries that hold it
  __device__ __forceinline__ AdapterBlocks(const AdapterList& list, int u) : list(list) {
    c = list.n ? u / list.n : 0;
    d = u - c * list.n;
    held = list.row_of(d >> 5);
  }
  __device__ __forceinline__ int adapter() const { return __shfl_sync(0xffffffffu, held, d & 31); }
  __device__ __forceinline__ void next() {
    if (++d == list.n) {
      d = 0;
      ++c;
    }
    if ((d & 31) == 0) held = list.row_of(d >> 5);
  }
};

// The ranks from r0 on of kRows rows' sums (m, m + 32; past the last row: its own) as the 32-bit words of a block's row: the
// leading bits of each, then what they leave, twice over for FP32 results; zeros past the rank.
template <bool kF32, int kRows>
__device__ __forceinline__ void split_sums(const LinearParams& p, int64_t m, int r0, uint32_t (&w)[kRows][32]) {
  using Terms = SumTerms<kF32>;
  constexpr int kFours = Terms::kRanks / 4, kWords = Terms::kRanks / 2;
  const int left = p.lora_rank - r0;
  float4 sum[kRows][kFours] = {};
  for (int c = 0; c < p.lora_parts; ++c) {
    float4 v[kRows][kFours];  // on their way together
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float* s = p.lora_s + c * p.lora_part + min(m + 32 * i, p.M - 1) * p.lora_rank + r0;
#pragma unroll
      for (int j = 0; j < kFours; ++j) v[i][j] = 4 * j < left ? reinterpret_cast<const float4*>(s)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int j = 0; j < kFours; ++j)
        sum[i][j] = make_float4(sum[i][j].x + v[i][j].x, sum[i][j].y + v[i][j].y, sum[i][j].z + v[i][j].z, sum[i][j].w + v[i][j].w);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int j = 0; j < kFours; ++j) {
      float f[4] = {sum[i][j].x, sum[i][j].y, sum[i][j].z, sum[i][j].w};
#pragma unroll
      for (int t = 0; t + 1 < Terms::kTerms; ++t) {
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[k] = __float_as_uint(f[k]) & 0xffff0000u;
          f[k] = isfinite(f[k]) ? f[k] - __uint_as_float(h[k]) : 0.f;
        }
        w[i][t * kWords + 2 * j] = h[0] >> 16 | h[1];
        w[i][t * kWords + 2 * j + 1] = h[2] >> 16 | h[3];
      }
      w[i][(Terms::kTerms - 1) * kWords + 2 * j] = pack_bf16(f[0], f[1]);
      w[i][(Terms::kTerms - 1) * kWords + 2 * j + 1] = pack_bf16(f[2], f[3]);
    }
}

// 2^-126, of the same sign, in place of what is not finite in the first 16 steps elements of rows r0 .. r1 - 1, of 128 bytes each
// (128-byte swizzle).
__device__ __noinline__ void replace_not_finite(uint8_t* at, int r0, int r1, int steps) {
  for (int r = r0 + (int)(threadIdx.x & 31); r < r1; r += 32)
    for (int c = 0; c < 2 * steps; ++c) {
      uint32_t* w = reinterpret_cast<uint32_t*>(at + r * 128 + ((c ^ (r & 7)) << 4));
      for (int k = 0; k < 4; ++k) {
        if ((w[k] & 0x7f80u) == 0x7f80u) w[k] = (w[k] & 0xffff8000u) | 0x80u;
        if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] = (w[k] & 0x8000ffffu) | 0x800000u;
      }
    }
}

// A CTA's kWarps adapter warps (this one: `part`) through a tile's blocks u0 .. u1 - 1, kKps to a stage, from `stage` on (a stage whose
// factors have landed is free).  x_at, w_at: where a block's rows of x and of W lie in its stage; x_rows (128 at most) of
// them are written, which are p's from row0 on; to_rank: the CTA that issues the products, or -1.
template <int kKps, bool kF32, int kWarps>
__device__ __forceinline__ bool build_adapters(const LinearParams& p, AdapterShared& a, uint8_t* smem, int stage_bytes, int block_bytes,
                                               int n_stages, int x_at, int x_rows, int w_at, int w_rows, int64_t row0,
                                               int part, const AdapterList& list, int u0, int u1, int to_rank, int& stage,
                                               uint32_t& loaded_bits, const Ctl& ctl) {
  if (u0 >= u1) return true;
  const int lane = threadIdx.x & 31, ranks = p.lora_rank;
  constexpr int kRows = 4 / kWarps;  // a lane's
  const int r0 = 32 * kRows * part + lane;
  int own[kRows];  // the adapters of this lane's rows
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t m = row0 + r0 + 32 * i;
    own[i] = m < p.M ? p.lora_ids[m] : -1;
  }
  using Terms = SumTerms<kF32>;
  AdapterBlocks at(list, u0);
  uint32_t words[kRows][32];
  split_sums<kF32, kRows>(p, row0 + r0, Terms::kRanks * at.c, words);
  int c_held = at.c;
  const uint32_t smem0 = ptx::smem_u32(smem) + x_at + r0 * 128, turn = lane & 7;
  const int w1 = (part + 1) * w_rows / kWarps, w0 = w1 - w_rows / kWarps + lane;  // w_rows: multiples of 16, 128 at most
  for (int u = u0; u < u1; u += kKps) {
    const uint32_t xb = smem0 + stage * stage_bytes;
    bool found = false;  // an infinity or NaN in the stage's factors
#pragma unroll
    for (int h = 0; h < kKps; ++h) {
      if (u + h >= u1) break;
      const int steps = Terms::steps(ranks, Terms::kRanks * at.c), adapter = at.adapter();
      if (at.c != c_held) {
        c_held = at.c;
        split_sums<kF32, kRows>(p, row0 + r0, Terms::kRanks * at.c, words);
      }
      if (h == 0) {
        if (!warp_wait_quick(ptx::smem_u32(&a.loaded[stage]), loaded_bits >> stage & 1, ctl)) return false;
        loaded_bits ^= 1u << stage;
      }
      uint8_t* wb = smem + stage * stage_bytes + h * block_bytes + w_at;
      __nv_bfloat162 most = __float2bfloat162_rn(0.f);  // the largest, NaN before infinity
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = w0 + 32 * i;  // a row of W, on its way while rows of x are written
        uint4 v[Terms::kPieces];
#pragma unroll
        for (int k = 0; k < Terms::kPieces; ++k)
          v[k] = r < w1 && k < 2 * steps ? *reinterpret_cast<const uint4*>(wb + r * 128 + ((k ^ (r & 7)) << 4)) : make_uint4(0, 0, 0, 0);
        if (r0 + 32 * i < x_rows) {
          const uint32_t to = xb + h * block_bytes + i * 4096, keep = own[i] == adapter ? 0xffffffffu : 0u;
#pragma unroll
          for (int k = 0; k < Terms::kPieces; ++k) {
            if (k >= 2 * steps) break;
#pragma unroll
            for (int t = 0; t < Terms::kTerms; ++t) {
              const int piece = t * Terms::kPieces + k;
              ptx::st_shared_v4(to + ((piece ^ turn) << 4), words[i][4 * piece] & keep, words[i][4 * piece + 1] & keep,
                                words[i][4 * piece + 2] & keep, words[i][4 * piece + 3] & keep);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < Terms::kPieces; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));
        }
      }
      const uint32_t bits = *reinterpret_cast<const uint32_t*>(&most);
      if (__any_sync(0xffffffffu, (bits & 0x7f80u) == 0x7f80u || (bits & 0x7f800000u) == 0x7f800000u)) {
        replace_not_finite(wb, w1 - w_rows / kWarps, w1, steps);
        found = true;
      }
      at.next();
    }
    ptx::fence_proxy_async_smem();
    if (found) {
      const uint32_t flag_at = ptx::smem_u32(&a.not_finite);
      if (lane < p.split) ptx::st_cluster_u32(p.split > 1 ? ptx::map_to_rank(flag_at, lane) : flag_at, 1u);
      __threadfence();
    }
    __syncwarp();
    if (lane == 0) {
      const uint32_t bar = ptx::smem_u32(&a.built[stage]);
      if (to_rank >= 0) ptx::mbar_arrive_remote(ptx::map_to_rank(bar, to_rank));
      else ptx::mbar_arrive(bar);
    }
    if (++stage == n_stages) stage = 0;
  }
  return true;
}

}  // namespace

// ============================================================================ direct form
// A warp multiplies 16 rows of W (with the gated activation 8 gate rows and the 8 up rows of the same columns) by the
// rows of x over its share of the K range, both read straight into the operand registers of mma.sync: lane l holds
// 8 consecutive elements of rows l / 4 and l / 4 + 8, its K slots of two products (A and B permute K alike).  The 16
// warps of a CTA are `groups` row groups times 16 / groups shares of K, interleaved in blocks of 32, so that the CTA
// reads each row in long pieces; their sums meet in shared memory in the order of the shares.
template <bool kGated, int kTiles, bool kF32, bool kLora>
__global__ void __launch_bounds__(512, 1) linear_direct_kernel(const __grid_constant__ LinearParams p) {
  constexpr int kTok = 8 * kTiles;
  constexpr int kU = kTiles == 1 ? 4 : (kTiles == 2 ? 2 : 1);  // blocks of 32 K of an operand set
  __shared__ float part[16][16][kTok + 1];
  [[maybe_unused]] __shared__ uint32_t s_err;
  [[maybe_unused]] __shared__ __align__(16) float s_parts[2][16][16], s_sums[32];  // lora_own
  // kLora: the launch before is the adapters' first factors, which began after all before it had ended; what it computes
  // is not read until the weights' products are done
  if (!kLora || p.lora_own) ptx::griddep_wait();
  if (kLora && threadIdx.x == 0) s_err = 0;
  ptx::griddep_launch_dependents();
  if (!kLora && blockIdx.x == 0 && threadIdx.x == 0) {  // no wait here can give up
    p.hdr[0] = 1;
    p.hdr[1] = 0;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = p.group_m, splits = 16 / groups, grp = warp % groups, split = warp / groups;
  constexpr int kCols = kGated ? 8 : 16;  // columns of y per group
  const int64_t n0 = ((int64_t)blockIdx.x * groups + grp) * kCols;
  const int M = (int)p.M;
  if constexpr (kLora && kTiles == 1) {
    // One or two tokens' sums, 16 ranks to each of two units: every CTA makes them for itself, its warps sharing the K range.
    // A launch is saved: one token, 2048 x 2048, 9.7 -> 6.6 us a call, which the host bounds.
    if (p.lora_own) {
      const int rc = (p.lora_rank + 15) / 16, row = lane >> 2;
      const __nv_bfloat16* xr = p.x + (int64_t)min(row, M - 1) * p.ldx;
      for (int u = 0; u < M * rc; ++u) {
        const int a = p.lora_ids[u / rc], r0 = u % rc * 16;
        if ((uint32_t)a >= (uint32_t)p.lora_count) continue;
        const __nv_bfloat16* ar = p.lora_a + ((int64_t)a * p.lora_rank + r0) * p.K;
        const __nv_bfloat16 *ra = ar + min(row, p.lora_rank - r0 - 1) * p.K, *rb = ar + min(row + 8, p.lora_rank - r0 - 1) * p.K;
        float acc[4] = {};
        for (int64_t k0 = warp * 32; k0 < p.K; k0 += 4 * 512) {
          uint4 wa[4], wb[4], x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t k = k0 + i * 512 + (lane & 3) * 8, at = k < p.K ? k : 0;
            wa[i] = ptx::ld_nc_v4(ra + at);
            wb[i] = ptx::ld_nc_v4(rb + at);
            x[i] = ptx::ld_nc_v4(xr + at);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (k0 + i * 512 + (lane & 3) * 8 >= p.K) wa[i] = wb[i] = x[i] = make_uint4(0, 0, 0, 0);
            ptx::mma_16816(acc, wa[i].x, wb[i].x, wa[i].y, wb[i].y, x[i].x, x[i].y);
            ptx::mma_16816(acc, wa[i].z, wb[i].z, wa[i].w, wb[i].w, x[i].z, x[i].w);
          }
        }
        // column u / rc of the products, 0 or 1, is lane 4 row's
        if ((lane & 3) == 0) {
          s_parts[u][warp][row] = u / rc ? acc[1] : acc[0];
          s_parts[u][warp][row + 8] = u / rc ? acc[3] : acc[2];
        }
      }
    }
  }
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
  if (kLora && !p.lora_own) ptx::griddep_wait();
  __syncthreads();
  if constexpr (kLora && kTiles == 1) {
    if (p.lora_own) {
      const int rc = (p.lora_rank + 15) / 16;
      if (tid < M * p.lora_rank) {
        const int t = tid / p.lora_rank, r = tid - t * p.lora_rank, a = p.lora_ids[t];
        if ((uint32_t)a < (uint32_t)p.lora_count) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < 16; ++w) v += s_parts[t * rc + r / 16][w][r % 16];
          s_sums[tid] = p.lora_scale ? v * p.lora_scale[a] : v;
        }
      }
      __syncthreads();
    }
  }
  if constexpr (kLora) {  // no wait here can give up
    if (blockIdx.x == 0 && warp == 0) {
      if (lane < M) adapter_of(p, lane, &s_err);
      __syncwarp();
      if (lane == 0) {
        p.hdr[0] = 1;
        p.hdr[1] = s_err;
      }
    }
  }
  for (int i = tid; i < groups * kCols * M; i += 512) {  // columns fastest
    const int c = i % (groups * kCols), t = i / (groups * kCols), g = c / kCols, r = c - g * kCols;
    const int64_t n = ((int64_t)blockIdx.x * groups + g) * kCols + r;
    if (n >= p.N) continue;
    float v = 0.f, u = 0.f;
    for (int k = 0; k < splits; ++k) {
      v += part[k * groups + g][r][t];
      if constexpr (kGated) u += part[k * groups + g][8 + r][t];
    }
    if constexpr (kLora) {
      const int a = p.lora_ids[t];
      float more[1] = {0.f}, more_up[1] = {0.f};
      const float* s = p.lora_own ? &s_sums[t * p.lora_rank] : p.lora_s + (int64_t)t * p.lora_rank;
      const int parts = p.lora_own ? 1 : p.lora_parts;
      add_adapter(p, a, s, parts, p.lora_part, n, 1, more);
      v += more[0];
      if constexpr (kGated) {
        add_adapter(p, a, s, parts, p.lora_part, p.N + n, 1, more_up);
        u += more_up[0];
      }
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
template <int kAct, int kKps, bool kF32, bool kLora>
__global__ void __launch_bounds__(lin::kPairThreads + (kLora ? 32 * lin::kLoraWarps<kF32> : 0), 1)
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
  [[maybe_unused]] AdapterShared& ad = *reinterpret_cast<AdapterShared*>(smem + lin::kPairTurnOff + 8 * 32 * 33 * 4);
  using Terms = SumTerms<kF32>;
  [[maybe_unused]] const int rank_chunks = Terms::blocks(p.lora_rank);  // kLora: blocks of an adapter
  [[maybe_unused]] const bool apart = Terms::apart(p.lora_rank);

  if (threadIdx.x == 0) {
    for (int s = 0; s < n_stages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&accf[b]), 1 + p.test_stall);
      ptx::mbar_init(ptx::smem_u32(&acce[b]), 16);
    }
    if constexpr (kLora) init_adapters(ad, n_stages, 2 * lin::kLoraWarps<kF32>);
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
  if (!kLora || !p.lora_early) ptx::griddep_wait();  // lora_early: who reads the sums or lists waits before it does
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
      [[maybe_unused]] AdapterList list;
      if (kLora && t != first) list.load(p, mt);  // of the first tile when the sums are there
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
      if constexpr (kLora) {
        if (!ok) break;
        if (t == first) {
          if (p.lora_early) ptx::griddep_wait();
          list.load(p, mt);
        }
        const int units = list.n * rank_chunks;
        AdapterBlocks next(list, 0);
        for (int u = 0; u < units; u += kKps) {
          if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
            ok = false;
            break;
          }
          const uint32_t lb = ptx::smem_u32(&ad.loaded[stage]);
          int adapter[kKps], rank0[kKps];
#pragma unroll
          for (int i = 0; i < kKps; ++i) {
            rank0[i] = Terms::kRanks * next.c;
            adapter[i] = next.adapter();
            next.next();
          }
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(lb, min(kKps, units - u) * BN * 64);
#pragma unroll
            for (int i = 0; i < kKps; ++i)
              if (u + i < units)
                ptx::tma_load_3d(sb + i * block_bytes + lin::kTileBytes, &maps.b, rank0[i], yn, adapter[i], lb, pol);
          }
          sb += stage_bytes;
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
            sb = smem_base;
          }
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
    if (kLora && !ok) {
      let_loads_land();
    } else if (!ok && rank == 0) {  // aborted: let what is in flight land (both CTAs' loads count on rank 0's barriers)
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
      [[maybe_unused]] uint32_t full_bits = 0, built_bits = 0;  // kLora: a barrier's phase by its own uses
      bool ok = true;
      for (int t = first, left = KB; ok && t < tiles; t += left == KB ? pairs : 0) {  // left: stages left of the tile
        const int buf = acc_i & 1, n = kF32 ? min(per, left) : KB;
        if (!__all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(&acce[buf]), ((acc_i >> 1) & 1) ^ 1, ctl))) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + buf * 256;
        [[maybe_unused]] int count = 0, mt, nt;
        if constexpr (kLora) {
          tile_at(t, mt, nt);
          if (n == left && t != first) count = adapters_of(p.lora_lists + (int64_t)mt * kLoraListInts);
        }
        uint32_t accumulate = 0;
        for (int kb = 0; kb < n; ++kb) {
          if (!warp_wait_quick(full0 + 8 * stage, kLora ? full_bits >> stage & 1 : phase, ctl)) {
            ok = false;
            break;
          }
          if (kLora) full_bits ^= 1u << stage;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
#pragma unroll
            for (int i = 0; i < kKps; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::tc_mma_f16_pair_lo(d, lo + i * lo_block + 2 * q, lo + i * lo_block + (lin::kTileBytes >> 4) + 2 * q, desc_hi,
                                        idesc, i + q > 0 ? 1u : accumulate);
            ptx::tc_commit_pair(empty0 + 8 * stage);
            if (kb == n - 1 && (!(kLora && n == left) || apart)) ptx::tc_commit_pair(ptx::smem_u32(&accf[buf]));
          }
          accumulate = 1;
          lo += lo_step;
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
            lo = lo0;
          }
        }
        if constexpr (kLora) {
          if (ok && n == left) {  // the tile's last accumulator takes the adapters, or the next one
            if (t == first) {
              if (p.lora_early) ptx::griddep_wait();
              count = adapters_of(p.lora_lists + (int64_t)mt * kLoraListInts);
            }
            const int units = count * rank_chunks;
            uint32_t to = d;
            if (apart && units > 0) {
              ++acc_i;
              if (!__all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(&acce[acc_i & 1]), ((acc_i >> 1) & 1) ^ 1, ctl))) break;
              ptx::tc_fence_after();
              to = tmem_base + (acc_i & 1) * 256;
              accumulate = 0;
            }
            for (int u = 0; u < units; u += kKps) {
              if (!(ok = __all_sync(0xffffffffu, wait_bar_cluster(ptx::smem_u32(&ad.built[stage]), built_bits >> stage & 1, ctl)))) break;
              built_bits ^= 1u << stage;
              ptx::tc_fence_after();
              if (ptx::elect_one()) {
                for (int i = 0; i < kKps && u + i < units; ++i) {
                  const int steps = Terms::steps(p.lora_rank, u + i >= count * (rank_chunks - 1) ? Terms::kRanks * (rank_chunks - 1) : 0);
                  const uint32_t xa = lo + i * lo_block, wb = xa + (lin::kTileBytes >> 4);
                  for (int q = 0; q < steps; ++q)
#pragma unroll
                    for (int t = 0; t < Terms::kTerms; ++t)
                      ptx::tc_mma_f16_pair_lo(to, xa + t * Terms::kPieces + 2 * q, wb + 2 * q, desc_hi, idesc, kF32 && i + q + t == 0 ? accumulate : 1u);
                }
                ptx::tc_commit_pair(empty0 + 8 * stage);
              }
              accumulate = 1;
              lo += lo_step;
              if (++stage == n_stages) {
                stage = 0;
                phase ^= 1;
                lo = lo0;
              }
            }
            if (!ok) break;
            if ((!apart || units > 0) && ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(&accf[acc_i & 1]));
          }
        }
        ++acc_i;
        if (kF32) left = left > n ? left - n : KB;
      }
      if (ptx::elect_one()) ptx::tc_commit_pair(ptx::smem_u32(drain));
      wait_bar_drain(ptx::smem_u32(drain), 0);
    }
    __syncwarp();
  } else if (kLora && warp >= lin::kLoraWarp) {
    if constexpr (kLora) {
      const int part = warp - lin::kLoraWarp;
      int stage = 0;
      uint32_t loaded_bits = 0;
      if (p.lora_early) ptx::griddep_wait();
      if (part == 0)
        for (int i = blockIdx.x * 32 + lane; i < p.lora_err_count; i += gridDim.x * 32)
          if (const uint32_t e = p.lora_errs[i]) atomicOr(s_err, e);
      for (int t = first; t < tiles; t += pairs) {
        int mt, nt;
        tile_at(t, mt, nt);
        AdapterList list;
        list.load(p, mt);
        stage = (stage + KB) % n_stages;
        if (!build_adapters<kKps, kF32, lin::kLoraWarps<kF32>>(p, ad, smem, stage_bytes, block_bytes, n_stages, 0, 128, lin::kTileBytes, BN / 2,
                                  (int64_t)mt * 256 + 128 * rank, part, list, 0, list.n * rank_chunks, 0, stage, loaded_bits, ctl))
          break;
      }
    }
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
        if constexpr (kLora) {
          if (nt == 0 && i == 0 && half == 0 && m0 + lane < p.M) adapter_of(p, m0 + lane, s_err);  // reported once
          const int64_t n = n0 + 32 * half + 64 * i;
          if (*(volatile int32_t*)&ad.not_finite && m0 + lane < p.M && n < p.N) {
            const int a = p.lora_ids[m0 + lane], left = (int)min(p.N - n, (int64_t)32);
            const float* s = p.lora_s + (m0 + lane) * p.lora_rank;
            add_adapter<32, true>(p, a, s, p.lora_parts, p.lora_part, n, left, v);
            if constexpr (kGated) add_adapter<32, true>(p, a, s, p.lora_parts, p.lora_part, p.N + n, left, u);
          }
          __syncwarp();
        }
        if (p.bias) add_bias32(bias[i], v, turn);
        if constexpr (kGated) {
          if (p.bias) add_bias32(bias_up[i], u, turn);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = silu<!kF32>(v[j]) * u[j];
        } else {
          if constexpr (kLora) {
            activate_all<!kF32>(p.act, v);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = activate<!kF32>(kAct, v[j]);
          }
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
        for (int kb = 0, end = KB; kb < end; kb += per) {
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
          if constexpr (kLora) {
            if (apart && end == KB && kb + per >= KB) {  // the adapters' own
              if (t == first && p.lora_early) ptx::griddep_wait();
              if (adapters_of(p.lora_lists + (int64_t)mt * kLoraListInts)) end = kb + per + 1;
            }
          }
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
template <int kAct, bool kF32, bool kLora>
__global__ void __launch_bounds__(lin::kThreads + (kLora ? 32 * lin::kLoraWarps<kF32> : 0), 1)
    linear_stream_kernel(const __grid_constant__ LinearMaps maps, const __grid_constant__ LinearParams p) {
  constexpr bool kGated = kAct == GMMFR_ACT_SWIGLU;
  constexpr int kCols = kGated ? 64 : 128;  // columns of y per tile
  constexpr int kEpi = lin::kThreads - 64, kKps = lin::kStreamKps;  // kEpi: the epilogue's threads
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
  [[maybe_unused]] AdapterShared& ad = *reinterpret_cast<AdapterShared*>(smem + lin::kStreamArena + lin::kStreamBars * 8 + 32);
  using Terms = SumTerms<kF32>;
  [[maybe_unused]] const int rank_chunks = Terms::blocks(p.lora_rank);  // kLora: blocks of an adapter
  [[maybe_unused]] const bool apart = Terms::apart(p.lora_rank);
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
    if constexpr (kLora) init_adapters(ad, n_stages, lin::kLoraWarps<kF32>);
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
  if (!kLora && !p.beside) ptx::griddep_wait();  // kLora: as in the direct form, who reads the sums or lists waits
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
      if constexpr (kLora) {  // one list serves all tiles
        if (!ok) break;
        if (t == first && !p.beside) ptx::griddep_wait();
        AdapterList list;
        list.load(p, 0);
        const int n = list.n, u0 = n * rank_chunks * (int)rank / S, u1 = n * rank_chunks * ((int)rank + 1) / S;
        AdapterBlocks next(list, u0);
        for (int u = u0; u < u1; u += kKps) {
          if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
            ok = false;
            break;
          }
          const uint32_t lb = ptx::smem_u32(&ad.loaded[stage]);
          int adapter[kKps], rank0[kKps];
#pragma unroll
          for (int h = 0; h < kKps; ++h) {
            rank0[h] = Terms::kRanks * next.c;
            adapter[h] = next.adapter();
            next.next();
          }
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(lb, min(kKps, u1 - u) * lin::kTileBytes);
#pragma unroll
            for (int h = 0; h < kKps; ++h)
              if (u + h < u1) {
                const uint32_t to = sb + h * block_bytes;
                ptx::tma_load_3d(to, &maps.b, rank0[h], y, adapter[h], lb, pol_w);
                if constexpr (kGated) ptx::tma_load_3d(to + 64 * 128, &maps.b, rank0[h], y_up, adapter[h], lb, pol_w);
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
    }
    for (int s = 0; ok && s < n_stages; ++s) {  // no load is in flight at exit
      ok = warp_wait_quick(ptx::smem_u32(&empty[stage]), phase ^ 1, ctl);
      if (++stage == n_stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (kLora && !ok) let_loads_land();
    else if (!ok)  // aborted: let what is in flight land
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
    [[maybe_unused]] uint32_t full_bits = 0, built_bits = 0;  // kLora: a barrier's phase by its own uses
    bool ok = true;
    for (int t = first, k0 = kb0; ok && t < tiles; t += k0 == kb0 ? clusters : 0) {
      const int k1 = kF32 ? min(k0 + per, kb1) : kb1;
      if (!warp_wait_quick(ptx::smem_u32(&acce[acc_of(acc_i)]), phase_of(acc_i) ^ 1, ctl)) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem_base + acc_of(acc_i) * acc_cols;
      uint32_t accumulate = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!warp_wait_quick(full0 + 8 * stage, kLora ? full_bits >> stage & 1 : phase, ctl)) {
          ok = false;
          break;
        }
        if (kLora) full_bits ^= 1u << stage;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
#pragma unroll
          for (int h = 0; h < kKps; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              ptx::tc_mma_f16_lo(d, lo + h * lo_block + 2 * q, lo + h * lo_block + (lin::kTileBytes >> 4) + 2 * q, desc_hi, idesc,
                                 h + q > 0 ? 1u : accumulate);
          ptx::tc_commit(empty0 + 8 * stage);
          if (kb == k1 - 1 && (!(kLora && k1 == kb1) || apart)) ptx::tc_commit(ptx::smem_u32(&accf[acc_of(acc_i)]));
        }
        accumulate = 1;
        lo += lo_step;
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
          lo = lo0;
        }
      }
      if constexpr (kLora) {
        if (ok && k1 == kb1) {  // the tile's last accumulator takes the adapters, or the next one
          if (t == first && !p.beside) ptx::griddep_wait();
          const int count = adapters_of(p.lora_lists), u0 = count * rank_chunks * (int)rank / S, u1 = count * rank_chunks * ((int)rank + 1) / S;
          uint32_t to = d;
          if (apart && u0 < u1) {
            ++acc_i;
            if (!warp_wait_quick(ptx::smem_u32(&acce[acc_of(acc_i)]), phase_of(acc_i) ^ 1, ctl)) break;
            ptx::tc_fence_after();
            to = tmem_base + acc_of(acc_i) * acc_cols;
            accumulate = 0;
          }
          for (int u = u0; u < u1; u += kKps) {
            if (!(ok = warp_wait_quick(ptx::smem_u32(&ad.built[stage]), built_bits >> stage & 1, ctl))) break;
            built_bits ^= 1u << stage;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
              for (int h = 0; h < kKps && u + h < u1; ++h) {
                const int steps = Terms::steps(p.lora_rank, u + h >= count * (rank_chunks - 1) ? Terms::kRanks * (rank_chunks - 1) : 0);
                const uint32_t wa = lo + h * lo_block, xb = wa + (lin::kTileBytes >> 4);
                for (int q = 0; q < steps; ++q)
#pragma unroll
                  for (int t = 0; t < Terms::kTerms; ++t)
                    ptx::tc_mma_f16_lo(to, wa + 2 * q, xb + t * Terms::kPieces + 2 * q, desc_hi, idesc, kF32 && h + q + t == 0 ? accumulate : 1u);
              }
              ptx::tc_commit(empty0 + 8 * stage);
            }
            accumulate = 1;
            lo += lo_step;
            if (++stage == n_stages) {
              stage = 0;
              phase ^= 1;
              lo = lo0;
            }
          }
          if (!ok) break;
          if ((!apart || u0 < u1) && ptx::elect_one()) ptx::tc_commit(ptx::smem_u32(&accf[acc_of(acc_i)]));
        }
      }
      ++acc_i;
      if (kF32) k0 = k1 == kb1 ? kb0 : k1;
    }
    if (ptx::elect_one()) ptx::tc_commit(ptx::smem_u32(drain));
    wait_bar_drain(ptx::smem_u32(drain), 0);
    __syncwarp();
  } else if (kLora && warp >= lin::kLoraWarp) {
    if constexpr (kLora) {
      const int part = warp - lin::kLoraWarp;
      int stage = 0;
      uint32_t loaded_bits = 0;
      if (!p.beside) ptx::griddep_wait();
      AdapterList list;
      list.load(p, 0);
      for (int t = first; t < tiles; t += clusters) {
        stage = (stage + kb1 - kb0) % n_stages;
        if (!build_adapters<kKps, kF32, lin::kLoraWarps<kF32>>(p, ad, smem, stage_bytes, block_bytes, n_stages, lin::kTileBytes, npad, 0, 128, 0, part, list,
                                  list.n * rank_chunks * (int)rank / S, list.n * rank_chunks * ((int)rank + 1) / S, -1, stage, loaded_bits,
                                  ctl))
          break;
      }
    }
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
        for (int kb = kb0, end = kb1; ok && kb < end; kb += per) {
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
          if constexpr (kLora) {
            if (apart && end == kb1 && kb + per >= kb1) {  // the adapters' own
              if (t == first && !p.beside) ptx::griddep_wait();
              const int blocks = adapters_of(p.lora_lists) * rank_chunks;
              if (blocks * (int)rank / S < blocks * ((int)rank + 1) / S) end = kb + per + 1;
            }
          }
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
          float g[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
          if constexpr (kLora) {
            if (t == 0 && c == 0) adapter_of(p, tok, s_err);  // reported once
            if (*(volatile int32_t*)&ad.not_finite) {
              const float* s = p.lora_s + (int64_t)tok * p.lora_rank;
              add_adapter<4, true>(p, p.lora_ids[tok], s, p.lora_parts, p.lora_part, n, cols, f);
              if constexpr (kGated) add_adapter<4, true>(p, p.lora_ids[tok], s, p.lora_parts, p.lora_part, p.N + n, cols, g);
            }
          }
          if constexpr (kLora && !kGated) {
            activate_all<false>(p.act, f);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (kGated) f[k] = silu(f[k]) * (g[k] + bias_up[k]);
              else f[k] = activate(kAct, f[k]);
            }
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

// ============================================================================ launch
template <int kAct, bool kF32, bool kLora>
static cudaError_t launch_one(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  auto kernel = p.form == kLinearStream ? linear_stream_kernel<kAct, kF32, kLora>
                                        : (p.kps == 1 ? linear_pair_kernel<kAct, 1, kF32, kLora> : linear_pair_kernel<kAct, 2, kF32, kLora>);
  constexpr int kMore = kLora ? (int)sizeof(AdapterShared) : 0, kPairBytes = lin::kPairSmem + kMore;
  constexpr int kStreamBytes = lin::kStreamSmem + kMore;
  static_assert(kStreamBytes <= 232448 && kPairBytes <= 232448, "shared memory budget");
  const int smem = p.form == kLinearStream ? kStreamBytes : kPairBytes;
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(linear_stream_kernel<kAct, kF32, kLora>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(linear_pair_kernel<kAct, 1, kF32, kLora>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(linear_pair_kernel<kAct, 2, kF32, kLora>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)p.grid);
  lc.blockDim = dim3((p.form == kLinearStream ? lin::kThreads : lin::kPairThreads) + (kLora ? 32 * lin::kLoraWarps<kF32> : 0));
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

template <bool kF32, bool kLora>
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
    constexpr decltype(&linear_direct_kernel<true, 1, kF32, kLora>) kernels[2][3] = {
        {linear_direct_kernel<false, 1, kF32, kLora>, linear_direct_kernel<false, 2, kF32, kLora>, linear_direct_kernel<false, 4, kF32, kLora>},
        {linear_direct_kernel<true, 1, kF32, kLora>, linear_direct_kernel<true, 2, kF32, kLora>, linear_direct_kernel<true, 4, kF32, kLora>}};
    return cudaLaunchKernelEx(&lc, kernels[p.act == GMMFR_ACT_SWIGLU][tiles], p);
  }
  if constexpr (kLora) {
    return p.act == GMMFR_ACT_SWIGLU ? launch_one<GMMFR_ACT_SWIGLU, kF32, true>(maps, p, s) : launch_one<GMMFR_ACT_NONE, kF32, true>(maps, p, s);
  } else switch (p.act) {
    case GMMFR_ACT_RELU: return launch_one<GMMFR_ACT_RELU, kF32, kLora>(maps, p, s);
    case GMMFR_ACT_GELU: return launch_one<GMMFR_ACT_GELU, kF32, kLora>(maps, p, s);
    case GMMFR_ACT_GELU_TANH: return launch_one<GMMFR_ACT_GELU_TANH, kF32, kLora>(maps, p, s);
    case GMMFR_ACT_SILU: return launch_one<GMMFR_ACT_SILU, kF32, kLora>(maps, p, s);
    case GMMFR_ACT_SWIGLU: return launch_one<GMMFR_ACT_SWIGLU, kF32, kLora>(maps, p, s);
    default: return launch_one<GMMFR_ACT_NONE, kF32, kLora>(maps, p, s);
  }
}

}  // namespace gmmfr
