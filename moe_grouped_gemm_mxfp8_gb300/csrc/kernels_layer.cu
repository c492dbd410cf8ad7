// A whole mixture-of-experts layer for a few tokens (at most 64), in two kernels.
//
//   front   the gate; the tokens as images of the products' B operand; counters to zero
//   layer   one persistent CTA per SM; two runs of weight tiles
//             up          x times the gate/up tiles of the shared expert and of the chosen ones
//             down        column tile by column tile: sw times the down tiles of every chosen expert and of
//                         the shared one, one long sum over (expert, intermediate index)
//           each run cut into equal contiguous ranges over the CTAs.
//
// The weights are the 128-row operand of tcgen05.mma (prepared tiles, one bulk copy each), the tokens the N-wide
// one: all T of them for every expert (T padded to 16), since the time goes to the weights' bytes and a token
// that did not choose the expert costs only tensor-core slots that would idle.  Its row of sw is zero, which lets
// the down run add all experts of a column tile into the same accumulator, the router's weight being folded into
// sw (in FP32, before its rounding).  Zero times an infinite or NaN weight is NaN: sums that come out NaN are made
// again from the experts that the token chose (own_sums).
// The weights' producer never waits for a token: the first down tiles are requested while other CTAs still finish
// the up run.
//
// A column tile cut between CTAs is joined through the workspace: each piece stores its FP32 sums, and
//   up     one of its CTAs adds the pieces in CTA order, applies SwiGLU and stores sw;
//   down   every CTA with a piece waits for the others at its end and adds its share of the tile.
// Both orders are fixed, so results are the same bits every time.
//
// H = 2048, 256 experts of 512 with a shared one, 8 per token, BF16: 64 tokens (1408 MB) 229 us, 6.1 TB/s, 92% of a copy's
// rate; 13 tokens that share experts (491 MB) 87.8 us, 5.6 TB/s.  One token (58 MB) 28 us, 2.1 TB/s: latencies, one
// after the other: the gate 6, launch, set-up and first copy 4, the stream 10, the two joins and the up run's
// hand-over 8; the same 18 us or so stand in the larger calls.
// MXFP8, 16 experts of 7168 x 2048 with a shared one of 4096, 40 tokens (819 MB): 151 us, 5.4 TB/s; 16 of it between
// the runs, while the units with all 40 tokens are finished.
//
// sw is rounded to what the tensor cores take: BF16, or with MXFP8 weights a sum of two E4M3 numbers with
// their block scales (hi + lo, about as exact as BF16), and the tokens likewise: BF16's eight bits split exactly
// into hi and lo, so that MXFP8 weights meet unrounded activations (down to 2^-14 of the block's largest; what is
// smaller is off by at most 2^-22 of it).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "epilogue.cuh"
#include "gate_select.cuh"
#include "ops.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace gmmfr {

// MXFP8 tiles (include/gmmfr.h, gmmfr_ffn_prepare_weights_mx): the code of row r, K byte c of a tile
// at r * 128 + ((c / 16) ^ (r % 8)) * 16 + c % 16, the scale of row r, 32-block q at
// 16384 + 16 * (r % 32) + 4 * (r / 32) + q.  Codes past the matrix are 0, their scales 127 (1.0).
__global__ void __launch_bounds__(256) ffn_prep_mx_kernel(FfnPrepMxParams p) {
  const int64_t t1 = (int64_t)p.E * p.NT1 * p.KB1, t2 = (int64_t)p.E * p.NT2 * p.KB2;
  for (int64_t tile = blockIdx.x; tile < t1 + t2; tile += gridDim.x) {
    const bool first = tile < t1;
    const int64_t lt = first ? tile : tile - t1;
    const int KB = first ? p.KB1 : p.KB2, NT = first ? p.NT1 : p.NT2;
    const int64_t kb = lt % KB, j = (lt / KB) % NT, e = lt / ((int64_t)KB * NT);
    const int64_t K = first ? p.H : p.I, N = first ? 2 * p.I : p.H;
    const uint8_t* src = (first ? p.w13 : p.w2) + e * K * N;
    const int64_t Ks = (K + 63) / 64;
    const uint8_t* ssrc = (first ? p.s13 : p.s2) + e * Ks * N * 2;
    uint8_t* dst = p.prepared + tile * kPrepTileBytes;
    auto column = [&](int r) -> int64_t {  // the matrix column of tile row r, -1 past the matrix
      if (!first) return j * 128 + r < N ? j * 128 + r : -1;
      const int64_t i = j * 64 + (r & 63);
      return i < p.I ? (r < 64 ? i : p.I + i) : -1;
    };
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int id = threadIdx.x + it * 256;
      const int r = id & 127, c = id >> 7;
      const int64_t n = column(r);
      uint8_t b[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t k = kb * 128 + c * 16 + i;
        b[i] = n >= 0 && k < K ? src[k * N + n] : 0;
      }
      *reinterpret_cast<uint4*>(dst + r * 128 + ((c ^ (r & 7)) << 4)) = *reinterpret_cast<const uint4*>(b);
    }
    for (int id = threadIdx.x; id < kSfChunk; id += 256) {
      const int r = id & 127, q = id >> 7;
      const int64_t n = column(r), g = kb * 4 + q;
      dst[kWTileBytes + 16 * (r & 31) + 4 * (r >> 5) + q] =
          n >= 0 && g * 32 < K ? ssrc[((g >> 1) * N + n) * 2 + (g & 1)] : 127;
    }
  }
}

cudaError_t launch_ffn_prep_mx(const FfnPrepMxParams& p, cudaStream_t s) {
  const int64_t tiles = (int64_t)p.E * p.NT1 * p.KB1 + (int64_t)p.E * p.NT2 * p.KB2;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t grid = tiles < (int64_t)sms * 8 ? tiles : (int64_t)sms * 8;
  ffn_prep_mx_kernel<<<(unsigned)grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

namespace layer {

constexpr int kThreads = 256;  // warp 0 weights, 1 MMA, 2..5 epilogue, 6 tokens' producer
// HBM gives more to rings that are not too deep (13 tokens, 256 experts of 2048: 4, 6, 8, 10 stages take 91.9, 88.9, 89.4,
// 91.5 us; 64 tokens, 7 and 8 stages: 230 and 236).
constexpr int kMaxStages = 6;
constexpr int kFrontAhead = 16 << 20;  // bytes that HBM has time for while the router works
constexpr int kRound = 4;  // tokens whose SwiGLU values are made at a time
// A stage: weight tile (with MXFP8 its 512 scale bytes), then the tokens' image: BF16 npad rows of 128 bytes;
// MXFP8 the scale chunk of hi and lo (512 bytes), npad rows of hi codes, npad of lo.
__host__ __device__ constexpr int tile_bytes(bool mx) { return mx ? kPrepTileBytes : kWTileBytes; }
__host__ __device__ constexpr int rows_off(bool mx) { return mx ? kPrepTileBytes + kSfChunk : kWTileBytes; }
__host__ __device__ constexpr int image_bytes(bool mx, int npad) { return mx ? kSfChunk + 256 * npad : 128 * npad; }
__host__ __device__ constexpr int stage_bytes(bool mx, int npad) { return tile_bytes(mx) + image_bytes(mx, npad); }
constexpr int kArena = 180 * 1024;
__host__ __device__ constexpr int n_stages(bool mx, int npad) {
  return kArena / stage_bytes(mx, npad) < kMaxStages ? kArena / stage_bytes(mx, npad) : kMaxStages;
}
static_assert(stage_bytes(true, 8) % 1024 == 0 && stage_bytes(false, 16) % 1024 == 0 && rows_off(true) % 1024 == 0,
              "swizzled operands need 1024-byte alignment");
constexpr int kBarOff = kArena;
constexpr int kNumBars = 2 * kMaxStages + 5;
constexpr int kMiscOff = kBarOff + kNumBars * 8 + 8;             // int32 misc[16]
constexpr int kMaskOff = kMiscOff + 64;                          // uint64 mask[1024]: tokens of each expert
constexpr int kActOff = kMaskOff + 8 * kMaxExperts;              // uint16 act[1024]: the chosen experts
constexpr int kIdsOff = kActOff + 2 * kMaxExperts;               // uint16 ids[64 * 32]
constexpr int kWtOff = kIdsOff + 2 * kLayerMaxTokens * kMaxTopk; // float weights[64 * 32]
constexpr int kXchgOff = kWtOff + 4 * kLayerMaxTokens * kMaxTopk;  // float [kRound][2][32]: values handed over for SwiGLU
constexpr int kTokWOff = kXchgOff + kRound * 2 * 32 * 4;             // float [64]: the unit's router weights
constexpr int kSmemBytes = kTokWOff + 4 * kLayerMaxTokens + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
// TMEM: two accumulators of acc_cols columns (MXFP8: the products with hi, then those with lo), then with MXFP8 the
// scale columns of every stage
__host__ __device__ constexpr int acc_cols(bool mx, int npad) { return mx ? 2 * npad : npad; }
__host__ __device__ constexpr int tmem_cols(bool mx) { return mx ? 512 : 128; }
static_assert(2 * acc_cols(true, 64) + 8 * n_stages(true, 64) <= tmem_cols(true) &&
                  2 * acc_cols(true, 8) + 8 * n_stages(true, 8) <= tmem_cols(true) && 2 * acc_cols(false, 64) <= tmem_cols(false),
              "TMEM");

}  // namespace layer

namespace {

// 16-byte chunk c of row t of a 128-byte-row image with the 128-byte swizzle.
__device__ __forceinline__ int image_chunk(int t, int c) { return t * 128 + ((c ^ (t & 7)) << 4); }
// Scale byte of row t, 32-block q of a tile (the layout tcgen05.cp 32x128b.warpx4 spreads over TMEM).
__device__ __forceinline__ int scale_at(int t, int q) { return 16 * (t & 31) + 4 * (t >> 5) + q; }

// The power of two that puts a block with largest magnitude bits `amax` into E4M3's upper range: hi codes stand
// for x / 2^(e-7) (below 256 of E4M3's 448), lo codes for the rest in units of 2^(e-12).  Blocks below 2^-100
// keep that unit.  A block with an infinity or NaN gets the NaN scale: its products are NaN.
struct BlockScale {
  float inv_hi, unit_hi, inv_lo;
  uint32_t byte_hi, byte_lo;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax) {
  BlockScale b;
  int e = (int)(amax >> 23) - 127;
  const bool finite = e < 128;
  e = e < -100 ? -100 : (finite ? e : 0);
  b.inv_hi = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
  b.unit_hi = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
  b.inv_lo = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
  b.byte_hi = finite ? (uint32_t)(127 + e - 7) : 255u;
  b.byte_lo = finite ? (uint32_t)(127 + e - 12) : 255u;
  return b;
}
__device__ __forceinline__ void split_e4m3(float x, const BlockScale& b, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float_to_fp8(x * b.inv_hi, __NV_SATFINITE, __NV_E4M3);
  const float h = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)hi, __NV_E4M3)));
  lo = __nv_cvt_float_to_fp8((x - h * b.unit_hi) * b.inv_lo, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_add(uint32_t* p, uint32_t v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Bounded wait until *p reaches n.
__device__ __forceinline__ bool wait_count(const uint32_t* p, uint32_t n, const Ctl& c) {
  Deadline d;
  while (ld_acquire(p) < n)
    if (!d.go_on(c)) return false;
  return true;
}

// Tokens c0 .. c0 + 15 of this thread's accumulator row (MXFP8: the sums with hi and with lo).
template <bool kMx>
__device__ __forceinline__ void load_acc16(uint32_t taddr, int npad, float (&v)[16]) {
  uint32_t r[16];
  ptx::tmem_ld_32x32b_x16(taddr, r);
  if constexpr (kMx) {
    uint32_t l[16];
    ptx::tmem_ld_32x32b_x16(taddr + npad, l);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]) + __uint_as_float(l[i]);
  } else {
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  }
}

// One run of U tiles in units of K tiles, cut evenly over the first G CTAs: CTA b has [U b / G, U (b + 1) / G).  A
// small run leaves some CTAs out: fewer than four tiles each save less in streaming than their joins cost.
// (The host refuses sizes whose U * G passes 32 bits.)
struct Run {
  uint32_t U, K, G;
  __device__ Run(uint32_t U_, uint32_t K_, uint32_t ctas) : U(U_), K(K_), G(min(ctas, max(1u, U_ / 4))) {}
  __device__ uint32_t lo(uint32_t b) const { return b < G ? U * b / G : U; }
  __device__ uint32_t owner(uint32_t x) const { return ((x + 1) * G - 1) / U; }
};
// The pieces of unit u: those of n consecutive CTAs from b0 (every CTA of the run has a tile at least).  A CTA's pieces
// of cut units lie in its two slots: 0 where its range begins in the unit, 1 where it ends there; so only the first
// piece of a unit can lie in slot 1.
struct Pieces {
  uint32_t b0, n, first_slot, x0;
  __device__ Pieces(const Run& r, uint32_t u) : x0(u * r.K) {
    b0 = r.owner(x0);
    n = r.owner(x0 + r.K - 1) - b0 + 1;
    first_slot = r.lo(b0) >= x0 ? 0 : 1;
  }
  __device__ uint32_t slot(uint32_t i) const { return (b0 + i) * 2 + (i == 0 ? first_slot : 0); }
};

// The pieces of one CTA: units (or parts of units) of the two runs in order; every role walks them.
struct Walk {
  const Run *up, *down;
  uint32_t pos, end, end2;
  uint32_t unit, k0, k1;
  bool is_down;  // of the current piece
  __device__ Walk(const Run& up_, const Run& down_) : up(&up_), down(&down_), is_down(false) {
    pos = up->lo(blockIdx.x);
    end = up->lo(blockIdx.x + 1);
  }
  __device__ bool next() {
    if (pos == end) {
      if (is_down) return false;
      is_down = true;
      pos = down->lo(blockIdx.x);
      end = down->lo(blockIdx.x + 1);
      if (pos == end) return false;
    }
    const uint32_t K = is_down ? down->K : up->K;
    unit = pos / K;
    k0 = pos - unit * K;
    k1 = min(K, k0 + (end - pos));
    pos += k1 - k0;
    return true;
  }
};

// One E8M0 scale, and 32 K elements of a row in MXFP8: codes in two 16-byte chunks of an image, for a sum in FP32.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}
__device__ __forceinline__ float scaled(float s, uint32_t a, uint32_t b) {  // s 2^(a - 127) 2^(b - 127)
  return a == 255u || b == 255u ? __int_as_float(0x7fffffff) : ldexpf(s, (int)(a + b) - 254);
}

// sum over k of tiles[r, k] sw[t, k] over KB tiles of consecutive K
template <bool kMx>
__device__ float row_product(const uint8_t* tiles, int r, const uint8_t* images, int t, int KB, int npad) {
  float s = 0.f;
  const int img = layer::image_bytes(kMx, npad), tile = layer::tile_bytes(kMx);
#pragma unroll 1
  for (int kb = 0; kb < KB; ++kb, tiles += tile, images += img) {
    if constexpr (!kMx) {
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(tiles + image_chunk(r, c));
        const uint4 x4 = *reinterpret_cast<const uint4*>(images + image_chunk(t, c));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w}, x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = fmaf(__uint_as_float(w[i] << 16), __uint_as_float(x[i] << 16), s);
          s = fmaf(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(x[i] & 0xffff0000u), s);
        }
      }
    } else {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float hi = 0.f, lo = 0.f;
#pragma unroll 1
        for (int c = 2 * q; c < 2 * q + 2; ++c) {
          const uint8_t* w = tiles + image_chunk(r, c);
          const uint8_t* x = images + kSfChunk + image_chunk(t, c);
#pragma unroll 1
          for (int i = 0; i < 16; ++i) {
            const float v = e4m3_value(w[i]);
            hi = fmaf(v, e4m3_value(x[i]), hi);
            lo = fmaf(v, e4m3_value(x[npad * 128 + i]), lo);
          }
        }
        const uint32_t b = tiles[kWTileBytes + scale_at(r, q)];
        s += scaled(hi, b, images[scale_at(t, q)]) + scaled(lo, b, images[scale_at(npad + t, q)]);
      }
    }
  }
  return s;
}

// Columns n .. n + 3 of token t's result, without the residual, of which s holds the accumulated sums: those that are NaN
// made again from the experts that t chose and the shared one alone.  A token with a NaN among its own SwiGLU values keeps
// them; another's stay NaN when a down weight of its own experts made them, and else it was an infinite or NaN weight of an
// expert that only other tokens chose.  A rare call, kept out of line and small rather than fast: all of 64 x 7168 results
// of 16 experts of 2048 take 20 ms (BF16) or 53 (MXFP8).
template <bool kMx>
__device__ __noinline__ float4 own_sums(const LayerParams& p, const uint16_t* s_act, const uint16_t* s_ids, int A, int n_units, int t,
                                        int64_t n0, float4 s) {
  // every unit's sw is there (the sums were made of them), and with this read they are visible to this thread too
  if (ld_acquire(p.up_done) < (uint32_t)n_units || __ldcg(p.nan_rows + t) != 0) return s;
  const int topk = p.gate.rule.topk, tile = layer::tile_bytes(kMx);
  const int64_t img = layer::image_bytes(kMx, p.npad);
  float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    if (f[i] == f[i]) continue;
    const int j = (int)((n0 + i) >> 7), r = (int)((n0 + i) & 127);
    float own = 0.f;
#pragma unroll 1
    for (int k = 0; k <= topk; ++k) {
      const uint8_t *tiles = p.shared2 + (int64_t)j * p.KB2s * tile, *images = p.swimg_s;  // last
      if (k < topk) {
        const int e = s_ids[t * topk + k];
        int a = 0;  // its place among the chosen experts, which are in order
        while (a < A - 1 && s_act[a] != e) ++a;
        tiles = p.prepared2 + ((int64_t)e * p.NT2 + j) * p.KB2 * tile;
        images = p.swimg + a * p.KB2 * img;
      }
      own += row_product<kMx>(tiles, r, images, t, k < topk ? p.KB2 : p.KB2s, p.npad);
    }
    f[i] = own;
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}

}  // namespace

// ============================================================================ front
// The first T / 8 clusters are the router (gate_select.cuh); the others make the token images and zero the counters.
template <bool kMx, int kThr>
__global__ void __launch_bounds__(kThr) layer_front_kernel(const __grid_constant__ LayerParams p) {
  __shared__ gate::Smem<1, kThr> sm;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const GateParams& g = p.gate;
  const int T = (int)g.T;
  const int lane = threadIdx.x & 31;
  const int routers = (T + 7) / 8 * gate::kCluster;
  if ((int)blockIdx.x < routers) {
    gate_cluster<1, kThr, 1>(g, (int64_t)(blockIdx.x / gate::kCluster) * 8, sm, ptx::cluster_rank());
    return;
  }
  const int block = blockIdx.x - routers, blocks = gridDim.x - routers, warps = blocks * (kThr / 32);
  const int tid = threadIdx.x * blocks + block, threads = blocks * kThr;
  for (int i = tid; i < p.n_counters; i += threads) p.counters[i] = 0;
  // The shared expert's gate and up tiles, whoever the router chooses, into L2 while it works (17 tokens, 60 experts of 3536,
  // shared 688: 55.4 -> 53.0 us).  Of more than fit in that time a part would run a few CTAs ahead of the others and gain
  // nothing (40 tokens MXFP8, 60 MB: 12 of them ahead 152.7 us, none 152.2).
  const int tile = layer::tile_bytes(kMx), shared_tiles = p.NT1s * p.KB1;
  if (threadIdx.x == 0 && (int64_t)shared_tiles * tile <= layer::kFrontAhead)
    for (int i = block; i < shared_tiles; i += blocks) ptx::bulk_prefetch_l2(p.shared + (int64_t)i * tile, tile);
  // images: 8 elements of a row per thread, zero past H (their weights are zero, but 0 x NaN is not)
  const int img = layer::image_bytes(kMx, p.npad);
  const int per_row = p.KB1 * (kMx ? 16 : 8);
  // a warp's 32 items are consecutive 8-element chunks of a row (per_row is a multiple of 8: quads never straddle)
  const int items = T * per_row, w_items = (items + 31) / 32;
  for (int wi = block + threadIdx.x / 32 * blocks; wi < w_items; wi += warps) {
    const int it = wi * 32 + lane;
    const bool in = it < items;
    const int t = in ? it / per_row : 0, c = in ? it - t * per_row : 0;
    const int64_t h = (int64_t)c * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in && h < g.H) v = *reinterpret_cast<const uint4*>(g.x + (int64_t)t * g.ldx + h);
    if constexpr (!kMx) {
      if (in) *reinterpret_cast<uint4*>(p.ximg + (int64_t)(c >> 3) * img + image_chunk(t, c & 7)) = v;
    } else {
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      uint32_t amax = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        amax = max(amax, (u[q] << 16) & 0x7fffffffu);
        amax = max(amax, u[q] & 0x7fff0000u);
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // four lanes hold a block of 32
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const BlockScale b = block_scale(amax);
      uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint32_t a, r;
        split_e4m3(__uint_as_float((q & 1) ? u[q >> 1] & 0xffff0000u : u[q >> 1] << 16), b, a, r);
        hi[q >> 2] |= a << (8 * (q & 3));
        lo[q >> 2] |= r << (8 * (q & 3));
      }
      if (in) {
        uint8_t* dst = p.ximg + (int64_t)(c >> 4) * img;
        const int at = image_chunk(t, (c & 15) >> 1) + (c & 1) * 8;
        *reinterpret_cast<uint2*>(dst + kSfChunk + at) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(dst + kSfChunk + p.npad * 128 + at) = make_uint2(lo[0], lo[1]);
        if ((c & 3) == 0) {
          dst[scale_at(t, (c & 15) >> 2)] = (uint8_t)b.byte_hi;
          dst[scale_at(p.npad + t, (c & 15) >> 2)] = (uint8_t)b.byte_lo;
        }
      }
    }
  }
}

// ============================================================================ layer
// Loops of unknown length are kept rolled: in a small call every instruction comes from memory the first time, and the
// shorter code is up to 5% faster there (39 tokens, 20 experts of 728: 32.2 -> 30.5 us) and nowhere slower.
template <bool kMx>
__global__ void __launch_bounds__(layer::kThreads, 2) layer_kernel(const __grid_constant__ LayerParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + layer::kBarOff);  // both producers' copies landed
  uint64_t* empty = full + layer::kMaxStages;
  uint64_t* accf = empty + layer::kMaxStages;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  int32_t* misc = reinterpret_cast<int32_t*>(smem + layer::kMiscOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&misc[0]);
  int* abort_flag = &misc[1];
  uint32_t* s_err = reinterpret_cast<uint32_t*>(&misc[2]);
  int* s_warp_sum = &misc[4];  // [8]
  unsigned long long* s_mask = reinterpret_cast<unsigned long long*>(smem + layer::kMaskOff);
  uint16_t* s_act = reinterpret_cast<uint16_t*>(smem + layer::kActOff);
  uint16_t* s_ids = reinterpret_cast<uint16_t*>(smem + layer::kIdsOff);
  float* s_wt = reinterpret_cast<float*>(smem + layer::kWtOff);
  float* xchg = reinterpret_cast<float*>(smem + layer::kXchgOff);
  float* s_tokw = reinterpret_cast<float*>(smem + layer::kTokWOff);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
  const GateParams& g = p.gate;
  const int T = (int)g.T, E = g.rule.E, topk = g.rule.topk, G = gridDim.x;
  const int npad = p.npad, acc = layer::acc_cols(kMx, npad), img = layer::image_bytes(kMx, npad);
  const int tile = layer::tile_bytes(kMx), stage_bytes = layer::stage_bytes(kMx, npad), n_stages = layer::n_stages(kMx, npad);
  const uint32_t smem_base = ptx::smem_u32(smem);

  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int s = 0; s < n_stages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&full[s]), 2);
      ptx::mbar_init(ptx::smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&accf[b]), 1 + p.test_stall);
      ptx::mbar_init(ptx::smem_u32(&acce[b]), 4);
    }
    ptx::mbar_init(ptx::smem_u32(drain), 1);
    *abort_flag = 0;
    *s_err = 0;
    ptx::fence_mbar_init();
  }
#pragma unroll 1
  for (int e = threadIdx.x; e < E; e += layer::kThreads) s_mask[e] = 0;
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), layer::tmem_cols(kMx));
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Ctl ctl{abort_flag, s_err, p.timeout_ns};

  ptx::griddep_wait();

  // ---------------------------------------------------------------- the chosen experts
#pragma unroll 1
  for (int i = threadIdx.x; i < T * topk; i += layer::kThreads) {
    const int e = static_cast<const int32_t*>(g.ids)[i];  // in [0, E): the front kernel's
    s_ids[i] = (uint16_t)e;
    s_wt[i] = g.weights[i];
    atomicOr(&s_mask[e], 1ull << (i / topk));
  }
  __syncthreads();
  // the chosen experts in index order: four experts per thread
  int A;
  {
    const int e0 = threadIdx.x * 4;
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += e0 + i < E && s_mask[e0 + i] != 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) s_warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - n, all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      before += w < warp ? s_warp_sum[w] : 0;
      all += s_warp_sum[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < E && s_mask[e0 + i] != 0) s_act[before++] = (uint16_t)(e0 + i);
    A = __shfl_sync(0xffffffffu, all, 0);  // uniform, so that what the roles derive from it is
  }
  __syncthreads();
  const int D = A * p.KB2 + p.KB2s;  // tiles of one column tile of the down run
  const int n_units = A * p.NT1 + p.NT1s;  // the shared expert's first
  const Run up((uint32_t)n_units * p.KB1, (uint32_t)p.KB1, (uint32_t)G), down((uint32_t)p.NT2 * D, (uint32_t)D, (uint32_t)G);
  Walk walk(up, down);
  // Aborted: lets a producer's copies in flight land.  The other producer's may never be asked for, which leaves a stage
  // short of its arrival; what was in flight has landed by the time such a wait gives up, whichever the stage.
  auto let_land = [&](int stage, uint32_t phase) {
#pragma unroll 1
    for (int s = 0; s < n_stages; ++s)
      if (!wait_bar_drain(ptx::smem_u32(&full[s]), s < stage ? phase : phase ^ 1)) break;
  };
  if (warp == 0) {
    // -------------------------------------------------------------- weights
    {
      const uint64_t pol = ptx::l2_evict_first_policy();
      const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
      int stage = 0;
      uint32_t phase = 0, sb = smem_base;
      bool ok = true;
      while (ok && walk.next()) {
        // the piece's tiles lie in runs of consecutive ones: `src` walks a run of `left` tiles
        const uint8_t* src = nullptr;
        int left = 0;
#pragma unroll 1
        for (int k = walk.k0; k < (int)walk.k1; ++k) {
          if (left == 0) {
            if (!walk.is_down) {
              const int u = (int)walk.unit - p.NT1s;
              if (u < 0) {
                src = p.shared + ((int64_t)walk.unit * p.KB1 + k) * tile;
              } else {
                const int a = u / p.NT1;
                src = p.prepared + (((int64_t)s_act[a] * p.NT1 + (u - a * p.NT1)) * p.KB1 + k) * tile;
              }
              left = p.KB1 - k;
            } else if (k < A * p.KB2) {
              const int a = k / p.KB2, kb = k - a * p.KB2;
              src = p.prepared2 + (((int64_t)s_act[a] * p.NT2 + walk.unit) * p.KB2 + kb) * tile;
              left = p.KB2 - kb;
            } else {
              src = p.shared2 + ((int64_t)walk.unit * p.KB2s + (k - A * p.KB2)) * tile;
              left = D - k;
            }
          }
          if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
            ok = false;
            break;
          }
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(full0 + 8 * stage, tile);
            ptx::bulk_g2s(sb, src, tile, full0 + 8 * stage, pol);
          }
          src += tile;
          --left;
          sb += stage_bytes;
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
            sb = smem_base;
          }
        }
      }
#pragma unroll 1
      for (int s = 0; ok && s < n_stages; ++s) {  // no copy is in flight at exit
        ok = warp_wait_quick(ptx::smem_u32(&empty[stage]), phase ^ 1, ctl);
        if (++stage == n_stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) let_land(stage, phase);
    }
    __syncwarp();
  } else if (warp == 6) {
    // -------------------------------------------------------------- the tokens' images
    {
      const uint64_t pol = ptx::l2_evict_last_policy();
      const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
      int stage = 0;
      uint32_t phase = 0, sb = smem_base + tile;
      const uint32_t bytes = img - (npad - T) * 128;  // without the rows past the tokens (their columns are not read)
      bool ok = true, sw_ready = false;
      while (ok && walk.next()) {
        if (walk.is_down && !sw_ready) {  // every unit of the up run has stored its sw
          ok = __all_sync(0xffffffffu, lane != 0 || wait_count(p.up_done, n_units, ctl)) != 0;
          asm volatile("fence.proxy.async;" ::: "memory");
          sw_ready = true;
          if (!ok) break;
        }
        // the shared expert's images follow the chosen ones' in the down run, in a buffer of their own
        const int past = walk.is_down ? (int)walk.k0 - A * p.KB2 : -1;
        const uint8_t* src = past >= 0 ? p.swimg_s + (int64_t)past * img
                                       : (walk.is_down ? p.swimg : p.ximg) + (int64_t)walk.k0 * img;
#pragma unroll 1
        for (int k = walk.k0; k < (int)walk.k1; ++k) {
          if (walk.is_down && past < 0 && k == A * p.KB2) src = p.swimg_s;
          if (!warp_wait_quick(empty0 + 8 * stage, phase ^ 1, ctl)) {
            ok = false;
            break;
          }
          if (ptx::elect_one()) {
            ptx::mbar_arrive_expect_tx(full0 + 8 * stage, bytes);
            ptx::bulk_g2s(sb, src, bytes, full0 + 8 * stage, pol);
          }
          src += img;
          sb += stage_bytes;
          if (++stage == n_stages) {
            stage = 0;
            phase ^= 1;
            sb = smem_base + tile;
          }
        }
      }
      if (!ok) let_land(stage, phase);  // (else the weights' producer sees every stage released)
    }
    __syncwarp();
  } else if (warp == 1) {
    // -------------------------------------------------------------- products
    {
      // kind::f16: FP32 accumulator, BF16 operands; kind::mxf8f6f4: E4M3 operands with E8M0 scales
      const uint32_t idesc = (kMx ? (1u << 23) : (1u << 4) | (1u << 7) | (1u << 10)) | ((128u >> 4) << 24) | ((uint32_t)(acc >> 3) << 17);
      const uint32_t sf0 = tmem_base + 2 * acc;
      // the start address is a field of 16-byte units in the low word: stages stay below 2^18 bytes
      const uint64_t da0 = ptx::smem_desc(smem_base, 16, 1024, ptx::kSwizzle128B);
      const uint64_t ds0 = ptx::smem_desc(smem_base + kWTileBytes, 0, 128, ptx::kSwizzleNone);
      const uint32_t hi = (uint32_t)(da0 >> 32), s_hi = (uint32_t)(ds0 >> 32), s_lo0 = (uint32_t)ds0 - (uint32_t)da0;
      const uint32_t lo0 = (uint32_t)da0, lo_step = (uint32_t)stage_bytes >> 4;
      const uint32_t full0 = ptx::smem_u32(full), empty0 = ptx::smem_u32(empty);
      constexpr uint32_t kB = layer::rows_off(kMx) >> 4;
      int stage = 0, acc_i = 0;
      uint32_t phase = 0, lo = lo0;
      bool ok = true;
      while (ok && walk.next()) {
        const int buf = acc_i & 1;
        if (!warp_wait_quick(ptx::smem_u32(&acce[buf]), ((acc_i >> 1) & 1) ^ 1, ctl)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + buf * acc;
        uint32_t accumulate = 0;
#pragma unroll 1
        for (int k = walk.k0; k < (int)walk.k1; ++k) {
          if (!warp_wait_quick(full0 + 8 * stage, phase, ctl)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            if constexpr (!kMx) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::tc_mma_f16_lo(d, lo + 2 * q, lo + kB + 2 * q, hi, idesc, q > 0 ? 1u : accumulate);
            } else {
              const uint32_t sfa = sf0 + 8 * stage;
              ptx::tc_cp_sf_lo(sfa, lo + s_lo0, s_hi);                         // the weights' scales
              ptx::tc_cp_sf_lo(sfa + 4, lo + s_lo0 + (kSfChunk >> 4), s_hi);  // the tokens'
#pragma unroll
              for (int q = 0; q < 4; ++q)
                ptx::tc_mma_mxf8_lo(d, lo + 2 * q, lo + kB + 2 * q, hi, idesc | ((uint32_t)q << 4) | ((uint32_t)q << 29), sfa,
                                    sfa + 4, q > 0 ? 1u : accumulate);
            }
            ptx::tc_commit(empty0 + 8 * stage);
            if (k == (int)walk.k1 - 1) ptx::tc_commit(ptx::smem_u32(&accf[buf]));
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
      }
      if (ptx::elect_one()) ptx::tc_commit(ptx::smem_u32(drain));
      wait_bar_drain(ptx::smem_u32(drain), 0);
    }
    __syncwarp();
  } else if (warp < 6) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, ep = threadIdx.x - 64;
    const int row = q * 32 + lane;  // this thread's TMEM lane: row of the weight tile
    const int64_t slot_floats = (int64_t)T * 128;
    int acc_i = 0;
    int cut0 = 0, cut1 = 0, n_cut = 0;  // column tiles of the down run that this CTA has a piece of
    bool ok = true, left = false;       // left: gave up, all four warps together
    // A cut unit of the up run is finished by the CTA of its second piece, whose range begins inside the unit: a CTA
    // owes at most one, after its own pieces (its others are waited for by others).  That code runs once before, on no
    // pieces at all (it leaves zeros, which the real pass overwrites): its instructions come from memory the first
    // time, which here costs nothing (nothing has arrived yet) and later 1.5 us on the way of every CTA.
    const uint32_t begin = up.lo(blockIdx.x);
    int owed_unit = -1;
    if (begin < up.lo(blockIdx.x + 1)) {
      const Pieces first(up, begin / up.K);
      if (blockIdx.x - first.b0 == 1) owed_unit = (int)(begin / up.K);
    }
    bool rehearse = owed_unit >= 0;
    bool more = walk.next();
    while (more || owed_unit >= 0) {
      const bool owed = owed_unit >= 0 && (rehearse || !more || walk.is_down);
      const int buf = acc_i & 1;
      const bool is_down = !owed && walk.is_down;
      const uint32_t unit = owed ? (uint32_t)owed_unit : walk.unit;
      const Run& run = is_down ? down : up;
      const bool routed = !is_down && (int)unit >= p.NT1s;
      const int a = routed ? ((int)unit - p.NT1s) / p.NT1 : 0;
      const int j = routed ? (int)unit - p.NT1s - a * p.NT1 : (int)unit;  // column tile
      const int e = routed ? s_act[a] : 0;
      const unsigned long long mask = routed ? s_mask[e] : (T == 64 ? ~0ull : (1ull << T) - 1);
      const bool whole = !owed && walk.k1 - walk.k0 == run.K;
      const Pieces pieces(run, unit);
      if (!is_down && ep < T) {  // the router's weight of each token for this expert
        float w = routed ? 0.f : 1.f;
        if (routed)
#pragma unroll 1
          for (int k = 0; k < topk; ++k) w = s_ids[ep * topk + k] == e ? s_wt[ep * topk + k] : w;
        s_tokw[ep] = w;
      }
      if (!owed) ok = warp_wait_quick(ptx::smem_u32(&accf[buf]), (acc_i >> 1) & 1, ctl);
      else if (!rehearse && ep == 0) ok = wait_count(p.up_cnt + unit, pieces.n, ctl);
      left = !ptx::bar_all(1, 128, ok);  // the four warps leave together: they share named barriers
      if (left) break;
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + buf * acc;
      if (!whole && !owed) {
        // this CTA's range begins in the unit (slot 0) or ends there (slot 1)
        const uint32_t at = blockIdx.x * 2 + (run.lo(blockIdx.x) >= pieces.x0 ? 0 : 1);
        float* slot = (is_down ? p.slots_down : p.slots_up) + (int64_t)at * slot_floats;
#pragma unroll 1
        for (int c0 = 0; c0 < T; c0 += 16) {
          if (((mask >> c0) & 0xffff) == 0) continue;
          float v[16];
          load_acc16<kMx>(taddr + c0, npad, v);
#pragma unroll
          for (int jj = 0; jj < 16; ++jj)
            if ((mask >> (c0 + jj)) & 1) __stcg(slot + (c0 + jj) * 128 + row, v[jj]);
        }
        ptx::bar_sync(1, 128);  // the pieces' stores, then one thread's release
        if (ep == 0) red_release_add((is_down ? p.down_cnt : p.up_cnt) + unit, 1);
        if (is_down) {
          if (n_cut++ == 0) cut0 = unit;
          else cut1 = unit;
        }
      } else if (is_down) {  // a column tile of this CTA alone
#pragma unroll 1
        for (int c0 = 0; c0 < T; c0 += 16) {
          float v[16];
          load_acc16<kMx>(taddr + c0, npad, v);
          const int64_t n = (int64_t)j * 128 + row;
          uint32_t nans = 0;
#pragma unroll
          for (int jj = 0; jj < 16; ++jj) {
            const int t = c0 + jj;
            if (t < T && n < g.H) {
              if (v[jj] != v[jj]) {
                nans |= 1u << jj;
                continue;
              }
              float o = v[jj];
              if (p.residual) o += __bfloat162float(p.residual[t * p.ld_residual + n]);
              p.out[t * p.ld_out + n] = __float2bfloat16_rn(o);
            }
          }
#pragma unroll 1
          for (; nans; nans &= nans - 1) {
            const int t = c0 + __ffs((int)nans) - 1;
            float o = own_sums<kMx>(p, s_act, s_ids, A, n_units, t, n, make_float4(__int_as_float(0x7fffffff), 0.f, 0.f, 0.f)).x;
            if (p.residual) o += __bfloat162float(p.residual[t * p.ld_residual + n]);
            p.out[t * p.ld_out + n] = __float2bfloat16_rn(o);
          }
          __syncwarp();
        }
      } else {
        const uint32_t n_pieces = rehearse ? 0 : pieces.n;
        // SwiGLU: rows 0..63 of the tile hold gate columns, 64..127 the up columns of the same indices
        uint8_t* dst = routed ? p.swimg + (int64_t)a * p.KB2 * img : p.swimg_s;
        dst += (int64_t)(kMx ? j >> 1 : j) * img;
        const bool pad_half = kMx && (j & 1) == 0 && j + 1 == (routed ? p.NT1 : p.NT1s);  // no unit fills the tile's other half
        // rows of tokens that did not choose the expert: zeros, in 16-byte chunks (MXFP8: of hi and of lo)
#pragma unroll 1
        for (int i = ep; i < T * 8; i += 128) {
          const int t = i >> 3, c = i & 7;
          if ((mask >> t) & 1) continue;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          if constexpr (!kMx) {
            *reinterpret_cast<uint4*>(dst + image_chunk(t, c)) = zero;
          } else {
            uint8_t* at = dst + kSfChunk + (c >> 2) * npad * 128;
            *reinterpret_cast<uint4*>(at + image_chunk(t, (j & 1) * 4 + (c & 3))) = zero;
            if ((c & 3) < 2) dst[scale_at((c >> 2) * npad + t, (j & 1) * 2 + (c & 3))] = 127;
          }
        }
        if (pad_half) {
#pragma unroll 1
          for (int i = ep; i < T * 8; i += 128) {
            const int t = i >> 3, c = i & 7;
            uint8_t* at = dst + kSfChunk + (c >> 2) * npad * 128;
            *reinterpret_cast<uint4*>(at + image_chunk(t, 4 + (c & 3))) = make_uint4(0, 0, 0, 0);
            if ((c & 3) < 2) dst[scale_at((c >> 2) * npad + t, 2 + (c & 3))] = 127;
          }
        }
        // the others
        auto store_sw = [&](int t, int col, float sw) {  // col: intermediate index within the unit, a lane each
          if constexpr (!kMx) {
            if (sw != sw && !rehearse) p.nan_rows[t] = 1;
            *reinterpret_cast<__nv_bfloat16*>(dst + image_chunk(t, col >> 3) + (col & 7) * 2) = __float2bfloat16_rn(sw);
          } else {
            const BlockScale b = block_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(sw) & 0x7fffffffu));
            uint32_t hi, lo;
            split_e4m3(sw, b, hi, lo);
            const int c = (j & 1) * 64 + col;
            uint8_t* at = dst + kSfChunk + image_chunk(t, c >> 4) + (c & 15);
            at[0] = (uint8_t)hi;
            at[npad * 128] = (uint8_t)lo;
            if (lane == 0) {
              dst[scale_at(t, c >> 5)] = (uint8_t)b.byte_hi;
              dst[scale_at(npad + t, c >> 5)] = (uint8_t)b.byte_lo;
              if (b.byte_hi == 255u) p.nan_rows[t] = 1;
            }
          }
        };
        if (owed) {
          // from the slots: a thread takes both rows of an index, for every other token
          const int col = ep & 63;
          unsigned long long m = mask;
          if (ep >= 64) m &= m - 1;  // the second, fourth, ...
          while (m) {
            constexpr int kTok = 4;
            int tok[kTok];
            float gate_v[kTok] = {}, up_v[kTok] = {};
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
              tok[i] = m ? __ffsll((long long)m) - 1 : -1;
              m &= m - 1;
              m &= m - 1;
            }
#pragma unroll 4
            for (uint32_t k = 0; k < n_pieces; ++k) {
              const float* slot = p.slots_up + (int64_t)pieces.slot(k) * slot_floats + col;
#pragma unroll
              for (int i = 0; i < kTok; ++i) {
                if (tok[i] >= 0) {
                  gate_v[i] += __ldcg(slot + tok[i] * 128);
                  up_v[i] += __ldcg(slot + tok[i] * 128 + 64);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < kTok; ++i)
              if (tok[i] >= 0) store_sw(tok[i], col, silu(gate_v[i]) * up_v[i] * s_tokw[tok[i]]);
          }
        } else {
          // from TMEM, kRound tokens at a time: warps 4, 5 (gate rows) take the even ones, warps 2, 3 (up rows) the odd,
          // each handing the other what it needs
          constexpr int kRound = layer::kRound;
          const int half = q >= 2, col = (q & 1) * 32 + lane;
          for (unsigned long long m = mask; m;) {
            int tok[kRound];
            uint32_t r[kRound], l[kRound];
            float v[kRound];
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
              tok[i] = m ? __ffsll((long long)m) - 1 : -1;
              m &= m - 1;
              if (tok[i] >= 0) {
                r[i] = ptx::tmem_ld_32x32b_x1(taddr + tok[i]);
                if constexpr (kMx) l[i] = ptx::tmem_ld_32x32b_x1(taddr + npad + tok[i]);
              }
            }
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
              v[i] = kMx ? __uint_as_float(r[i]) + __uint_as_float(l[i]) : __uint_as_float(r[i]);
              if ((i & 1) != half) xchg[(i * 2 + (q & 1)) * 32 + lane] = v[i];
            }
            ptx::bar_sync(1, 128);
#pragma unroll
            for (int i = 0; i < kRound / 2; ++i) {
              const int t = half ? tok[2 * i + 1] : tok[2 * i];
              const float mine = half ? v[2 * i + 1] : v[2 * i], other = xchg[((2 * i + half) * 2 + (q & 1)) * 32 + lane];
              if (t >= 0) store_sw(t, col, silu(half ? other : mine) * (half ? mine : other) * s_tokw[t]);
            }
            if (m) ptx::bar_sync(1, 128);  // xchg is written again
          }
        }
        asm volatile("fence.proxy.async;" ::: "memory");  // sw is read by bulk copies
        ptx::bar_sync(1, 128);
        if (ep == 0 && !rehearse) red_release_add(p.up_done, 1);
      }
      if (owed) {
        if (!rehearse) owed_unit = -1;
        rehearse = false;
      } else {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&acce[buf]));
        ++acc_i;
        more = walk.next();
      }
    }
    // the cut column tiles (at most two): this CTA's share of each, once all its pieces are there
    const bool vec = ((reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.residual)) & 7) == 0 &&
                     ((p.ld_out | p.ld_residual) & 3) == 0;
    if (!left && n_cut > 0) {
      const Pieces pa(down, cut0), pb(down, n_cut > 1 ? cut1 : cut0);
      if (ep == 0) ok = wait_count(p.down_cnt + cut0, pa.n, ctl);
      if (ep == 32 && n_cut > 1) ok = wait_count(p.down_cnt + cut1, pb.n, ctl);
      if (ptx::bar_all(1, 128, ok)) {
        const int total = T * 32, a_lo = total * (int)(blockIdx.x - pa.b0) / (int)pa.n,
                  a_n = total * (int)(blockIdx.x - pa.b0 + 1) / (int)pa.n - a_lo,
                  b_lo = total * (int)(blockIdx.x - pb.b0) / (int)pb.n,
                  b_n = n_cut > 1 ? total * (int)(blockIdx.x - pb.b0 + 1) / (int)pb.n - b_lo : 0;
#pragma unroll 1
        for (int x = ep; x < a_n + b_n; x += 128) {
          const bool in_a = x < a_n;
          const int i = in_a ? a_lo + x : b_lo + x - a_n, j = in_a ? cut0 : cut1, n = in_a ? pa.n : pb.n;
          const uint32_t b0 = in_a ? pa.b0 : pb.b0, first_slot = in_a ? pa.first_slot : pb.first_slot;
          const int t = i >> 5, r4 = (i & 31) * 4;
          const int64_t col = (int64_t)j * 128 + r4;
          if (col >= g.H) continue;
          const float* slot = p.slots_down + (int64_t)(b0 * 2) * slot_floats + t * 128 + r4;
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int kJoin = kMx ? 4 : 8;
#pragma unroll kJoin
          for (int k = 0; k < n; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(slot + (int64_t)(2 * k + (k == 0 ? first_slot : 0)) * slot_floats));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
          }
          const float all = s.x + s.y + s.z + s.w;
          if (all != all) s = own_sums<kMx>(p, s_act, s_ids, A, n_units, t, col, s);
          __nv_bfloat16* o = p.out + t * p.ld_out + col;
          const __nv_bfloat16* res = p.residual ? p.residual + t * p.ld_residual + col : nullptr;
          if (vec) {
            if (res) {
              const uint2 r = *reinterpret_cast<const uint2*>(res);
              s.x += __uint_as_float(r.x << 16);
              s.y += __uint_as_float(r.x & 0xffff0000u);
              s.z += __uint_as_float(r.y << 16);
              s.w += __uint_as_float(r.y & 0xffff0000u);
            }
            const __nv_bfloat162 a = __floats2bfloat162_rn(s.x, s.y), b = __floats2bfloat162_rn(s.z, s.w);
            *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
          } else {
            const float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = __float2bfloat16_rn(res ? f[k] + __bfloat162float(res[k]) : f[k]);
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, layer::tmem_cols(kMx));
  }
  if (threadIdx.x == 0) {
    p.hdr[1 + blockIdx.x] = *s_err;
    if (blockIdx.x == 0) p.hdr[0] = gridDim.x;
  }
}

template <bool kMx>
static cudaError_t launch_layer_of(const LayerParams& p, int sms, cudaStream_t s) {
  static int configured_device = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (configured_device != dev) {
    cudaError_t e = cudaFuncSetAttribute(layer_kernel<kMx>, cudaFuncAttributeMaxDynamicSharedMemorySize, layer::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeCooperative;  // CTAs wait for one another: all must be resident
  attr[1].val.cooperative = 1;
  lc.stream = s;
  // the router's clusters (one per 8 tokens, at most 8) and the images': about as many as run at once
  lc.gridDim = dim3((unsigned)std::max<int64_t>(15, (p.gate.T + 7) / 8 + 7) * gate::kCluster);
  const int threads = gate::cluster_threads(p.gate.T, p.gate.H, p.gate.rule.E);
  lc.blockDim = dim3((unsigned)threads);
  cudaLaunchAttribute fattr[2];
  fattr[0] = attr[0];
  fattr[1].id = cudaLaunchAttributeClusterDimension;
  fattr[1].val.clusterDim.x = gate::kCluster;
  fattr[1].val.clusterDim.y = fattr[1].val.clusterDim.z = 1;
  lc.attrs = fattr;
  lc.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&lc, threads == gate::kSmall ? layer_front_kernel<kMx, gate::kSmall> : layer_front_kernel<kMx, gate::kLarge>, p);
  if (e != cudaSuccess) return e;
  lc.gridDim = dim3((unsigned)(sms < kLayerMaxCtas ? sms : kLayerMaxCtas));
  lc.blockDim = dim3(layer::kThreads);
  lc.dynamicSmemBytes = layer::kSmemBytes;
  lc.attrs = attr;
  return cudaLaunchKernelEx(&lc, layer_kernel<kMx>, p);
}

cudaError_t launch_layer(const LayerParams& p, int sms, cudaStream_t s) {
  return p.mx ? launch_layer_of<true>(p, sms, s) : launch_layer_of<false>(p, sms, s);
}

int64_t layer_image_bytes(bool mx, int64_t npad) { return layer::image_bytes(mx, (int)npad); }

}  // namespace gmmfr
