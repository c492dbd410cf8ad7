// A whole mixture-of-experts layer for a few tokens: the gate, then for every token and chosen
// expert (and the shared expert) the gate/up product with SwiGLU, then the down product summed over
// the token's experts.  Weights are the prepared tiles of the grouped FFN (BF16: 64 K per 128-byte row)
// or their MXFP8 form (128 K codes per row and 512 scale bytes per tile).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "epilogue.cuh"
#include "ops.cuh"
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

namespace {
// Sum over k of tile row r of the K blocks [0, KB) with v[k]; one lane's share (the warp adds up).
__device__ __forceinline__ float row_dot(const uint8_t* tiles, int mx, int64_t KB, int64_t K, int r, int lane,
                                         const __nv_bfloat16* xb, const float* xf) {
  const int kt = mx ? 128 : 64;
  const int64_t tb = mx ? kPrepTileBytes : kWTileBytes;
  float acc = 0.f;
  for (int64_t k = lane; k < KB * kt; k += 32) {
    if (k >= K) break;
    const uint8_t* tile = tiles + (k / kt) * tb;
    const int c = (int)(k % kt);
    float w;
    if (mx) {
      __nv_fp8_e4m3 code;
      code.__x = tile[r * 128 + (((c >> 4) ^ (r & 7)) << 4) + (c & 15)];
      w = (float)code * exp2f((float)tile[kWTileBytes + 16 * (r & 31) + 4 * (r >> 5) + (c >> 5)] - 127.f);
    } else {
      w = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(tile + r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2));
    }
    acc = fmaf(w, xb ? __bfloat162float(xb[k]) : xf[k], acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  return acc;
}
}  // namespace

// One warp per (token, choice, intermediate index); choice topk is the shared expert.
__global__ void __launch_bounds__(256) layer_up_kernel(LayerParams p) {
  const int lane = threadIdx.x & 31;
  const GateParams& g = p.gate;
  const int64_t topk = g.rule.topk;
  const int64_t n_routed = g.T * topk * p.I;
  const int64_t o = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= n_routed + g.T * p.shared_I) return;
  const bool routed = o < n_routed;
  const int64_t I = routed ? p.I : p.shared_I;
  const int64_t pair = (routed ? o : o - n_routed) / I, i = (routed ? o : o - n_routed) % I;
  const int64_t t = routed ? pair / topk : pair;
  const int64_t e = routed ? static_cast<const int32_t*>(g.ids)[pair] : 0;
  const int64_t kt = p.mx ? 128 : 64, tb = p.mx ? kPrepTileBytes : kWTileBytes;
  const int64_t NT = (I + 63) / 64, KB = (g.H + kt - 1) / kt;
  const uint8_t* tiles = (routed ? p.prepared : p.shared) + (e * NT + i / 64) * KB * tb;
  const float gate = row_dot(tiles, p.mx, KB, g.H, (int)(i & 63), lane, g.x + t * g.ldx, nullptr);
  const float up = row_dot(tiles, p.mx, KB, g.H, (int)(i & 63) + 64, lane, g.x + t * g.ldx, nullptr);
  if (lane == 0) p.sw[o] = silu(gate) * up * (routed ? g.weights[pair] : 1.f);
}

// One warp per (token, output column).
__global__ void __launch_bounds__(256) layer_down_kernel(LayerParams p) {
  const int lane = threadIdx.x & 31;
  const GateParams& g = p.gate;
  const int64_t topk = g.rule.topk;
  const int64_t o = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (o >= g.T * g.H) return;
  const int64_t t = o / g.H, n = o % g.H;
  const int64_t kt = p.mx ? 128 : 64, tb = p.mx ? kPrepTileBytes : kWTileBytes;
  const int64_t NT2 = (g.H + 127) / 128, KBh = (g.H + kt - 1) / kt;
  float acc = 0.f;
  for (int64_t k = 0; k <= topk; ++k) {
    const bool routed = k < topk;
    const int64_t I = routed ? p.I : p.shared_I;
    if (I == 0) continue;
    const int64_t e = routed ? static_cast<const int32_t*>(g.ids)[t * topk + k] : 0;
    const int64_t E = routed ? g.rule.E : 1, KB = (I + kt - 1) / kt;
    const uint8_t* base = (routed ? p.prepared : p.shared) + E * ((I + 63) / 64) * KBh * tb;
    const float* sw = routed ? p.sw + (t * topk + k) * I : p.sw + g.T * topk * p.I + t * I;
    acc += row_dot(base + (e * NT2 + n / 128) * KB * tb, p.mx, KB, I, (int)(n & 127), lane, nullptr, sw);
  }
  if (lane == 0) {
    if (p.residual) acc += __bfloat162float(p.residual[t * p.ld_residual + n]);
    p.out[t * p.ld_out + n] = __float2bfloat16_rn(acc);
  }
}

cudaError_t launch_layer(const LayerParams& p, cudaStream_t s) {
  const GateParams& g = p.gate;
  if (g.T == 0) return cudaSuccess;
  if (cudaError_t e = launch_gate(g, s)) return e;
  const int64_t up = g.T * (g.rule.topk * p.I + p.shared_I);
  layer_up_kernel<<<(unsigned)((up + 7) / 8), 256, 0, s>>>(p);
  if (cudaError_t e = cudaGetLastError()) return e;
  layer_down_kernel<<<(unsigned)((g.T * g.H + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gmmfr
