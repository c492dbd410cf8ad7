// The dense product with low-rank adapters of many requests (forms: linear_forms.cuh, with kLora), and the sums that it
// starts from: s[t] = scale_a (A_a x[t]) for the adapter a of row t.
//
// The sums take r (16, say) rows of K for every adapter in use and every row of x once.  A cluster of CTAs takes a tile of
// 8 or 32 rows of x and shares its K range; the adapters of the tile's rows are shared out over each CTA's warps, or the
// warps share an adapter's K when the adapters are few, so that one decoded token's 16 x 4096 factor is on its way all at
// once.  Products by mma.sync: they wait for memory, and a tile's rows have up to as many adapters as there are rows.  The
// product's launch follows at once and begins with its weights; only its epilogue waits for the sums.
#include "linear_forms.cuh"

namespace gmmfr {
namespace lora {
constexpr int kThreads = 256;
constexpr int kRanks = 32;  // rows of a first factor at a time
}  // namespace lora

template <int kTiles>
__global__ void __launch_bounds__(lora::kThreads) lora_sums_kernel(const __grid_constant__ LoraParams p) {
  constexpr int kTok = 8 * kTiles, kU = kTiles == 1 ? 4 : 2, kRt = lora::kRanks / 16;
  __shared__ __align__(16) float part[8][kTok][lora::kRanks];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = p.split;
  const uint32_t crank = C > 1 ? ptx::cluster_rank() : 0u;
  const int64_t t0 = (int64_t)(blockIdx.x / C) * kTok;
  // the launch after this one reads x and its weights without waiting for this one: it may start when all before has ended
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // lane t has row t0 + t's adapter; the first row of each adapter stands for it
  int id = -1;
  if (lane < kTok && t0 + lane < p.M) {
    id = p.ids[t0 + lane];
    if ((uint32_t)id >= (uint32_t)p.count) id = -1;
  }
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  const uint32_t firsts = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
  const int adapters = __popc(firsts);
  const int groups = adapters <= 1 ? 1 : (adapters <= 2 ? 2 : (adapters <= 4 ? 4 : 8)), splits = 8 / groups;
  const int group = warp / splits, split = warp - group * splits;
  const int blocks = (int)((p.K + 31) / 32);
  const int b_begin = (int)((int64_t)blocks * crank / C) + split, b_end = (int)((int64_t)blocks * (crank + 1) / C);
  const __nv_bfloat16* xr[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) xr[i] = p.x + min(t0 + 8 * i + (lane >> 2), p.M - 1) * p.ldx;  // past the end: not stored
  for (int r0 = 0; r0 < p.rank; r0 += lora::kRanks) {
    uint32_t left = firsts;
    for (int d = 0; d < adapters; ++d, left &= left - 1) {
      if (d % groups != group) continue;
      const int first = __ffs(left) - 1;
      const int a = __shfl_sync(0xffffffffu, id, first);
      const uint32_t mine = __shfl_sync(0xffffffffu, same, first);
      const __nv_bfloat16* ar = p.a + ((int64_t)a * p.rank + r0 + (lane >> 2)) * p.K;
      float acc[kTiles][kRt][4] = {};
      for (int b0 = b_begin; b0 < b_end; b0 += kU * splits) {
        uint4 w[kU][kRt][2], x[kU][kTiles];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int64_t k = (int64_t)(b0 + u * splits) * 32 + (lane & 3) * 8;
          const bool in = b0 + u * splits < b_end && k < p.K;
#pragma unroll
          for (int i = 0; i < kRt; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[u][i][h] = in && r0 + 16 * i + 8 * h + (lane >> 2) < p.rank
                               ? __ldg(reinterpret_cast<const uint4*>(ar + (16 * i + 8 * h) * p.K + k))
                               : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
            x[u][i] = in ? __ldg(reinterpret_cast<const uint4*>(xr[i] + k)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < kRt; ++j) {
              ptx::mma_16816(acc[i][j], w[u][j][0].x, w[u][j][1].x, w[u][j][0].y, w[u][j][1].y, x[u][i].x, x[u][i].y);
              ptx::mma_16816(acc[i][j], w[u][j][0].z, w[u][j][1].z, w[u][j][0].w, w[u][j][1].w, x[u][i].z, x[u][i].w);
            }
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tok = 8 * i + (lane & 3) * 2 + (c & 1);
          if (mine >> tok & 1)
#pragma unroll
            for (int j = 0; j < kRt; ++j) part[split][tok][16 * j + 8 * (c >> 1) + (lane >> 2)] = acc[i][j][c];
        }
    }
    __syncthreads();
    // the splits' sums in order, then the cluster's CTAs'
    constexpr int kFours = kTok * lora::kRanks / 4;
    float4* mine4 = reinterpret_cast<float4*>(&part[0][0][0]);
    for (int i = threadIdx.x; i < kFours; i += lora::kThreads) {
      float4 v = mine4[i];
      for (int s = 1; s < splits; ++s) {
        const float4 z = mine4[s * kFours + i];
        v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
      }
      mine4[i] = v;
    }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
    for (int i = crank * lora::kThreads + threadIdx.x; i < kFours; i += C * lora::kThreads) {
      const int tok = i / (lora::kRanks / 4), r = r0 + i % (lora::kRanks / 4) * 4;
      if (t0 + tok >= p.M || r >= p.rank) continue;
      const int a = p.ids[t0 + tok];
      if ((uint32_t)a >= (uint32_t)p.count) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = ptx::smem_u32(&mine4[i]);
      for (int c = 0; c < C; ++c) {
        const float4 z = ptx::ld_cluster_v4(C > 1 ? ptx::map_to_rank(at, c) : at);
        v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
      }
      const float scale = p.scale ? p.scale[a] : 1.f;
      *reinterpret_cast<float4*>(p.s + (t0 + tok) * p.rank + r) = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
  }
}

cudaError_t launch_lora_sums(LoraParams p, int sms, cudaStream_t s) {
  // small tiles while they leave room for all of a cluster; large ones read the factors less often
  const int tok = p.M <= 128 ? 8 : 32;
  const int64_t tiles = (p.M + tok - 1) / tok;
  p.split = 1;
  while (p.split < 8 && (tok == 8 || tiles * p.split < 2 * sms) && 2 * p.split * 32 <= p.K) p.split *= 2;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(tiles * p.split));
  lc.blockDim = dim3(lora::kThreads);
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = p.split > 1 ? 2 : 1;
  return tok == 8 ? cudaLaunchKernelEx(&lc, lora_sums_kernel<1>, p) : cudaLaunchKernelEx(&lc, lora_sums_kernel<4>, p);
}

cudaError_t launch_lora_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  return p.out_f32 ? launch_form<true, true>(maps, p, s) : launch_form<false, true>(maps, p, s);
}

}  // namespace gmmfr
