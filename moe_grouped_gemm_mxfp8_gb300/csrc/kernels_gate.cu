// The router: logits = x W^T (FP32 sums of BF16 products), then the selection of each token.
//   gate_logits  one warp per (expert, up to 8 tokens): the weight row is read once for them
//   gate_select  one warp per token (gate_select.cuh)
#include "gate_select.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace gmmfr {

namespace {
constexpr int kGateTok = 8;  // tokens a warp carries through one weight row

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
}  // namespace

__global__ void __launch_bounds__(256) gate_logits_kernel(GateParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = (int64_t)blockIdx.x * 8 + warp;
  const int64_t t0 = (int64_t)blockIdx.y * kGateTok;
  if (e >= p.rule.E) return;
  float acc[kGateTok] = {};
  for (int64_t h = lane * 8; h < p.H; h += 256) {
    float w[8];
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.weight + e * p.H + h), w);
#pragma unroll
    for (int i = 0; i < kGateTok; ++i) {
      if (t0 + i < p.T) {
        float x[8];
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(p.x + (t0 + i) * p.ldx + h), x);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i] = fmaf(w[q], x[q], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kGateTok; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    if (lane == 0 && t0 + i < p.T) p.logits[(t0 + i) * p.rule.E + e] = acc[i];
  }
}

template <int kPer>
__global__ void __launch_bounds__(128) gate_select_kernel(GateParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * 4 + warp;
  if (t >= p.T) return;
  int id;
  float w;
  gate_select_warp<kPer>(p.rule, p.logits + t * p.rule.E, p.select_bias, lane, id, w);
  if (lane < p.rule.topk) {
    const int64_t o = t * p.rule.topk + lane;
    if (p.ids_i64) static_cast<int64_t*>(p.ids)[o] = id;
    else static_cast<int32_t*>(p.ids)[o] = id;
    p.weights[o] = w;
  }
}

__global__ void __launch_bounds__(gate::kThreads) gate_cluster_kernel(const __grid_constant__ GateParams p) {
  __shared__ gate::Smem sm;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  gate_cluster(p, (int64_t)(blockIdx.x / gate::kCluster) * gate::kTok, sm, ptx::cluster_rank());
}

cudaError_t launch_gate(const GateParams& p, cudaStream_t s) {
  if (p.T == 0) return cudaSuccess;
  if (p.T <= kGateClusterTokens) {
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = gate::kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 2;
    lc.stream = s;
    lc.gridDim = dim3((unsigned)((p.T + gate::kTok - 1) / gate::kTok * gate::kCluster));
    lc.blockDim = dim3(gate::kThreads);
    return cudaLaunchKernelEx(&lc, gate_cluster_kernel, p);
  }
  const int64_t per_launch = (int64_t)65535 * kGateTok;  // grid.y limit
  for (int64_t t = 0; t < p.T; t += per_launch) {
    GateParams q = p;
    q.x += t * p.ldx;
    q.logits += t * p.rule.E;
    q.T = p.T - t < per_launch ? p.T - t : per_launch;
    gate_logits_kernel<<<dim3((unsigned)((p.rule.E + 7) / 8), (unsigned)((q.T + kGateTok - 1) / kGateTok)), 256, 0, s>>>(q);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  const unsigned grid = (unsigned)((p.T + 3) / 4);
  if (p.rule.E <= 32) gate_select_kernel<1><<<grid, 128, 0, s>>>(p);
  else if (p.rule.E <= 64) gate_select_kernel<2><<<grid, 128, 0, s>>>(p);
  else if (p.rule.E <= 128) gate_select_kernel<4><<<grid, 128, 0, s>>>(p);
  else if (p.rule.E <= 256) gate_select_kernel<8><<<grid, 128, 0, s>>>(p);
  else if (p.rule.E <= 512) gate_select_kernel<16><<<grid, 128, 0, s>>>(p);
  else gate_select_kernel<32><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gmmfr
