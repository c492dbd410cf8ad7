// The dense product with its epilogue: y = act(x W^T + bias) + residual.
#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "ops.cuh"
#include "ptx.cuh"

namespace gmmfr {

// Plain form for rows of any alignment: 64 x 64 outputs per CTA, 16 K at a time through shared
// memory, 4 x 4 FP32 sums per thread (twice that with the gated activation).
template <bool kGated>
__global__ void __launch_bounds__(256) linear_plain_kernel(LinearParams p) {
  __shared__ float sx[16][64 + 4];
  __shared__ float sw[kGated ? 2 : 1][16][64 + 4];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  float acc[kGated ? 2 : 1][4][4] = {};
  const int lk = tid & 15, lr = tid >> 4;
  for (int64_t k0 = 0; k0 < p.K; k0 += 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = lr + 16 * i;
      const bool k_ok = k0 + lk < p.K;
      sx[lk][r] = k_ok && m0 + r < p.M ? __bfloat162float(p.x[(m0 + r) * p.ldx + k0 + lk]) : 0.f;
#pragma unroll
      for (int g = 0; g < (kGated ? 2 : 1); ++g)
        sw[g][lk][r] = k_ok && n0 + r < p.N ? __bfloat162float(p.w[(g * p.N + n0 + r) * p.ldw + k0 + lk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float4 a = *reinterpret_cast<const float4*>(&sx[k][ty * 4]);
      const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int g = 0; g < (kGated ? 2 : 1); ++g) {
        const float4 b = *reinterpret_cast<const float4*>(&sw[g][k][tx * 4]);
        const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[g][i][j] = fmaf(av[i], bv[j], acc[g][i][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= p.M) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (n >= p.N) break;
      float v = acc[0][i][j];
      if (p.bias) v += __bfloat162float(p.bias[n]);
      if constexpr (kGated) {
        float u = acc[1][i][j];
        if (p.bias) u += __bfloat162float(p.bias[p.N + n]);
        v = silu(v) * u;
      } else {
        v = activate(p.act, v);
      }
      if (p.residual) v += __bfloat162float(p.residual[m * p.ldr + n]);
      if (p.out_f32) static_cast<float*>(p.out)[m * p.ldo + n] = v;
      else static_cast<__nv_bfloat16*>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
    }
  }
}

cudaError_t launch_linear(const LinearParams& p, cudaStream_t s) {
  if (p.M == 0 || p.N == 0) return cudaSuccess;
  const int64_t per_launch = (int64_t)65535 * 64;  // grid.y limit
  for (int64_t m = 0; m < p.M; m += per_launch) {
    LinearParams q = p;
    q.x += m * p.ldx;
    if (q.residual) q.residual += m * p.ldr;
    q.out = static_cast<uint8_t*>(p.out) + m * p.ldo * (p.out_f32 ? 4 : 2);
    q.M = p.M - m < per_launch ? p.M - m : per_launch;
    const dim3 grid((unsigned)((q.N + 63) / 64), (unsigned)((q.M + 63) / 64));
    if (p.act == GMMFR_ACT_SWIGLU) linear_plain_kernel<true><<<grid, 256, 0, s>>>(q);
    else linear_plain_kernel<false><<<grid, 256, 0, s>>>(q);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  return cudaSuccess;
}

}  // namespace gmmfr
