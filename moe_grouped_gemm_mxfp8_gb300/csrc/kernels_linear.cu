// The dense product (forms: linear_forms.cuh): its plan, and the copies of rows that TMA cannot read in place.
// Rows of x or W that do not start on 16-byte boundaries (a TMA rule) are first copied to a pitch that does.
#include "linear_forms.cuh"

namespace gmmfr {

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

// ============================================================================ plan
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
    auto kernel = linear_stream_kernel<GMMFR_ACT_NONE, false, false>;
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
    // With adapters also by what its epilogue takes from the second factors: 32 rows of 2048, rank 64 (4.2 M) 9.8 us, the
    // stream form 12.5; 25 gated of 2 x 4160, rank 64 (13 M) 16.8 and 12.4.
    const int64_t factors = p.lora_ids ? p.M * p.lora_rows * p.lora_rank : 0;
    if ((p.M == 1 || p.M * p.group_m * 16 * p.K <= 1900000) && factors <= 8000000) {
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
    if (tail.lora_ids) {
      tail.lora_ids += at;
      tail.lora_s += at * tail.lora_rank;
      tail.lora_lists += at / 256 * kLoraListInts;
    }
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

cudaError_t launch_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  return p.out_f32 ? launch_form<true, false>(maps, p, s) : launch_form<false, false>(maps, p, s);
}

}  // namespace gmmfr
