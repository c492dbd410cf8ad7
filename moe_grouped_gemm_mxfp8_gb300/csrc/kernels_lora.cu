// The dense product with low-rank adapters of many requests (forms: linear_forms.cuh, with kLora), and the sums that it
// starts from: s[t] = scale_a (A_a x[t]) for the adapter a of row t.
//
// The sums read r (16, say) rows of K for every adapter in use, and the rows of x.  Both kernels multiply by mma.sync: they wait
// for memory, and an adapter has a few rows at a time.  A lane loads 16 bytes of a row at a time straight into operand
// registers; the CTAs of a cluster and their warps share the K range, and their sums meet in shared memory in their order.
//   few   up to 128 rows: a cluster for each adapter and 16 of its ranks, its rows gathered, so that every factor is read once
//         and all of them are on their way at once
//   many  a cluster for 64 rows of x, whose warps share the adapters of those rows when there are several
// CTAs beside them list the adapters of each 256 rows, and scan those adapters' second factors for infinities and NaN (which
// also brings them into L2).  The product's launch follows at once and begins with its weights; only its adapters wait.
#include "linear_forms.cuh"

namespace gmmfr {
namespace lora {
constexpr int kThreads = 256;
constexpr int kFewRows = 128, kManyRows = 64;
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
  for (int j = 0; j < tid; j += 4) {
    const int4 v = *reinterpret_cast<const int4*>(&s_id[j]);
    first &= v.x != id && (v.y != id || j + 1 >= tid) && (v.z != id || j + 2 >= tid) && (v.w != id || j + 3 >= tid);
  }
  return first;
}

__device__ __forceinline__ int adapter_at(const LoraParams& p, int64_t m) {
  const int id = m < p.M ? p.ids[m] : -1;
  return (uint32_t)id < (uint32_t)p.count ? id : -1;
}

// Part `i` of the lists and scans: list i / scans, share i % scans of its adapters' second factors taken together.
__device__ void list_and_scan(const LoraParams& p, int64_t i) {
  static_assert(lora::kThreads == 256, "a thread for each of a list's rows");
  __shared__ __align__(16) int l_id[256];
  __shared__ int l_list[256];
  __shared__ uint32_t l_first[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t block = i / p.scans;
  const int share = (int)(i - block * p.scans);
  const int id = adapter_at(p, block * 256 + tid);
  l_id[tid] = id;
  __syncthreads();
  const bool first = first_of(l_id, tid, id);
  const uint32_t b = __ballot_sync(0xffffffffu, first);
  if (lane == 0) l_first[warp] = b;
  __syncthreads();
  int n = 0, at = __popc(b & ((1u << lane) - 1));
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int c = __popc(l_first[w]);
    if (w < warp) at += c;
    n += c;
  }
  int32_t* list = p.lists + block * kLoraListInts;
  if (first) {
    l_list[at] = id;
    if (share == 0) list[4 + at] = id;
  }
  if (share == 0 && tid == 0) list[0] = n;
  __syncthreads();
  const int64_t pieces = p.rows * p.rank / 8, from = n * pieces * share / p.scans, to = n * pieces * (share + 1) / p.scans;
  bool found = false;
  for (int64_t d = from / pieces; d * pieces < to; ++d) {
    const uint4* f = reinterpret_cast<const uint4*>(p.b) + l_list[d] * pieces;
    const int64_t end = min(to - d * pieces, pieces);
#pragma unroll 4
    for (int64_t k = max(from - d * pieces, (int64_t)0) + tid; k < end; k += lora::kThreads) {
      const uint4 v = __ldg(f + k);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) found |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
    }
  }
  found = __syncthreads_or(found);
  if (tid == 0) p.flags[i] = found;
}

}  // namespace

// ============================================================================ few rows
// Cluster (d, r): the d-th adapter in the order of the rows, ranks 16 r and up.
__global__ void __launch_bounds__(lora::kThreads) lora_sums_few_kernel(const __grid_constant__ LoraParams p) {
  constexpr int kU = 4;
  __shared__ __align__(16) int s_id[lora::kFewRows];
  __shared__ uint32_t s_first[4], s_mine[4];
  __shared__ int s_row[lora::kFewRows];
  __shared__ __align__(16) float part[8][8][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.split, rc = (p.rank + 15) / 16;
  const uint32_t crank = C > 1 ? ptx::cluster_rank() : 0u;
  const int units = (int)min(p.M, (int64_t)p.count) * rc, unit = blockIdx.x / C, d = unit / rc, r0 = unit % rc * 16;
  // the launch after this one reads x and its weights without waiting for this one: it may start when all before has ended
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (unit >= units) {
    const int i = blockIdx.x - units * C;
    if (i < p.scans) list_and_scan(p, i);
    return;
  }
  int id = -1;
  if (tid < lora::kFewRows) s_id[tid] = id = adapter_at(p, tid);
  __syncthreads();
  if (tid < lora::kFewRows) {
    const uint32_t b = __ballot_sync(0xffffffffu, first_of(s_id, tid, id));
    if (lane == 0) s_first[warp] = b;
  }
  __syncthreads();
  // the d-th first row's adapter, and its rows
  int a = -1;
  {
    int skip = d;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t b = s_first[w];
      const int n = __popc(b);
      if (a < 0 && skip < n) {
        for (int i = 0; i < skip; ++i) b &= b - 1;
        a = s_id[32 * w + __ffs(b) - 1];
      }
      skip -= n;
    }
  }
  if (a < 0) return;  // fewer adapters: the whole cluster leaves
  if (tid < lora::kFewRows) {
    const uint32_t b = __ballot_sync(0xffffffffu, id == a);
    if (lane == 0) s_mine[warp] = b;
  }
  __syncthreads();
  const int n0 = __popc(s_mine[0]), n1 = n0 + __popc(s_mine[1]), n2 = n1 + __popc(s_mine[2]), rows = n2 + __popc(s_mine[3]);
  if (tid < lora::kFewRows && id == a)
    s_row[(warp == 0 ? 0 : (warp == 1 ? n0 : (warp == 2 ? n1 : n2))) + __popc(s_mine[warp] & ((1u << lane) - 1))] = tid;
  __syncthreads();
  const float scale = p.scale ? p.scale[a] : 1.f;
  const int blocks = (int)((p.K + 31) / 32);
  const int b_begin = (int)((int64_t)blocks * crank / C) + warp, b_end = (int)((int64_t)blocks * (crank + 1) / C);
  const __nv_bfloat16* ar = p.a + ((int64_t)a * p.rank + r0) * p.K;
  for (int t0 = 0; t0 < rows; t0 += 8) {
    const __nv_bfloat16* const xr[1] = {p.x + (int64_t)s_row[min(t0 + (lane >> 2), rows - 1)] * p.ldx};
    float acc[1][1][4] = {};
    for (int b0 = b_begin; b0 < b_end; b0 += 8 * kU) {
      SumOperands<1, 1> o[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t k = (int64_t)(b0 + 8 * u) * 32 + (lane & 3) * 8;
        o[u].load(ar, p.rank - r0, p.K, xr, k, b0 + 8 * u < b_end && k < p.K);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        o[u].keep(b0 + 8 * u < b_end && (int64_t)(b0 + 8 * u) * 32 + (lane & 3) * 8 < p.K);
        o[u].multiply(acc);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) part[warp][(lane & 3) * 2 + (c & 1)][8 * (c >> 1) + (lane >> 2)] = acc[0][0][c];
    __syncthreads();
    // 128 sums: the warps' parts in order, then the cluster's CTAs'
    float* sums = &part[0][0][0];
    if (tid < 32) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(sums + w * 128 + 4 * tid);
        v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
      }
      *reinterpret_cast<float4*>(sums + 4 * tid) = v;
    }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
    const int i = crank * 32 / C + tid;  // this CTA's share of the 32 x 4
    if (tid < 32 / C && t0 + i / 4 < rows && r0 + i % 4 * 4 < p.rank) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = ptx::smem_u32(sums + 4 * i);
      for (int c = 0; c < C; ++c) {
        const float4 z = ptx::ld_cluster_v4(C > 1 ? ptx::map_to_rank(at, c) : at);
        v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
      }
      *reinterpret_cast<float4*>(p.s + (int64_t)s_row[t0 + i / 4] * p.rank + r0 + i % 4 * 4) =
          make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
  }
}

// ============================================================================ many rows
// `depth` clusters take 64 rows and share their adapters; each warp of a CTA takes kRt times 16 ranks of an adapter at a time,
// its K range split further when the adapters are fewer than the warps.  An adapter's rows are gathered, 32 at a time.
template <int kRt>
__global__ void __launch_bounds__(lora::kThreads, kRt == 1 ? 2 : 1) lora_sums_many_kernel(const __grid_constant__ LoraParams p) {
  constexpr int kTiles = 4, kRanks = 16 * kRt, kRows = lora::kManyRows;
  __shared__ __align__(16) int s_id[kRows];
  __shared__ uint32_t s_first[2];
  extern __shared__ __align__(16) float part[];  // [8][kRows][kRanks]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.split;
  const uint32_t crank = C > 1 ? ptx::cluster_rank() : 0u;
  const int64_t tiles = (p.M + kRows - 1) / kRows, unit = blockIdx.x / C;
  ptx::griddep_wait();  // as above
  ptx::griddep_launch_dependents();
  if (unit >= tiles * p.depth) {
    const int64_t i = blockIdx.x - tiles * p.depth * C;
    if (i < p.scans * ((p.M + 255) / 256)) list_and_scan(p, i);
    return;
  }
  const int64_t row0 = unit % tiles * kRows;
  const int turn = (int)(unit / tiles);
  int id = -1;
  if (tid < kRows) s_id[tid] = id = adapter_at(p, row0 + tid);
  __syncthreads();
  if (tid < kRows) {
    const uint32_t b = __ballot_sync(0xffffffffu, first_of(s_id, tid, id));
    if (lane == 0) s_first[warp] = b;
  }
  __syncthreads();
  uint64_t firsts = 0;  // this cluster's: every depth-th
  {
    uint64_t b = s_first[0] | (uint64_t)s_first[1] << 32;
    for (int d = 0; b; ++d, b &= b - 1)
      if (d % p.depth == turn) firsts |= b & -b;
  }
  if (!firsts) return;  // the whole cluster leaves
  const int adapters = __popcll(firsts);
  const int groups = adapters <= 1 ? 1 : (adapters <= 2 ? 2 : (adapters <= 4 ? 4 : 8)), splits = 8 / groups;
  const int group = warp / splits, split = warp - group * splits;
  const int blocks = (int)((p.K + 31) / 32);
  const int b_begin = (int)((int64_t)blocks * crank / C) + split, b_end = (int)((int64_t)blocks * (crank + 1) / C);
  for (int r0 = 0; r0 < p.rank; r0 += kRanks) {
    uint64_t left = firsts;
    for (int d = 0; d < adapters; ++d, left &= left - 1) {
      if (d % groups != group) continue;
      const int a = s_id[__ffsll(left) - 1];
      const __nv_bfloat16* ar = p.a + ((int64_t)a * p.rank + r0) * p.K;
      uint64_t mine = __ballot_sync(0xffffffffu, s_id[lane] == a) | (uint64_t)__ballot_sync(0xffffffffu, s_id[32 + lane] == a) << 32;
#pragma unroll 1
      while (mine) {
        // up to 32 rows: lane l's are the (8 i + l / 4)-th
        int row[kTiles];
        const __nv_bfloat16* xr[kTiles];
        const int n = __popcll(mine);
        if (n == kRows || (mine << 32 == 0 && n == 32)) {  // all, or the last 32 behind them
#pragma unroll
          for (int i = 0; i < kTiles; ++i) row[i] = kRows - n + 8 * i + (lane >> 2);
        } else {
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            int skip = min(8 * i + (lane >> 2), n - 1), at = 0;  // past the last one: it again, and not stored
#pragma unroll
            for (int half = 32; half >= 1; half >>= 1) {
              const int below = __popcll(mine >> at & ((1ull << half) - 1));
              if (skip >= below) {
                skip -= below;
                at += half;
              }
            }
            row[i] = at;
          }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) xr[i] = p.x + (row0 + row[i]) * p.ldx;
        float acc[kTiles][kRt][4] = {};
        // two sets of operands: one is on its way while the other is multiplied
        SumOperands<kTiles, kRt> even, odd;
        auto load = [&](SumOperands<kTiles, kRt>& o, int b) {
          const int64_t k = (int64_t)b * 32 + (lane & 3) * 8;
          o.load(ar, p.rank - r0, p.K, xr, k, k < p.K);
        };
        auto multiply = [&](SumOperands<kTiles, kRt>& o, int b) {
          o.keep((int64_t)b * 32 + (lane & 3) * 8 < p.K);
          o.multiply(acc);
        };
        if (b_begin < b_end) load(even, b_begin);
        for (int b = b_begin; b < b_end; b += 2 * splits) {
          const bool more = b + splits < b_end;
          if (more) load(odd, b + splits);
          multiply(even, b);
          if (!more) break;
          if (b + 2 * splits < b_end) load(even, b + 2 * splits);
          multiply(odd, b + splits);
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // columns 2 (lane % 4) + c of the products
            const int to = __shfl_sync(0xffffffffu, row[i], ((lane & 3) * 2 + c) * 4);
            if (8 * i + (lane & 3) * 2 + c < n)
#pragma unroll
              for (int j = 0; j < kRt; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) part[(split * kRows + to) * kRanks + 16 * j + 8 * h + (lane >> 2)] = acc[i][j][2 * h + c];
          }
#pragma unroll
        for (int i = 0; i < 8 * kTiles; ++i) mine &= mine - 1;
      }
    }
    __syncthreads();
    // the splits' sums in order, then the cluster's CTAs'
    constexpr int kFours = kRows * kRanks / 4;
    float4* fours = reinterpret_cast<float4*>(part);
    if (splits > 1)
      for (int i = tid; i < kFours; i += lora::kThreads) {
        float4 v = fours[i];
        for (int s = 1; s < splits; ++s) {
          const float4 z = fours[s * kFours + i];
          v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
        }
        fours[i] = v;
      }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
    for (int i = crank * lora::kThreads + tid; i < kFours; i += C * lora::kThreads) {
      const int row = i / (kRanks / 4), r = r0 + i % (kRanks / 4) * 4, a = s_id[row];
      if (a < 0 || r >= p.rank) continue;
      if (adapters < 64 && p.depth > 1) {  // another cluster's
        bool here = false;
        for (uint64_t f = firsts; f; f &= f - 1) here |= s_id[__ffsll(f) - 1] == a;
        if (!here) continue;
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t at = ptx::smem_u32(&fours[i]);
      for (int c = 0; c < C; ++c) {
        const float4 z = ptx::ld_cluster_v4(C > 1 ? ptx::map_to_rank(at, c) : at);
        v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
      }
      const float scale = p.scale ? p.scale[a] : 1.f;
      *reinterpret_cast<float4*>(p.s + (row0 + row) * p.rank + r) = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
  }
}

cudaError_t launch_lora_sums(LoraParams p, int sms, cudaStream_t s) {
  const bool few = p.M <= lora::kFewRows;
  const int64_t tiles = (p.M + lora::kManyRows - 1) / lora::kManyRows;
  const int64_t ranks = (p.rank + 15) / 16;
  int64_t units = few ? std::min<int64_t>(p.M, p.count) * ranks : tiles;
  // few: as wide as clusters go; many: twice the SMs' number of CTAs, of at least 256 K each, and where that leaves SMs idle
  // more clusters for the tiles that have several adapters
  p.split = 1;
  while (p.split < 8 && (few ? 2 * p.split * 32 <= p.K : units * p.split < 2 * sms && 2 * p.split * 256 <= p.K)) p.split *= 2;
  p.depth = 1;
  if (!few) {
    while (p.depth < 8 && 2 * p.depth <= p.count && tiles * p.split * p.depth * 2 <= 4 * sms) p.depth *= 2;
    units = tiles * p.depth;
  }
  const int64_t scans = p.scans * ((p.M + 255) / 256);
  const int smem = few ? 0 : 8 * lora::kManyRows * (p.rank <= 16 ? 16 : 32) * 4;
  auto kernel = few ? lora_sums_few_kernel : (p.rank <= 16 ? lora_sums_many_kernel<1> : lora_sums_many_kernel<2>);
  if (smem > 48 * 1024) {
    static std::atomic<int> configured_device{-1};
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device.load(std::memory_order_relaxed) != dev) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      configured_device.store(dev, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)((units + (scans + p.split - 1) / p.split) * p.split));
  lc.blockDim = dim3(lora::kThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, p);
}

cudaError_t launch_lora_linear(const LinearMaps& maps, const LinearParams& p, cudaStream_t s) {
  return p.out_f32 ? launch_form<true, true>(maps, p, s) : launch_form<false, true>(maps, p, s);
}

}  // namespace gmmfr
