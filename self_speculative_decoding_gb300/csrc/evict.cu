// Eviction from a K/V cache by accumulated attention weight (sm_103a).
//
// Per K/V head, of the rows 0 .. n-1 the first `sinks`, the last `recent` and
// the heaviest of the rest stay, `keep` in all, in their order; a tie goes to
// the lower row.  One kernel finds the rows (the weight of the last row that
// stays, by radix selection on the weights' bits, then the rows' places by
// prefix sums), one copies them.
#include <cooperative_groups.h>

#include "kernels.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 49152;     // weights of a CTA that fit its shared memory
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;

// Weights as unsigned keys in the same order: -0 as +0, NaN as -infinity.
SSD_DI uint32_t weight_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the block's lower threads of x (exclusive), and the total.
SSD_DI int block_scan(int x, int* wsum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, v, d);
    if (lane >= d) v += y;
  }
  if (lane == 31) wsum[warp] = v;
  __syncthreads();
  int w = wsum[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(~0u, w, 31);
  const int below = __shfl_sync(~0u, w, warp ? warp - 1 : 0);
  __syncthreads();
  return (warp ? below : 0) + v - x;
}

// Cluster = one K/V head, its middle rows divided among the CTAs.  Each keeps
// its weights' keys in shared memory (re-reading them from L2 where a head
// has more than a cluster holds); 11 + 11 + 10 bits of the cut are found from
// histograms summed over the cluster.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[3][kBins];
  __shared__ int wsum[kSelWarps];
  __shared__ uint32_t s_bin;
  __shared__ int s_need;
  __shared__ int s_count[2];
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const float* w = a.weight + (size_t)blockIdx.y * a.max_seq;
  int32_t* kept = a.kept + (size_t)blockIdx.y * a.keep;
  const int lo = a.sinks, hi = a.n - a.recent, want = a.keep - a.sinks - a.recent;
  const int share = (hi - lo + nc - 1) / nc;
  const int c0 = min(lo + rank * share, hi), len = min(share, hi - c0);
  const bool held = share <= kSelKeys;
  auto key = [&](int i) { return held ? keys[i] : weight_key(w[c0 + i]); };
  if (held)
    for (int i = tid; i < len; i += kSelThreads) keys[i] = weight_key(w[c0 + i]);
  if (rank == 0) {
    for (int i = tid; i < a.sinks; i += kSelThreads) kept[i] = i;
    for (int i = tid; i < a.recent; i += kSelThreads) kept[a.keep - a.recent + i] = hi + i;
  }
  if (want == 0) return;  // the whole cluster
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  // ---- the want-th largest key, and how many rows at it stay
  uint32_t cut = 0;
  int need = want;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024u : 2048u;
    const int above = shift + (pass == 2 ? 10 : 11);
    for (int i = tid; i < len; i += kSelThreads) {
      const uint32_t u = key(i);
      if (pass == 0 || (u >> above) == (cut >> above)) atomicAdd(&hist[pass][(u >> shift) & (bins - 1)], 1);
    }
    cluster.sync();
    // thread t takes the bins 2047 - 2 t and 2046 - 2 t, so that lower threads
    // hold larger keys
    const int b1 = kBins - 1 - 2 * tid;
    int2 h = make_int2(0, 0);
    for (int c = 0; c < nc; ++c) {
      const int* other = cluster.map_shared_rank(&hist[pass][0], c);
      h.x += other[b1];
      h.y += other[b1 - 1];
    }
    int total;
    const int before = block_scan(h.x + h.y, wsum, total);
    if (before < need && before + h.x + h.y >= need) {
      const bool first = before + h.x >= need;
      s_bin = (uint32_t)(first ? b1 : b1 - 1);
      s_need = need - before - (first ? 0 : h.x);
    }
    __syncthreads();
    cut |= s_bin << shift;
    need = s_need;
    __syncthreads();
  }
  // ---- places: rows over the cut, and the lowest `need` rows at it
  const int per = ((len + kSelThreads - 1) / kSelThreads) | 1;  // odd: no bank conflicts
  const int i0 = min(tid * per, len), i1 = min(i0 + per, len);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t u = key(i);
    gt += u > cut;
    eq += u == cut;
  }
  int tg, te;
  int g = block_scan(gt, wsum, tg), e = block_scan(eq, wsum, te);
  if (tid == 0) {
    s_count[0] = tg;
    s_count[1] = te;
  }
  cluster.sync();
  for (int c = 0; c < rank; ++c) {
    const int* other = cluster.map_shared_rank(&s_count[0], c);
    g += other[0];
    e += other[1];
  }
  for (int i = i0; i < i1; ++i) {
    const uint32_t u = key(i);
    if (u > cut || (u == cut && e < need)) kept[a.sinks + g + min(e, need)] = c0 + i;
    g += u > cut;
    e += u == cut;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// CTA = a run of rows that stay: all of their 16-byte units in flight at once.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 4;       // units per thread, of K and of V
__global__ void __launch_bounds__(kCopyThreads) evict_gather_kernel(const EvictArgs a, int rows) {
  __shared__ int32_t src_row[kCopyThreads * kCopyUnits];
  pdl_wait();
  const int h = blockIdx.y, j0 = blockIdx.x * rows, tid = threadIdx.x;
  const int cnt = min(rows, a.keep - j0);
  for (int j = tid; j < cnt; j += kCopyThreads) {
    const int i = a.kept[(size_t)h * a.keep + j0 + j];
    src_row[j] = i;
    if (a.weight_out)
      a.weight_out[(size_t)h * a.max_out + j0 + j] = a.weight[(size_t)h * a.max_seq + i];
  }
  __syncthreads();
  const uint4* k = a.k + (size_t)h * a.max_seq * a.units;
  const uint4* v = a.v + (size_t)h * a.max_seq * a.units;
  const size_t o = ((size_t)h * a.max_out + j0) * a.units;
  const unsigned n = (unsigned)cnt * a.units;
  for (unsigned e0 = 0; e0 < n; e0 += kCopyThreads * kCopyUnits) {
    uint4 x[kCopyUnits], y[kCopyUnits];
#pragma unroll
    for (int q = 0; q < kCopyUnits; ++q) {
      const unsigned e = e0 + q * kCopyThreads + tid;
      if (e >= n) continue;
      const unsigned j = e / (unsigned)a.units, u = e - j * a.units;
      const size_t s = (size_t)src_row[j] * a.units + u;
      x[q] = __ldcs(k + s);
      y[q] = __ldcs(v + s);
    }
#pragma unroll
    for (int q = 0; q < kCopyUnits; ++q) {
      const unsigned e = e0 + q * kCopyThreads + tid;
      if (e >= n) continue;
      a.k_out[o + e] = x[q];
      a.v_out[o + e] = y[q];
    }
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  // a CTA per 4096 middle rows up to the portable cluster size: fewer leave
  // SMs idle, more only exchange histograms
  int nc = 1;
  while (nc < kMaxCluster && (long long)nc * 4096 < a.n) nc *= 2;
  const int share = (a.n - a.sinks - a.recent + nc - 1) / nc;
  const size_t smem = share <= kSelKeys ? (size_t)share * 4 : 0;
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e = cudaFuncSetAttribute(
        evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
    if (e != cudaSuccess) return e;
    if (dv >= 0) ready[dv] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)nc, (unsigned)a.Hkv);
  lc.blockDim = dim3(kSelThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&lc, evict_select_kernel, a);
  if (e != cudaSuccess) return e;
  int rows = kCopyThreads * kCopyUnits / a.units;
  if (rows < 1) rows = 1;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)((a.keep + rows - 1) / rows), (unsigned)a.Hkv);
  lc.blockDim = dim3(kCopyThreads);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, evict_gather_kernel, a, rows);
}

}  // namespace ssd
