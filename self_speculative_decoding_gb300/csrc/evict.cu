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
constexpr int kCopies = 8;          // of the first histogram: lane l counts in copy l % 8
constexpr int kSelKeys = 33792;     // weights of a CTA that fit its shared memory
constexpr int kRankKeys = 512;      // at most so many middle rows are ranked by counting
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kFusedRows = 512;     // rows and 16-byte units that a selecting CTA copies itself
constexpr int kFusedUnits = 4096;

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

// Rows j0 .. j0 + cnt - 1 of a head's output: all of a thread's 16-byte units
// in flight at once.
constexpr int kCopyUnits = 4;       // units per thread and turn, of K and of V
template <int kThreads>
SSD_DI void copy_rows(const EvictArgs& a, int h, int j0, int cnt, int32_t* src_row) {
  const int tid = threadIdx.x;
  for (int j = tid; j < cnt; j += kThreads) {
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
  for (unsigned e0 = 0; e0 < n; e0 += kThreads * kCopyUnits) {
    uint4 x[kCopyUnits], y[kCopyUnits];
#pragma unroll
    for (int q = 0; q < kCopyUnits; ++q) {
      const unsigned e = e0 + q * kThreads + tid;
      if (e >= n) continue;
      const unsigned j = e / (unsigned)a.units, u = e - j * a.units;
      const size_t s = (size_t)src_row[j] * a.units + u;
      x[q] = __ldcs(k + s);
      y[q] = __ldcs(v + s);
    }
#pragma unroll
    for (int q = 0; q < kCopyUnits; ++q) {
      const unsigned e = e0 + q * kThreads + tid;
      if (e >= n) continue;
      a.k_out[o + e] = x[q];
      a.v_out[o + e] = y[q];
    }
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = kCopyThreads * kCopyUnits;
__global__ void __launch_bounds__(kCopyThreads) evict_gather_kernel(const EvictArgs a, int rows) {
  __shared__ int32_t src_row[kCopyRows];
  pdl_wait();
  const int j0 = blockIdx.x * rows;
  copy_rows<kCopyThreads>(a, blockIdx.y, j0, min(rows, a.keep - j0), src_row);
}

// Cluster = one K/V head, its middle rows divided among the CTAs.  Each keeps
// its weights' keys in shared memory (re-reading them from L2 where a head
// has more than a cluster holds); 11 + 11 + 10 bits of the cut are found from
// histograms summed over the cluster.  Weights share few exponents, so the
// first histogram has eight copies: lanes of a warp rarely meet in one.
// With `fused` (one CTA per head, few rows) the CTA copies the rows too.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int fused) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int32_t src_row[kFusedRows];
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
  if (rank == 0) {
    for (int i = tid; i < a.sinks; i += kSelThreads) kept[i] = i;
    for (int i = tid; i < a.recent; i += kSelThreads) kept[a.keep - a.recent + i] = hi + i;
  }
  if (nc == 1 && len <= kRankKeys) {
    // few rows: each counts the rows before it in the order
    if (tid < kRankKeys) smem[tid] = tid < len ? weight_key(w[c0 + tid]) : 0u;  // 0: under every key
    __syncthreads();
    const uint32_t u = tid < len ? smem[tid] : 0u;
    int before = tid < len ? 0 : want;
    for (int j = 0; j < len && tid < len; j += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(smem + j);
      before += (o.x > u || (o.x == u && j < tid)) + (o.y > u || (o.y == u && j + 1 < tid)) +
                (o.z > u || (o.z == u && j + 2 < tid)) + (o.w > u || (o.w == u && j + 3 < tid));
    }
    int total;
    const int at = block_scan(before < want, wsum, total);
    if (before < want) kept[a.sinks + at] = c0 + tid;
  } else if (want > 0) {
    int* hist = reinterpret_cast<int*>(smem);    // [bin][copy]
    int* sums = hist + kCopies * kBins;          // [pass][bin]
    uint32_t* keys = smem + (kCopies + 3) * kBins;
    const bool held = share <= kSelKeys;
    auto key = [&](int i) { return held ? keys[i] : weight_key(w[c0 + i]); };
    for (int i = tid; i < (kCopies + 3) * kBins / 4; i += kSelThreads)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (held)
      for (int i = tid; i < len; i += kSelThreads) keys[i] = weight_key(w[c0 + i]);
    __syncthreads();
    // ---- the want-th largest key, and how many rows at it stay
    uint32_t cut = 0;
    int need = want;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      const int above = shift + (pass == 2 ? 10 : 11);
      int* sum = sums + pass * kBins;
      if (pass == 0) {
        for (int i = tid; i < len; i += kSelThreads)
          atomicAdd(&hist[(key(i) >> 21) * kCopies + (tid & (kCopies - 1))], 1);
        __syncthreads();
        for (int i = tid; i < kBins; i += kSelThreads) {
          const int4 x = reinterpret_cast<const int4*>(hist)[2 * i];
          const int4 y = reinterpret_cast<const int4*>(hist)[2 * i + 1];
          sum[i] = (x.x + x.y + x.z + x.w) + (y.x + y.y + y.z + y.w);
        }
      } else {
        for (int i = tid; i < len; i += kSelThreads) {
          const uint32_t u = key(i);
          if ((u >> above) == (cut >> above)) atomicAdd(&sum[(u >> shift) & mask], 1);
        }
      }
      if (nc > 1)
        cluster.sync();
      else
        __syncthreads();
      // thread t takes the bins 2047 - 2 t and 2046 - 2 t, so that lower
      // threads hold larger keys
      const int b1 = kBins - 1 - 2 * tid;
      int2 h = make_int2(0, 0);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < nc) {
          const int2 o = *reinterpret_cast<const int2*>(cluster.map_shared_rank(sum, c) + b1 - 1);
          h.x += o.y;
          h.y += o.x;
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
    if (nc > 1) {
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
    }
    for (int i = i0; i < i1; ++i) {
      const uint32_t u = key(i);
      if (u > cut || (u == cut && e < need)) kept[a.sinks + g + min(e, need)] = c0 + i;
      g += u > cut;
      e += u == cut;
    }
    if (nc > 1) cluster.sync();  // no CTA leaves while another reads its shared memory
  }
  if (fused) {
    __syncthreads();             // the CTA's own entries of kept
    copy_rows<kSelThreads>(a, blockIdx.y, 0, a.keep, src_row);
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  const int middle = a.n - a.sinks - a.recent, want = a.keep - a.sinks - a.recent;
  // Few rows that stay: the selecting CTA copies them (one launch).
  const bool few = (long long)a.keep * a.units <= kFusedUnits && a.keep <= kFusedRows;
  // A CTA per 8192 middle rows up to the portable cluster size: the exchange
  // of histograms costs a cluster more than a CTA's longer runs (40 heads of
  // 4095 rows: 12 us with one CTA per head, 25 us with four).
  int nc = 1;
  while (nc < kMaxCluster && (long long)nc * 8192 < middle) nc *= 2;
  const bool fused = few && nc == 1;
  const int share = (middle + nc - 1) / nc;
  const bool ranked = want == 0 || (nc == 1 && share <= kRankKeys);
  const size_t smem = ranked ? kRankKeys * 4
                             : ((size_t)(kCopies + 3) * kBins + (share <= kSelKeys ? share : 0)) * 4;
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e =
        cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ((kCopies + 3) * kBins + kSelKeys) * 4);
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
  cudaError_t e = cudaLaunchKernelEx(&lc, evict_select_kernel, a, (int)fused);
  if (e != cudaSuccess || fused) return e;
  int rows = kCopyRows / a.units;
  if (rows < 1) rows = 1;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3((unsigned)((a.keep + rows - 1) / rows), (unsigned)a.Hkv);
  lc.blockDim = dim3(kCopyThreads);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, evict_gather_kernel, a, rows);
}

}  // namespace ssd
