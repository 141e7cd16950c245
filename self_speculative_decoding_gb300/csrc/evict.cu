// Eviction from a K/V cache by accumulated attention weight (sm_103a).
//
// Per K/V head, of the rows 0 .. n-1 the first `sinks`, the last `recent` and
// the heaviest of the rest stay, `keep` in all, in their order; a tie goes to
// the lower row.  One kernel finds the rows (the weight of the last row that
// stays, by radix selection on the weights' bits, then the rows' places by
// prefix sums), one copies them.
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "tree.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCopies = 8;          // of the first histogram: lane l counts in copy l % 8
constexpr int kItems = 16;          // keys per thread that stay in shared memory
constexpr int kChunk = kSelThreads * kItems;
static_assert(kChunk < 1 << 15, "two counts of a chunk's rows share a word");
constexpr int kRankKeys = 512;      // at most so many middle rows are ranked by counting
constexpr int kMaxCluster = 8;
constexpr int kWords = 1024;        // of a histogram of 2048 bins
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

// log2 of the rows per thread of a chunk: 4, 8 or 16.
SSD_HD int key_log(int share) {
  return share <= 4 * kSelThreads ? 2 : share <= 8 * kSelThreads ? 3 : 4;
}

// Rows j0 .. j0 + cnt - 1 of a head's output: all of a thread's 16-byte units
// in flight at once.
constexpr int kCopyUnits = 4;       // units per thread and turn, of K and of V
template <int kThreads>
SSD_DI void copy_rows(const EvictArgs& a, int h, int j0, int cnt, int32_t* src_row) {
  const int tid = threadIdx.x;
  for (int j = tid; j < cnt; j += kThreads) {
    // the first and the last rows are known without the selection
    const int o = j0 + j, last = o - (a.keep - a.recent);
    const int i = o < a.sinks ? o : last >= 0 ? a.n - a.recent + last : a.kept[(size_t)h * a.keep + o];
    src_row[j] = i;
    if (o < a.sinks || last >= 0) a.kept[(size_t)h * a.keep + o] = i;
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

// The kept rows of a head in turn to CTAs of 1024 units of K and of V, read once
// (past the caches) and written once: bound by memory, 8 heads of 16384 rows
// 20.4 us (134 MB, 6.6 TB/s), 40 heads of 2048 rows 14.7 (84 MB, 5.7 TB/s).
constexpr int kCopyThreads = 256;
constexpr int kCopyRows = kCopyThreads * kCopyUnits;
__global__ void __launch_bounds__(kCopyThreads) evict_gather_kernel(const EvictArgs a, int rows) {
  __shared__ int32_t src_row[kCopyRows];
  // (rows that are known are copied while the selection runs)
  const int j0 = blockIdx.x * rows, cnt = min(rows, a.keep - j0);
  const bool known = j0 + cnt <= a.sinks || j0 >= a.keep - a.recent;
  if (!known) pdl_wait();
  copy_rows<kCopyThreads>(a, blockIdx.y, j0, cnt, src_row);
  if (known) pdl_wait();
}

// Cluster = one K/V head, its middle rows divided among the CTAs (`share`
// each), the weights' keys in shared memory (a CTA with more than 16384 reads
// them again from L2).  11 + 11 + 10 bits of the cut are found from histograms
// summed over the cluster; a pass whose bin stays as a whole is the last.
// Counts are 16 bits, two to a word, which halves what the CTAs read of each
// other (a word each, `wide`, where a CTA has more rows than 16 bits count).
// Weights share few exponents, so the first histogram has eight copies: lanes
// of a warp rarely meet in one.  What the lower CTAs have over the cut comes
// out of the same sums, so that the places need no further exchange.
// With `fused` (one CTA per head, few rows) the CTA copies the rows too.
// Bound by latency: barriers, reads of the others' sums, and code that runs
// only once.  Hence short loops over keys in shared memory and places counted
// per thread over rows that lie together: 8 heads of 131072 rows took 36.9 us
// with the copy (20.4) against 40.8 with the keys in registers, unrolled loops
// and places from ballots, 40 heads of 4095 rows 16.9 against 17.9, in turns in
// one process (processes differ: 36.5 to 41.4 and 17.2 to 20.0 us).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int share,
                                                                  int fused) {
  extern __shared__ __align__(16) uint32_t smem[];
  __shared__ int32_t src_row[kFusedRows];
  __shared__ int wsum[kSelWarps];
  __shared__ uint32_t s_bin;
  __shared__ int s_need;
  __shared__ int s_all;
  __shared__ int s_over;         // rows of the lower CTAs over the cut's bin,
  __shared__ int s_with;         // and in it
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const float* w = a.weight + (size_t)blockIdx.y * a.max_seq;
  int32_t* kept = a.kept + (size_t)blockIdx.y * a.keep;
  const int lo = a.sinks, hi = a.n - a.recent, want = a.keep - a.sinks - a.recent;
  const int c0 = min(lo + rank * share, hi), len = min(share, hi - c0);
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
    const bool wide = share > 65535;
    const int words = wide ? 2 * kWords : kWords;
    uint32_t* hist = smem;                       // [word][copy]
    uint32_t* sums = hist + kCopies * words;     // [pass][word]
    // a chunk's keys: thread t has rows t << lg .. ((t + 1) << lg) - 1, four
    // words more behind every thread's eight or sixteen (no bank conflicts)
    uint32_t* keys = sums + 3 * words;
    const int lg = key_log(share), pad = lg > 2 ? 4 : 0, stride = (1 << lg) + pad;
    const bool again = len > kChunk;             // the chunks take turns in it
    auto fetch = [&](int base) {
      const int cnt = min(kChunk, len - base);
      for (int i0 = tid; i0 < cnt; i0 += 8 * kSelThreads) {
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int i = i0 + q * kSelThreads;
          x[q] = i < cnt ? w[c0 + base + i] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int i = i0 + q * kSelThreads;
          if (i < cnt) keys[i + (i >> lg) * pad] = __float_as_uint(x[q]);
        }
      }
    };
    // four keys from the thread's row j on, 0 beyond the chunk's cnt rows
    auto raw = [&](int j, int cnt) {
      uint4 x = *reinterpret_cast<const uint4*>(keys + tid * stride + j);
      const int left = cnt - (tid << lg) - j;
      x.x = left > 0 ? weight_key(__uint_as_float(x.x)) : 0u;
      x.y = left > 1 ? weight_key(__uint_as_float(x.y)) : 0u;
      x.z = left > 2 ? weight_key(__uint_as_float(x.z)) : 0u;
      x.w = left > 3 ? weight_key(__uint_as_float(x.w)) : 0u;
      return x;
    };
    auto four = [&](int j, int cnt) {
      return again ? raw(j, cnt) : *reinterpret_cast<const uint4*>(keys + tid * stride + j);
    };
    if (tid == 0) s_over = 0;
    for (int i = tid; i < (kCopies + 3) * words / 4; i += kSelThreads)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (!again) fetch(0);
    __syncthreads();
    // ---- the want-th largest key, and how many rows at it stay
    uint32_t cut = 0;
    int need = want;
    bool exact = false;
#pragma unroll 1
    for (int pass = 0; pass < 3 && !exact; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      const int above = shift + (pass == 2 ? 10 : 11);
      uint32_t* sum = sums + pass * words;
      for (int base = 0; base < len; base += kChunk) {
        const int cnt = min(kChunk, len - base);
        if (again) {
          __syncthreads();                       // the chunk before is read
          fetch(base);
          __syncthreads();
        }
        for (int j = 0; j < 1 << lg; j += 4) {
          uint4 x;
          if (pass == 0) {                       // keys take the place of the weights
            x = raw(j, cnt);
            *reinterpret_cast<uint4*>(keys + tid * stride + j) = x;
          } else {
            x = four(j, cnt);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t k = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
            const uint32_t bin = (k >> shift) & mask;
            const uint32_t at = wide ? bin : bin >> 1, one = wide ? 1u : 1u << (16 * (bin & 1));
            if (pass == 0) {
              if (k) atomicAdd(&hist[at * kCopies + (tid & (kCopies - 1))], one);
            } else if ((k >> above) == (cut >> above)) {
              atomicAdd(&sum[at], one);
            }
          }
        }
      }
      if (pass == 0) {
        __syncthreads();
        for (int i = tid; i < words; i += kSelThreads) {
          const uint4 x = reinterpret_cast<const uint4*>(hist)[2 * i];
          const uint4 y = reinterpret_cast<const uint4*>(hist)[2 * i + 1];
          sum[i] = (x.x + x.y + x.z + x.w) + (y.x + y.y + y.z + y.w);
        }
      }
      if (nc > 1)
        cluster.sync();
      else
        __syncthreads();
      // thread t takes the bins 2047 - 2 t and 2046 - 2 t, so that lower
      // threads hold larger keys
      const int pair = kWords - 1 - tid;
      int hi_n = 0, lo_n = 0;
      uint2 o[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        o[c] = make_uint2(0u, 0u);
        if (c >= nc) continue;
        const uint32_t* from = nc > 1 ? cluster.map_shared_rank(sum, c) : sum;
        if (wide)
          o[c] = reinterpret_cast<const uint2*>(from)[pair];
        else
          o[c].x = from[pair];
      }
      int hi_low = 0, lo_low = 0;                // of the lower CTAs
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const int h = (int)(wide ? o[c].y : o[c].x >> 16);
        const int l = (int)(wide ? o[c].x : o[c].x & 0xffffu);
        hi_n += h;
        lo_n += l;
        if (c < rank) {
          hi_low += h;
          lo_low += l;
        }
      }
      int total;
      const int before = block_scan(hi_n + lo_n, wsum, total);
      if (before < need && before + hi_n + lo_n >= need) {
        const bool first = before + hi_n >= need;
        s_bin = (uint32_t)(2 * pair + first);
        s_need = need - before - (first ? 0 : hi_n);
        s_all = s_need == (first ? hi_n : lo_n);
        s_with = first ? hi_low : lo_low;
      }
      __syncthreads();
      if (rank) {
        const uint32_t b = s_bin;
        const int over = __reduce_add_sync(~0u, ((uint32_t)(2 * pair + 1) > b ? hi_low : 0) +
                                                    ((uint32_t)(2 * pair) > b ? lo_low : 0));
        if (lane == 0 && over) atomicAdd(&s_over, over);
      }
      cut |= s_bin << shift;
      need = s_need;
      exact = s_all;
    }
    if (nc > 1) cluster.barrier_arrive();        // the others' sums are read
    __syncthreads();
    // rows over and at the cut before this CTA's
    int g = s_over + (exact ? s_with : 0), e = s_with;
    if (exact) {                                 // the last bin stays as a whole
      cut -= 1;                                  // (bin 0 of every pass is no key)
      need = 0;
    }
    // ---- places: rows over the cut, and the lowest `need` rows at it; each
    // thread's counted (over: low half, at: high half; each below 2^15), then
    // placed from where the threads before it end
    for (int base = 0; base < len; base += kChunk) {
      const int cnt = min(kChunk, len - base);
      if (again) {
        __syncthreads();
        fetch(base);
        __syncthreads();
      }
      int mine = 0;
      for (int j = 0; j < 1 << lg; j += 4) {
        const uint4 x = four(j, cnt);
        mine += (x.x > cut) + (x.y > cut) + (x.z > cut) + (x.w > cut);
        mine += ((x.x == cut) + (x.y == cut) + (x.z == cut) + (x.w == cut)) << 16;
      }
      int total;
      const uint32_t at = (uint32_t)block_scan(mine, wsum, total);
      int over = g + (int)(at & 0xffffu), with = e + (int)(at >> 16);
      for (int j = 0; j < 1 << lg; j += 4) {
        const uint4 x = four(j, cnt);
        const int i0 = c0 + base + (tid << lg) + j;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
          if (k > cut || (k == cut && with < need)) kept[a.sinks + over + min(with, need)] = i0 + i;
          over += k > cut;
          with += k == cut;
        }
      }
      g += total & 0xffff;
      e += (int)((uint32_t)total >> 16);
    }
    if (nc > 1) cluster.barrier_wait();          // no CTA leaves while another reads its sums
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
  // A CTA per 4096 middle rows up to the portable cluster size (8 heads of 16000
  // rows 18.9 us so, 20.9 with one per 8192; 40 heads of 4095 rows 16.4 with one,
  // 18 with two CTAs a head, in turns in one process), while no SM gets a second one (32 heads of 32768 rows 31.7
  // us with four CTAs a head, 49.5 with eight; 40 heads of 20000 rows 25.1 with
  // two, 29 with four) or a CTA has more rows than it holds (80 heads of 65536
  // rows 72 us with four, 95 with one, 104 with eight).
  int nc = 1;
  while (nc < kMaxCluster && (long long)nc * 4096 < middle &&
         (2LL * nc * a.Hkv <= tree_sms() || (long long)nc * kChunk < middle))
    nc *= 2;
  const bool fused = few && nc == 1;
  const int share = (middle + nc - 1) / nc;
  const bool ranked = want == 0 || (nc == 1 && share <= kRankKeys);
  const size_t hist = (size_t)(kCopies + 3) * kWords * 4;
  const int lg = key_log(share);
  const size_t held = (size_t)kSelThreads * ((1 << lg) + (lg > 2 ? 4 : 0)) * 4;
  const size_t smem = ranked ? kRankKeys * 4 : (share > 65535 ? 2 * hist : hist) + held;
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e = cudaFuncSetAttribute(
        evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)(2 * hist) + kSelThreads * (kItems + 4) * 4);
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
  cudaError_t e = cudaLaunchKernelEx(&lc, evict_select_kernel, a, share, (int)fused);
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
