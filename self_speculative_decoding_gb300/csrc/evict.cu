// Eviction from a K/V cache by accumulated attention weight (sm_103a).
//
// Per K/V head, of the rows 0 .. n-1 the first `sinks`, the last `recent` and
// the heaviest of the rest stay, `keep` in all, in their order; a tie goes to
// the lower row.  One kernel finds the rows (the weight of the last row that
// stays, by radix selection on the weights' bits), one copies them.
#include "kernels.cuh"

namespace ssd {
namespace {

constexpr int kSelThreads = 1024;

// Weights as unsigned keys in the same order: -0 as +0, NaN as -infinity.
SSD_DI uint32_t weight_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// CTA = one K/V head.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int wsum[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* w = a.weight + (size_t)blockIdx.x * a.max_seq;
  int32_t* kept = a.kept + (size_t)blockIdx.x * a.keep;
  const int lo = a.sinks, hi = a.n - a.recent, want = a.keep - a.sinks - a.recent;
  // the want-th largest key of [lo, hi), eight bits at a time
  if (tid == 0) {
    s_prefix = 0;
    s_need = want;
  }
  for (int shift = 24; shift >= 0 && want > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t u = weight_key(w[i]);
      if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(u >> shift) & 255u], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int need = s_need, b = 255;
      while (b > 0 && hist[b] < need) need -= hist[b--];
      s_need = need;
      s_prefix = prefix | ((uint32_t)b << shift);
    }
    __syncthreads();
  }
  __syncthreads();
  const uint32_t cut = s_prefix;
  const int ties = s_need;  // rows of weight `cut` that stay: the lowest ones
  for (int i = tid; i < a.sinks; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < a.recent; i += kSelThreads) kept[a.keep - a.recent + i] = hi + i;
  int above = 0, equal = 0;  // rows before this tile over the cut, and at it
  for (int base = lo; base < hi && want > 0; base += kSelThreads) {
    const int i = base + tid;
    const uint32_t u = i < hi ? weight_key(w[i]) : 0u;
    const bool gt = i < hi && u > cut, eq = i < hi && u == cut;
    const uint32_t mg = __ballot_sync(~0u, gt), me = __ballot_sync(~0u, eq);
    if (lane == 0) {
      wsum[0][warp] = __popc(mg);
      wsum[1][warp] = __popc(me);
    }
    __syncthreads();
    int g = above, e = equal;
    for (int x = 0; x < kSelThreads / 32; ++x) {
      if (x < warp) {
        g += wsum[0][x];
        e += wsum[1][x];
      }
      above += wsum[0][x];
      equal += wsum[1][x];
    }
    g += __popc(mg & ((1u << lane) - 1u));
    e += __popc(me & ((1u << lane) - 1u));
    if (gt || (eq && e < ties)) kept[a.sinks + g + min(e, ties)] = i;
    __syncthreads();
  }
}

// Warp = one row that stays: 16-byte units of its K and V row.
__global__ void __launch_bounds__(256) evict_gather_kernel(const EvictArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 8 + warp, h = blockIdx.y;
  if (j >= a.keep) return;
  const int i = a.kept[(size_t)h * a.keep + j];
  const size_t src = ((size_t)h * a.max_seq + i) * a.units, dst = ((size_t)h * a.max_out + j) * a.units;
  for (int u = lane; u < a.units; u += 32) {
    a.k_out[dst + u] = a.k[src + u];
    a.v_out[dst + u] = a.v[src + u];
  }
  if (lane == 0 && a.weight_out)
    a.weight_out[(size_t)h * a.max_out + j] = a.weight[(size_t)h * a.max_seq + i];
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  evict_select_kernel<<<a.Hkv, kSelThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_gather_kernel<<<dim3((a.keep + 7) / 8, a.Hkv), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssd
