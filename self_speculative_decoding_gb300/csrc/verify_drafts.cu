// Verification of drafted tokens from given random numbers (sm_103a).
//
// Draft j of a sequence, token y, stays while u_j q_j(y) < p_j(y) (in 64 bits,
// where the product is exact).  At the first that does not, a token is drawn
// from r = max(p_j - q_j, 0), or from p_j where that is empty; after the last,
// from r = p_d: the lowest v with  sum_{w <= v} r_w > U sum r.
//
// Sums keep the rounding errors of their fp32 additions beside them (Knuth's
// two-sum), which leaves about 2^-45 of the sum: a token changes hands only if U
// lies that near to a border.
#include <cooperative_groups.h>

#include "batch.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// s + e = a + b exactly.
SSD_DI void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// What one entry adds: max(p - q, 0) as a value and its rounding error.
SSD_DI void rest_of(float p, float q, float& r, float& e) {
  two_sum(p, -q, r, e);
  if (!(r > 0.f)) r = e = 0.f;                   // (NaN too)
}

// A cluster per sequence, a slice of the vocabulary per CTA and a run of it per
// warp.  Each CTA tests the drafts by itself; the sums meet once.
__global__ void __launch_bounds__(kThreads) verify_drafts_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int s_taken;
  __shared__ double s_warp[kWarps];
  __shared__ double s_cta[2][kMaxCluster];       // each CTA's sum, from the CTAs themselves
  cluster.barrier_arrive();                      // (all CTAs run before one writes to another)
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / size;
  const int count = a.counts ? min(max(a.counts[b], 0), a.d) : a.d;
  if (tid == 0) s_taken = count;
  __syncthreads();
  for (int j = tid; j < count; j += kThreads) {
    const int y = a.drafts[(size_t)b * a.d + j];
    bool good = y >= 0 && y < a.V;
    if (good) {
      const double p = a.p[((size_t)b * (a.d + 1) + j) * a.V + y];
      const double q = a.q ? a.q[((size_t)b * a.d + j) * a.V + y] : 1.f;
      good = (double)a.accept_u[(size_t)b * a.d + j] * q < p;
    }
    if (!good) atomicMin(&s_taken, j);
  }
  __syncthreads();
  const int taken = s_taken;
  const float* p = a.p + ((size_t)b * (a.d + 1) + taken) * a.V;
  const float* q = a.q && taken < count ? a.q + ((size_t)b * a.d + taken) * a.V : nullptr;
  // without probabilities of the drafts the rejected token alone is left out
  const int out = !a.q && taken < count ? a.drafts[(size_t)b * a.d + taken] : -1;
  bool plain = taken == count;                   // r = p
  const int slice = (a.V + size - 1) / size, lo = min(rank * slice, a.V), hi = min(lo + slice, a.V);
  const int run = (hi - lo + kWarps - 1) / kWarps, w0 = min(lo + warp * run, hi), w1 = min(w0 + run, hi);
  auto entry = [&](int v, float& r, float& e) {
    rest_of(p[v], plain ? 0.f : q ? q[v] : v == out ? p[v] : 0.f, r, e);
  };
  double total = 0.0, before = 0.0, mine = 0.0;
  int last = -1;                                 // the last CTA with anything
  for (int turn = 0; turn < 2; ++turn) {
    float s = 0.f, c = 0.f;
#pragma unroll 4
    for (int v = w0 + lane; v < w1; v += 32) {
      float r, e, t;
      entry(v, r, e);
      two_sum(s, r, s, t);
      c += t + e;
    }
    double x = (double)s + (double)c;
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    mine = 0.0;
    for (int i = 0; i < kWarps; ++i) mine += s_warp[i];
    if (turn == 0) cluster.barrier_wait();
    if (tid < size) cluster.map_shared_rank(&s_cta[turn][rank], tid)[0] = mine;
    cluster.sync();
    total = 0.0;
    last = -1;
    for (int i = 0; i < size; ++i) {
      if (i == rank) before = total;
      total += s_cta[turn][i];
      if (s_cta[turn][i] > 0.0) last = i;
    }
    if (plain || total > 0.0) break;
    plain = true;                                // nothing is left: from p itself
    __syncthreads();
  }
  // the CTA, then the warp, then the entry in which the sum passes the target
  const double target = (double)a.sample_u[b] * total;
  int owner = total < INFINITY ? last : -1;
  if (owner >= 0) {
    double sum = 0.0;
    for (int i = 0; i < size; ++i) {
      sum += s_cta[plain && taken < count ? 1 : 0][i];
      if (sum > target) {
        owner = i;
        break;
      }
    }
  }
  int32_t* tokens = a.tokens + (size_t)b * (a.d + 1);
  if (rank == 0) {
    for (int j = tid; j <= a.d; j += kThreads)
      if (j != taken) tokens[j] = j < taken ? a.drafts[(size_t)b * a.d + j] : -1;
    if (tid == 0) {
      a.n[b] = taken + (owner >= 0 ? 1 : 0);
      if (owner < 0) tokens[taken] = -1;         // no probability anywhere
    }
  }
  if (rank != owner) return;
  double sum = before;
  int w = -1, lastw = -1;
  for (int i = 0; i < kWarps; ++i) {
    if (s_warp[i] > 0.0) lastw = i;
    if (sum + s_warp[i] > target) {
      w = i;
      break;
    }
    sum += s_warp[i];
  }
  const bool found = w >= 0;
  if (warp != (found ? w : lastw)) return;
  int token = -1;
  for (int v0 = w0; v0 < w1 && token < 0; v0 += 32) {
    float r = 0.f, e = 0.f;
    if (v0 + lane < w1) entry(v0 + lane, r, e);
    double x = (double)r + (double)e;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    const unsigned past = __ballot_sync(~0u, found && v0 + lane < w1 && r > 0.f && sum + x > target);
    if (past) token = v0 + __ffs(past) - 1;
    sum += __shfl_sync(~0u, x, 31);
  }
  if (token < 0) {                               // U at the sum's very end: the last entry with anything
    for (int v0 = w0; v0 < w1; v0 += 32) {
      float r = 0.f, e = 0.f;
      if (v0 + lane < w1) entry(v0 + lane, r, e);
      const unsigned any = __ballot_sync(~0u, r > 0.f);
      if (any) token = v0 + 31 - __clz(any);
    }
  }
  if (lane == 0) tokens[taken] = token;
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
  int size = 1;
  while (size < kMaxCluster && a.V > size * 4096) size *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)size, 1, 1};
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(a.B * size));
  lc.blockDim = dim3(kThreads);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, verify_drafts_kernel, a);
}

}  // namespace ssd
