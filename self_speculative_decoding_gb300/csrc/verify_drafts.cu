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
#include "tree.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;

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

// Sum over the warp's lower lanes and itself, in 64 bits.
SSD_DI double scan(double x, int lanes) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    if (d >= lanes) break;
    const double y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The row that a token is drawn from: max(p - q, 0), p, or p without one token.
struct Rest {
  const float *p, *q;
  int out;
};

constexpr int kBatch = 8;                        // entries of a lane in flight at once

// A lane's entries v0 + k step < v1, k < kBatch, as values and rounding errors.
SSD_DI void get_batch(const Rest& rest, int v0, int step, int v1, float (&r)[kBatch], float (&e)[kBatch]) {
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int v = v0 + k * step;
    r[k] = v < v1 ? rest.p[v] : 0.f;
    e[k] = v < v1 && rest.q ? rest.q[v] : v == rest.out ? r[k] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kBatch; ++k) rest_of(r[k], e[k], r[k], e[k]);
}

// A cluster per sequence, a slice of the vocabulary per CTA and a run of it per
// warp.  Each CTA tests the drafts by itself; the sums meet once.  Then one warp
// walks its run again, 8 entries in a row to a lane.
// Bound by latency: the drafts, their probabilities, the row's entries, the
// cluster's exchange and the walk one behind the other.
__global__ void __launch_bounds__(kThreads, 3) verify_drafts_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  cluster.barrier_arrive();                      // (all CTAs run before one writes to another)
  __shared__ double s_warp[kWarps];              // sums of the warps, then of those up to each
  __shared__ double s_cta[2][kMaxCluster];       // each CTA's sum, from the CTAs themselves
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / size;
  const int count = a.counts ? min(max(a.counts[b], 0), a.d) : a.d;
  const float sample = a.sample_u[b];
  // the drafts in order, 32 at a time (by each warp for itself)
  int taken = count;
#pragma unroll 1
  for (int j0 = 0; j0 < count; j0 += 32) {
    const int j = j0 + lane;
    bool good = true;
    if (j < count) {
      const float u = a.accept_u[(size_t)b * a.d + j];
      const int y = a.drafts[(size_t)b * a.d + j];
      good = y >= 0 && y < a.V;
      if (good) {
        const float p = a.p[((size_t)b * (a.d + 1) + j) * a.V + y];
        const float q = a.q ? a.q[((size_t)b * a.d + j) * a.V + y] : 1.f;
        good = (double)u * (double)q < (double)p;
      }
    }
    const unsigned bad = __ballot_sync(~0u, !good);
    if (bad) {
      taken = j0 + __ffs(bad) - 1;
      break;
    }
  }
  bool plain = taken == count;                   // r = p
  Rest rest;
  rest.p = a.p + ((size_t)b * (a.d + 1) + taken) * a.V;
  rest.q = a.q && !plain ? a.q + ((size_t)b * a.d + taken) * a.V : nullptr;
  // without probabilities of the drafts the rejected token alone is left out
  rest.out = !a.q && !plain ? a.drafts[(size_t)b * a.d + taken] : -1;
  const int slice = (a.V + size - 1) / size, lo = (int)min((long long)rank * slice, (long long)a.V);
  const int hi = min(lo, a.V - slice) + slice;
  const int run = (hi - lo + kWarps - 1) / kWarps, w0 = min(lo + warp * run, hi), w1 = min(w0 + run, hi);
  double total = 0.0, before = 0.0, mine = 0.0;
  int owner = -1, turn = 0;
  while (true) {
    float s = 0.f, c = 0.f;
#pragma unroll 1
    for (int v = w0 + lane; v - lane < w1; v += 32 * kBatch) {
      float r[kBatch], e[kBatch];
      get_batch(rest, v, 32, w1, r, e);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float t;
        two_sum(s, r[k], s, t);
        c += t + e[k];
      }
    }
    double x = (double)s + (double)c;
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
      const double up = scan(lane < kWarps ? s_warp[lane] : 0.0, kWarps);
      mine = __shfl_sync(~0u, up, kWarps - 1);
      if (turn == 0) cluster.barrier_wait();
      if (lane < size) *cluster.map_shared_rank(&s_cta[turn][rank], lane) = mine;
      __syncwarp();
      if (lane < kWarps) s_warp[lane] = up;
    } else if (turn == 0) {
      cluster.barrier_wait();
    }
    cluster.sync();
    // the first CTA whose sums pass the target, or the last that has any
    const double sums = scan(lane < size ? s_cta[turn][lane] : 0.0, kMaxCluster);
    total = __shfl_sync(~0u, sums, size - 1);
    const unsigned any = __ballot_sync(~0u, lane < size && s_cta[turn][lane < size ? lane : 0] > 0.0);
    const unsigned past = __ballot_sync(~0u, lane < size && sums > (double)sample * total);
    owner = past ? __ffs(past) - 1 : any ? 31 - __clz(any) : -1;
    before = __shfl_sync(~0u, sums, rank ? rank - 1 : 0);
    if (rank == 0) before = 0.0;
    if (plain || total > 0.0) break;
    plain = true;                                // nothing is left: from p itself
    rest.q = nullptr;
    rest.out = -1;
    turn = 1;
    __syncthreads();
  }
  if (!(total < INFINITY)) owner = -1;
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
  // the warp, then the lane, then the entry in which the sum passes the target
  const double target = (double)sample * total;
  const double up = lane < kWarps ? s_warp[lane] : 0.0;
  const unsigned past = __ballot_sync(~0u, lane < kWarps && before + up > target);
  const double lower = __shfl_up_sync(~0u, up, 1);
  const unsigned any = __ballot_sync(~0u, lane < kWarps && up > (lane ? lower : 0.0));
  const bool found = past != 0;
  if (warp != (found ? __ffs(past) - 1 : any ? 31 - __clz(any) : 0)) return;
  double sum = before + (warp ? s_warp[warp - 1] : 0.0);
  int token = -1;
#pragma unroll 1
  for (int base = w0; base < w1; base += 32 * kBatch) {
    const int v0 = base + lane * kBatch;
    float r[kBatch], e[kBatch], s = 0.f, c = 0.f;
    get_batch(rest, v0, 1, w1, r, e);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      float t;
      two_sum(s, r[k], s, t);
      c += t + e[k];
    }
    const double x = (double)s + (double)c, to = scan(x, 32);
    const unsigned here = __ballot_sync(~0u, found && x > 0.0 && sum + to > target);
    const unsigned some = __ballot_sync(~0u, x > 0.0);
    double at = sum + (to - x);
    int first = -1, last = -1;                   // the lane's first past the target, its last over 0
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      at += (double)r[k] + (double)e[k];
      if (r[k] > 0.f) {
        last = v0 + k;
        if (first < 0 && at > target) first = v0 + k;
      }
    }
    if (here && first >= 0) last = first;
    if (some) token = __shfl_sync(~0u, last, here ? __ffs(here) - 1 : 31 - __clz(some));
    if (here) break;
    sum += __shfl_sync(~0u, to, 31);
  }
  if (lane == 0) tokens[taken] = token;
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
  // as many CTAs to a sequence as have 2048 entries each and are resident together
  // (three of an SM)
  int size = 1;
  while (size < kMaxCluster && a.V > size * 2048 && a.B * size * 2 <= 3 * tree_sms()) size *= 2;
  if (size > 8) {
    static bool ready[kDeviceSlots] = {};
    const int dv = device_slot();
    if (dv < 0 || !ready[dv]) {
      const cudaError_t e = cudaFuncSetAttribute(verify_drafts_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dv >= 0) ready[dv] = true;
    }
  }
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
