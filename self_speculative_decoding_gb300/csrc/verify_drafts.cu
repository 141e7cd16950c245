// Verification of drafted tokens from given random numbers (sm_103a).
//
// Draft j of a sequence, token y, stays while u_j q_j(y) < p_j(y) (in 64 bits,
// where the product is exact).  At the first that does not, a token is drawn
// from r = max(p_j - q_j, 0), or from p_j where that is empty; after the last,
// from r = p_d: the lowest v with  sum_{w <= v} r_w > U sum r.
//
// Sums keep the rounding errors of their fp32 additions beside them (Knuth's
// two-sum), which leaves 2^-41 of the sum, and 2^-49 for each of a thread's entries: a
// token changes hands only if U lies that near to a border.
#include <cooperative_groups.h>

#include <cfloat>

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

// u q < p without rounding: the product's rounding error decides where the rounded
// product is p (u and p scaled, so that the error of a small product is a normal number; a
// product that overflows is above any p).  In 64 bits it took 0.6 us more.
SSD_DI bool less(float u, float q, float p) {
  const float up = p < 0x1p60f ? 0x1p64f : 1.f;
  u *= up;
  p *= up;
  const float h = __fmul_rn(u, q), l = __fmaf_rn(u, q, -h);
  return h < p || (h == p && l < 0.f);
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
// FULL: all are below v1.
template <bool FULL>
SSD_DI void get_entries(const Rest& rest, int v0, int step, int v1, float (&r)[kBatch], float (&e)[kBatch]) {
  const float *p = rest.p + v0, *q = rest.q + v0;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) r[k] = FULL || v0 + k * step < v1 ? p[k * step] : 0.f;
  if (rest.q) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) e[k] = FULL || v0 + k * step < v1 ? q[k * step] : 0.f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) rest_of(r[k], e[k], r[k], e[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      r[k] = r[k] > 0.f && v0 + k * step != rest.out ? r[k] : 0.f;  // (NaN too)
      e[k] = 0.f;
    }
  }
}
SSD_DI void get_batch(const Rest& rest, int v0, int step, int end, int v1, float (&r)[kBatch], float (&e)[kBatch]) {
  if (end <= v1) get_entries<true>(rest, v0, step, v1, r, e);
  else get_entries<false>(rest, v0, step, v1, r, e);
}

// A warp's sum of the entries w0 .. w1 - 1.  The errors of a batch add up in fp32 (2^-42 of
// the batch's sum), the batches in a pair of fp32 (2^-46 of the sum each).  One error for all
// of a lane's entries would be off by the square of their number; the pair's sums in 64
// bits took 16 x 32000 entries from 9 to 15 us, pairs of pairs from 9.0 to 9.5.
static __device__ __noinline__ float2 sum_run(const Rest& rest, int w0, int w1) {
  const int lane = threadIdx.x & 31;
  float s = 0.f, c = 0.f, t;
#pragma unroll 1
  for (int v = w0; v < w1; v += 32 * kBatch) {
    float r[kBatch], e[kBatch];
    get_batch(rest, v + lane, 32, v + 32 * kBatch, w1, r, e);
    float bs = r[0], bc = e[0];
#pragma unroll
    for (int k = 1; k < kBatch; ++k) {
      two_sum(bs, r[k], bs, t);
      bc += t + e[k];
    }
    two_sum(s, bs, s, t);
    two_sum(s, c + (t + bc), s, c);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    two_sum(s, __shfl_xor_sync(~0u, s, d), s, t);
    c += __shfl_xor_sync(~0u, c, d) + t;
  }
  return make_float2(s, c);
}

// A cluster per sequence, a slice of the vocabulary per CTA and a run of it per
// warp.  Each CTA tests the drafts by itself; the sums meet once.  Then the CTA in
// whose slice the token lies searches it.
// Bound by latency: the drafts, their probabilities, the row's entries, the
// cluster's exchange and the search one behind the other.  48 sequences x 128003
// entries: 49 MB in 20 us, 2.5 TB/s (7.3 us at a copy's rate); 16 x 32000 without q
// 8.7 us; one x 1024 6.2 us.
__global__ void __launch_bounds__(kThreads, 3) verify_drafts_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  cluster.barrier_arrive();                      // (all CTAs run before one writes to another)
  __shared__ float2 s_part[kWarps];              // sums of the warps
  __shared__ double s_warp[kWarps];              // of those up to each
  __shared__ double s_before, s_total;           // of the CTAs below, of all
  __shared__ int s_owner;
  __shared__ int s_pick;                         // of the search (late warps may still read the owner)
  __shared__ double s_low;
  __shared__ double s_cta[2][kMaxCluster];       // each CTA's sum, from the CTAs themselves
  const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / size;
  pdl_wait();
  pdl_trigger();
  const int count = a.counts ? min(max(a.counts[b], 0), a.d) : a.d;
  const float sample = fmaxf(a.sample_u[b], 0.f);  // (NaN too: with it no sum would pass)
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
        good = less(u, q, p);
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
  double total;
  int owner, turn = 0;
  while (true) {
    const float2 own = sum_run(rest, w0, w1);
    if (lane == 0) s_part[warp] = own;
    __syncthreads();
    if (turn == 0) cluster.barrier_wait();
    if (warp == 0) {
      const float2 part = lane < kWarps ? s_part[lane] : make_float2(0.f, 0.f);
      const double up = scan((double)part.x + (double)part.y, kWarps);
      if (lane < kWarps) s_warp[lane] = up;
      const double mine = __shfl_sync(~0u, up, kWarps - 1);
      if (lane < size) *cluster.map_shared_rank(&s_cta[turn][rank], lane) = mine;
    }
    cluster.sync();
    if (warp == 0) {
      // the first CTA whose sums pass the target, or the last that has any
      const double x = lane < size ? s_cta[turn][lane] : 0.0, sums = scan(x, kMaxCluster);
      const double all = __shfl_sync(~0u, sums, size - 1);
      const unsigned any = __ballot_sync(~0u, x > 0.0), past = __ballot_sync(~0u, lane < size && sums > (double)sample * all);
      const double below = __shfl_sync(~0u, sums, rank ? rank - 1 : 0);
      if (lane == 0) {
        s_before = rank ? below : 0.0;
        s_total = all;
        s_owner = !(all <= (double)FLT_MAX) ? -1 : past ? __ffs(past) - 1 : any ? 31 - __clz(any) : -1;
      }
    }
    __syncthreads();
    total = s_total;
    owner = s_owner;
    if (plain || total > 0.0) break;
    plain = true;                                // nothing is left: from p itself
    rest.q = nullptr;
    rest.out = -1;
    turn = 1;
    __syncthreads();
  }
  int32_t* tokens = a.tokens + (size_t)b * (a.d + 1);
  if (rank == 0 && warp == 1) {
    for (int j = lane; j <= a.d; j += 32)
      if (j != taken) tokens[j] = j < taken ? a.drafts[(size_t)b * a.d + j] : -1;
    if (lane == 0) {
      a.n[b] = taken + (owner >= 0 ? 1 : 0);
      if (owner < 0) tokens[taken] = -1;         // no probability anywhere
    }
  }
  if (rank != owner) return;
  // the warp's run in which the sum passes the target, a 16th of that, and so on,
  // all warps together; the last 128 entries by one
  const double target = (double)sample * total;
  int x0 = lo, x1 = hi;
  double below = s_before;
#pragma unroll 1
  while (true) {
    const int part = (x1 - x0 + kWarps - 1) / kWarps;
    if (warp == 0) {                             // (s_warp: the sums up to each warp's part)
      const double up = lane < kWarps ? s_warp[lane] : 0.0, lower = __shfl_up_sync(~0u, up, 1);
      const unsigned past = __ballot_sync(~0u, lane < kWarps && below + up > target);
      const unsigned any = __ballot_sync(~0u, lane < kWarps && up > (lane ? lower : 0.0));
      const int w = past ? __ffs(past) - 1 : any ? 31 - __clz(any) : 0;
      if (lane == w) {
        s_pick = w;
        s_low = below + (w ? lower : 0.0);
      }
    }
    __syncthreads();
    const int w = s_pick;
    below = s_low;
    x0 = min(x0 + w * part, x1);
    x1 = min(x0 + part, x1);
    if (x1 - x0 <= 128) break;
    const int next = (x1 - x0 + kWarps - 1) / kWarps, y0 = min(x0 + warp * next, x1);
    const float2 own = sum_run(rest, y0, min(y0 + next, x1));
    if (lane == 0) s_part[warp] = own;
    __syncthreads();
    if (warp == 0) {
      const float2 y = lane < kWarps ? s_part[lane] : make_float2(0.f, 0.f);
      const double up = scan((double)y.x + (double)y.y, kWarps);
      if (lane < kWarps) s_warp[lane] = up;
      __syncwarp();
    }
  }
  if (warp != 0) return;
  const int v0 = x0 + lane * 4;
  double at[4], sum = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float r = 0.f, e = 0.f;
    if (v0 + k < x1) {
      const float pk = rest.p[v0 + k];
      rest_of(pk, rest.q ? rest.q[v0 + k] : v0 + k == rest.out ? pk : 0.f, r, e);
    }
    at[k] = (double)r + (double)e;
    sum += at[k];
  }
  const double to = scan(sum, 32);
  double up = below + (to - sum);
  int first = -1, last = -1;                     // the lane's first past the target, its last over 0
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    up += at[k];
    if (at[k] > 0.0) {
      last = v0 + k;
      if (first < 0 && up > target) first = v0 + k;
    }
  }
  const unsigned here = __ballot_sync(~0u, first >= 0), some = __ballot_sync(~0u, last >= 0);
  const int token = here ? __shfl_sync(~0u, first, __ffs(here) - 1) : some ? __shfl_sync(~0u, last, 31 - __clz(some)) : -1;
  if (lane == 0) tokens[taken] = token;
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
  // As many CTAs to a sequence as have 2048 entries each and an SM for each, and
  // three of an SM where they have 16000 entries.  (us with 1, 2, 4, 8, 16 CTAs:
  // one sequence of 32000 entries 12.9, 10.5, 9.1, 8.5, 7.1; 16 of them 13.4, 10.9,
  // 9.6, 10.0, 10.1; 48 of them 13.6, 11.0, 11.9, 12.4, 18.2; 48 of 128003 39, 25,
  // 20, 18.7, 27; 128 of 32000 15.2, 15.3, 20, 25, 42)
  int size = 1;
  while (size < kMaxCluster && a.V > size * 2048 &&
         (a.B * size * 2 <= tree_sms() || (a.V > size * 16000 && a.B * size * 2 <= 3 * tree_sms())))
    size *= 2;
  if (size > 8) {
    static bool ready[kDeviceSlots] = {};
    const int dv = device_slot();
    if (dv < 0 || !ready[dv]) {
      const cudaError_t e = cudaFuncSetAttribute(verify_drafts_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dv >= 0) ready[dv] = true;
    }
  }
  return launch_early(verify_drafts_kernel, (unsigned)(a.B * size), kThreads, 0, s, size, a);
}

}  // namespace ssd
