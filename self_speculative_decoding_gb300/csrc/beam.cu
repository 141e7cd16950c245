// Beam selection over beams x vocabulary, and the reordering of the beams'
// caches (sm_103a).
//
// Candidate (b, v) scores score_b + (z_bv - lse_b), summed in 64 bits: the
// 32-bit terms add without rounding that could reorder them.  Within a beam
// the order is that of the logits, so each piece of a row is cut down to its
// W largest logits first; the pieces' lists are then merged by score.  Ties
// go to the lower beam, then to the lower token.
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "tree.cuh"

namespace ssd {
namespace {

constexpr int kPieceThreads = 512;
constexpr int kPieceItems = 44;
constexpr int kPieceMax = kPieceThreads * kPieceItems;  // logits per CTA at most
constexpr int kMergeThreads = 1024;
constexpr int kMaxCluster = 8;      // portable cluster size
constexpr int kList = 1024;         // candidates over the threshold that are ranked at once

// Floats as unsigned integers in the same order (-0 as +0; no NaN).
SSD_DI uint32_t float_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
SSD_DI float order_float(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// (logit, token) as one key: larger logit first, then lower token; 0 stands
// for no candidate (NaN and -infinity are none).
SSD_DI uint64_t logit_key(float z, int token) {
  if (!(z > -INFINITY)) return 0;
  return ((uint64_t)float_order(z) << 32) | (uint32_t)~token;
}
SSD_DI float key_logit(uint64_t k) { return order_float((uint32_t)(k >> 32)); }
SSD_DI int key_token(uint64_t k) { return (int)~(uint32_t)k; }

// A value that W of the block's threads reach (each with the maximum of its
// own, not NaN) and that few others do: the W-th largest to its first kBits
// bits, one vote of the block for each; -infinity where fewer than W have any.
template <int kBits>
SSD_DI float block_cut(float mine, int W) {
  const uint32_t o = float_order(mine);
  uint32_t t = 0;
#pragma unroll 1
  for (int bit = 31; bit >= 32 - kBits; --bit) {
    const uint32_t c = t | (1u << bit);
    if (__syncthreads_count(o >= c) >= W) t = c;
  }
  return t > float_order(-INFINITY) ? order_float(t) : -INFINITY;
}

// Sum of the block's values; `turn` (0, 1, 0, ...) differs from the last call's.
SSD_DI int block_sum(int x, int turn) {
  constexpr int kWarps = kPieceThreads / 32;
  __shared__ int part[2][kWarps];
  const int all = __reduce_add_sync(~0u, x);
  if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = all;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += part[turn][i];
  return sum;
}

// Piece `piece` of row b: its W largest keys to its list, largest first.  The
// logits stay in registers; what reaches the W-th largest of the threads'
// maxima is listed and ranked.
template <int kItems>
SSD_DI void piece_items(const BeamArgs& a, int len, int piece, int b, uint64_t* out,
                        uint64_t* list, int& s_n) {
  const int tid = threadIdx.x;
  if (a.done && a.done[b]) return;               // the merge does not read its lists
  const int v0 = piece * len, n = min(len, a.V - v0);
  const float* row = a.logits + (size_t)b * a.V + v0;
  float z[kItems];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int v = i * kPieceThreads + tid;
    z[i] = v < n ? __ldcs(row + v) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) mx = fmaxf(mx, z[i]);  // ignores NaN
  if (tid == 0) s_n = 0;
  const float cut = block_cut<24>(mx, a.W);
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (z[i] >= cut && z[i] > -INFINITY) {
      const int at = atomicAdd(&s_n, 1);
      if (at < kList) list[at] = logit_key(z[i], v0 + i * kPieceThreads + tid);
    }
  __syncthreads();
  int cnt = s_n;
  if (cnt > kList) {
    // many equal logits (a vocabulary masked by the type's lowest value): the
    // W-th largest exactly, by its bits, then of its equals the lowest tokens
    uint32_t t = 0;
    int turn = 0, over = 0, m = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit, turn ^= 1) {
      const float c = order_float(t | (1u << bit));
      int k = 0;
#pragma unroll
      for (int i = 0; i < kItems; ++i) k += z[i] >= c;
      if (block_sum(k, turn) >= a.W) t |= 1u << bit;
    }
    const float last = order_float(t);
#pragma unroll
    for (int i = 0; i < kItems; ++i) over += z[i] > last;
    const int need = a.W - block_sum(over, turn);
    turn ^= 1;
#pragma unroll 1
    for (int bit = 14; bit >= 0; --bit, turn ^= 1) {  // (a piece has under 2^15 logits)
      const int c = m | (1 << bit);
      int k = 0;
#pragma unroll
      for (int i = 0; i < kItems; ++i) k += z[i] == last && i * kPieceThreads + tid < c;
      if (block_sum(k, turn) < need) m = c;
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int v = i * kPieceThreads + tid;
      if (z[i] > last || (z[i] == last && v <= m)) list[atomicAdd(&s_n, 1)] = logit_key(z[i], v0 + v);
    }
    __syncthreads();
    cnt = s_n;
  }
  // keys differ, so each key's rank is its place
  // (counted by four threads together)
  for (int i = tid >> 2; i < ((cnt + 7) & ~7); i += kPieceThreads / 4) {
    const uint64_t k = i < cnt ? list[i] : 0;
    int rank = 0;
    for (int j = tid & 3; j < cnt; j += 4) rank += list[j] > k;
    rank += __shfl_xor_sync(~0u, rank, 1);
    rank += __shfl_xor_sync(~0u, rank, 2);
    if ((tid & 3) == 0 && i < cnt && rank < a.W) out[rank] = k;
  }
  for (int i = cnt + tid; i < a.W; i += kPieceThreads) out[i] = 0;
}

// A short piece has code of its own: what runs once is bound by its fetching
// (4 beams of 1024 logits 9.6 us with the long one and 8.1 when that changed,
// 8.2 in the present build).
constexpr int kFewItems = 4;
SSD_DI void piece_body(const BeamArgs& a, int len, int piece, int b, uint64_t* out,
                       uint64_t* list) {
  __shared__ int s_n;
  if (len <= kFewItems * kPieceThreads)
    piece_items<kFewItems>(a, len, piece, b, out, list, s_n);
  else
    piece_items<kPieceItems>(a, len, piece, b, out, list, s_n);
}

// CTA = (piece of a row, beam).  48 rows of 128003 logits (24.6 MB) take 11 us
// (12 alone and cold):
// the loads 6 of them (4 bytes each, since rows begin anywhere; all of a
// thread's in flight at once), then the threshold, the list and its ranks.
__global__ void __launch_bounds__(kPieceThreads, 2) beam_piece_kernel(const BeamArgs a, int len) {
  __shared__ uint64_t list[kList];
  pdl_trigger();
  piece_body(a, len, blockIdx.x, blockIdx.y,
             a.lists + ((size_t)blockIdx.y * gridDim.x + blockIdx.x) * a.W, list);
}

// A candidate in the whole order: the 64-bit score as an ordered integer
// (64-bit arithmetic runs at a 64th of the 32-bit rate: it is kept to the few
// candidates over the threshold, and comparisons are integers').
struct Cand {
  uint64_t s;
  uint64_t k;
  int b;
};
SSD_DI bool before(const Cand& x, const Cand& y) {
  if (x.s != y.s) return x.s > y.s;
  if (x.b != y.b) return x.b < y.b;
  return x.k > y.k;
}
SSD_DI uint64_t ordered(double s) {
  const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
SSD_DI double unordered(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? (o & ~(1ull << 63)) : ~o));
}

// What the scores of a beam's candidates share, in shared memory.
struct Beam {
  float score, lse;
  int ended;
};

// Entry d of list i, 0 where there is none (an ended beam has one entry, 1).
SSD_DI uint64_t entry(const BeamArgs& a, const Beam* beams, int pieces, int i, int d) {
  const int b = i / pieces;
  if (beams[b].ended) return (uint64_t)(d == 0 && i == b * pieces);
  return a.lists[(size_t)i * a.W + d];
}

// The candidate of an entry; false where its score is NaN or -infinity.
SSD_DI bool score(const Beam& m, uint64_t k, int b, Cand& c) {
  const double sc = (double)m.score;
  const double s = m.ended ? sc : sc + ((double)key_logit(k) - (double)m.lse);
  c.s = ordered(s);
  c.k = k;
  c.b = b;
  return s > -INFINITY;
}

// Bounds of that score in 32-bit arithmetic: either sum is off by half a step of
// its result, 2^-24 (twice that is taken; the bounds are rounded too).  All is
// taken by a quarter, so that no sum leaves the 32-bit range (z - lse may); what
// the last product makes an infinity lies beyond every 32-bit value.  A quarter
// is exact but for the last steps above zero (1e-44).  A sum that is infinite has
// an infinite term, and NaN is no candidate.
SSD_DI void score_bounds(const Beam& m, uint64_t k, float& lower, float& upper) {
  const float d = m.ended ? 0.f : 0.25f * key_logit(k) - 0.25f * m.lse;
  const float f = 0.25f * m.score + d;
  const float e = fmaf(fabsf(d), 1.2e-7f, fmaf(fabsf(f), 1.2e-7f, 1e-44f));
  const bool finite = fabsf(f) < INFINITY;
  lower = finite ? 4.f * (f - e) : f > 0.f ? INFINITY : -INFINITY;
  upper = finite ? 4.f * (f + e) : lower;
}

SSD_DI void put(const BeamArgs& a, const Beam* beams, int w, const Cand& c, bool got) {
  const bool ended = got && beams[c.b].ended;
  const int token = !got ? -1 : ended ? a.end_id : key_token(c.k);
  a.tokens[w] = token;
  a.parents[w] = got ? c.b : -1;
  a.scores_out[w] = got ? (float)unordered(c.s) : -INFINITY;
  if (a.done_out) a.done_out[w] = !got || token == a.end_id;
}

// One CTA: the W best of all lists, which are sorted.  The W-th largest of the
// threads' maxima over the lists' first eight entries (of lower bounds of their
// scores) is a threshold that W candidates reach; the entries of each list
// whose upper bound reaches it are collected and ranked by the whole order,
// eight threads to a candidate (48 beams of 128003 logits 16.5 us in all; when
// that changed, 18.3 after 21.2 with one thread to each).  Where a few lists hold most of the best, too many
// reach it: then every entry that does counts towards a second threshold (128
// of 128 uneven beams of 32000 logits 21 us; one maximum after the other, what
// is left for more than 1024 equal scores, took 715).
// Bound by latency, about 6 us for 288 lists: two rounds of reads of L2, the
// threshold and the ranks; holding the lists' first entries in shared memory
// was slower (22.1 against 21.2 at the time).  WAIT: the lists come from the kernel before.
template <int kThreads, bool WAIT>
SSD_DI void merge_body(const BeamArgs& a, int pieces, Cand* list) {
  __shared__ Beam beams[256];
  __shared__ uint32_t gm[kThreads];
  __shared__ int s_n;
  const int tid = threadIdx.x, lists = a.B * pieces;
  if (tid < a.B) {
    beams[tid].score = a.scores[tid];
    beams[tid].lse = a.lse ? a.lse[(size_t)tid * a.lse_stride] : 0.f;
    beams[tid].ended = a.done && a.done[tid];
  }
  gm[tid] = 0u;
  if (WAIT) pdl_wait();                          // (the beams are not the pieces' work)
  __syncthreads();
  // eight lanes go through a list together
  float mx = -INFINITY;
#pragma unroll 2
  for (int i = tid >> 3; i < lists; i += kThreads / 8) {
    const int d = tid & 7;
    const uint64_t k = d < a.W ? entry(a, beams, pieces, i, d) : 0;
    float lo, up;
    score_bounds(beams[i / pieces], k, lo, up);
    if (k) mx = fmaxf(mx, lo);
  }
  float cut = block_cut<32>(mx, a.W);
  int cnt = 0;
#pragma unroll 1
  for (int turn = 0; turn < 3; ++turn) {
    // 0 and 2: collect; 1: the second threshold
    if (tid == 0) s_n = 0;
    __syncthreads();
    for (int i = tid >> 3; i < lists; i += kThreads / 8) {
      for (int d0 = 0; d0 < a.W; d0 += 8) {
        const int d = d0 + (tid & 7);
        bool in = false;
        const uint64_t k = d < a.W ? entry(a, beams, pieces, i, d) : 0;
        if (k) {
          float lo, up;
          score_bounds(beams[i / pieces], k, lo, up);
          in = up >= cut;
          Cand c;
          if (in && turn == 1) {
            // (a multiple of W by itself would meet few places where W is even)
            const uint32_t place = ((uint32_t)i * (uint32_t)a.W + (uint32_t)d) * 2654435769u;
            atomicMax(&gm[place / (0x80000000u / (kThreads / 2))], float_order(lo));
          } else if (in && score(beams[i / pieces], k, i / pieces, c)) {
            const int at = atomicAdd(&s_n, 1);
            if (at < kList) list[at] = c;
          }
        }
        const unsigned group = 0xffu << (tid & 24);
        if (__ballot_sync(group, in) != group) break;
      }
    }
    __syncthreads();
    if (turn == 1) {
      const uint32_t o = gm[tid];
      cut = fmaxf(cut, block_cut<32>(o ? order_float(o) : -INFINITY, a.W));
      continue;
    }
    cnt = s_n;
    if (cnt <= kList) break;
    __syncthreads();                             // s_n is read
  }
  if (cnt <= kList) {
    for (int i = tid >> 3; i < ((cnt + 3) & ~3); i += kThreads / 8) {
      const Cand c = list[min(i, cnt - 1)];
      int rank = 0;
      for (int j = tid & 7; j < cnt; j += 8) rank += before(list[j], c);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) rank += __shfl_xor_sync(~0u, rank, d);
      if ((tid & 7) == 0 && i < cnt && rank < a.W) put(a, beams, rank, c, true);
    }
    for (int w = cnt + tid; w < a.W; w += kThreads) put(a, beams, w, Cand{}, false);
    return;
  }
  // many equal scores: W maxima in turn; each thread has the first candidate of
  // its lists that is left (a list of its own: entry `next`)
  const Cand none = {0, 0, 1 << 30};
  Cand own = none, last = {~0ull, ~0ull, -1};
  int next = 0;
  auto find = [&]() {
    own = none;
    for (int i = tid; i < lists; i += kThreads) {
      const int b = i / pieces;
      Cand x;
      int d = next;
      if (lists > kThreads) {                    // the first entry after the last candidate
        int top = a.W;
        d = 0;
        while (d < top) {
          const int mid = (d + top) >> 1;
          const uint64_t k = entry(a, beams, pieces, i, mid);
          if (k && score(beams[b], k, b, x) && !before(last, x))
            d = mid + 1;
          else
            top = mid;
        }
      }
      const uint64_t k = d < a.W ? entry(a, beams, pieces, i, d) : 0;
      if (k && score(beams[b], k, b, x) && before(x, own)) own = x;
    }
  };
  find();
#pragma unroll 1
  for (int w = 0; w < a.W; ++w) {
    Cand c = own;
    for (int d = 16; d; d >>= 1) {
      Cand x;
      x.s = __shfl_xor_sync(~0u, c.s, d);
      x.k = __shfl_xor_sync(~0u, c.k, d);
      x.b = __shfl_xor_sync(~0u, c.b, d);
      if (before(x, c)) c = x;
    }
    __syncthreads();
    if ((tid & 31) == 0) list[tid >> 5] = c;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i)
      if (before(list[i], c)) c = list[i];
    if (tid == 0) put(a, beams, w, c, c.k != 0);
    last = c;
    if (c.k && own.k == c.k && own.b == c.b) {
      ++next;
      find();
    }
  }
}

__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamArgs a, int pieces) {
  __shared__ Cand list[kList];
  merge_body<kMergeThreads, true>(a, pieces, list);
}

// Few pieces: one cluster holds them all, and its first CTA merges the lists
// out of the others' shared memory (one launch instead of two, no workspace).
__global__ void __launch_bounds__(kPieceThreads, 1) beam_cluster_kernel(const BeamArgs a, int len) {
  constexpr int kMost = 256;                     // W at most
  __shared__ uint64_t mine[kMost];
  __shared__ uint64_t all[kMaxCluster * kMost];
  __shared__ Cand list[kList];                   // and the piece's keys before
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  piece_body(a, len, blockIdx.x, blockIdx.y, mine, reinterpret_cast<uint64_t*>(list));
  cluster.sync();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < (int)cluster.num_blocks() * a.W; i += kPieceThreads)
      all[i] = cluster.map_shared_rank(mine, i / a.W)[i % a.W];
  cluster.sync();                                // no list is gone while it is read
  if (blockIdx.x || blockIdx.y) return;
  BeamArgs b = a;
  b.lists = all;
  merge_body<kPieceThreads, false>(b, gridDim.x, list);
}

// Reordering by source: a tile of 1024 16-byte units of one group's rows is
// read once and written to every state that takes it (read once per taker, 8
// beams of 32 layers at 1025 rows took 319 us; the copies of a source lie too
// far apart for L2).
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 4;       // per thread, of K and of V
__global__ void __launch_bounds__(kCopyThreads) beam_reorder_kernel(const ReorderArgs a) {
  const size_t span = (size_t)(a.stop - a.start) * a.units;  // units per group
  const size_t per = (span + kCopyThreads * kCopyUnits - 1) / (kCopyThreads * kCopyUnits);
  const size_t tiles = (size_t)a.B * a.groups * per, len = (size_t)a.max_seq * a.units;
  for (size_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const size_t grp = i / per;                  // (source state, group)
    const int p = (int)(grp / a.groups);
    const size_t u0 = (i - grp * per) * (kCopyThreads * kCopyUnits) + threadIdx.x;
    const size_t src = grp * len + (size_t)a.start * a.units + u0;
    uint4 x[kCopyUnits], y[kCopyUnits];
    bool read = false;
    for (int w = 0; w < a.W; ++w) {
      if (__ldg(a.parents + w) != p) continue;
      if (!read) {
        read = true;
#pragma unroll
        for (int q = 0; q < kCopyUnits; ++q) {
          if (u0 + q * kCopyThreads >= span) continue;
          x[q] = __ldcs(a.k + src + q * kCopyThreads);
          if (a.v) y[q] = __ldcs(a.v + src + q * kCopyThreads);
        }
      }
      const size_t dst = src + ((size_t)w - (size_t)p) * a.groups * len;
#pragma unroll
      for (int q = 0; q < kCopyUnits; ++q) {
        if (u0 + q * kCopyThreads >= span) continue;
        __stcs(a.k_out + dst + q * kCopyThreads, x[q]);
        if (a.v) __stcs(a.v_out + dst + q * kCopyThreads, y[q]);
      }
    }
  }
}

}  // namespace

// Pieces per row, and their length: as few as hold a row in registers, and
// more while they leave SMs idle and a piece is over 2048 logits.
static int beam_pieces(int B, int V, int& len) {
  int p = V / kPieceMax + (V % kPieceMax != 0);
  while ((long long)B * p < tree_sms() && V / (2 * p) >= 2048) p *= 2;
  len = V / p + (V % p != 0);
  return p;
}

size_t beam_select_workspace(int B, int V, int W) {
  int len;
  const size_t lists = (size_t)B * beam_pieces(B, V, len);
  return lists <= kMaxCluster ? 0 : lists * W * sizeof(uint64_t);
}

cudaError_t launch_beam_select(const BeamArgs& a, cudaStream_t s) {
  int len;
  const int pieces = beam_pieces(a.B, a.V, len);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(pieces, a.B);
  lc.blockDim = dim3(kPieceThreads);
  lc.stream = s;
  lc.attrs = attr;
  if (pieces * a.B <= kMaxCluster) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = pieces;
    attr[0].val.clusterDim.y = a.B;
    attr[0].val.clusterDim.z = 1;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, beam_cluster_kernel, a, len);
  }
  cudaError_t e = cudaLaunchKernelEx(&lc, beam_piece_kernel, a, len);
  if (e != cudaSuccess) return e;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.gridDim = dim3(1);
  lc.blockDim = dim3(kMergeThreads);
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, beam_merge_kernel, a, pieces);
}

cudaError_t launch_beam_reorder(const ReorderArgs& a, cudaStream_t s) {
  const size_t span = (size_t)(a.stop - a.start) * a.units;
  const size_t tiles = (size_t)a.B * a.groups * ((span + kCopyThreads * kCopyUnits - 1) /
                                                 (kCopyThreads * kCopyUnits));
  beam_reorder_kernel<<<(unsigned)(tiles < (1u << 20) ? tiles : 1u << 20), kCopyThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssd
