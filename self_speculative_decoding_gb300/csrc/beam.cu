// Beam selection over beams x vocabulary, and the reordering of the beams'
// caches (sm_103a).
//
// Candidate (b, v) scores score_b + (z_bv - lse_b), summed in 64 bits: the
// 32-bit terms add without rounding that could reorder them.  Within a beam
// the order is that of the logits, so each piece of a row is cut down to its
// W largest logits first; the pieces' lists are then merged by score.  Ties
// go to the lower beam, then to the lower token.
#include "kernels.cuh"

namespace ssd {
namespace {

constexpr int kPieceThreads = 256;
constexpr int kPieceItems = 16;
constexpr int kPiece = kPieceThreads * kPieceItems;  // logits per CTA
constexpr int kMergeThreads = 1024;

// (logit, token) as one key: larger logit first, then lower token; 0 stands
// for no candidate (NaN and -infinity are none).
SSD_DI uint64_t logit_key(float z, int token) {
  if (!(z > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(z + 0.f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)o << 32) | (uint32_t)~token;
}
SSD_DI float key_logit(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
SSD_DI int key_token(uint64_t k) { return (int)~(uint32_t)k; }

// CTA = (piece of a row, beam): the piece's W largest keys, by W maxima.
__global__ void __launch_bounds__(kPieceThreads) beam_piece_kernel(const BeamArgs a) {
  __shared__ uint64_t best[kPieceThreads / 32];
  const int b = blockIdx.y, tid = threadIdx.x;
  uint64_t* list = a.lists + ((size_t)b * gridDim.x + blockIdx.x) * a.W;
  if (a.done && a.done[b]) {
    for (int i = tid; i < a.W; i += kPieceThreads) list[i] = 0;
    return;
  }
  uint64_t key[kPieceItems];
  const float* z = a.logits + (size_t)b * a.V;
#pragma unroll
  for (int i = 0; i < kPieceItems; ++i) {
    const int v = blockIdx.x * kPiece + i * kPieceThreads + tid;
    key[i] = v < a.V ? logit_key(z[v], v) : 0;
  }
  for (int w = 0; w < a.W; ++w) {
    uint64_t m = 0;
#pragma unroll
    for (int i = 0; i < kPieceItems; ++i) m = max(m, key[i]);
    for (int d = 16; d; d >>= 1) m = max(m, __shfl_xor_sync(~0u, m, d));
    if ((tid & 31) == 0) best[tid >> 5] = m;
    __syncthreads();
    for (int i = 0; i < kPieceThreads / 32; ++i) m = max(m, best[i]);
    __syncthreads();
    if (tid == 0) list[w] = m;
#pragma unroll
    for (int i = 0; i < kPieceItems; ++i)
      if (key[i] == m) key[i] = 0;
  }
}

struct Cand {
  double s;
  uint64_t k;
  int b;
};
SSD_DI bool before(const Cand& x, const Cand& y) {
  if (x.s != y.s) return x.s > y.s;
  if (x.b != y.b) return x.b < y.b;
  return x.k > y.k;
}

// One CTA: W maxima over all lists.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamArgs a, int pieces) {
  __shared__ double bs[kMergeThreads / 32];
  __shared__ uint64_t bk[kMergeThreads / 32];
  __shared__ int bb[kMergeThreads / 32];
  const int tid = threadIdx.x, per = pieces * a.W, n = a.B * per;
  const Cand none = {-INFINITY, 0, 1 << 30};
  Cand last = {INFINITY, ~0ull, -1};  // the candidate taken before
  for (int w = 0; w < a.W; ++w) {
    Cand c = none;
    for (int i = tid; i < n; i += kMergeThreads) {
      const int b = i / per;
      const bool ended = a.done && a.done[b];
      const uint64_t k = ended ? (i == b * per ? (uint64_t)1 : 0) : a.lists[i];
      if (!k) continue;
      Cand x;
      x.s = ended ? (double)a.scores[b]
                  : (double)a.scores[b] +
                        ((double)key_logit(k) - (a.lse ? (double)a.lse[(size_t)b * a.lse_stride] : 0.0));
      x.k = k;
      x.b = b;
      if (x.s > -INFINITY && before(last, x) && before(x, c)) c = x;
    }
    for (int d = 16; d; d >>= 1) {
      Cand x;
      x.s = __shfl_xor_sync(~0u, c.s, d);
      x.k = __shfl_xor_sync(~0u, c.k, d);
      x.b = __shfl_xor_sync(~0u, c.b, d);
      if (before(x, c)) c = x;
    }
    if ((tid & 31) == 0) {
      bs[tid >> 5] = c.s;
      bk[tid >> 5] = c.k;
      bb[tid >> 5] = c.b;
    }
    __syncthreads();
    for (int i = 0; i < kMergeThreads / 32; ++i) {
      const Cand x = {bs[i], bk[i], bb[i]};
      if (before(x, c)) c = x;
    }
    __syncthreads();
    if (tid == 0) {
      const bool got = c.k != 0;
      const bool ended = got && a.done && a.done[c.b];
      const int token = !got ? -1 : ended ? a.end_id : key_token(c.k);
      a.tokens[w] = token;
      a.parents[w] = got ? c.b : -1;
      a.scores_out[w] = got ? (float)c.s : -INFINITY;
      if (a.done_out) a.done_out[w] = !got || token == a.end_id;
    }
    last = c;
  }
}

// Units of 16 bytes of the rows start .. stop-1 of every group of every state.
__global__ void __launch_bounds__(256) beam_reorder_kernel(const ReorderArgs a) {
  const size_t span = (size_t)(a.stop - a.start) * a.units;  // units per group
  const size_t n = (size_t)a.W * a.groups * span;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (size_t)gridDim.x * blockDim.x) {
    const size_t grp = i / span, u = i - grp * span;
    const int w = (int)(grp / a.groups), p = a.parents[w];
    if (p < 0 || p >= a.B) continue;
    const size_t at = (size_t)a.start * a.units + u, len = (size_t)a.max_seq * a.units;
    const size_t src = ((size_t)p * a.groups + grp % a.groups) * len + at, dst = grp * len + at;
    a.k_out[dst] = a.k[src];
    if (a.v) a.v_out[dst] = a.v[src];
  }
}

}  // namespace

size_t beam_select_workspace(int B, int V, int W) {
  return (size_t)B * ((V + kPiece - 1) / kPiece) * W * sizeof(uint64_t);
}

cudaError_t launch_beam_select(const BeamArgs& a, cudaStream_t s) {
  const int pieces = (a.V + kPiece - 1) / kPiece;
  beam_piece_kernel<<<dim3(pieces, a.B), kPieceThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  beam_merge_kernel<<<1, kMergeThreads, 0, s>>>(a, pieces);
  return cudaGetLastError();
}

cudaError_t launch_beam_reorder(const ReorderArgs& a, cudaStream_t s) {
  beam_reorder_kernel<<<1216, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssd
