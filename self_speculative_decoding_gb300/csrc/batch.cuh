// Calls of many sequences at once: the norms and rotation of new tokens with
// their append, the move of cache rows to 8 bits, attention over the cache
// that results, and the verification of drafts.  Arguments and launches.
//
// A layer's caches of B sequences: row p of sequence b lies at row p % rows of
// k, v (bf16 [B][Hkv][rows][dh]: all rows, or a ring of the newest), and, once it
// has been moved, also at row p of k8, v8 (e4m3 [B][Hkv][max_seq][dh], with a
// scale for each block of rows and head).  What differs between sequences
// (lengths, counts) is read from device memory, so that a captured graph serves
// every round.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace ssd {

constexpr int kBatchMaxSeqs = 512;

struct RopeAppendArgs {
  const float* qkv = nullptr;          // [B][T][(H + 2 Hkv) dh] raw projections
  const int32_t* lengths = nullptr;    // [B] rows before the call
  const int32_t* counts = nullptr;     // [B] tokens of the call, nullable: T
  const int32_t* positions = nullptr;  // [B] position of the first token, nullable: lengths
  const float* q_gain = nullptr;       // [dh] nullable: q as it is
  const float* k_gain = nullptr;
  float eps = 0.f;
  int B = 0, T = 0, H = 0, Hkv = 0, dh = 0;
  int rows = 0;
  size_t seq_stride = 0;               // elements between two sequences of k and of v
  bf16* k = nullptr;
  bf16* v = nullptr;
  bf16* q = nullptr;                   // [B][T][H][dh]
  uint64_t turns[64];                  // theta^(-2 i / dh) / (2 pi) in 2^-64 of a turn
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s);

struct QuantizeArgs {
  const bf16* k = nullptr;
  const bf16* v = nullptr;
  const int32_t* held = nullptr;       // [B] rows in 8 bits before the call
  const int32_t* lengths = nullptr;    // [B] rows that may be moved
  int B = 0, Hkv = 0, dh = 0, rows = 0, block = 0, max_seq = 0;
  size_t seq_stride = 0, seq8_stride = 0, scale_stride = 0;
  uint8_t* k8 = nullptr;
  uint8_t* v8 = nullptr;
  float* k_scale = nullptr;            // [B][Hkv][max_seq / block]
  float* v_scale = nullptr;
  int32_t* held_out = nullptr;
};
cudaError_t launch_cache_quantize(const QuantizeArgs& a, cudaStream_t s);

struct CacheAttnArgs {
  const bf16* q = nullptr;             // [B][T][H][dh]
  const int32_t* lengths = nullptr;
  const int32_t* counts = nullptr;     // nullable
  const int32_t* held = nullptr;       // nullable: no row in 8 bits
  const bf16* k = nullptr;
  const bf16* v = nullptr;
  const uint8_t* k8 = nullptr;
  const uint8_t* v8 = nullptr;
  const float* k_scale = nullptr;
  const float* v_scale = nullptr;
  int B = 0, T = 0, H = 0, Hkv = 0, G = 0, dh = 0, rows = 0, max_seq = 0, block = 32;
  int window = 0, sinks = 0;           // window 0: all rows
  size_t seq_stride = 0, seq8_stride = 0, scale_stride = 0;
  float scale_log2 = 0.f;              // |scale| of the scores times log2(e)
  bool negate = false;                 // the scale is below 0: q with the other sign
  bf16* out = nullptr;                 // [B][T][H][dh]
  // workspace: partial results of the pairs (sequence, K/V head) that several
  // CTAs share, two places for each CTA
  int ctas = 0;
  float* part_o = nullptr;             // [2 ctas][T G][dh] unnormalised outputs
  float* part_m = nullptr;             // [2 ctas][T G] base-2 maximum of the row's scores
  float* part_l = nullptr;             // [2 ctas][T G] sum of 2^(score - maximum)
  int4* shared = nullptr;              // [ctas] (sequence, head, last CTA, -) of the pair that goes on
                                       // behind the CTA's last tile; sequence -1: none
  int give_up = -1;                    // self-test: this CTA acts as after a wait that gave up
};
size_t cache_attn_workspace(CacheAttnArgs& a, void* base);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s);

struct VerifyArgs {
  const float* p = nullptr;            // [B][d + 1][V]
  const float* q = nullptr;            // [B][d][V], nullable: the drafts were certain
  const int32_t* drafts = nullptr;     // [B][d]
  const int32_t* counts = nullptr;     // nullable: d
  const float* accept_u = nullptr;     // [B][d]
  const float* sample_u = nullptr;     // [B]
  int B = 0, d = 0, V = 0;
  int32_t* tokens = nullptr;           // [B][d + 1]
  int32_t* n = nullptr;                // [B]
};
cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s);

// A launch whose CTAs may start while the kernel before ends; the kernel waits for
// that one (pdl_wait) before it touches memory, and lets the next start likewise.
template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                                A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&lc, kernel, static_cast<A&&>(args)...);
}

// Tokens of sequence b in a call (none where its numbers make no sense).
SSD_DI int batch_count(const int32_t* counts, const int32_t* lengths, int b, int T) {
  const int n = lengths[b];
  const int c = counts ? min(max(counts[b], 0), T) : T;
  return n < 0 || n > INT32_MAX - T ? 0 : c;
}

// What an attention call reads of a sequence: rows [0, sinks) and [low, end),
// of which those below `held` are in 8 bits.  count < 0: the numbers make no
// sense, or the ring no longer holds a row that is needed.
struct SeqRange {
  int length, count, held, low, sinks, end;
};
SSD_DI SeqRange seq_range(const CacheAttnArgs& a, int length, int count, int held) {
  SeqRange r = {0, 0, 0, 0, 0, 0};
  if (length < 0 || length > INT32_MAX - a.T - 256 || count < 0 || count > a.T || held < 0 ||
      held > a.max_seq || held > length + count) {
    r.count = -1;
    return r;
  }
  if (count == 0) return r;
  r.length = length;
  r.count = count;
  r.held = held;
  r.end = length + count;
  r.low = a.window ? max(0, length + 1 - a.window) : 0;
  r.sinks = min(a.sinks, r.low);
  if (r.sinks == r.low) r.sinks = r.low = 0;     // one run of rows
  // rows from `held` on come from the ring, which has the newest only (and whose end
  // no tile of 128 may cross)
  const int first = r.sinks > held ? held : max(r.low, held);
  if (r.end - first > a.rows || (a.rows % 128 && r.end > a.rows && r.end > first)) {
    r = SeqRange{0, -1, 0, 0, 0, 0};
  }
  return r;
}

}  // namespace ssd
