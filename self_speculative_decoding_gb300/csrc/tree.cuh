// Attention of a tree of drafted tokens over a cache: arguments, the layout
// of the caller's workspace and the launches (tree.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace ssd {

constexpr int kTreeMaxNodes = 1024;  // nodes (rows) of one tree
constexpr int kTreeKeys = 128;       // keys per block
constexpr int kTreeMaxHalf = 64;     // dh / 2 at most
// Up to so many rows per K/V head, the weights are summed from scores that the
// attention stores (4 bytes per row and key, against a second read of K and a
// second pass of products).  Both grow with the context and the heads, so that
// the rows alone decide: us of a call so | by a second pass, for 8, 16, 32 and
// 64 rows per head, 128 elements each,
//    8 heads,   4000 keys   14 | 18,   16 | 18,   20 | 18,   28 | 19
//    8 heads, 131072 keys  115 | 138, 132 | 138, 168 | 131, 257 | 135
//   40 heads,  32768 keys  141 | 168, 162 | 168, 210 | 165, 307 | 171
// and of 64 elements 4 heads, 131072 keys 53 | 59, 65 | 59, 89 | 54, 140 | 57.
constexpr int kTreeScoreRows = 16;

struct TreeArgs {
  const float* qkv = nullptr;        // [T][(H + 2 Hkv) dh] raw projections
  const int32_t* parents = nullptr;  // [T]
  int T = 0, n = 0, pos0 = 0, H = 0, Hkv = 0, G = 0, dh = 0, max_seq = 0;
  bf16* kc = nullptr;                // [Hkv][max_seq][dh]
  bf16* vc = nullptr;
  const float* w_in = nullptr;       // [Hkv][max_seq], nullable
  float* w_out = nullptr;            // nullable: no weights
  bf16* out = nullptr;               // [T][H dh]
  float scale_log2 = 0.f;            // log2(e) / sqrt(dh)
  // workspace
  uint32_t* anc = nullptr;           // [T][anc_words] ancestors-and-self bits
  int32_t* depth = nullptr;          // [T] ancestors above the node, -1 absent
  uint8_t* vbad = nullptr;           // [Hkv][T rounded up to 4] the node's V row holds inf or NaN
  bf16* q = nullptr;                 // [2][Hkv][T G][dh]: the rotated query's high and low part
  bf16* kt = nullptr;                // [Hkv][T][dh] the tree's K rows
  bf16* vt = nullptr;                // [Hkv][T][dh] its V rows, inf and NaN as 0
  float* lse = nullptr;              // [Hkv][T G] base-2 log-sum-exp of a row's scores
  float* part_o = nullptr;           // [slots][dh / 4][128 rows][4] unnormalised outputs
  float* part_m = nullptr;           // [slots][128] base-2 maximum of the row's scores
  float* part_l = nullptr;           // [slots][128] sum of 2^(score - maximum)
  float* part_s = nullptr;           // [Hkv][nb][rows][128] masked scores (few rows with weights)
  int* err = nullptr;                // non-zero: a bounded wait gave up
  int anc_words = 0;
  int row_kt = 0, row_vt = 0;        // first row of kt and vt in the workspace's matrix
  // the rows in tiles of 128, the keys in blocks of 128 (the context's, then
  // the tree's); a unit = (head, split, item): a run of key blocks for one tile
  // (two = 0: blocks in turn to two streams) or a pair of tiles (two = 1: one
  // stream each); with one split a unit's result is final
  int tiles = 0, two = 0, items = 0, nb_ctx = 0, nb = 0, splits = 0, units = 0, ctas = 0;
  double inv_freq[kTreeMaxHalf];     // theta^(-2 i / dh) / pi
  // self-test: this CTA of the attention acts as after a wait that gave up, this
  // CTA's waits of the weights' kernel give up at once (-1: none)
  int give_up = -1, give_up_weights = -1;
};

SSD_HD int tree_anc_words(int T) { return 4 * ((T + kTreeKeys - 1) / kTreeKeys); }

SSD_HD size_t tree_vbad_stride(int T) { return ((size_t)T + 3) & ~(size_t)3; }

// Sets the work split and the workspace pointers of `a` (sizes already set)
// from base and returns the bytes used; with base NULL only the size.
size_t tree_workspace(TreeArgs& a, void* base);
cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s);
void tree_split(TreeArgs& a);        // tree_attn_tc.cu
int tree_slots(const TreeArgs& a);
int tree_sms();                      // SMs of the current device
// Tensor maps of 128-row boxes: the caches ([Hkv][max_seq][dh], rows < n of
// each head seen, the others read as zero), and the workspace's rows (the two
// planes of q, kt and vt one behind the other, seen as one matrix: a box that
// runs over the end of a head reads rows of what follows, all finite, whose
// results nothing takes).
struct TreeMaps {
  CUtensorMap k, v, ws;
};
cudaError_t launch_tree_attn_tc(const TreeArgs& a, const TreeMaps& m, cudaStream_t s);
cudaError_t launch_tree_weight_tc(const TreeArgs& a, const TreeMaps& m, cudaStream_t s);

// ---- device helpers of the two tensor-core kernels

// A ring's slot and the parity of its use.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  SSD_DI Ring next() const {
    Ring r = *this;
    if (++r.slot == N) {
      r.slot = 0;
      r.phase ^= 1u;
    }
    return r;
  }
};

// The warp's number as a value that the compiler knows to be the same in all
// lanes: branches on it keep the warp together.
SSD_DI int tree_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

SSD_DI bool tree_flagged(const int* f) { return *reinterpret_cast<const volatile int*>(f) != 0; }

SSD_DI bool tree_try(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Bounded wait for one or two barriers at once (b NULL: one); false if it ran
// out or the CTA is flagged.
SSD_DI bool tree_wait(const int* fail, int polls, uint64_t* a, uint32_t pa, uint64_t* b = nullptr,
                      uint32_t pb = 0) {
  bool da = false, db = b == nullptr;
  for (int i = 0; i < polls; ++i) {
    if (!da) da = tree_try(a, pa);
    if (!db) db = tree_try(b, pb);
    if (da && db) return true;
    if ((i & 63) == 63 && tree_flagged(fail)) return false;
  }
  return false;
}

// 2^x on the special-function unit (relative error about 2^-22).
SSD_DI float tree_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of fp32 values in one instruction, and the maximum of three.
SSD_DI uint64_t tree_pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
SSD_DI void tree_unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
SSD_DI uint64_t tree_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SSD_DI uint64_t tree_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SSD_DI float tree_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The matrix instructions are issued by one elected lane of a warp that runs
// its loop together (in one lane's own branch an instruction took 95 cycles to
// issue, of the 64 that it runs).  The matrix pipe holds hardly more than the
// instruction that runs, so what the warp does between two groups is time
// lost: about 95 cycles a wait, 42 a commit, 90 a look at the failure flag.
// Hence the flag is looked at only while a wait lasts, and the weights' kernel
// waits for two barriers at once (in the attention, whose streams take turns,
// that was slower: 954 against 850 us for 256 nodes over 131000 rows).  A warp
// for each stream was no way out (1145 against 885 us): the streams' products
// then interleave, and both wait for their softmax at the same time.
SSD_DI uint32_t tree_elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// D += A B, both operands in shared memory / A in tensor memory.
SSD_DI void tree_mma_ss(uint32_t lead, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
SSD_DI void tree_mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
SSD_DI void tree_commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar)),
      "r"(lead)
      : "memory");
}

}  // namespace ssd
