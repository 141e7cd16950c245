// Attention of a few tokens per sequence over rows held in 8 bits and in bf16,
// on the 5th-generation tensor cores (sm_103a).
//
// The R = T G query rows of a sequence and K/V head (G query heads share it), 128
// at most, are the narrow side of every product, tiles of 128 cache rows the wide
// one (tensor memory lanes), so that the matrix pipe's work goes by R:
//
//   S = K q^T               8-bit rows: q = (q0 + q1) 2^-a with two e4m3 parts, which
//                           hold every bit of a bf16 number, so that the products
//                           with the stored bytes are exact; bf16 rows: q itself
//   P = 2^(S c - m) v_scale one thread per key, 16 bits, to shared memory
//   O += V^T P              8-bit rows: V widened to fp16, P in fp16; bf16 rows: both bf16
//
// A thread has one key and all rows: scores up to m + 10 (a factor of 1024, which the
// sums and P carry; with a small scale so much more, which the sums do) need no look at
// other threads but one vote of four warps for 8 rows; where a score passes that, m is
// raised and O rescaled.  (With m + 8, 72 rows took 127 us instead of 120.)
//
// K and q enter the matrix instructions as they are: a tile of K costs no thread
// anything.  V cannot: P needs more than e4m3's range and bits (a first row that
// takes most of the weight leaves the others small), and both operands of a
// 16-bit product are 16 bits wide, so four warps widen V on its way.  fp16 has
// less range than P: P is held in units of 2^-7 vref 2^m, vref a power of two not
// below any value scale so far (two binades of room make it grow seldom), and m
// follows the largest of score + log2(4 scale / vref) over the row's keys: 11 bits down to
// 2^-18 of the row's largest weight (probability times scale) and steps of 2^-28 below,
// while a sequence's scales lie within 2^40 of each other and scores below 2^21; beyond
// that the steps are 2^-28 of the largest scale times the largest probability.  (m from
// the scores alone loses what lies 2^-26 below another row's scale.  It costs 8 x 2
// tokens of 40 heads 47.6 -> 48.5 us, the others under 1 %.)
//
// Work: the tiles of all sequences and heads in one line, divided evenly among
// the CTAs (one per SM); a pair of sequence and head that several CTAs share is
// joined by a second kernel in a fixed order.  The division is computed from the
// lengths on the device, so that a graph follows them.
//
// The softmax is a chain of latencies (scores out of tensor memory, a vote, the
// exponentials) and no unit's full load, so that two or three groups of four warps
// share it: 8 rows of a tile each, in turn, or with up to 8 rows every other tile (each
// with maxima and outputs of its own, joined in the end).  The matrix
// instructions' chain of waits and issues is shared by two warps likewise.
//
// Measured (graphs of calls over inputs larger than L2; bytes of the rows read at
// 6.7 TB/s would be the floor):
//   1 sequence x 1 token, 64 / 8 heads, 131000 rows       52 us   5.2 TB/s (floor 40)
//   8 x 2 tokens, 40 / 40 heads, 4095 rows, window 2048   49 us   3.6 TB/s (floor 26)
//   16 x 9 tokens, 64 / 8 heads, up to 16385 rows        120 us   2.7 TB/s (floor 48)
// One token is bound by the copies and by the CTAs that end last, many heads by the
// start and the end of each pair (a few thousand cycles in which nothing streams),
// 72 rows by the softmax: some 700 cycles for 8 rows of a tile in each of three warps of
// a scheduler, whose issue slots are taken for 57% of the time, and the matrix pipe is
// busy for 19%.
//
// The groups' warps come first, then four that widen V, one that copies K, one that
// copies V, one for the products K q^T and one for V^T P.  Every wait is
// bounded: one that gives up sets the CTA's flag, every role runs out, and the
// CTA's rows become NaN.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "batch.cuh"
#include "tc_dev.cuh"
#include "tree.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kKeys = 128;
constexpr int kWiden = 128;                      // threads that widen V
constexpr int kPolls = 1 << 22;
constexpr int kUnit = 16 * 1024;                 // 128 rows of up to 128 bytes, swizzled
constexpr int kRaise = 10;                       // P: 2^5 where m is raised, 2^15 before it is again
constexpr float kNone = -3.402823466e38f;        // the maximum of a row that has seen no key: no score is below

// A condition that seldom holds: its code lies apart from the loop's.
SSD_DI bool seldom(bool x) { return __builtin_expect(x, false); }

// Shared memory: q in e4m3 parts and in bf16, P, V in 16 bits, rings of K and V.
struct Layout {
  int rows;                                      // padded to 16
  int q16, p, wide, kring, vring, rest, bytes;   // offsets
  int p_bufs, k_units, v_units;
};
constexpr int kSmemMost = 227 * 1024 - 1024;     // (from a 1024-byte boundary)
constexpr int kPlaces = 20 * 80;                 // of up to 20 warps
constexpr int kSmall = (4 * 128 + 4 * 128) * 4 + 512 + kPlaces + 96;  // per-row values, barriers, places
__host__ __device__ inline Layout layout_of(int rows, int dh, int B) {
  Layout l;
  l.rows = (rows + 15) / 16 * 16;
  const int q8 = 2 * l.rows * dh, q16 = 2 * l.rows * dh, p = l.rows * 256, wide = dh / 64 * kUnit;
  const int plan = (16 * B + 8 + 127) / 128 * 128;
  const int fixed = (q8 + q16 + 2 * wide + kSmall + plan + 1023) / 1024 * 1024;
  l.k_units = dh / 64;                           // (a tile of bf16 rows)
  l.v_units = 1;
  l.p_bufs = 1;
  int left = kSmemMost - fixed - p - (l.k_units + l.v_units) * kUnit;
  if (left >= p + kUnit) {
    l.p_bufs = 2;
    left -= p;
  }
  for (; left >= kUnit && l.v_units < 6; left -= kUnit) {
    if (l.k_units <= l.v_units) ++l.k_units;
    else ++l.v_units;
  }
  l.q16 = q8;
  l.p = l.q16 + q16;
  l.wide = (l.p + l.p_bufs * p + 1023) / 1024 * 1024;
  l.kring = l.wide + 2 * wide;
  l.vring = l.kring + l.k_units * kUnit;
  l.rest = l.vring + l.v_units * kUnit;
  l.bytes = l.rest + kSmall + plan + 1024;
  return l;
}

SSD_DI void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
// V tile in panels of 64 columns as the MN-major A operand (with 64 columns the
// second panel is whatever follows: lanes that nobody reads).
SSD_DI uint64_t v_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kUnit >> 4) << 16;             // leading offset: next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;              // stride offset: next 8 keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;                        // 128-byte swizzle
  return d;
}
// P in panels of 16 rows as the MN-major B operand: 32 bytes per key, swizzled.
constexpr int kPanel = kKeys * 32;
SSD_DI uint64_t p_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kPanel >> 4) << 16;            // leading offset: next 16 rows
  d |= (uint64_t)(256 >> 4) << 32;               // stride offset: next 8 keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)6 << 61;                        // 32-byte swizzle
  return d;
}
// fp32 D; e4m3 (or, with bits 7 and 10, as bf16 of the 16-bit kind) A and B, K-major.
SSD_DI uint32_t idesc_e4m3(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24); }
SSD_DI void mma_ss_e4m3(uint32_t lead, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
// tree_wait, in a loop that stays one.  (A sleeping hint of 2 us costs 72 rows 6
// us of 147, a loop that polls faster 10, naps in the warps that copy or widen none.)
SSD_DI bool wait_for(const int* fail, uint64_t* a, uint32_t pa) {
  if (!seldom(!tree_try(a, pa))) return true;
#pragma unroll 1
  for (int i = 0; i < kPolls; ++i) {
    if (tree_try(a, pa)) return true;
    if (seldom((i & 63) == 63) && tree_flagged(fail)) return false;
  }
  return false;
}
// The same for two barriers, or the first alone: one latency for both where they are over.
SSD_DI bool wait_for_both(const int* fail, uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, bool two) {
  const bool da = tree_try(a, pa), db = tree_try(two ? b : a, two ? pb : pa);
  if (!seldom(!(da && db))) return true;
  return wait_for(fail, a, pa) && (!two || wait_for(fail, b, pb));
}
// The barrier of a group of four softmax warps.
SSD_DI void bar_group(int group) { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); }
// Of both groups.
SSD_DI void bar_both() { asm volatile("bar.sync 4, 256;" ::: "memory"); }
// 8 columns of the thread's tensor memory lane.
SSD_DI void tmem_ld8_nw(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
SSD_DI void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
SSD_DI void tmem_pin8(uint32_t (&r)[8]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
// 8 values of each lane joined over the warp by halving: lane l ends with value
// l / 4 in v[0].
template <class F>
SSD_DI void over_lanes(float (&v)[8], F join) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 16; w > 2; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int e = 0; e < w / 4; ++e) {
      const float got = __shfl_xor_sync(~0u, up ? v[e] : v[e + w / 4], w);
      v[e] = join(up ? v[e + w / 4] : v[e], got);
    }
  }
  v[0] = join(v[0], __shfl_xor_sync(~0u, v[0], 2));
  v[0] = join(v[0], __shfl_xor_sync(~0u, v[0], 1));
}
// Whether any thread of the group says so.
SSD_DI bool any_group(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(group + 1)
      : "memory");
  return r != 0;
}

// ---- division of the work

// What runs once per sequence or run of tiles is kept out of line (code beyond 32
// KB is fetched at 2.4 cycles an instruction, beyond 128 KB at 6), and what it
// finds lies in shared memory, a place for each warp: with a block's shared memory
// this large there is next to no L1 cache, and each value that the stack holds
// costs a trip to L2.
SSD_DI int cdiv_keys(int x) { return (x + kKeys - 1) / kKeys; }
// Tiles in 8 bits: the first rows, then the run; and in bf16 the same.
SSD_DI int tiles_eight(const SeqRange& r) {
  return cdiv_keys(min(r.sinks, r.held)) + (r.low < r.held ? cdiv_keys(r.held) - r.low / kKeys : 0);
}
SSD_DI int tiles_of(const SeqRange& r) {
  const int first = max(r.low, r.held);
  return tiles_eight(r) + (r.sinks > r.held ? cdiv_keys(r.sinks) - r.held / kKeys : 0) +
         (r.end > first ? cdiv_keys(r.end) - first / kKeys : 0);
}
// A place in a pair's tiles: rows p0 .. p0 + 127, of which [rs, re) count; all
// tokens see all of them where f0 <= p0 and p0 + 128 <= f1.
struct Walk {
  int p0, rs, re, f0, f1;
  int i, left;                                   // the tile's number, tiles to the end of its run
  bool eight;
  SSD_DI bool edge() const { return p0 < f0 || p0 + kKeys > f1; }
};

static __device__ __noinline__ void find_run(const SeqRange& r, int window, int tile, Walk& w) {
  const int first = max(r.low, r.held);
  int i = tile, start = 0, n;
  bool whole = true;                             // (first rows: all tokens see them)
  w.i = tile;
  w.eight = true;
  w.rs = 0;
  w.re = min(r.sinks, r.held);
  n = cdiv_keys(w.re);
  if (i >= n) {
    i -= n;
    whole = false;
    w.rs = r.low;
    w.re = r.held;
    start = r.low / kKeys;
    n = r.low < r.held ? cdiv_keys(r.held) - start : 0;
    if (i >= n) {
      i -= n;
      whole = true;
      w.eight = false;
      w.rs = r.held;
      w.re = r.sinks;
      start = r.held / kKeys;
      n = r.sinks > r.held ? cdiv_keys(r.sinks) - start : 0;
      if (i >= n) {
        i -= n;
        whole = false;
        w.rs = first;
        w.re = r.end;
        start = first / kKeys;
        n = cdiv_keys(r.end) - start;
      }
    }
  }
  w.p0 = (start + i) * kKeys;
  w.left = n - i;
  w.f0 = window && !whole ? max(w.rs, r.end - window) : w.rs;
  w.f1 = min(w.re, r.length + 1);
}

// What the CTA's threads know of the sequences, in shared memory.
struct Plan {
  int* first;                                    // [B + 1] tiles (of one head) before sequence b: all lie
                                                 // in the caches, so that 31 bits count them
  int *length, *held;                            // [B]
  short *some, *count;                           // [B + 1] sequences with any tiles before b; [B]
  long long begin, end;                          // the CTA's tiles
  long long total;                               // units
  int ctas;                                      // that share them
  int start;                                     // units for the start of a pair

  SSD_DI long long units(int b) const { return (long long)first[b] + start * some[b]; }  // before b, of one head
};
// The work is divided in units of a tile.  A pair's start counts as several (q, the
// first scores and the result's way out are no tile's work, and take as long as
// kStart tiles), but at most as a quarter of a CTA's tiles: with less
// to do than that the CTAs' tiles, and not their starts, differ.  (0, 3, 5, 8: 8 x 2
// tokens of 40 heads 70, 62, 59, 60 us; 16 x 9 tokens 162, 155, 154, 154)
constexpr int kStart = 5;
// (64-bit divisions cost a thousand cycles where they are cold)
SSD_DI long long cta_start(long long total, int ctas, int cta) {
  if (cta >= ctas) return total;
  if (total < 1 << 20) return (unsigned)total * (unsigned)cta / (unsigned)ctas;  // (at most 1024 CTAs)
  return total * cta / ctas;
}
// The CTA that has the last tile of a pair.
static __device__ __noinline__ int last_cta(const CacheAttnArgs& a, const Plan& p, int b, int h) {
  const long long unit = p.units(b) * a.Hkv + (h + 1) * (p.units(b + 1) - p.units(b)) - 1;
  int cta = (int)(unit * p.ctas / p.total);
  while (cta_start(p.total, p.ctas, cta + 1) <= unit) ++cta;
  return cta;
}
// Tiles before unit `at`.
static __device__ __noinline__ long long tiles_before(const CacheAttnArgs& a, const Plan& p, long long at) {
  if (at >= p.total) return (long long)p.first[a.B] * a.Hkv;
  int lo = 0, hi = a.B - 1;                      // the last b whose units begin at or before `at`
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.units(mid) * a.Hkv <= at) lo = mid;
    else hi = mid - 1;
  }
  const int n = p.first[lo + 1] - p.first[lo];
  const long long local = at - p.units(lo) * a.Hkv;
  const int w = n + p.start, h = local < 0x7fffffff ? (int)((unsigned)local / (unsigned)w) : (int)(local / w);
  return (long long)p.first[lo] * a.Hkv + (long long)h * n + max((int)(local - (long long)h * w) - p.start, 0);
}
// A run of a pair's tiles within the CTA's.
struct Segment {
  int b, h, i0, n;                               // tiles i0 .. i0 + n - 1 of the pair
  int eight;                                     // of which so many are in 8 bits (the first ones)
  bool whole, head;                              // all of them; the pair began in an earlier CTA
  SeqRange r;
};
// A warp's own copies of what it works on.
struct Place {
  Segment s;
  Walk w;
};
// The segment at tile `at`, the CTA's first.
static __device__ __noinline__ void first_segment(const CacheAttnArgs& a, const Plan& p, long long at, Place& to) {
  int lo = 0, hi = a.B - 1;                      // the last b with first[b] Hkv <= at
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if ((long long)p.first[mid] * a.Hkv <= at) lo = mid;
    else hi = mid - 1;
  }
  const int n = p.first[lo + 1] - p.first[lo];
  const long long local = at - (long long)p.first[lo] * a.Hkv, left = p.end - at;
  const int h = local < 0x7fffffff ? (int)((unsigned)local / (unsigned)n) : (int)(local / n);
  const int i0 = (int)(local - (long long)h * n), m = n - i0 < left ? n - i0 : (int)left;
  to.s.b = lo;
  to.s.h = h;
  to.s.i0 = i0;
  to.s.n = m;
  to.s.whole = m == n;
  to.s.head = i0 > 0;
  to.s.r = seq_range(a, p.length[lo], p.count[lo], p.held[lo]);
  to.s.eight = max(0, min(m, tiles_eight(to.s.r) - i0));
  find_run(to.s.r, a.window, i0, to.w);
}
// The segment behind the one that a warp has, at tile `at`: the next head or the
// next sequence with any tiles.
static __device__ __noinline__ void next_segment(const CacheAttnArgs& a, const Plan& p, long long at, Place& to) {
  __syncwarp();
  int b = to.s.b, h = to.s.h + 1;
  __syncwarp();
  if (h == a.Hkv) {
    h = 0;
    do ++b;
    while (p.first[b + 1] == p.first[b]);
    to.s.b = b;
    to.s.r = seq_range(a, p.length[b], p.count[b], p.held[b]);
  }
  const int n = p.first[b + 1] - p.first[b];
  const long long left = p.end - at;
  const int m = n < left ? n : (int)left;
  to.s.h = h;
  to.s.i0 = 0;
  to.s.n = m;
  to.s.whole = m == n;
  to.s.head = false;
  __syncwarp();
  to.s.eight = min(m, tiles_eight(to.s.r));
  find_run(to.s.r, a.window, 0, to.w);
  __syncwarp();
}

// One tile on.
SSD_DI void step(Walk& w, Place& place, int window) {
  ++w.i;
  w.p0 += kKeys;
  if (seldom(--w.left == 0)) {
    __syncwarp();
    find_run(place.s.r, window, w.i, place.w);
    __syncwarp();
    w = place.w;
  }
}

// ---- values

// The two e4m3 in the low half of x as two fp16 (exact).
SSD_DI uint32_t widen(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
SSD_DI uint4 widen(uint32_t x, uint32_t y) { return make_uint4(widen(x), widen(x >> 16), widen(y), widen(y >> 16)); }
// Two 16-bit numbers with what is not finite (all of the exponent's bits `e`
// set) as 0; `bad` if there was any.
SSD_DI uint32_t finite_only(uint32_t x, uint32_t e, bool& bad) {
  if ((x & e & 0xffffu) == (e & 0xffffu)) {
    x &= 0xffff0000u;
    bad = true;
  }
  if ((x & e & 0xffff0000u) == (e & 0xffff0000u)) {
    x &= 0xffffu;
    bad = true;
  }
  return x;
}
SSD_DI uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The smallest power of two that is not below |x| (x finite and not 0), 2^-126 at least;
// and its exponent, from 1 on (0 for 0).
SSD_DI float power_above(float x) {
  return __uint_as_float((__float_as_uint(fabsf(x)) + 0x7fffffu) & 0x7f800000u);
}
SSD_DI int exponent_above(float x) { return (int)((__float_as_uint(fabsf(x)) + 0x7fffffu) >> 23) & 0xff; }
// A row's maximum follows a value scale down to kBelow binades below vref / 4, and comes down
// by kDown in all where vref grows.  With kRaise and 31 for a sum of rows these stay in
// fp32's range.
constexpr int kBelow = 42, kDown = 42;
// kRaise for a tile: what its scores may pass a maximum by.  (log2(vref / scale) from the
// numbers' bits, to 0.09.)
SSD_DI float raise_of(bool eight, float scale, float vref) {
  const float far = (float)((int)__float_as_uint(vref) - (int)__float_as_uint(fabsf(scale)));
  return eight ? fminf(fmaf(far, 0x1p-23f, kRaise - 2), kBelow + kRaise) : kRaise;
}
constexpr float kTiny = 0x1p-24f;
constexpr float kFar = 0x1p22f;                  // from here on a maximum is the score alone: its steps are 1/2

// How a row of V goes into the products: 0 as zeros (it is outside the tile's
// run), 1 without what is not finite (0 x infinity is NaN, and some token of the
// sequence does not see it), 2 as it is.
SSD_DI int row_kind(const CacheAttnArgs& a, const SeqRange& r, const Walk& t, int j) {
  if (j < t.rs || j >= t.re) return 0;
  if (j > r.length) return 1;
  return a.window && j >= a.sinks && j <= r.end - 1 - a.window ? 1 : 2;
}
// What the products left out in column c of the segment's V rows that the token
// in row pos sees.
static __device__ __noinline__ float not_finite(const CacheAttnArgs& a, const Segment& s, int pos, int c) {
  float sum = 0.f;
  Walk t;
  for (int i = 0; i < s.n; ++i) {
    find_run(s.r, a.window, s.i0 + i, t);
    for (int j = max(t.p0, t.rs); j < min(t.p0 + kKeys, t.re); ++j) {
      if (row_kind(a, s.r, t, j) != 1 || j > pos || (a.window && j >= a.sinks && j <= pos - a.window)) continue;
      float x;
      if (t.eight) {
        const uint8_t code = a.v8[(size_t)s.b * a.seq8_stride + ((size_t)s.h * a.max_seq + j) * a.dh + c];
        x = (code & 0x7f) == 0x7f ? NAN : 0.f;
      } else {
        x = __bfloat162float(a.v[(size_t)s.b * a.seq_stride + ((size_t)s.h * a.rows + j % a.rows) * a.dh + c]);
      }
      if (!isfinite(x)) sum += x;
    }
  }
  return sum;
}
// Whether V rows j .. j + 31 of the pair, as far as they lie in [rs, re), hold zeros alone.
SSD_DI bool rows_are_zero(const CacheAttnArgs& a, const Segment& s, int j, int rs, int re) {
  j += threadIdx.x & 31;
  uint32_t any = 0;
  if (j >= rs && j < re) {
    const uint4* row = reinterpret_cast<const uint4*>(a.v8 + (size_t)s.b * a.seq8_stride + ((size_t)s.h * a.max_seq + j) * a.dh);
#pragma unroll 1
    for (int i = 0; !any && i < a.dh / 16; ++i) any |= (row[i].x | row[i].y | row[i].z | row[i].w) & 0x7f7f7f7fu;
  }
  return !__any_sync(~0u, any);
}
// The CTA's rows as NaN: a wait gave up, and none is sure.
static __device__ __noinline__ void mark_rows(const CacheAttnArgs& a, const Plan& plan, Place& place) {
  const int rows = a.T * a.G;
  __syncthreads();
  if (plan.begin < plan.end) first_segment(a, plan, plan.begin, place);
  for (long long at = plan.begin; at < plan.end;) {
    __syncwarp();
    const Segment& s = place.s;
    const size_t slot = (size_t)blockIdx.x * 2 + (s.head ? 0 : 1);
    if (!s.whole && !s.head && threadIdx.x == 0)
      a.shared[blockIdx.x] = make_int4(s.b, s.h, last_cta(a, plan, s.b, s.h), 0);
    for (int i = threadIdx.x; i < rows * a.dh; i += blockDim.x) {
      const int r = i / a.dh, tk = r / a.G;
      if (s.whole) {
        if (tk < s.r.count)
          a.out[(((size_t)s.b * a.T + tk) * a.H + s.h * a.G + r % a.G) * a.dh + i % a.dh] = __float2bfloat16(NAN);
      } else if (i % a.dh == 0) {
        a.part_m[slot * rows + r] = 0.f;
        a.part_l[slot * rows + r] = tk < s.r.count ? NAN : 0.f;
      }
    }
    at += s.n;
    if (at < plan.end) next_segment(a, plan, at, place);
  }
}

// SMALL: up to 16 rows, whose parts of q make one product (twice as wide) and
// whose state the groups keep in registers.  (16 sequences of 8192 rows, 8 and 16
// query rows a pair: 54.8 and 59.2 us, with the kernel for more rows 58.8 and 63.9)
// TURNS: up to 8 rows, the groups take the tiles in turn.  (the same with 8 rows 52.7
// us, one sequence of 131000 rows 52.3 -> 51.2; four of 300 rows 10.3 -> 10.7, which
// the lengths on the device decide and the launch cannot know)
// More rows: three groups, or two where that leaves none with more than two chunks
// (25 to 32 rows).  (16 sequences of 8192 rows, 24, 32 and 40 query rows: three groups
// 68.7, 81.3 and 85.0 us, two 73.7, 77.9 and 89.2; 72 rows: three 134, two 149, four, of 80
// registers a thread, 155; all before the loop for plain 8-bit tiles, below)
constexpr int threads_of(int groups) { return (4 * groups + 8) * 32; }
template <int DH, int kGroups, bool SMALL, bool TURNS>
__global__ void __launch_bounds__(threads_of(kGroups), 1)
    cache_attn_tc_kernel(const __grid_constant__ CUtensorMap mK8, const __grid_constant__ CUtensorMap mV8,
                         const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                         const __grid_constant__ CacheAttnArgs a, const Layout lay) {
  constexpr int kThreads = threads_of(kGroups);
  constexpr int kWidenWarp = 4 * kGroups, kCopyWarp = kWidenWarp + 4, kMmaWarp = kCopyWarp + 2;
  constexpr int P = DH / 64;                     // 16-bit panels of 64 columns
  constexpr int kWide = P * kUnit;               // a V tile in 16 bits
  const int NP = SMALL ? 16 : lay.rows;
  const uint32_t scols = SMALL ? 32 : NP;        // TMEM: S0, S1, O, sums
  const uint32_t col_o = 2 * scols, col_l = col_o + NP;
  extern __shared__ unsigned char sm_raw[];
  // (an offset, and not a rounded address: the compiler keeps sight of shared memory)
  unsigned char* sm = sm_raw + (-smem_addr(sm_raw) & 1023u);
  unsigned char *q8 = sm, *q16 = sm + lay.q16, *psm = sm + lay.p, *wide = sm + lay.wide;
  unsigned char *kring = sm + lay.kring, *vring = sm + lay.vring;
  float* row_c = reinterpret_cast<float*>(sm + lay.rest);  // [128] what a row's 8-bit scores are multiplied by
  float* row_nm = row_c + 128;                   // [128] minus its maximum
  float* row_f = row_nm + 128;                   // [128] what O is multiplied by in the end
  float* part = row_f + 128;                     // [16][4][8] of chunks' warps; of groups' while tiles go on
  int* row_at = reinterpret_cast<int*>(part + 4 * 128);  // [128] a row's place among the sequence's heads
  uint64_t* bars = reinterpret_cast<uint64_t*>(row_c + 8 * 128);
  uint64_t* kfull = bars;                        // [8] each
  uint64_t* kempty = kfull + 8;
  uint64_t* vfull = kempty + 8;
  uint64_t* vempty = vfull + 8;
  uint64_t* wfull = vempty + 8;                  // [2] V in 16 bits
  uint64_t* wempty = wfull + 2;                  // [2] the tile's products V^T P done
  uint64_t* sfull = wempty + 2;                  // [2]
  uint64_t* pready = sfull + 2;                  // [2]
  uint64_t* qready = pready + 2;
  uint64_t* mdone = qready + 1;                  // [2]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(mdone + 2);
  int* fail = reinterpret_cast<int*>(tslot + 1);
  int* odd = fail + 1;                           // a V element that is not finite was left out
  Plan& plan = *reinterpret_cast<Plan*>(bars + 46);
  Place* places = reinterpret_cast<Place*>(bars + 64);  // of the warps
  int* first = reinterpret_cast<int*>(reinterpret_cast<unsigned char*>(row_c) + kSmall);  // the plan's arrays
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.T * a.G, chunks = (rows + 7) / 8;
  const int active = TURNS ? kGroups : min(kGroups, chunks);  // groups with any rows

  // ---- set-up
  if (warp == kMmaWarp) {
    // (kfull, kempty, vfull, vempty: 8 each; wfull, wempty, sfull, pready: 2; qready; mdone: 2)
    if (lane < 24) mbar_init(bars + lane, 1);
    else mbar_init(bars + lane, kWiden / 32);
    if (lane < 11)
      mbar_init(bars + 32 + lane, lane < 2                ? kWiden / 32
                                  : lane == 6 || lane == 7 ? (TURNS ? 4 : 4 * active)
                                  : lane == 8              ? (TURNS ? 4 : 4 * active)
                                                           : 1);
    if (lane == 0) {
      *fail = (int)blockIdx.x == a.give_up;
      *odd = 0;
      plan.first = first;
      plan.length = first + a.B + 1;
      plan.held = plan.length + a.B;
      plan.some = reinterpret_cast<short*>(plan.held + a.B);
      plan.count = plan.some + a.B + 1;
    }
    fence_mbar_init();
  }
  if (warp == kCopyWarp && lane < 4) {
    const CUtensorMap* m = lane == 0 ? &mK8 : lane == 1 ? &mV8 : lane == 2 ? &mK : &mV;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  pdl_wait();                                    // (up to here beside the kernel before; nothing is held)
  if (warp == 0) tmem_alloc(tslot, 512);
#pragma unroll 1
  for (int b = tid; b < a.B; b += kThreads) {
    const int n = a.lengths[b], h = a.held ? a.held[b] : 0;
    const int c = a.counts ? min(max(a.counts[b], -1), 129) : a.T;  // (129: too many, like all above)
    first[a.B + 1 + b] = n;
    first[2 * a.B + 1 + b] = h;
    reinterpret_cast<short*>(first + 3 * a.B + 1)[a.B + 1 + b] = (short)c;
    first[b + 1] = tiles_of(seq_range(a, n, c, h));
  }
  if (tid < rows) row_at[tid] = tid / a.G * a.H + tid % a.G;
  // the rows beyond
  if (tid >= rows && tid < 128) row_c[tid] = 0.f;
#pragma unroll 1
  for (int i = tid; i < lay.p / 16; i += kThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == kWidenWarp) {
    int sum = 0, some = 0;
    if (lane == 0) first[0] = plan.some[0] = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int x = b0 + lane < a.B ? first[b0 + lane + 1] : 0;
      const uint32_t any = __ballot_sync(~0u, x > 0);
      if (b0 + lane < a.B) plan.some[b0 + lane + 1] = (short)(some + __popc(any & (~0u >> (31 - lane))));
      some += __popc(any);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
      }
      if (b0 + lane < a.B) first[b0 + lane + 1] = sum + x;
      sum += __shfl_sync(~0u, x, 31);
    }
    const long long tiles = (long long)sum * a.Hkv;
    const int ctas = (int)min((long long)gridDim.x, tiles);
    if (lane == 0) {
      int start = kStart;                        // (as long as a CTA has four times as many tiles)
      while (start && tiles < 4ll * start * ctas) --start;
      plan.start = start;
      plan.total = tiles + (long long)start * some * a.Hkv;
      plan.ctas = ctas;
    }
    __syncwarp();
    if (lane < 2)
      (lane ? plan.end : plan.begin) = tiles_before(a, plan, cta_start(plan.total, ctas, blockIdx.x + lane));
    __syncwarp();
    if (plan.begin < plan.end && lane == 0) first_segment(a, plan, plan.begin, places[0]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tslot);
  const long long begin = plan.begin, end = plan.end;
  Place& place = places[warp];
  static_assert(sizeof(Place) % 4 == 0 && sizeof(Place) <= 128, "a word per lane");
  static_assert(sizeof(Place) * (kThreads / 32) <= kPlaces, "a place per warp");
  if (warp && lane < (int)sizeof(Place) / 4)
    reinterpret_cast<int*>(&place)[lane] = reinterpret_cast<const int*>(places)[lane];
  __syncthreads();                               // (the first warp's own may change from here on)
  auto give_up = [&](bool ok) {
    if (!ok) atomicExch(fail, 1);
  };

  if (warp == kCopyWarp || warp == kCopyWarp + 1) {
    // ---- copies of K (first warp) or V tiles, in units of 128 rows of up to
    // 128 bytes: one for a tile of 8-bit rows, a panel of 64 columns each for bf16
    // (the warp runs together up to the copies themselves)
    {
      const bool is_v = warp > kCopyWarp;
      const int units = is_v ? lay.v_units : lay.k_units;
      unsigned char* ring = is_v ? vring : kring;
      uint64_t *full = is_v ? vfull : kfull, *empty = is_v ? vempty : kempty;
      const CUtensorMap *m8 = is_v ? &mV8 : &mK8, *m16 = is_v ? &mV : &mK;
      int issued = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = !tree_flagged(fail);
#pragma unroll 1
      for (long long at = begin; ok && at < end;) {
        if (at != begin) next_segment(a, plan, at, place);
        const int sn = place.s.n, sb = place.s.b, sh = place.s.h;
        Walk t = place.w;
        if (!is_v)                               // q on its way, while the pair before is at work
#pragma unroll 1
          for (int i = lane; i < rows * P; i += 32) {
            const bf16* at_q = a.q + ((size_t)sb * a.T * a.H + (size_t)sh * a.G + row_at[i / P]) * DH + i % P * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at_q));
          }
#pragma unroll 1
        for (int i = 0; ok && i < sn; ++i) {
#pragma unroll 1
          for (int u = 0; ok && u < (t.eight ? 1 : P); ++u) {
            if (issued >= units) ok = wait_for(fail, &empty[slot], phase ^ 1u);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], t.eight ? 128u * DH : (uint32_t)kUnit);
            if (lane != 0) {
            } else if (t.eight) tma_load_4d(ring + slot * kUnit, m8, 0, t.p0, sh, sb, &full[slot]);
            else tma_load_4d(ring + slot * kUnit, m16, u * 64, t.p0 % a.rows, sh, sb, &full[slot]);
            ++issued;
            if (++slot == units) {
              slot = 0;
              phase ^= 1u;
            }
          }
          if (i + 1 < sn) step(t, place, a.window);
        }
        at += sn;
      }
      give_up(ok);
      if (is_v && lane == 0) {
        // the pair that goes on in the next CTA, and which one has its last tile
        const Segment& s = place.s;
        const bool goes_on = begin < end && !s.whole && !s.head;
        a.shared[blockIdx.x] = goes_on ? make_int4(s.b, s.h, last_cta(a, plan, s.b, s.h), 0) : make_int4(-1, 0, 0, 0);
      }
      // what is still in flight lands before the memory is released
#pragma unroll 1
      for (int i = max(0, issued - units); i < issued; ++i)
        mbar_wait_n(&full[i % units], (uint32_t)((i / units) & 1), kPolls);
    }
  } else if (warp >= kMmaWarp) {
    // ---- products: the warp runs together, one lane issues
    const uint32_t lead = tree_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    bool ok = !tree_flagged(fail);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && wait_for(fail, bar, parity));
      tc_fence_after();
    };
    auto wait_both = [&](uint64_t* a0, uint32_t p0, uint64_t* a1, uint32_t p1, bool two) {
      ok = __all_sync(0xffffffffu, ok && wait_for_both(fail, a0, p0, a1, p1, two));
      tc_fence_after();
    };
    uint32_t n = 0;                              // tiles so far
    if (warp == kMmaWarp) {
      // scores: K q^T
      const uint32_t kr = smem_addr(kring), qa8 = smem_addr(q8), qa16 = smem_addr(q16);
      const uint32_t id8 = idesc_e4m3((int)scols), id16 = idesc_e4m3(NP) | 1u << 7 | 1u << 10;
      const uint64_t low = (uint64_t)((uint32_t)(NP * DH) >> 4);
      uint32_t kphase = 0, segments = 0;
      int kslot = 0;
      auto next_k = [&]() {
        if (++kslot == lay.k_units) {
          kslot = 0;
          kphase ^= 1u;
        }
      };
#pragma unroll 1
      for (long long pos = begin; ok && pos < end; ++segments) {
        if (pos != begin) next_segment(a, plan, pos, place);
        const int sn = place.s.n, in_eight = place.s.eight;
        wait(qready, segments & 1u);
#pragma unroll 1
        for (int i = 0; ok && i < sn; ++i, ++n) {
          const uint32_t buf = n & 1u, d = tm + buf * scols;
          // the softmax has read what was in this place
          wait_both(&kfull[kslot], kphase, &pready[buf], ((n >> 1) & 1u) ^ 1u, n >= 2);
          if (!ok) break;
          if (!seldom(i >= in_eight)) {
            const uint32_t kb = kr + (uint32_t)kslot * kUnit;
            const uint64_t kd = DH == 128 ? sw128_desc(kb) : sw64_desc(kb);
            const uint64_t qd = DH == 128 ? sw128_desc(qa8) : sw64_desc(qa8);
            // (the low part first)
            if (!SMALL)
#pragma unroll
              for (int ks = 0; ks < DH / 32; ++ks)
                mma_ss_e4m3(lead, d, kd + 2 * ks, qd + low + 2 * ks, id8, ks > 0 ? 1u : 0u);
#pragma unroll
            for (int ks = 0; ks < DH / 32; ++ks)
              mma_ss_e4m3(lead, d, kd + 2 * ks, qd + 2 * ks, id8, !SMALL || ks > 0 ? 1u : 0u);
            tree_commit(lead, &sfull[buf]);
            tree_commit(lead, &kempty[kslot]);
            next_k();
          } else {
#pragma unroll 1
            for (int u = 0; ok && u < P; ++u) {
              if (u) wait(&kfull[kslot], kphase);
              if (!ok) break;
              const uint64_t kd = sw128_desc(kr + (uint32_t)kslot * kUnit);
              const uint64_t qd = sw128_desc(qa16 + (uint32_t)(u * NP) * 128);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) tree_mma_ss(lead, d, kd + 2 * ks, qd + 2 * ks, id16, u || ks > 0 ? 1u : 0u);
              if (u + 1 == P) tree_commit(lead, &sfull[buf]);
              tree_commit(lead, &kempty[kslot]);
              next_k();
            }
          }
        }
        pos += sn;
      }
    } else {
      // values: V^T P
      const uint32_t wr = smem_addr(wide), pr = smem_addr(psm);
      // (both operands MN-major; fp16, bf16)
      const uint32_t idp8 = idesc_e4m3(NP) | 3u << 15, idp16 = idp8 | 1u << 7 | 1u << 10;
#pragma unroll 1
      for (long long pos = begin; ok && pos < end;) {
        if (pos != begin) next_segment(a, plan, pos, place);
        const int sn = place.s.n, in_eight = place.s.eight;
#pragma unroll 1
        for (int i = 0; ok && i < sn; ++i, ++n) {
          const uint32_t buf = n & 1u, ph = (n >> 1) & 1u;
          wait_both(&pready[buf], ph, &wfull[buf], ph, true);
          if (!ok) break;
          const uint64_t vd = v_desc(wr + buf * (uint32_t)kWide);
          const uint64_t pd = p_desc(pr + (lay.p_bufs == 2 ? buf * (uint32_t)NP * 256u : 0u));
          const uint32_t idp = i < in_eight ? idp8 : idp16, d = tm + col_o + (TURNS ? buf * 16u : 0u);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tree_mma_ss(lead, d, vd + 128 * ks, pd + 32 * ks, idp, (i > (TURNS ? 1 : 0) || ks > 0) ? 1u : 0u);
          tree_commit(lead, &wempty[buf]);
        }
        pos += sn;
      }
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
    tree_commit(lead, &mdone[warp - kMmaWarp]);
    mbar_wait_n(&mdone[warp - kMmaWarp], 0u, kPolls);
  } else if (warp >= kWidenWarp) {
    // ---- V to 16 bits in the products' layout
    const int cw = warp - kWidenWarp, ct = tid - kWidenWarp * 32;
#pragma unroll 1
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      if (first[b + 1] != first[b]) continue;
      // a sequence without tokens, or without sense
      const float x = seq_range(a, plan.length[b], plan.count[b], plan.held[b]).count < 0 ? NAN : 0.f;
      const uint32_t w = pack_bf16x2(x, x);
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)b * a.T * a.H * DH);
#pragma unroll 1
      for (size_t i = ct; i < (size_t)a.T * a.H * DH / 8; i += kWiden) o[i] = make_uint4(w, w, w, w);
    }
    int slot = 0;
    uint32_t phase = 0, n = 0;
    bool ok = !tree_flagged(fail);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && wait_for(fail, bar, parity));
    };
    auto freed = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(&vempty[slot]);
      if (++slot == lay.v_units) {
        slot = 0;
        phase ^= 1u;
      }
    };
#pragma unroll 1
    for (long long pos = begin; ok && pos < end;) {
      if (pos != begin) next_segment(a, plan, pos, place);
      const int sn = place.s.n;
      Walk t = place.w;
#pragma unroll 1
      for (int i = 0; ok && i < sn; ++i, ++n) {
        if (i) step(t, place, a.window);
        const bool edge = t.edge();
        const uint32_t buf = n & 1u;
        unsigned char* to = wide + buf * kWide;
        ok = __all_sync(0xffffffffu, ok && wait_for_both(fail, &vfull[slot], phase, &wempty[buf],
                                                         ((n >> 1) & 1u) ^ 1u, n >= 2));
        if (!ok) break;
        // (a warp has rows 32 cw .. + 31 of the tile)
        if (!seldom(!t.eight)) {
          // eight lanes read 16 bytes each of two rows four apart, and write the
          // first half of theirs while the others write the second: all banks
          const unsigned char* from = vring + slot * kUnit + (cw * 32) * DH;
          unsigned char* rows_to = to + cw * 32 * 128;
          const int c = lane & 3, half = (lane >> 2) & 1, k7 = (lane >> 3) + 4 * half;
          const int a0 = ((2 * c + half) ^ k7) << 4, a1 = ((2 * c + 1 - half) ^ k7) << 4;
#pragma unroll 1
          for (int r0 = 0; r0 < 32; r0 += 16) {
            uint4 xs[2 * P];
#pragma unroll
            for (int it = 0; it < 2 * P; ++it) {
              const int key = r0 + (P == 2 ? it >> 1 : it) * 8 + k7, panel = P == 2 ? it & 1 : 0;
              xs[it] = *reinterpret_cast<const uint4*>(
                  from + (DH == 128 ? key * 128 + (((panel * 4 + c) ^ k7) << 4)
                                    : key * 64 + ((c ^ ((key >> 1) & 3)) << 4)));
            }
#pragma unroll
            for (int it = 0; it < 2 * P; ++it) {
              const int key = r0 + (P == 2 ? it >> 1 : it) * 8 + k7, panel = P == 2 ? it & 1 : 0;
              const uint4 x = xs[it];
              const uint32_t u0 = half ? x.z : x.x, u1 = half ? x.w : x.y, v0 = half ? x.x : x.z, v1 = half ? x.y : x.w;
              unsigned char* row = rows_to + panel * kUnit + key * 128;
              *reinterpret_cast<uint4*>(row + a0) = widen(u0, u1);
              *reinterpret_cast<uint4*>(row + a1) = widen(v0, v1);
            }
          }
          freed();
        } else {
#pragma unroll 1
          for (int u = 0; ok && u < P; ++u) {
            if (u) wait_w(&vfull[slot], phase);
            if (!ok) break;
            const uint4* from = reinterpret_cast<const uint4*>(vring + slot * kUnit) + cw * 256 + lane;
            uint4* rows_to = reinterpret_cast<uint4*>(to + u * kUnit) + cw * 256 + lane;
#pragma unroll
            for (int it = 0; it < 8; ++it) rows_to[it * 32] = from[it * 32];
            freed();
          }
          if (!ok) break;
        }
        if (seldom(edge)) {
          // rows that not all tokens see, two at a time
          const int kd = row_kind(a, place.s.r, t, t.p0 + cw * 32 + lane);
          __syncwarp();
#pragma unroll 1
          for (int kind = 0; kind < 2; ++kind) {
            uint32_t left = __ballot_sync(~0u, kd == kind);
#pragma unroll 1
            while (left) {
              const uint32_t rest = left & (left - 1), one = lane < 16 || !rest ? left : rest;
              left = rest & (rest - 1);
              uint4* x = reinterpret_cast<uint4*>(to + ((lane >> 3) & 1) * kUnit + (cw * 32 + __ffs(one) - 1) * 128) +
                         (lane & 7);
              if (P == 1 && (lane & 8)) continue;
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (kind) {
                const uint32_t e = t.eight ? 0x7c007c00u : 0x7f807f80u;
                bool bad = false;
                v = *x;
                v = make_uint4(finite_only(v.x, e, bad), finite_only(v.y, e, bad), finite_only(v.z, e, bad),
                               finite_only(v.w, e, bad));
                if (bad) atomicExch(odd, 1);
              }
              *x = v;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&wfull[buf]);
      }
      pos += sn;
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
  } else {
    // ---- softmax and results: one thread per key of a tile and group, then per
    // column of V; group g has rows 8 q .. 8 q + 7 for q = g, g + groups, ..., or all
    // rows of tiles n = g, g + groups, ...
    const int group = warp >> 2, w4 = warp & 3, key = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)(w4 * 32) << 16);
    const int nblk = a.max_seq / a.block, shift = 31 - __clz(a.block);
    float* gpart = part + group * 32;
    uint32_t n = 0;                              // tiles so far
    // A wait that gives up is the last that this warp makes; it goes on without
    // (its results are marked in the end), as the others count on it at their
    // common barriers.
    bool ok = !tree_flagged(fail);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) {
      if (ok) {
        ok = __all_sync(0xffffffffu, wait_for(fail, bar, parity));
        if (seldom(!ok) && lane == 0) atomicExch(fail, 1);
      }
      tc_fence_after();
    };
    // The products V^T P of tile `done` - 1 (the barrier's phase before has been
    // waited for, so that its parity tells).
    auto wait_values = [&](uint32_t done) { wait_w(&wempty[(done - 1) & 1u], ((done - 1) >> 1) & 1u); };
    const int q0 = TURNS ? 0 : group, q_step = TURNS ? 1 : kGroups;
    const int s0 = TURNS ? group : 0;            // where the rows' state lies: chunk s0 + q
    const uint32_t col_mine = col_o + (TURNS ? group * 16u : 0u);
    // Columns of O of 8 rows times f and all.
    auto rescale = [&](int q, const float (&f)[8], float all) {
      uint32_t o[8];
      tmem_ld8_nw(trow + col_mine + q * 8, o);
      tmem_wait_ld();
      tmem_pin8(o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (f[e] * all));
      tmem_st8(trow + col_mine + q * 8, o);
      tmem_wait_st();
    };
#pragma unroll 1
    for (long long at = group < active ? begin : end; at < end;) {
      if (at != begin) next_segment(a, plan, at, place);
      const Segment& s = place.s;
      const int sn = s.n;
      // ---- the query's parts: bf16, and e4m3 twice under a power of two
      {
        constexpr int kEach = DH / 8;            // threads per row, 8 elements each
        const int c = key % kEach, live = s.r.count * a.G;
        const bf16* src = a.q + ((size_t)s.b * a.T * a.H + (size_t)s.h * a.G) * DH + c * 8;
        auto fetch_q = [&](int row) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (row < live && key / kEach < 8 && !(TURNS && group))
            x = *reinterpret_cast<const uint4*>(src + (size_t)row_at[row] * DH);
          return x;
        };
        uint4 coming = fetch_q(q0 * 8 + key / kEach);
#pragma unroll 1
        for (int r0 = q0 * 8; r0 < (TURNS && group ? 0 : chunks * 8); r0 += q_step * 8) {
          {
            const int row = r0 + key / kEach;
            const uint4 x = coming;
            if (!SMALL) coming = fetch_q(row + q_step * 8);
            uint32_t w[4] = {x.x, x.y, x.z, x.w}, most = 0, hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k) most = __vmaxu2(most, w[k] & 0x7fff7fffu);
            most = max(most & 0xffffu, most >> 16);
#pragma unroll
            for (int d = kEach / 2; d; d >>= 1) most = max(most, __shfl_xor_sync(~0u, most, d));
            const int e = min(134 - (int)(most >> 7), 120);  // |q| 2^e below 256
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (a.negate) w[k] ^= 0x80008000u;
              // (a query that is not finite: NaN, as an infinite element may make all scores -infinity)
              if (most >= 0x7f80u) w[k] = 0x7fff7fffu;
              const float2 f = make_float2(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
              const uint32_t h = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
              const __half2 b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
              const float2 d = __half22float2(b);
              const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(f.x - d.x, f.y - d.y), __NV_SATFINITE, __NV_E4M3);
              hi[k >> 1] |= h << (16 * (k & 1));
              lo[k >> 1] |= l << (16 * (k & 1));
            }
            auto place = [&](int r) {
              return DH == 128 ? r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8
                               : r * 64 + (((c >> 1) ^ ((r >> 1) & 3)) << 4) + (c & 1) * 8;
            };
            if (row < rows && key / kEach < 8) {
              *reinterpret_cast<uint2*>(q8 + place(row)) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(q8 + place(NP + row)) = make_uint2(lo[0], lo[1]);
              *reinterpret_cast<uint4*>(q16 + (c >> 3) * NP * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
              if (c == 0)
                row_c[row] = most < 0x7f80u ? a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23) : NAN;
            }
          }
          if (key < 8) row_nm[r0 + key] = -kNone;
        }
        if (TURNS && group && key < 8) row_nm[8 + key] = -kNone;
        fence_proxy_async_smem();
        if (TURNS) bar_both();
        else bar_group(group);
        if (lane == 0 && (!TURNS || group == 0)) mbar_arrive_cta(qready);
      }
      // ---- tiles
      // O holds sums of 2^(score - m) v 2^7 / vref.  m follows the largest score + log2(scale /
      // (vref / 4)) of the row's keys, so that what P holds of a row's largest weight depends
      // on no scale without weight.
      float vref = 0.f, unit = 0.f;              // (unit = 2^7 / vref)
      float c[8], nm[8], ls[8];                  // of the chunk; the sums of SMALL
      auto state = [&](int q) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 u = *reinterpret_cast<const float4*>(row_c + q * 8 + e);
          const float4 w = *reinterpret_cast<const float4*>(row_nm + (s0 + q) * 8 + e);
          c[e] = u.x, c[e + 1] = u.y, c[e + 2] = u.z, c[e + 3] = u.w;
          nm[e] = w.x, nm[e + 1] = w.y, nm[e + 2] = w.z, nm[e + 3] = w.w;
        }
      };
      if (SMALL) {
        state(q0);
#pragma unroll
        for (int e = 0; e < 8; ++e) ls[e] = 0.f;
      } else {
        const uint32_t zero[8] = {};
#pragma unroll 1
        for (int q = q0; q < chunks; q += q_step) tmem_st8(trow + col_l + q * 8, zero);
        tmem_wait_st();
      }
      const float* kscale = a.k_scale + (size_t)s.b * a.scale_stride + (size_t)s.h * nblk;
      const float* vscale = a.v_scale + (size_t)s.b * a.scale_stride + (size_t)s.h * nblk;
      float ks = 1.f, vs = 1.f;                  // of the tile to come, the warp's 32 keys
      auto fetch = [&](const Walk& t) {
        const int blk = min((t.p0 + w4 * 32) >> shift, nblk - 1);
        if (t.eight) {
          ks = kscale[blk];
          vs = vscale[blk];
        }
      };
      Walk t = place.w;
      // (TURNS: the tiles that the other group takes are passed by)
      int i = TURNS ? (int)((n ^ (uint32_t)group) & 1u) : 0;
      const int i_first = i;
      if (TURNS) {
        n += i;
        if (i && i < sn) step(t, place, a.window);
      }
      if (i < sn) fetch(t);
#pragma unroll 1
      for (; i < sn; i += TURNS ? 2 : 1, n += TURNS ? 2 : 1) {
        const uint32_t buf = n & 1u;
        const bool eight = t.eight, edge = t.edge();
        const float kc = ks;
        float vc = eight ? vs : 1.f;
        // the rows that see the thread's key: [r0, r1); the warp's scale passes vref
        // (if any of its keys counts)
        int r0 = 0, r1 = NP;
        // (bf16 rows: a unit far below their values' would take P and O out of fp32's range)
        bool over = eight ? fabsf(vc) > vref && fabsf(vc) < 0x1p124f : vref < kTiny && vref != 0.f;
        if (seldom(edge)) {
          const int j = t.p0 + key;
          r0 = max(j - s.r.length, 0) * a.G;
          r1 = s.r.count * a.G;
          if (a.window && j >= a.sinks) {
            const long long last = (long long)j + a.window - s.r.length;
            if (last < s.r.count) r1 = last < 0 ? 0 : (int)last * a.G;
          }
          if (j < t.rs || j >= t.re) r1 = 0;
          over = over && t.p0 + w4 * 32 < t.re && t.p0 + w4 * 32 + 32 > t.rs;
        }
        // (a scale of 1 may be that of zeros, whose weight is none; where all scales are 1 a pair's
        // first tile is looked at for nothing, 1 us of 51 of one token over 131000 rows)
        if (seldom(over && eight && vc == 1.f) && rows_are_zero(a, s, t.p0 + w4 * 32, t.rs, t.re)) {
          over = false;
          vc = 0.f;
        }
        if (i + (TURNS ? 2 : 1) < sn) {
          if (TURNS) step(t, place, a.window);
          step(t, place, a.window);
          fetch(t);
        }
        // the scores are there, P's place is free
        if (ok) {
          ok = __all_sync(0xffffffffu, wait_for_both(fail, &sfull[buf], (n >> 1) & 1u, &wempty[buf],
                                                     ((n >> 1) & 1u) ^ 1u, n >= 2));
          if (seldom(!ok) && lane == 0) atomicExch(fail, 1);
        }
        tc_fence_after();
        if (!SMALL && lay.p_bufs == 1 && n > 0) wait_values(n);  // (its only one)
        float pv = vc * unit;
        float most_over = raise_of(eight, vc, vref);
        // vref's change: its inverse, what maxima come down by, so far (in the place of a chunk of
        // the group's own, or of none)
        float* grown = part + (group + (TURNS ? 4 : kGroups)) * 32;
        unsigned char* pto = psm + (lay.p_bufs == 2 ? buf * NP * 256 : 0) + key * 32;
        // More than 16 rows: the loop a second time for what nearly all tiles are, 8-bit rows
        // that all tokens see, without the questions after the others.  (72 rows 134.2 ->
        // 122.6 us; for few rows the longer code costs a window 12.1 -> 12.7 us and takes
        // two tokens of 40 heads from 48.3 to 47.6)
        auto tile = [&](auto plain) {
          const bool in_eight = SMALL ? eight : decltype(plain)::value || eight;
          const bool at_edge = SMALL ? edge : !decltype(plain)::value && edge;
          // the tokens that see the key, of chunk q's rows
          auto seen_of = [&](int q) {
            const int m0 = max(r0 - q * 8, 0), m1 = min(r1 - q * 8, 8);
            return m1 > m0 ? ((1u << m1) - 1u) & ~((1u << m0) - 1u) : 0u;
          };
          bool force = over || vref == 0.f;
          uint32_t x[8], y[8];                     // products; SMALL: their second parts, else the sums
          tmem_ld8_nw(trow + buf * scols + q0 * 8, x);
          if (SMALL) tmem_ld8_nw(trow + buf * scols + q0 * 8 + 16, y);
          tmem_wait_ld();
          tmem_pin8(x);
          if (SMALL) tmem_pin8(y);
#pragma unroll 1
          for (int q = q0; q < chunks; q += q_step) {
            const uint32_t scol = trow + buf * scols + q * 8;
            if (!SMALL) {
              tmem_ld8_nw(trow + col_l + q * 8, y);  // (needed in the end)
              state(q);
            }
            // scores (of the products' two parts), as multiples of what the exponential
            // takes, minus m
            float d[8];
            auto scores = [&](bool from_m) {
              const float2 k2 = make_float2(kc, kc), s2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                float2 v = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                if (in_eight) {
                  if (SMALL) v = __fadd2_rn(v, make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])));
                  v = __fmul2_rn(v, __fmul2_rn(make_float2(c[e], c[e + 1]), k2));
                } else {
                  v = __fmul2_rn(v, s2);
                }
                // (not fused: m is a rounded product, and so is at most kRaise below any)
                if (from_m) v = __fadd2_rn(v, make_float2(nm[e], nm[e + 1]));
                d[e] = v.x;
                d[e + 1] = v.y;
              }
              if (seldom(at_edge)) {
                const uint32_t seen = seen_of(q);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (!((seen >> e) & 1u)) d[e] = -INFINITY;
              }
            };
            scores(true);
            const float top = tree_max3(tree_max3(d[0], d[1], d[2]), tree_max3(d[3], d[4], d[5]), fmaxf(d[6], d[7]));
            if (seldom(any_group(group, top > most_over || force))) {
              if (q == q0) {
                // the largest of the four warps' scales
                if (lane == 0) gpart[w4] = over ? fabsf(vc) : 0.f;
                bar_group(group);
                const float most = fmaxf(fmaxf(gpart[0], gpart[1]), fmaxf(gpart[2], gpart[3]));
                if (most > vref || vref == 0.f) {
                  // (2^7 / next: finite; 1 for bf16 rows alone)
                  const float next = most > 0.f ? fmaxf(power_above(most) * 4.f, 0x1p-119f) : eight ? 1.f : 0x1p7f;
                  force = vref != 0.f;           // (then all chunks of this tile come through here)
                  if (key == 0) {
                    const float down = force ? grown[2] : 0.f;
                    const float by = force ? (float)(exponent_above(next) - exponent_above(vref)) : 0.f;
                    if (force) {
                      grown[0] = vref / next;
                      grown[1] = fminf(by, kDown - down);
                    }
                    grown[2] = fminf(down + by, kDown);
                  }
                  vref = next;
                  unit = __uint_as_float((261u << 23) - __float_as_uint(next));
                  pv = vc * unit;
                  most_over = raise_of(eight, vc, vref);
                } else {
                  force = false;
                }
                bar_group(group);
              }
              // the rows' largest scores of all keys, and what their scales lie below vref; those
              // that pass m + kRaise become m
              tmem_ld8_nw(scol, x);
              if (SMALL) tmem_ld8_nw(scol + 16, y);
              tmem_wait_ld();
              tmem_pin8(x);
              tmem_pin8(y);
              scores(false);
              over_lanes(d, [](float u, float w) { return fmaxf(u, w); });
              if (!(lane & 3)) gpart[w4 * 8 + (lane >> 2)] = fabsf(d[0]) < kFar ? d[0] + (kRaise - most_over) : d[0];
              bar_group(group);
              if (key < 8) {
                const int at_row = (s0 + q) * 8 + key;
                const float old = -row_nm[at_row], low = force && fabsf(old) < kFar ? old - grown[1] : old;
                const float z = fmaxf(fmaxf(gpart[key], gpart[8 + key]), fmaxf(gpart[16 + key], gpart[24 + key]));
                const float m = z > low + kRaise ? z : low;
                row_f[at_row] = tree_ex2(old - m);
                row_nm[at_row] = -m;
              }
              bar_group(group);
              float g[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                g[e] = row_f[(s0 + q) * 8 + e];
                nm[e] = row_nm[(s0 + q) * 8 + e];
                if (SMALL) ls[e] *= g[e];
                else y[e] = __float_as_uint(__uint_as_float(y[e]) * g[e]);
              }
              if (i > i_first) {                   // (O as the tile before left it)
                if (!TURNS) wait_values(n);
                rescale(q, g, force ? grown[0] : 1.f);
              }
              tmem_ld8_nw(scol, x);
              if (SMALL) tmem_ld8_nw(scol + 16, y);
              tmem_wait_ld();
              tmem_pin8(x);
              if (SMALL) tmem_pin8(y);
              scores(true);
            }
            // (the next chunk's products come in behind the exponentials)
            if (!SMALL) tmem_ld8_nw(scol + (q + q_step < chunks ? q_step * 8 : 0), x);
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = tree_ex2(d[e]);
            if (SMALL)
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 v = __fadd2_rn(make_float2(ls[e], ls[e + 1]), make_float2(d[e], d[e + 1]));
                ls[e] = v.x;
                ls[e + 1] = v.y;
              }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = __fmul2_rn(make_float2(d[2 * e], d[2 * e + 1]), make_float2(pv, pv));
              pk[e] = in_eight ? pack_f16x2(v.x, v.y) : pack_bf16x2(v.x, v.y);
            }
            if (seldom(at_edge)) {                    // (a scale that is none of the row's)
              const uint32_t seen = seen_of(q);
#pragma unroll
              for (int e = 0; e < 8; e += 2)
                pk[e / 2] &= ((seen >> e) & 1u ? 0x0000ffffu : 0u) | ((seen >> e) & 2u ? 0xffff0000u : 0u);
            }
            *reinterpret_cast<uint4*>(pto + (q >> 1) * kPanel + (((q & 1) ^ ((key >> 2) & 1)) << 4)) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
            if (!SMALL) {
              tmem_wait_ld();
              tmem_pin8(x);
              tmem_pin8(y);
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 v = __fadd2_rn(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])),
                                            make_float2(d[e], d[e + 1]));
                y[e] = __float_as_uint(v.x);
                y[e + 1] = __float_as_uint(v.y);
              }
              tmem_st8(trow + col_l + q * 8, y);
            }
          }
        };
        if (SMALL || !seldom(!eight || edge)) tile(std::true_type{});
        else tile(std::false_type{});
        if (!SMALL) tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(&pready[buf]);
      }
      // ---- the run's result: final, or a part of the pair's
      const bool any = i_first < sn;             // (TURNS: the group had a tile)
      if (TURNS) {
        if (any) wait_values(n - 1);             // (n - 2 was the last)
        n = n - i + sn;                          // tiles so far, of both groups
      } else {
        wait_values(n);
      }
      const bool final = s.whole;
      const size_t slot = (size_t)blockIdx.x * 2 + (s.head ? 0 : 1);
      const size_t out0 = ((size_t)s.b * a.T * a.H + (size_t)s.h * a.G) * DH;
      const int live = s.r.count * a.G;          // rows with a token
      // the sums over the keys: a warp's, then (a thread per row) the four warps'
#pragma unroll 1
      for (int q = q0; q < chunks; q += q_step) {
        if (!SMALL) {
          uint32_t y[8];
          tmem_ld8_nw(trow + col_l + q * 8, y);
          tmem_wait_ld();
          tmem_pin8(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) ls[e] = __uint_as_float(y[e]);
        }
        over_lanes(ls, [](float u, float w) { return u + w; });
        if (!(lane & 3)) part[(s0 + q) * 32 + w4 * 8 + (lane >> 2)] = ls[0];
      }
      bar_group(group);
      const int mine = q0 + (key >> 3) * q_step, row = mine * 8 + (key & 7);  // the thread's chunk and row
      float m = kNone, l = 0.f;
      if (mine < chunks) {
        const float* p4 = part + (s0 + mine) * 32 + (key & 7);
        m = -row_nm[s0 * 8 + row];
        l = (p4[0] + p4[8]) + (p4[16] + p4[24]);
      }
      uint32_t o[8];
      auto fetch_o = [&](int q) {
        tmem_ld8_nw(trow + col_mine + q * 8, o);
        tmem_wait_ld();
        tmem_pin8(o);
      };
      if (TURNS) {
        // the second group's: its sums, and its outputs in the place of its P
        float* other = reinterpret_cast<float*>(psm + 4096);
        if (any) {
          fetch_o(0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0u;
        }
        if (group) {
          if (key < 8) part[64 + key] = l;
#pragma unroll
          for (int e = 0; e < 8; ++e) other[e * 128 + key] = __uint_as_float(o[e]) * (0x1p-7f * vref);
        }
        bar_both();
        if (group == 0) {
          float f[8];
          if (key < 8) {
            const float m1 = -row_nm[8 + key], top = fmaxf(m, m1);
            const float w0 = tree_ex2(m - top), w1 = tree_ex2(m1 - top);
            l = l * w0 + part[64 + key] * w1;
            m = top;
            row_f[key] = w0;
            row_f[8 + key] = w1;
          }
          bar_group(group);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f[e] = __uint_as_float(o[e]) * (0x1p-7f * vref * row_f[e]) + other[e * 128 + key] * row_f[8 + e];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(f[e]);
          bar_group(group);
        }
      }
      if (!TURNS || group == 0) {
        // (the segment's tiles are all behind: with TURNS the other group's since
        // bar_both, as it waited for its own before that)
        const bool bad = tree_flagged(odd);
        if (mine < chunks) {
          const float over_l = !final ? 1.f : l != 0.f ? __fdividef(1.f, l) : 0.f;
          row_f[row] = row < live ? over_l : 0.f;
          if (!final && row < rows) {
            a.part_m[slot * rows + row] = m;
            a.part_l[slot * rows + row] = row < live ? l : 0.f;
          }
        }
        bar_group(group);
        const float out_unit = TURNS ? 1.f : 0x1p-7f * vref;  // (apart: times 1 / l it may be no normal number)
        if (DH == 128 || w4 < 2)
#pragma unroll 1
          for (int q = q0; q < chunks; q += q_step) {
            if (!TURNS) fetch_o(q);
            bf16* out = a.out + out0 + key;
            float* po = a.part_o + (slot * rows + q * 8) * DH + key;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int row = q * 8 + e;
              const float w = row < live ? __uint_as_float(o[e]) * row_f[row] * out_unit : 0.f;
              if (row < rows && final) out[row_at[row] * DH] = __float2bfloat16(w);
              if (row < rows && !final) po[e * DH] = w;
            }
            if (bad)                             // what the products left out
#pragma unroll 1
              for (int e = 0; e < min(8, live - q * 8); ++e) {
                const int row = q * 8 + e;
                const float w = not_finite(a, s, s.r.length + row / a.G, key);
                if (w == 0.f) continue;          // (-0 stays: whether the flag is set here may be another pair's doing)
                if (final) out[row_at[row] * DH] = __float2bfloat16(__bfloat162float(out[row_at[row] * DH]) + w);
                else po[e * DH] += w;
              }
          }
      }
      if (TURNS) bar_both();                     // (its P's place is the second group's again)
      at += sn;
    }
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (tree_flagged(fail)) mark_rows(a, plan, place);
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins a pair that several CTAs share: CTA x = the first of them, thread = 16
// bytes of a row's output; the parts are added in order.  Bound by latency: the
// first parts are asked for together with the word that says how many there are.
// kBatch parts at once.
constexpr int kJoinThreads = 256;
template <int DH, int kBatch>
__global__ void __launch_bounds__(kJoinThreads) cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  const int rows = a.T * a.G, i = blockIdx.y * kJoinThreads + threadIdx.x, c0 = blockIdx.x;
  const int row = i / (DH / 4), col = i % (DH / 4) * 4, tok = row / a.G;
  if (row >= rows) return;
  float pm[kBatch], pl[kBatch], m = -INFINITY, l = 0.f;
  float4 v[kBatch], o = make_float4(0.f, 0.f, 0.f, 0.f);
  // the first CTA's second place, the others' first
  auto load = [&](int k0, int n) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = k0 + u;
      pm[u] = -INFINITY;
      pl[u] = 0.f;
      v[u] = o;
      if (k < n) {
        const size_t at = (k == 0 ? (size_t)c0 * 2 + 1 : (size_t)(c0 + k) * 2) * rows + row;
        pm[u] = a.part_m[at];
        pl[u] = a.part_l[at];
        v[u] = *reinterpret_cast<const float4*>(a.part_o + at * DH + col);
      }
    }
  };
  pdl_wait();
  pdl_trigger();
  const int4 pair = a.shared[c0];
  const int guess = min((int)gridDim.x - c0, kBatch);
  load(0, guess);                                // (what is there: some of it nobody wrote)
  if (pair.x < 0) return;
  const int n = pair.z - c0 + 1;
  if (n > guess) load(0, n);
  for (int k0 = 0;;) {
    float mn = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (k0 + u < n) mn = fmaxf(mn, pm[u]);
    const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(m - base);
    l *= old;
    o.x *= old;
    o.y *= old;
    o.z *= old;
    o.w *= old;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (k0 + u < n) {
        const float w = exp2f(pm[u] - base);
        l = fmaf(pl[u], w, l);
        o.x = fmaf(v[u].x, w, o.x);
        o.y = fmaf(v[u].y, w, o.y);
        o.z = fmaf(v[u].z, w, o.z);
        o.w = fmaf(v[u].w, w, o.w);
      }
    m = mn;
    if ((k0 += kBatch) >= n) break;
    load(k0, n);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;    // (NaN where a wait gave up)
  const size_t to = (((size_t)pair.x * a.T + tok) * a.H + pair.y * a.G + row % a.G) * DH + col;
  *reinterpret_cast<uint2*>(a.out + to) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

template <int DH, int GROUPS, bool SMALL, bool TURNS>
cudaError_t launch(const CacheAttnArgs& a, const CUtensorMap (&m)[4], cudaStream_t st) {
  const Layout lay = layout_of(a.T * a.G, DH, a.B);
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_tc_kernel<DH, GROUPS, SMALL, TURNS>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    if (dv >= 0) ready[dv] = true;
  }
  const cudaError_t e = launch_early(cache_attn_tc_kernel<DH, GROUPS, SMALL, TURNS>, a.ctas, threads_of(GROUPS),
                                     lay.bytes, st, 0, m[0], m[1], m[2], m[3], a, lay);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.ctas, (a.T * a.G * (DH / 4) + kJoinThreads - 1) / kJoinThreads);
  // A pair of few rows that 16 CTAs or more share (if the sequences are alike, and
  // long enough): its parts are asked for at once, in a short join.  Others two at a time: the
  // loads that go out unasked are traffic.  (20 at a time and 2, us: one sequence of
  // 131000 rows and 8 heads, 8 query rows each 52.1 and 53.8, 72 rows 127 and 115;
  // four of 20000 rows 39.9 and 38.5; 16 of 8192 rows 56.4 and 55.1)
  const long long tiles = ((long long)(a.k8 ? a.max_seq : 0) + a.rows) / kKeys, pairs = (long long)a.B * a.Hkv;
  const bool many = SMALL && a.ctas / pairs >= 16 && tiles >= 16;
  return many ? launch_early(cache_attn_join_kernel<DH, 20>, grid, kJoinThreads, 0, st, 0, a)
              : launch_early(cache_attn_join_kernel<DH, 2>, grid, kJoinThreads, 0, st, 0, a);
}

template <int DH>
cudaError_t launch_rows(const CacheAttnArgs& a, const CUtensorMap (&m)[4], cudaStream_t st) {
  const int rows = a.T * a.G;
  if (rows <= 8) return launch<DH, 2, true, true>(a, m, st);
  if (rows <= 16) return launch<DH, 2, true, false>(a, m, st);
  return rows > 24 && rows <= 32 ? launch<DH, 2, false, false>(a, m, st) : launch<DH, 3, false, false>(a, m, st);
}

}  // namespace

size_t cache_attn_workspace(CacheAttnArgs& a, void* base) {
  a.ctas = tree_sms();
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return base ? (void*)((char*)base + at) : nullptr;
  };
  const size_t rows = (size_t)a.T * a.G, places = (size_t)a.ctas * 2;
  a.part_o = (float*)take(places * rows * a.dh * 4);
  a.part_m = (float*)take(places * rows * 4);
  a.part_l = (float*)take(places * rows * 4);
  a.shared = (int4*)take((size_t)a.ctas * sizeof(int4));
  return off;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  EncodeTiled enc = tma_encoder();
  if (!enc) return cudaErrorNotSupported;
  // (columns, rows, heads, sequences) in boxes of 128 rows
  auto map = [&](CUtensorMap* m, bool eight, const void* base, int rows, size_t stride) {
    const size_t e = eight ? 1 : 2, row = a.dh * e;
    const cuuint64_t dims[4] = {(cuuint64_t)a.dh, (cuuint64_t)rows, (cuuint64_t)a.Hkv, (cuuint64_t)a.B};
    const cuuint64_t strides[3] = {row, row * rows, stride * e};
    const cuuint32_t box[4] = {eight ? (cuuint32_t)a.dh : 64u, 128, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               eight && a.dh == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  CUtensorMap m[4];
  if (!map(&m[2], false, a.k, a.rows, a.seq_stride) || !map(&m[3], false, a.v, a.rows, a.seq_stride))
    return cudaErrorInvalidValue;
  m[0] = m[2];                                   // (never read without 8-bit rows)
  m[1] = m[3];
  if (a.k8 && (!map(&m[0], true, a.k8, a.max_seq, a.seq8_stride) || !map(&m[1], true, a.v8, a.max_seq, a.seq8_stride)))
    return cudaErrorInvalidValue;
  return a.dh == 128 ? launch_rows<128>(a, m, s) : launch_rows<64>(a, m, s);
}

}  // namespace ssd
