// Attention of a few tokens per sequence over rows held in 8 bits and in bf16,
// on the 5th-generation tensor cores (sm_103a).
//
// The T G query rows of a sequence and K/V head (G query heads share it), 128 at
// most, are one tile, against tiles of 128 cache rows:
//
//   S = q K^T               8-bit rows: q = (q0 + q1) 2^-a with two e4m3 parts, which
//                           hold every bit of a bf16 number, so that the products
//                           with the stored bytes are exact; bf16 rows: q itself
//   P = 2^(S c - m) v_scale one thread per row, 16 bits over S's columns
//   O += P V                8-bit rows: V widened to fp16, P in fp16; bf16 rows: both bf16
//
// K and q enter the matrix instructions as they are: a tile of K costs no thread
// anything.  V cannot: P needs more than e4m3's range and bits (a first row that
// takes most of the weight leaves the others small), and both operands of a
// 16-bit product are 16 bits wide, so four warps widen V on its way: to fp16,
// which one instruction does for two values (bf16 takes four).  fp16 has less
// range than P: P is held in units of 2^-7 vref 2^m, vref a power of two not
// below any value scale so far, which keeps 11 bits down to 2^-18 of a row's
// largest weight and steps of 2^-28 below; two binades of room make it grow seldom.
//
// Rows of the tile: with up to 32 query rows the tile holds four copies of them,
// each of which keeps the keys of one quarter of the tile alone (64 rows: two
// copies, two halves): the softmax's work is divided among all four warps without
// an exchange, at the price of joining the copies at the end; the matrix pipe
// computes 128 rows in any case.
//
// Work: the tiles of all sequences and heads in one line, divided evenly among
// the CTAs (one per SM); a pair of sequence and head that several CTAs share is
// joined by a second kernel in a fixed order.  The division is computed from the
// lengths on the device, so that a graph follows them.
//
// Warps 0-3: softmax and results; 4-7: V to bf16; 8: copies of K; 9: copies of V;
// 10: matrix instructions.  Every wait is bounded: one that gives up sets the
// CTA's flag, every role runs out, and the CTA's rows become NaN.
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
constexpr int kThreads = 352;
constexpr int kPolls = 1 << 22;
constexpr int kUnit = 16 * 1024;                 // 128 rows of up to 128 bytes, swizzled
constexpr float kRaise = 8.f;
constexpr uint32_t kColO = 256, kColQ8 = 384, kColQ16 = 448;  // TMEM: S0, S1 (P over each), O, q

template <int DH>
struct Shape {
  static constexpr int kKUnits = DH == 128 ? 4 : 5;
  static constexpr int kVUnits = DH == 128 ? 3 : 4;
  static constexpr int kPanels = DH / 64;        // 16-bit panels of 64 columns
  static constexpr int kWide = kPanels * kUnit;  // a V tile in bf16
  static constexpr size_t kSmem = (size_t)(kKUnits + kVUnits) * kUnit + 2 * kWide + 4 * 32 * 33 * 4 + 6 * 128 * 4 + 512;
};

SSD_DI void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
SSD_DI void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
// V tile in panels of 64 columns as the MN-major B operand.
SSD_DI uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kUnit >> 4) << 16;             // leading offset: next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;              // stride offset: next 8 keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;                        // 128-byte swizzle
  return d;
}
// e4m3 A and B, fp32 D, both K-major; A in tensor memory.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
SSD_DI void mma_ts_e4m3(uint32_t lead, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
SSD_DI void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// ---- division of the work

// A tile: rows p0 .. p0 + 127, of which [rs, re) count.
struct Tile {
  int p0, rs, re;
  bool eight;
};
SSD_DI int cdiv_keys(int x) { return (x + kKeys - 1) / kKeys; }
SSD_DI int tiles_of(const SeqRange& r) {
  const int first = max(r.low, r.held);
  return cdiv_keys(min(r.sinks, r.held)) + (r.low < r.held ? cdiv_keys(r.held) - r.low / kKeys : 0) +
         (r.sinks > r.held ? cdiv_keys(r.sinks) - r.held / kKeys : 0) +
         (r.end > first ? cdiv_keys(r.end) - first / kKeys : 0);
}
// The i-th tile: first rows and the run in 8 bits, then the same in bf16.
SSD_DI Tile tile_at(const SeqRange& r, int i) {
  const int first = max(r.low, r.held);
  int n = cdiv_keys(min(r.sinks, r.held));
  if (i < n) return Tile{i * kKeys, 0, min(r.sinks, r.held), true};
  i -= n;
  n = r.low < r.held ? cdiv_keys(r.held) - r.low / kKeys : 0;
  if (i < n) return Tile{(r.low / kKeys + i) * kKeys, r.low, r.held, true};
  i -= n;
  n = r.sinks > r.held ? cdiv_keys(r.sinks) - r.held / kKeys : 0;
  if (i < n) return Tile{(r.held / kKeys + i) * kKeys, r.held, r.sinks, false};
  i -= n;
  return Tile{(first / kKeys + i) * kKeys, first, r.end, false};
}
// Whether some key of the tile is not seen by every token.
SSD_DI bool has_edge(const CacheAttnArgs& a, const SeqRange& r, const Tile& t) {
  return t.p0 < t.rs || t.p0 + kKeys > t.re || t.p0 + kKeys - 1 > r.length ||
         (a.window && t.p0 <= r.end - 1 - a.window && t.p0 + kKeys > a.sinks);
}
// Bits lo .. hi - 1 of a word, clipped.
SSD_DI uint32_t bits_between(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  if (hi <= lo) return 0u;
  return (0xffffffffu >> (32 - (hi - lo))) << lo;
}
// Which of the 32 keys from j on a token in row pos sees.
SSD_DI uint32_t seen_bits(const CacheAttnArgs& a, const Tile& t, int pos, int j) {
  uint32_t m = bits_between(t.rs - j, min(t.re, pos + 1) - j);
  if (a.window) m &= bits_between(0, a.sinks - j) | bits_between(pos - a.window + 1 - j, 32);
  return m;
}

// What the CTA's threads know of the sequences, in shared memory.
struct Plan {
  long long* first;                              // [B + 1] tiles (of one head) before sequence b
  int *length, *count, *held;                    // [B]
  long long begin, end;                          // the CTA's tiles
  long long total;
  int ctas;                                      // that have any
  SSD_DI long long start(int cta) const { return cta < ctas ? total * cta / ctas : total; }
  // The CTA that has a tile.
  SSD_DI int owner(long long tile) const {
    int cta = (int)(tile * ctas / total);
    while (start(cta + 1) <= tile) ++cta;
    return cta;
  }
};
// A run of a pair's tiles within the CTA's.
struct Segment {
  int b, h, i0, n;                               // tiles i0 .. i0 + n - 1 of the pair
  bool whole, head;                              // all of them; the pair began in an earlier CTA
  SeqRange r;
};
SSD_DI Segment segment_at(const CacheAttnArgs& a, const Plan& p, long long at) {
  Segment s;
  int lo = 0, hi = a.B - 1;                      // the last b with first[b] Hkv <= at
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.first[mid] * a.Hkv <= at) lo = mid;
    else hi = mid - 1;
  }
  s.b = lo;
  const int n = (int)(p.first[lo + 1] - p.first[lo]);
  const long long local = at - p.first[lo] * a.Hkv;
  s.h = (int)(local / n);
  s.i0 = (int)(local - (long long)s.h * n);
  const long long left = p.end - at;
  s.n = n - s.i0 < left ? n - s.i0 : (int)left;
  s.whole = s.n == n;
  s.head = s.i0 > 0;
  s.r = seq_range(a, p.length[lo], p.count[lo], p.held[lo]);
  return s;
}

// ---- values

// Two e4m3 (bytes lo and lo + 1 of x) to two fp16 of 2^-8 their value: the same
// sign, exponent and fraction at fp16's places (exact, fp16's range holds what
// e4m3's does; the code of NaN becomes 480 / 2^8).  Four integer instructions:
// the conversion instruction runs on the unit of the exponentials, far more
// slowly (a tile of 128 x 128 took 3000 cycles, against CYCLES so).
template <int LO>
SSD_DI uint32_t widen(uint32_t x) {
  const uint32_t h = __byte_perm(x, 0u, LO == 0 ? 0x1404 : 0x3424);
  return (h & 0x80008000u) | ((h >> 1) & 0x3fff3fffu);
}
constexpr uint32_t kWideNan = 0x3f80;            // what the code of NaN becomes, over all others
SSD_DI uint32_t larger(uint32_t most, uint32_t x) {
  const __half2 a = *reinterpret_cast<const __half2*>(&most), b = *reinterpret_cast<const __half2*>(&x);
  const __half2 m = __hmax2(a, __habs2(b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
// The NaN of two widened values as such.
SSD_DI uint32_t with_nan(uint32_t x) {
  if ((x & 0x7fffu) == kWideNan) x |= 0x7fffu;
  if ((x & 0x7fff0000u) == kWideNan << 16) x |= 0x7fff0000u;
  return x;
}
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
// The smallest power of two that is not below |x| (x finite and not 0), 2^-126 at least.
SSD_DI float power_above(float x) {
  return __uint_as_float((__float_as_uint(fabsf(x)) + 0x7fffffu) & 0x7f800000u);
}

// How a row of V goes into the products: 0 as zeros (it is outside the tile's
// run), 1 without what is not finite (0 x infinity is NaN, and some row of the
// products has a 0 there: a token that does not see it, or another copy), 2 as
// it is.
SSD_DI int row_kind(const CacheAttnArgs& a, const SeqRange& r, const Tile& t, int j) {
  if (j < t.rs || j >= t.re) return 0;
  if (!t.eight || j > r.length) return 1;
  return a.window && j >= a.sinks && j <= r.end - 1 - a.window ? 1 : 2;
}
// Adds to a row's n values from column c0 on what the products left out of the
// segment's V rows that the row's token, in row pos, sees.
static __device__ __noinline__ void add_not_finite(const CacheAttnArgs& a, const Segment& s, int pos, int c0, int n,
                                                   float* v) {
  for (int i = s.i0; i < s.i0 + s.n; ++i) {
    const Tile t = tile_at(s.r, i);
    for (int j = max(t.p0, t.rs); j < min(t.p0 + kKeys, t.re); ++j) {
      if (row_kind(a, s.r, t, j) != 1 || j > pos || (a.window && j >= a.sinks && j <= pos - a.window)) continue;
      for (int e = 0; e < n; ++e) {
        float x;
        if (t.eight) {
          const uint8_t code = a.v8[(size_t)s.b * a.seq8_stride + ((size_t)s.h * a.max_seq + j) * a.dh + c0 + e];
          x = (code & 0x7f) == 0x7f ? NAN : 0.f;
        } else {
          x = __bfloat162float(a.v[(size_t)s.b * a.seq_stride + ((size_t)s.h * a.rows + j % a.rows) * a.dh + c0 + e]);
        }
        if (!isfinite(x)) v[e] += x;
      }
    }
  }
}

template <int DH, int NCH>                       // NCH: chunks of 32 keys of a tile that a thread's row has
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_tc_kernel(const __grid_constant__ CUtensorMap mK8, const __grid_constant__ CUtensorMap mV8,
                         const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                         const __grid_constant__ CacheAttnArgs a) {
  using X = Shape<DH>;
  constexpr int kCopies = 4 / NCH;
  constexpr int KU = X::kKUnits, VU = X::kVUnits, P = X::kPanels;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* kring = sm;
  unsigned char* vring = kring + KU * kUnit;
  unsigned char* wide = vring + VU * kUnit;      // [2]
  float* merge = reinterpret_cast<float*>(wide + 2 * X::kWide);  // [4][32][33]
  float* xm = merge + 4 * 32 * 33;               // [128] per thread: maximum, sum
  float* xl = xm + 128;
  float* row_m = xl + 128;                       // [128] per row, of all copies
  float* row_l = row_m + 128;
  uint64_t* bars = reinterpret_cast<uint64_t*>(row_l + 128);
  uint64_t* kfull = bars;
  uint64_t* kempty = kfull + KU;
  uint64_t* vfull = kempty + KU;
  uint64_t* vempty = vfull + VU;
  uint64_t* wfull = vempty + VU;                 // [2] V in bf16
  uint64_t* wempty = wfull + 2;                  // [2] the tile's products P V done
  uint64_t* sfull = wempty + 2;                  // [2]
  uint64_t* pready = sfull + 2;                  // [2]
  uint64_t* qready = pready + 2;
  uint64_t* mdone = qready + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(mdone + 1);
  int* fail = reinterpret_cast<int*>(tslot + 1);
  int* odd = fail + 1;                           // a V element that is not finite was left out
  Plan plan;
  plan.first = reinterpret_cast<long long*>(reinterpret_cast<unsigned char*>(bars) + 512);
  plan.length = reinterpret_cast<int*>(plan.first + a.B + 1);
  plan.count = plan.length + a.B;
  plan.held = plan.count + a.B;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.T * a.G;

  // ---- set-up
  if (tid == 320) {
    for (int i = 0; i < KU; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < VU; ++i) {
      mbar_init(&vfull[i], 1);
      mbar_init(&vempty[i], 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&wfull[i], 128);
      mbar_init(&wempty[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&pready[i], 128);
    }
    mbar_init(qready, 128);
    mbar_init(mdone, 1);
    *fail = (int)blockIdx.x == a.give_up;
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  for (int b = tid; b < a.B; b += kThreads) {
    const int n = a.lengths[b], c = a.counts ? a.counts[b] : a.T, h = a.held ? a.held[b] : 0;
    plan.length[b] = n;
    plan.count[b] = c;
    plan.held[b] = h;
    plan.first[b + 1] = tiles_of(seq_range(a, n, c, h));
  }
  __syncthreads();
  if (warp == 4) {
    long long sum = 0;
    if (lane == 0) plan.first[0] = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      long long x = b0 + lane < a.B ? plan.first[b0 + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
      }
      if (b0 + lane < a.B) plan.first[b0 + lane + 1] = sum + x;
      sum += __shfl_sync(~0u, x, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tslot);
  plan.total = plan.first[a.B] * a.Hkv;
  plan.ctas = (int)min((long long)gridDim.x, plan.total);  // each with a tile at least
  plan.begin = plan.start(blockIdx.x);
  plan.end = plan.start(blockIdx.x + 1);
  auto give_up = [&](bool ok) {
    if (!ok) atomicExch(fail, 1);
  };

  if (warp == 8 || warp == 9) {
    // ---- copies of K (warp 8) or V (warp 9) tiles, in units of 128 rows of up to
    // 128 bytes: one for a tile of 8-bit rows, a panel of 64 columns each for bf16
    if (lane == 0) {
      const bool is_v = warp == 9;
      const int units = is_v ? VU : KU;
      unsigned char* ring = is_v ? vring : kring;
      uint64_t *full = is_v ? vfull : kfull, *empty = is_v ? vempty : kempty;
      const CUtensorMap *m8 = is_v ? &mV8 : &mK8, *m16 = is_v ? &mV : &mK;
      int issued = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = !tree_flagged(fail);
      for (long long at = plan.begin; ok && at < plan.end;) {
        const Segment s = segment_at(a, plan, at);
        for (int i = 0; ok && i < s.n; ++i) {
          const Tile t = tile_at(s.r, s.i0 + i);
          for (int u = 0; ok && u < (t.eight ? 1 : P); ++u) {
            if (issued >= units) ok = tree_wait(fail, kPolls, &empty[slot], phase ^ 1u);
            if (!ok) break;
            mbar_arrive_expect_tx(&full[slot], t.eight ? 128u * DH : (uint32_t)kUnit);
            if (t.eight) tma_load_4d(ring + slot * kUnit, m8, 0, t.p0, s.h, s.b, &full[slot]);
            else tma_load_4d(ring + slot * kUnit, m16, u * 64, t.p0 % a.rows, s.h, s.b, &full[slot]);
            ++issued;
            if (++slot == units) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
        at += s.n;
      }
      give_up(ok);
      // what is still in flight lands before the memory is released
      for (int i = max(0, issued - units); i < issued; ++i)
        mbar_wait_n(&full[i % units], (uint32_t)((i / units) & 1), kPolls);
    }
  } else if (warp == 10) {
    // ---- products: the warp runs together, one lane issues
    const uint32_t lead = tree_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t kr = smem_addr(kring), wr = smem_addr(wide);
    constexpr uint32_t id8 = idesc_e4m3(128, kKeys), id16 = idesc_bf16(128, kKeys);
    // (B is MN-major; fp16 in place of bf16 without bits 7 and 10)
    constexpr uint32_t idp16 = idesc_bf16(128, DH) | (1u << 16), idp8 = idp16 & ~(1u << 7 | 1u << 10);
    Ring<KU> at;
    int segments = 0;
    uint32_t n_s = 0, n_p = 0;                   // tiles whose scores / values were issued
    bool ok = !tree_flagged(fail);
    auto wait = [&](uint64_t* bar, uint32_t parity, uint64_t* other = nullptr, uint32_t other_parity = 0) {
      ok = __all_sync(0xffffffffu, ok && tree_wait(fail, kPolls, bar, parity, other, other_parity));
      tc_fence_after();
    };
    auto scores = [&](const Tile& t) {
      const uint32_t d = tm + (n_s & 1u) * 128;
      const Ring<KU> k0 = at, k1 = at.next();
      wait(&kfull[k0.slot], k0.phase);
      if (!t.eight && P == 2) wait(&kfull[k1.slot], k1.phase);
      if (!ok) return;
      const uint32_t kb = kr + (uint32_t)k0.slot * kUnit;
      if (t.eight) {
        const uint64_t desc = DH == 128 ? sw128_desc(kb) : sw64_desc(kb);
#pragma unroll
        for (int p = 1; p >= 0; --p)             // the low part first
#pragma unroll
          for (int ks = 0; ks < DH / 32; ++ks)
            mma_ts_e4m3(lead, d, tm + kColQ8 + (uint32_t)(p * (DH / 4) + ks * 8), desc + 2 * ks, id8,
                        (p == 0 || ks > 0) ? 1u : 0u);
      } else {
        const uint32_t kb1 = kr + (uint32_t)k1.slot * kUnit;
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks)
          tree_mma_ts(lead, d, tm + kColQ16 + (uint32_t)ks * 8, sw128_desc(ks < 4 ? kb : kb1) + 2 * (ks & 3), id16,
                      ks > 0 ? 1u : 0u);
      }
      tree_commit(lead, &sfull[n_s & 1u]);
      tree_commit(lead, &kempty[k0.slot]);
      at = at.next();
      if (!t.eight && P == 2) {
        tree_commit(lead, &kempty[k1.slot]);
        at = at.next();
      }
      ++n_s;
    };
    for (long long pos = plan.begin; ok && pos < plan.end; ++segments) {
      const Segment s = segment_at(a, plan, pos);
      wait(qready, (uint32_t)(segments & 1));
      if (ok) scores(tile_at(s.r, s.i0));
      for (int i = 0; ok && i < s.n; ++i) {
        if (i + 1 < s.n) scores(tile_at(s.r, s.i0 + i + 1));
        if (!ok) break;
        const uint32_t buf = n_p & 1u, ph = (n_p >> 1) & 1u;
        wait(&wfull[buf], ph, &pready[buf], ph);
        if (!ok) break;
        const uint32_t vb = wr + buf * (uint32_t)X::kWide;
        const bool eight = tile_at(s.r, s.i0 + i).eight;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tree_mma_ts(lead, tm + kColO, tm + buf * 128 + 8 * ks, mn_desc(vb + ks * 2048), eight ? idp8 : idp16,
                      (i > 0 || ks > 0) ? 1u : 0u);
        tree_commit(lead, &wempty[buf]);
        ++n_p;
      }
      pos += s.n;
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
    tree_commit(lead, mdone);
    mbar_wait_n(mdone, 0u, kPolls);
  } else if (warp >= 4) {
    // ---- V to bf16 in the products' layout
    const int cw = warp - 4, ct = tid - 128;
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      if (plan.first[b + 1] != plan.first[b]) continue;
      // a sequence without tokens, or without sense
      const float x = seq_range(a, plan.length[b], plan.count[b], plan.held[b]).count < 0 ? NAN : 0.f;
      const uint32_t w = pack_bf16x2(x, x);
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)b * a.T * a.H * DH);
      for (size_t i = ct; i < (size_t)a.T * a.H * DH / 8; i += 128) o[i] = make_uint4(w, w, w, w);
    }
    Ring<VU> at;
    uint32_t n = 0;
    bool ok = !tree_flagged(fail);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && tree_wait(fail, kPolls, bar, parity));
    };
    for (long long pos = plan.begin; ok && pos < plan.end;) {
      const Segment s = segment_at(a, plan, pos);
      for (int i = 0; ok && i < s.n; ++i, ++n) {
        const Tile t = tile_at(s.r, s.i0 + i);
        const bool edge = has_edge(a, s.r, t);
        const uint32_t buf = n & 1u;
        unsigned char* to = wide + buf * X::kWide;
        wait_w(&vfull[at.slot], at.phase);
        if (ok && n >= 2) wait_w(&wempty[buf], ((n >> 1) & 1u) ^ 1u);
        if (!ok) break;
        bool bad = false;
        const uint32_t exponent = t.eight ? 0x7c007c00u : 0x7f807f80u;
        auto fix = [&](uint4& x, int kd) {
          if (kd == 0) x = make_uint4(0u, 0u, 0u, 0u);
          if (kd == 1) {
            x.x = finite_only(x.x, exponent, bad);
            x.y = finite_only(x.y, exponent, bad);
            x.z = finite_only(x.z, exponent, bad);
            x.w = finite_only(x.w, exponent, bad);
          }
        };
        if (t.eight) {
          // eight lanes read 16 bytes each of two rows four apart, and write the
          // first half of theirs while the others write the second: all banks
          const unsigned char* from = vring + at.slot * kUnit;
          const int c = lane & 3, half = (lane >> 2) & 1, kq = lane >> 3;
          uint32_t most = 0;
          uint4 xs[4 * P];
#pragma unroll
          for (int it = 0; it < 4 * P; ++it) {
            const int panel = P == 2 ? it & 1 : 0, key = cw * 32 + (P == 2 ? it >> 1 : it) * 8 + kq + 4 * half;
            const int off = DH == 128 ? key * 128 + (((panel * 4 + c) ^ (key & 7)) << 4)
                                      : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
            xs[it] = *reinterpret_cast<const uint4*>(from + off);
          }
          auto store = [&](int it, const uint4& lo, const uint4& hi) {
            const int panel = P == 2 ? it & 1 : 0, key = cw * 32 + (P == 2 ? it >> 1 : it) * 8 + kq + 4 * half;
            unsigned char* row = to + panel * kUnit + key * 128;
            const int a0 = ((2 * c) ^ (key & 7)) << 4, a1 = ((2 * c + 1) ^ (key & 7)) << 4;
            *reinterpret_cast<uint4*>(row + (half ? a1 : a0)) = half ? hi : lo;
            *reinterpret_cast<uint4*>(row + (half ? a0 : a1)) = half ? lo : hi;
          };
#pragma unroll
          for (int it = 0; it < 4 * P; ++it) {
            const uint4 x = xs[it];
            const uint4 lo = make_uint4(widen<0>(x.x), widen<2>(x.x), widen<0>(x.y), widen<2>(x.y));
            const uint4 hi = make_uint4(widen<0>(x.z), widen<2>(x.z), widen<0>(x.w), widen<2>(x.w));
            most = larger(larger(larger(larger(most, lo.x), lo.y), lo.z), lo.w);
            most = larger(larger(larger(larger(most, hi.x), hi.y), hi.z), hi.w);
            store(it, lo, hi);
          }
          if (edge || (most & 0xffffu) >= kWideNan || most >> 16 >= kWideNan) {
#pragma unroll 1
            for (int it = 0; it < 4 * P; ++it) {
              const int panel = P == 2 ? it & 1 : 0, key = cw * 32 + (P == 2 ? it >> 1 : it) * 8 + kq + 4 * half;
              const int off = DH == 128 ? key * 128 + (((panel * 4 + c) ^ (key & 7)) << 4)
                                        : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
              const uint4 x = *reinterpret_cast<const uint4*>(from + off);
              uint4 lo = make_uint4(with_nan(widen<0>(x.x)), with_nan(widen<2>(x.x)), with_nan(widen<0>(x.y)),
                                    with_nan(widen<2>(x.y)));
              uint4 hi = make_uint4(with_nan(widen<0>(x.z)), with_nan(widen<2>(x.z)), with_nan(widen<0>(x.w)),
                                    with_nan(widen<2>(x.w)));
              const int kd = row_kind(a, s.r, t, t.p0 + key);
              fix(lo, kd);
              fix(hi, kd);
              store(it, lo, hi);
            }
          }
          mbar_arrive_cta(&vempty[at.slot]);
          at = at.next();
        } else {
#pragma unroll 1
          for (int u = 0; ok && u < P; ++u) {
            if (u) wait_w(&vfull[at.slot], at.phase);
            if (!ok) break;
            const unsigned char* from = vring + at.slot * kUnit;
#pragma unroll
            for (int it = 0; it < 8; ++it) {
              const int off = (it * 128 + ct) * 16;
              uint4 x = *reinterpret_cast<const uint4*>(from + off);
              fix(x, row_kind(a, s.r, t, t.p0 + (off >> 7)));
              *reinterpret_cast<uint4*>(to + u * kUnit + off) = x;
            }
            mbar_arrive_cta(&vempty[at.slot]);
            at = at.next();
          }
          if (!ok) break;
        }
        if (bad) atomicExch(odd, 1);
        fence_proxy_async_smem();
        mbar_arrive_cta(&wfull[buf]);
      }
      pos += s.n;
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
  } else {
    // ---- softmax and results: one thread per row of a copy
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    const int copy = kCopies == 4 ? warp : kCopies == 2 ? warp >> 1 : 0;
    const int row = kCopies == 4 ? lane : kCopies == 2 ? (warp & 1) * 32 + lane : tid;
    const int key0 = copy * NCH * 32;            // the thread's first key of a tile
    const bool live = row < rows;
    const bool warp_live = row - lane < rows;
    const int tok = live ? row / a.G : 0, g = live ? row - tok * a.G : 0;
    const int nblk = a.max_seq / a.block, shift = 31 - __clz(a.block);
    uint32_t n = 0;                              // tiles so far
    int4 go_on = make_int4(-1, 0, 0, 0);
    bool ok = !tree_flagged(fail);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && tree_wait(fail, kPolls, bar, parity));
      if (!ok && lane == 0) atomicExch(fail, 1);
      tc_fence_after();
    };
    // The products P V of the first `done` tiles: those of the last but two are
    // done (the scores that followed them are here), so that the last one's barrier
    // has one phase at most to go and its parity tells.
    auto wait_values = [&](uint32_t done) { wait_w(&wempty[(done - 1) & 1u], ((done - 1) >> 1) & 1u); };
    for (long long at = plan.begin; ok && at < plan.end;) {
      const Segment s = segment_at(a, plan, at);
      const int pos = s.r.length + tok;          // the row's own place
      const size_t out_row = ((size_t)(s.b * (long long)a.T + tok) * a.H + s.h * a.G + g) * DH;
      const bool present = live && tok < s.r.count;
      // ---- the query's parts: bf16, and e4m3 twice under a power of two
      float c16, c8;
      {
        uint32_t q[DH / 2];
        const uint4* src = reinterpret_cast<const uint4*>(a.q + out_row);
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < DH / 8; ++i) {
          const uint4 x = present ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          q[4 * i] = x.x;
          q[4 * i + 1] = x.y;
          q[4 * i + 2] = x.z;
          q[4 * i + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < DH / 2; ++i) most = __vmaxu2(most, q[i] & 0x7fff7fffu);
        most = max(most & 0xffffu, most >> 16);
        const int e = min(134 - (int)(most >> 7), 120);  // |q| 2^e below 256
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        const bool sane = most < 0x7f80u;
        c16 = sane ? a.scale_log2 : NAN;
        c8 = sane ? a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23) : NAN;
#pragma unroll
        for (int i = 0; i < DH / 2; i += 32) {
          uint32_t x[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = a.negate ? q[i + k] ^ 0x80008000u : q[i + k];
          tmem_st32(trow + kColQ16 + i, x);
        }
#pragma unroll
        for (int i = 0; i < DH / 4; i += 16) {
          uint32_t p0[16], p1[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            uint32_t w0 = 0, w1 = 0;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t w = a.negate ? q[2 * (i + k) + z] ^ 0x80008000u : q[2 * (i + k) + z];
              const float2 f = make_float2(bf16_lo(w) * up, bf16_hi(w) * up);
              const uint32_t h = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
              const __half2 b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h, __NV_E4M3);
              const float2 d = __half22float2(b);
              const uint32_t l =
                  __nv_cvt_float2_to_fp8x2(make_float2(f.x - d.x, f.y - d.y), __NV_SATFINITE, __NV_E4M3);
              w0 |= h << (16 * z);
              w1 |= l << (16 * z);
            }
            p0[k] = w0;
            p1[k] = w1;
          }
          tmem_st16(trow + kColQ8 + i, p0);
          tmem_st16(trow + kColQ8 + DH / 4 + i, p1);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_cta(qready);
      }
      // ---- tiles
      // O holds sums of 2^(score - m) v 2^-1 / vref: P has 2^7 of it and fp16 V 2^-8,
      // bf16 P 2^-1 by itself
      float m = -INFINITY, l = 0.f, vref = 0.f;
      const float* kscale = a.k_scale + (size_t)s.b * a.scale_stride + (size_t)s.h * nblk;
      const float* vscale = a.v_scale + (size_t)s.b * a.scale_stride + (size_t)s.h * nblk;
      float ks[NCH], vs[NCH];                    // of the tile to come
      auto fetch = [&](const Tile& t) {
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
          ks[q] = vs[q] = 1.f;
          if (t.eight) {
            const int blk = min((t.p0 + key0 + 32 * q) >> shift, nblk - 1);
            ks[q] = kscale[blk];
            vs[q] = vscale[blk];
          }
        }
      };
      Tile t = tile_at(s.r, s.i0);
      fetch(t);
      for (int i = 0; i < s.n; ++i, ++n) {
        const uint32_t buf = n & 1u;
        const uint32_t scol = trow + buf * 128;
        float c[NCH], v[NCH];
#pragma unroll
        for (int q = 0; q < NCH; ++q) {
          // (a scale of 0 must not meet the minus infinity of a key that is not
          // seen; scales below 0 are none)
          c[q] = t.eight ? (ks[q] >= 0.f ? fmaxf(c8 * ks[q], 1.2e-38f) : NAN) : c16;
          if (!(c8 == c8)) c[q] = NAN;
          v[q] = vs[q];
        }
        const Tile now = t;
        const bool edge = has_edge(a, s.r, now);
        if (i + 1 < s.n) {
          t = tile_at(s.r, s.i0 + i + 1);
          fetch(t);
        }
        wait_w(&sfull[buf], (n >> 1) & 1u);
        if (!ok) break;
        if (warp_live) {
          constexpr int kKept = NCH <= 2 ? NCH : 1;
          uint32_t sr[kKept][32];
          float bm = -INFINITY;
#pragma unroll
          for (int q = 0; q < NCH; ++q) {
            uint32_t(&x)[32] = sr[q % kKept];
            tmem_ld32_nw(scol + key0 + 32 * q, x);
            tmem_wait_ld();
            tmem_pin32(x);
            if (edge) {
              const uint32_t seen = present ? seen_bits(a, now, pos, now.p0 + key0 + 32 * q) : 0u;
              if (seen == 0u) {
                c[q] = 1.2e-38f;
                v[q] = 0.f;
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((seen >> e) & 1u)) x[e] = 0xff800000u;
              if (NCH > 2) tmem_st32(scol + key0 + 32 * q, x);
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx[(e >> 1) & 1] = tree_max3(mx[(e >> 1) & 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            bm = fmaxf(bm, fmaxf(mx[0], mx[1]) * c[q]);
          }
          if (NCH > 2 && edge) tmem_wait_st();
          const bool raise = bm > m + kRaise || (m == -INFINITY && bm > -INFINITY);
          float over = 0.f;                      // the largest scale over vref
#pragma unroll
          for (int q = 0; q < NCH; ++q)
            if (now.eight && fabsf(v[q]) > fmaxf(vref, over) && fabsf(v[q]) < 0x1p100f) over = fabsf(v[q]);
          if (__any_sync(0xffffffffu, raise || over > 0.f || vref == 0.f)) {
            float corr = raise ? tree_ex2(m - bm) : 1.f;
            if (raise) m = bm;
            l *= corr;
            if (over > 0.f || vref == 0.f) {
              const float next = over > 0.f ? power_above(over) * 4.f : 1.f;
              corr *= vref / next;               // (both are powers of two, or 0 at the start)
              vref = next;
            }
            if (i > 0) {
              wait_values(n);                    // O as the tile before left it
              if (!ok) break;
#pragma unroll 1
              for (int q = 0; q < DH / 16; ++q) {
                uint32_t o[16];
                tmem_ld16_nw(trow + kColO + q * 16, o);
                tmem_wait_ld();
                tmem_pin16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st16(trow + kColO + q * 16, o);
              }
            }
          }
          const float nm = m == -INFINITY ? 0.f : -m, unit = (now.eight ? 0x1p7f : 0x1p-1f) / vref;
          const uint64_t nm2 = tree_pack2(__float_as_uint(nm), __float_as_uint(nm));
          uint64_t ls2[2] = {0, 0};
          auto weights = [&](auto eight) {
#pragma unroll
            for (int q = 0; q < NCH; ++q) {
              uint32_t(&x)[32] = sr[q % kKept];
              if (NCH > 2) {
                tmem_ld32_nw(scol + key0 + 32 * q, x);
                tmem_wait_ld();
                tmem_pin32(x);
              }
              const uint64_t c2 = tree_pack2(__float_as_uint(c[q]), __float_as_uint(c[q]));
              const float pv = v[q] * unit;
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float p0, p1;
                tree_unpack2(tree_fma2(tree_pack2(x[2 * e], x[2 * e + 1]), c2, nm2), p0, p1);
                p0 = tree_ex2(p0);
                p1 = tree_ex2(p1);
                ls2[e & 1] = tree_add2(ls2[e & 1], tree_pack2(__float_as_uint(p0), __float_as_uint(p1)));
                pk[e] = decltype(eight)::value ? pack_f16x2(p0 * pv, p1 * pv) : pack_bf16x2(p0 * pv, p1 * pv);
              }
              tmem_st16(scol + (key0 + 32 * q) / 2, pk);
            }
          };
          if (now.eight) weights(std::true_type());
          else weights(std::false_type());
          // the other copies' keys
          if (kCopies > 1) {
            const uint32_t zero[16] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q * 32 < key0 || q * 32 >= key0 + NCH * 32) tmem_st16(scol + q * 16, zero);
          }
          float l0, l1;
          tree_unpack2(tree_add2(ls2[0], ls2[1]), l0, l1);
          l += l0 + l1;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive_cta(&pready[buf]);
      }
      if (!ok) break;
      // ---- the run's result: final, or a part of the pair's
      wait_values(n);
      if (!ok) break;
      const bool bad = tree_flagged(odd);
      const long long slot = (long long)blockIdx.x * 2 + (s.head ? 0 : 1);
      if (!s.whole && at + s.n == plan.end && s.i0 + s.n < (int)(plan.first[s.b + 1] - plan.first[s.b]) && !s.head) {
        // the pair's last tile: which CTA has it
        const long long last = plan.first[s.b] * a.Hkv +
                               (long long)(s.h + 1) * (plan.first[s.b + 1] - plan.first[s.b]) - 1;
        go_on = make_int4(s.b, s.h, plan.owner(last), 0);
      }
      float* po = a.part_o + (size_t)slot * rows * DH;
      float* pm = a.part_m + (size_t)slot * rows;
      float* pl = a.part_l + (size_t)slot * rows;
      if (kCopies == 1) {
        if (warp_live) {
          const float inv = vref * 2.f * (s.whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f);
          if (live && !s.whole) {
            pm[row] = m;
            pl[row] = l;
          }
#pragma unroll 1
          for (int q = 0; q < DH / 32; ++q) {
            uint32_t o[32];
            tmem_ld32_nw(trow + kColO + q * 32, o);
            tmem_wait_ld();
            tmem_pin32(o);
            if (!live) continue;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = present ? __uint_as_float(o[e + k]) * inv : 0.f;
              if (bad && present) add_not_finite(a, s, pos, q * 32 + e, 8, w);
              if (s.whole) {
                *reinterpret_cast<uint4*>(a.out + out_row + q * 32 + e) =
                    make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]),
                               pack_bf16x2(w[6], w[7]));
              } else {
                float4* d = reinterpret_cast<float4*>(po + (size_t)row * DH + q * 32 + e);
                d[0] = make_float4(w[0], w[1], w[2], w[3]);
                d[1] = make_float4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
      } else {
        // the copies of a row, under the largest of their maxima
        constexpr int kRows = 128 / kCopies;
        xm[tid] = m;
        xl[tid] = l;
        bar_softmax();
        float all = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) all = fmaxf(all, xm[k * kRows + row]);
        const float base = all == -INFINITY ? 0.f : all;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) sum += xl[k * kRows + row] * tree_ex2(xm[k * kRows + row] - base);
        const float w0 = tree_ex2(m - base) * (vref * 2.f);
        if (copy == 0) {
          row_m[row] = all;
          row_l[row] = sum;
          if (live && !s.whole) {
            pm[row] = all;
            pl[row] = sum;
          }
        }
#pragma unroll 1
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t o[32];
          tmem_ld32_nw(trow + kColO + q * 32, o);
          tmem_wait_ld();
          tmem_pin32(o);
          float* mine = merge + warp * 32 * 33 + lane * 33;
#pragma unroll
          for (int e = 0; e < 32; ++e) mine[e] = m == -INFINITY ? 0.f : __uint_as_float(o[e]) * w0;
          bar_softmax();
#pragma unroll
          for (int z = 0; z < kRows / 32; ++z) {
            const int rr = z * 32 + tid / 4, e0 = (tid & 3) * 8;
            if (rr < rows) {
              const int tk = rr / a.G, gg = rr - tk * a.G;
              const float lt = row_l[rr], inv = s.whole ? (lt != 0.f ? 1.f / lt : 0.f) : 1.f;
              const bool here = tk < s.r.count;
              float w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < kCopies; ++k) x += merge[(k * kRows + rr) * 33 + e0 + e];
                w[e] = here ? x * inv : 0.f;
              }
              if (bad && here) add_not_finite(a, s, s.r.length + tk, q * 32 + e0, 8, w);
              if (s.whole) {
                bf16* o8 = a.out + ((size_t)(s.b * (long long)a.T + tk) * a.H + s.h * a.G + gg) * DH + q * 32 + e0;
                *reinterpret_cast<uint4*>(o8) = make_uint4(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]),
                                                           pack_bf16x2(w[4], w[5]), pack_bf16x2(w[6], w[7]));
              } else {
                float4* d = reinterpret_cast<float4*>(po + (size_t)rr * DH + q * 32 + e0);
                d[0] = make_float4(w[0], w[1], w[2], w[3]);
                d[1] = make_float4(w[4], w[5], w[6], w[7]);
              }
            }
          }
          bar_softmax();
        }
      }
      at += s.n;
    }
    if (tid == 0) a.shared[blockIdx.x] = go_on;
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  // a wait gave up: none of the CTA's rows is sure
  if (tree_flagged(fail))
    for (long long at = plan.begin; at < plan.end;) {
      const Segment s = segment_at(a, plan, at);
      const long long slot = (long long)blockIdx.x * 2 + (s.head ? 0 : 1);
      if (!s.whole && !s.head && tid == 0) {
        const long long n = plan.first[s.b + 1] - plan.first[s.b];
        const long long last = plan.first[s.b] * a.Hkv + (long long)(s.h + 1) * n - 1;
        a.shared[blockIdx.x] = make_int4(s.b, s.h, plan.owner(last), 0);
      }
      for (int i = tid; i < rows * DH; i += kThreads) {
        const int r = i / DH, tk = r / a.G;
        if (s.whole) {
          if (tk < s.r.count)
            a.out[((size_t)(s.b * (long long)a.T + tk) * a.H + s.h * a.G + r % a.G) * DH + i % DH] = __float2bfloat16(NAN);
        } else if (i % DH == 0) {
          a.part_m[slot * rows + r] = 0.f;
          a.part_l[slot * rows + r] = NAN;
        }
      }
      at += s.n;
    }
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins a pair that several CTAs share: CTA x = the first of them, thread = 16
// bytes of a row's output; the parts are added in order, four in flight.
constexpr int kJoinThreads = 256;
template <int DH>
__global__ void __launch_bounds__(kJoinThreads) cache_attn_join_kernel(const __grid_constant__ CacheAttnArgs a) {
  pdl_wait();
  const int4 pair = a.shared[blockIdx.x];
  const int rows = a.T * a.G, i = blockIdx.y * kJoinThreads + threadIdx.x;
  const int row = i / (DH / 4), col = i % (DH / 4) * 4;
  if (pair.x < 0 || row >= rows) return;
  const int c0 = blockIdx.x, n = pair.z - c0 + 1;
  // the first CTA's second place, the others' first
  auto place = [&](int k) { return k == 0 ? (size_t)c0 * 2 + 1 : (size_t)(c0 + k) * 2; };
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    float pm[kBatch], pl[kBatch], mn = m;
    float4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool got = k0 + u < n;
      const size_t at = got ? place(k0 + u) * rows + row : 0;
      pm[u] = got ? a.part_m[at] : -INFINITY;
      pl[u] = got ? a.part_l[at] : 0.f;
      v[u] = got ? *reinterpret_cast<const float4*>(a.part_o + at * DH + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, pm[u]);
    const float base = mn == -INFINITY ? 0.f : mn, old = exp2f(m - base);
    l *= old;
    o.x *= old;
    o.y *= old;
    o.z *= old;
    o.w *= old;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (k0 + u >= n) break;
      const float w = exp2f(pm[u] - base);
      l = fmaf(pl[u], w, l);
      o.x = fmaf(v[u].x, w, o.x);
      o.y = fmaf(v[u].y, w, o.y);
      o.z = fmaf(v[u].z, w, o.z);
      o.w = fmaf(v[u].w, w, o.w);
    }
    m = mn;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;    // (NaN where a wait gave up)
  const int tok = row / a.G;
  const size_t to = ((size_t)(pair.x * (long long)a.T + tok) * a.H + pair.y * a.G + row % a.G) * DH + col;
  *reinterpret_cast<uint2*>(a.out + to) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

template <int DH, int NCH>
cudaError_t launch(const CacheAttnArgs& a, const CUtensorMap (&m)[4], cudaStream_t st) {
  const size_t most = Shape<DH>::kSmem + 1024 + 8 * (kBatchMaxSeqs + 1) + 12 * kBatchMaxSeqs;
  const size_t smem = Shape<DH>::kSmem + 1024 + 8 * ((size_t)a.B + 1) + 12 * (size_t)a.B;
  static_assert(Shape<DH>::kSmem + 1024 + 20 * kBatchMaxSeqs + 8 <= 227 * 1024, "shared memory");
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e = cudaFuncSetAttribute(cache_attn_tc_kernel<DH, NCH>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    if (dv >= 0) ready[dv] = true;
  }
  cache_attn_tc_kernel<DH, NCH><<<a.ctas, kThreads, smem, st>>>(m[0], m[1], m[2], m[3], a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(a.ctas, (a.T * a.G * (DH / 4) + kJoinThreads - 1) / kJoinThreads);
  lc.blockDim = dim3(kJoinThreads);
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, cache_attn_join_kernel<DH>, a);
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
  const int rows = a.T * a.G;
  if (a.dh == 128)
    return rows <= 32 ? launch<128, 1>(a, m, s) : rows <= 64 ? launch<128, 2>(a, m, s) : launch<128, 4>(a, m, s);
  return rows <= 32 ? launch<64, 1>(a, m, s) : rows <= 64 ? launch<64, 2>(a, m, s) : launch<64, 4>(a, m, s);
}

}  // namespace ssd
