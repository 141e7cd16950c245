// Tree attention on the 5th-generation tensor cores: a tile of 128 query rows
// (row = node G + head of the group) against blocks of 128 keys.
//
//   S = (Q_hi + Q_lo) K^T   tcgen05, fp32 in tensor memory
//   P = 2^(S c - m)         one thread per row, bf16 over S's columns
//   O += P V                tcgen05, P from tensor memory, V as it lies in the
//                           cache (key-major: the MN-major operand form)
//
// Two streams of (S, P, O) share the matrix pipe: while one stream's softmax
// runs, the other's products are issued.  With up to 128 rows the streams
// take the key blocks in turn (both of the one tile); with more, each takes a
// tile of its own and the pair reads every key block once.  m is raised, and
// O rescaled, only when a block's maximum passes it by 8 (a factor of 256,
// which fp32 sums and bf16 probabilities carry without loss).  P is rounded to
// bf16, half a step of 2^-8 each like the output's own, because a second part of
// it would cost another product as large as the three; its sum is of the
// unrounded values in fp32.  The keys are split into units over the SMs; a
// second kernel joins the units' partial results in a fixed order.
//
// With many rows the matrix pipe bounds it: 256 nodes of 64 / 8 heads over
// 131000 rows are 1.65 TFLOP in three products of one size (Q_hi K, Q_lo K,
// P V), 854 us at the 1931 TFLOP/s that a library product reaches in a burst;
// from a graph it takes 846 to 880 us, as a pass among others 931 to 959, where
// the power limit lowers the clock.  With few rows it is a stream's chain (copy,
// product, softmax, product) and the first copy's latency: 61 nodes of 40 heads
// over 2047 rows take 15 us for 7 us of bytes.  A thread's 128 scores at the 168
// registers that ten warps leave spill 24 to 64 bytes.
//
// Warps 0-3 and 4-7: the streams' softmax; warp 8: TMA copies; warp 9: MMA.
// Every wait is bounded: one that gives up sets the CTA's flag and every role
// runs out; then the CTA's own rows become NaN, or, with several splits, all
// rows that are joined after it, and so do the weights.
#include "tc_dev.cuh"
#include "tree.cuh"
#include "tree_join.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kThreads = 320;
constexpr int kPolls = 1 << 22;
constexpr int kRegion = 128 * 128;              // [128 rows][64] bf16, 128-byte swizzle
constexpr int kTileSmem = 224 * 1024;           // Q tiles, then the ring of K / V blocks
// K / V blocks in flight beside the Q tiles (two planes each).
__host__ __device__ constexpr int ring_stages(int dh, bool two) {
  const int item = dh / 64 * kRegion, n = kTileSmem / item - (two ? 4 : 2);
  return n < 12 ? n : 12;
}
constexpr uint32_t kColO = 256;                 // TMEM: S0, S1 (P over each), O0, O1
constexpr float kRaise = 8.f;

SSD_DI void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// V block [128 keys][dh] in 64-column regions as the MN-major B operand: 64
// contiguous columns per atom (next atom one region on), 8 keys per 1024 bytes.
SSD_DI uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kRegion >> 4) << 16;           // leading offset: next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;              // stride offset: next 8 keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;                        // 128-byte swizzle
  return d;
}
__host__ __device__ constexpr uint32_t idesc_pv(int N) {
  return idesc_bf16(128, N) | (1u << 16);        // B is MN-major
}
// Block range of a unit and its place.
struct Unit {
  int kvh, item, split, b0, nb;
};
SSD_DI Unit unit_of(const TreeArgs& a, int u) {
  Unit x;
  // items fastest, then splits: CTAs that run together read the same keys
  const int r = u / a.items;
  x.item = u - r * a.items;
  x.kvh = r / a.splits;
  x.split = r - x.kvh * a.splits;
  // nb / splits blocks each, one more for the first nb % splits
  const int len = a.nb / a.splits, more = a.nb - len * a.splits;
  x.b0 = x.split * len + min(x.split, more);
  x.nb = len + (x.split < more);
  return x;
}

// Scores of keys that the row does not see become -infinity, in tensor memory:
// a condition within the softmax became selections on every block.
__device__ __noinline__ void mask_scores(uint32_t col, uint4 mask) {
#pragma unroll 1
  for (int q = 0; q < 4; ++q) {
    const uint32_t w = q == 0 ? mask.x : q == 1 ? mask.y : q == 2 ? mask.z : mask.w;
    uint32_t v[32];
    tmem_ld32_nw(col + (uint32_t)q * 32, v);
    tmem_wait_ld();
    tmem_pin32(v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((w >> e) & 1u)) v[e] = 0xff800000u;
    tmem_st32(col + (uint32_t)q * 32, v);
  }
  tmem_wait_st();
}

template <int DH, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap mK,
                        const __grid_constant__ CUtensorMap mV,
                        const __grid_constant__ CUtensorMap mW,
                        const __grid_constant__ TreeArgs a) {
  constexpr int kRegs = DH / 64;                 // 64-column regions per row block
  constexpr int kItem = kRegs * kRegion;         // bytes of a K or V block, or a Q plane
  constexpr int kTiles = TWO ? 2 : 1;            // Q tiles of a unit
  constexpr int kStages = ring_stages(DH, TWO);
  constexpr int kLag = TWO ? 1 : 2;              // K blocks ahead of their V block
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  float* xm = reinterpret_cast<float*>(sm + kTileSmem);  // stream 1's maxima and sums
  float* xl = xm + 128;
  uint64_t* bars = reinterpret_cast<uint64_t*>(xl + 128);
  uint64_t* qfull = bars;
  uint64_t* qfree = bars + 1;
  uint64_t* sfull = bars + 2;                    // [2] S written
  uint64_t* pready = bars + 4;                   // [2] P written, O rescaled
  uint64_t* ofull = bars + 6;                    // [2] the unit's last product done
  uint64_t* mdone = bars + 8;
  uint64_t* given = bars + 9;                    // stream 1's statistics written
  uint64_t* taken = bars + 10;                   // and its output read by stream 0
  uint64_t* full = bars + 11;                    // [stages]
  uint64_t* empty = full + kStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(empty + kStages);
  int* fail = reinterpret_cast<int*>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.T * a.G;
  unsigned char* ring = sm + kTiles * 2 * kItem;

  // (the copying thread itself: its first copies need not wait for the others)
  if (tid == 256) {
    mbar_init(qfull, 1);
    mbar_init(qfree, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pready[s], 128);
      mbar_init(&ofull[s], 1);
    }
    mbar_init(mdone, 1);
    mbar_init(given, 128);
    mbar_init(taken, 128);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    // (self-test: every role as after a wait that gave up; a limit of its own on
    // each wait took the largest trees 1 % longer)
    *fail = (int)blockIdx.x == a.give_up;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  auto set_up = [&]() {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return *reinterpret_cast<volatile uint32_t*>(tslot);
  };

  if (warp == 8) {
    // ---- copies, in the order in which the products use them: K of the first
    // kLag blocks, then V of block i and K of block i + kLag in turn
    Ring<kStages> at;
    int issued = 0, units = 0;                   // copies / units so far
    auto is_ctx = [&](const Unit& x, int i, int& b, bool& is_v) {
      const int pro = min(kLag, x.nb), mid = 2 * (x.nb - pro);
      if (i < pro) {
        b = i;
        is_v = false;
      } else if (i - pro < mid) {
        is_v = ((i - pro) & 1) == 0;
        b = (i - pro) / 2 + (is_v ? 0 : kLag);
      } else {
        is_v = true;
        b = mid / 2 + (i - pro - mid);
      }
      b += x.b0;
      return b < a.nb_ctx;
    };
    auto copy = [&](const Unit& x, int b, bool is_v, bool ctx) {
      mbar_arrive_expect_tx(&full[at.slot], (uint32_t)kItem);
      const CUtensorMap* m = !ctx ? &mW : is_v ? &mV : &mK;
      const int row = ctx ? b * kTreeKeys
                          : (is_v ? a.row_vt : a.row_kt) + x.kvh * a.T + (b - a.nb_ctx) * kTreeKeys;
      for (int r = 0; r < kRegs; ++r)
        tma_load_3d(ring + at.slot * kItem + r * kRegion, m, r * 64, row, ctx ? x.kvh : 0,
                    &full[at.slot]);
      ++issued;
      at = at.next();
    };
    // the first copies of context blocks need neither the others' set-up nor
    // the preparation
    int b;
    bool is_v;
    if (lane == 0) {
      const Unit x = unit_of(a, blockIdx.x);
      while (issued < min(kStages, 2 * x.nb) && is_ctx(x, issued, b, is_v)) copy(x, b, is_v, true);
    }
    __syncwarp();
    set_up();
    if (lane == 0) {
      pdl_wait();                                // the queries come from the preparation
      bool ok = (int)blockIdx.x != a.give_up;
      for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x, ++units) {
        const Unit x = unit_of(a, u);
        bool q_sent = false;
        auto send_q = [&]() {
          if (units > 0 && !mbar_wait_n(qfree, (uint32_t)((units - 1) & 1), kPolls)) return false;
          mbar_arrive_expect_tx(qfull, (uint32_t)(kTiles * 2 * kItem));
          for (int t = 0; t < kTiles; ++t)
            for (int p = 0; p < 2; ++p)
              for (int r = 0; r < kRegs; ++r)
                tma_load_3d(sm + (t * 2 + p) * kItem + r * kRegion, &mW, r * 64,
                            (p * a.Hkv + x.kvh) * rows + (x.item * kTiles + t) * 128, 0, qfull);
          q_sent = true;
          return true;
        };
        for (int i = units > 0 ? 0 : issued; ok && i < 2 * x.nb; ++i) {
          const bool ctx = is_ctx(x, i, b, is_v);
          // a later unit's first blocks go out before its queries' place is
          // free (the slots they wait for need no query of this unit)
          if (!q_sent && (units == 0 || i >= kLag)) ok = send_q();
          if (ok && issued >= kStages) ok = mbar_wait_n(&empty[at.slot], at.phase ^ 1u, kPolls);
          if (!ok || tree_flagged(fail)) {
            ok = false;
            break;
          }
          copy(x, b, is_v, ctx);
        }
        if (ok && !q_sent) ok = send_q();
        if (!q_sent) break;
      }
      if (!ok) atomicExch(fail, 1);
      // what is still in flight lands before the memory is released
      for (int i = max(0, issued - kStages); i < issued; ++i)
        mbar_wait_n(&full[i % kStages], (uint32_t)((i / kStages) & 1), kPolls);
      if (units > 0) mbar_wait_n(qfull, (uint32_t)((units - 1) & 1), kPolls);
    }
  } else if (warp == 9) {
    // ---- products: the warp runs together, one lane issues
    const uint32_t tmem = set_up();
    pdl_wait();                                  // bounded waits begin after it
    const uint32_t lead = tree_elect();
    constexpr uint32_t ids = idesc_bf16(128, 128), idp = idesc_pv(DH);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t qa = smem_addr(sm), ra = smem_addr(ring);
    Ring<kStages> at;                            // the next K or V block
    int units = 0;
    uint32_t pphase[2] = {0, 0};                 // of the streams' P tiles
    bool ok = (int)blockIdx.x != a.give_up;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_n(bar, phase, kPolls));
      tc_fence_after();
    };
    auto landed = [&](const Ring<kStages>& r) {
      wait(&full[r.slot], r.phase);
      return ra + (uint32_t)r.slot * kItem;
    };
    auto scores = [&](int s, uint32_t kb) {
      const uint32_t q = qa + (uint32_t)(TWO ? s : 0) * 2 * kItem;
#pragma unroll
      for (int p = 1; p >= 0; --p)               // the low part first
#pragma unroll
        for (int ks = 0; ks < DH / 16; ++ks) {
          const uint32_t rg = (uint32_t)(ks >> 2) * kRegion;
          tree_mma_ss(lead, tm + (uint32_t)s * 128, sw128_desc(q + p * kItem + rg) + 2 * (ks & 3),
                      sw128_desc(kb + rg) + 2 * (ks & 3), ids, (p == 0 || ks > 0) ? 1u : 0u);
        }
      tree_commit(lead, &sfull[s]);
    };
    auto values = [&](int s, uint32_t vb, uint32_t acc) {
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        tree_mma_ts(lead, tm + kColO + (uint32_t)s * 128, tm + (uint32_t)s * 128 + 8 * ks,
                    mn_desc(vb + ks * 2048), idp, ks > 0 ? 1u : acc);
    };
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x, ++units) {
      const Unit x = unit_of(a, u);
      wait(qfull, (uint32_t)(units & 1));
      // the streams' block counts; a pair's second tile may lie beyond the rows
      const int cnt0 = TWO ? x.nb : (x.nb + 1) / 2;
      const int cnt1 = TWO ? (x.item * 2 + 1 < a.tiles ? x.nb : 0) : x.nb / 2;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!ok || !(s ? cnt1 : cnt0)) continue;
        const uint32_t kb = landed(at);
        if (!ok) continue;
        scores(s, kb);
        if (!TWO || s == 1 || !cnt1) {
          tree_commit(lead, &empty[at.slot]);
          at = at.next();
        }
      }
      for (int j = 0; ok && j < cnt0; ++j) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int cnt = s ? cnt1 : cnt0;
          if (!ok || j >= cnt) continue;
          // two tiles: V of block j and K of block j + 1 stay for both streams
          const bool last_user = !TWO || s == 1 || !cnt1, more = j + 1 < cnt;
          const Ring<kStages> v = at, k = at.next();
          const uint32_t vb = landed(v);
          wait(&pready[s], pphase[s]);
          pphase[s] ^= 1u;
          ok = __all_sync(0xffffffffu, ok && !tree_flagged(fail));
          if (!ok) continue;
          values(s, vb, j > 0 ? 1u : 0u);
          if (last_user) tree_commit(lead, &empty[v.slot]);
          if (!more) {
            tree_commit(lead, &ofull[s]);
            if (last_user) at = k;
            continue;
          }
          const uint32_t kb = landed(k);
          if (!ok) continue;
          scores(s, kb);
          if (last_user) {
            tree_commit(lead, &empty[k.slot]);
            at = k.next();
          }
        }
      }
      tree_commit(lead, qfree);
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
    tree_commit(lead, mdone);
    mbar_wait_n(mdone, 0u, kPolls);
  } else {
    // ---- softmax: stream s, one thread per row of its tile
    const uint32_t tmem = set_up();
    pdl_wait();
    const int s = warp >> 2, r = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t col_s = (uint32_t)s * 128, col_o = kColO + (uint32_t)s * 128;
    const float scale = a.scale_log2;
    int n_s = 0, n_own = 0, n_other = 0, units = 0;
    auto wait_w = [&](uint64_t* bar, uint32_t parity) -> bool {
      bool okw = !tree_flagged(fail) && mbar_wait_n(bar, parity, kPolls);
      okw = __all_sync(0xffffffffu, okw);
      if (!okw && lane == 0) atomicExch(fail, 1);
      return okw;
    };
    bool ok = true;
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x, ++units) {
      const Unit x = unit_of(a, u);
      const int tile = TWO ? x.item * 2 + s : x.item;
      const int cnt = TWO ? (tile < a.tiles ? x.nb : 0) : (x.nb + 1 - s) / 2;
      const int row = tile * 128 + r;
      const bool live = row < rows;
      const bool warp_live = tile * 128 + (r & ~31) < rows;
      const int t = live ? row / a.G : 0;
      const uint32_t* anc = a.anc + (size_t)t * a.anc_words;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < cnt; ++j) {
        ok = wait_w(&sfull[s], (uint32_t)(n_s++ & 1));
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          const int b = x.b0 + (TWO ? j : 2 * j + s);
          const int left = a.n - b * kTreeKeys;  // context keys from this block on
          if (b >= a.nb_ctx || left < kTreeKeys) {
            uint4 mask;
            if (b >= a.nb_ctx) {
              mask = live ? *reinterpret_cast<const uint4*>(anc + 4 * (b - a.nb_ctx))
                          : make_uint4(0u, 0u, 0u, 0u);
            } else {
              auto low = [&](int w) {
                const int k = left - 32 * w;
                return k >= 32 ? ~0u : (k > 0 ? (1u << k) - 1u : 0u);
              };
              mask = make_uint4(low(0), low(1), low(2), low(3));
            }
            mask_scores(trow + col_s, mask);
          }
          uint32_t sr[4][32];
#pragma unroll
          for (int q = 0; q < 2; ++q) tmem_ld32_nw(trow + col_s + q * 32, sr[q]);
          // the second half loads while the first half's maximum is taken
          tmem_wait_ld();
          tmem_pin32(sr[0]);
          tmem_pin32(sr[1]);
#pragma unroll
          for (int q = 2; q < 4; ++q) tmem_ld32_nw(trow + col_s + q * 32, sr[q]);
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int hlf = 0; hlf < 2; ++hlf) {
            if (hlf == 1) {
              tmem_wait_ld();
              tmem_pin32(sr[2]);
              tmem_pin32(sr[3]);
            }
#pragma unroll
            for (int q = 2 * hlf; q < 2 * hlf + 2; ++q)
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                mx[(e >> 1) & 3] = tree_max3(mx[(e >> 1) & 3], __uint_as_float(sr[q][e]),
                                        __uint_as_float(sr[q][e + 1]));
          }
          const float bm = fmaxf(tree_max3(mx[0], mx[1], mx[2]), mx[3]) * scale;
          const bool raise = bm > m + kRaise || (m == -INFINITY && bm > -INFINITY);
          if (__any_sync(0xffffffffu, raise)) {
            const float corr = raise ? tree_ex2(m - bm) : 1.f;
            if (raise) m = bm;
            l *= corr;
            if (j > 0) {  // the stream's products so far are done: S followed them
#pragma unroll 1
              for (int q = 0; q < DH / 16; ++q) {
                uint32_t o[16];
                tmem_ld16_nw(trow + col_o + q * 16, o);
                tmem_wait_ld();
                tmem_pin16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st16(trow + col_o + q * 16, o);
              }
            }
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          const uint64_t sc2 = tree_pack2(__float_as_uint(scale), __float_as_uint(scale));
          const uint64_t nm2 = tree_pack2(__float_as_uint(nm), __float_as_uint(nm));
          uint64_t ls2[2] = {0, 0};              // pairs of partial sums
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
            if (!TWO && a.part_s && live) {      // between the exponentials
              float4* ps = reinterpret_cast<float4*>(
                  a.part_s + (((size_t)x.kvh * a.nb + b) * rows + row) * kTreeKeys + q * 32);
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                ps[e >> 2] = make_float4(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1]),
                                         __uint_as_float(sr[q][e + 2]), __uint_as_float(sr[q][e + 3]));
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              tree_unpack2(tree_fma2(tree_pack2(sr[q][2 * e], sr[q][2 * e + 1]), sc2, nm2), p0, p1);
              p0 = tree_ex2(p0);
              p1 = tree_ex2(p1);
              ls2[e & 1] = tree_add2(ls2[e & 1], tree_pack2(__float_as_uint(p0), __float_as_uint(p1)));
              pk[e] = pack_bf16x2(p0, p1);
            }
            tmem_st16(trow + col_s + q * 16, pk);
          }
          float l0, l1;
          tree_unpack2(tree_add2(ls2[0], ls2[1]), l0, l1);
          l += l0 + l1;
          tmem_wait_st();
        }
        if (!TWO && s == 1 && j == 0 && units > 0) {
          // the unit before has been read: its first product may start
          ok = wait_w(taken, (uint32_t)((units - 1) & 1));
          if (!ok) break;
        }
        tc_fence_before();
        mbar_arrive_cta(&pready[s]);
      }
      if (!ok) break;
      // ---- the unit's result: a tile's two streams are joined (the other
      // stream's output lies in the same lanes), a pair's are two tiles
      const int cnt1 = x.nb / 2;                 // of stream 1, one tile
      const bool last = a.splits == 1;           // the row's final result
      const bool present = last && live && a.depth[t] >= 0;
      const bool bad = last && any_bad(a, x.kvh, lane);
      if (cnt > 0) ok = wait_w(&ofull[s], (uint32_t)(n_own++ & 1));
      if (!ok) break;
      if (!TWO && s == 1) {
        if (cnt == 0 && units > 0) {             // (no first product that waited)
          ok = wait_w(taken, (uint32_t)((units - 1) & 1));
          if (!ok) break;
        }
        xm[r] = m;
        xl[r] = l;
        mbar_arrive_cta(given);
        continue;
      }
      float w0 = 1.f, w1 = 0.f;
      if (!TWO) {
        if (cnt1 > 0) ok = wait_w(&ofull[1], (uint32_t)(n_other++ & 1));
        ok = ok && wait_w(given, (uint32_t)(units & 1));
        if (!ok) break;
        const float m1 = xm[r], mn = fmaxf(m, m1), base = mn == -INFINITY ? 0.f : mn;
        w0 = tree_ex2(m - base);
        w1 = tree_ex2(m1 - base);
        l = l * w0 + xl[r] * w1;
        m = mn;
      }
      tc_fence_after();
      if (warp_live) {
        const bool both = !TWO && cnt1 > 0;
        const int slot = TWO ? (x.kvh * a.splits + x.split) * (a.items * 2) + tile
                             : x.kvh * a.splits + x.split;
        float* po = a.part_o + (size_t)slot * DH * 128 + (size_t)r * 4;
        float lse = INFINITY, inv = 0.f;
        if (last) {
          lse = l != 0.f ? m + log2f(l) : INFINITY;
          inv = l != 0.f ? 1.f / l : 0.f;
        }
        bf16* out = a.out + ((size_t)t * a.H + x.kvh * a.G + row % a.G) * DH;
#pragma unroll 1
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t o[32];
          if (cnt > 0) {
            tmem_ld32_nw(trow + col_o + q * 32, o);
            tmem_wait_ld();
            tmem_pin32(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (both) {
            uint32_t o1[32];
            tmem_ld32_nw(trow + col_o + 128 + q * 32, o1);
            tmem_wait_ld();
            tmem_pin32(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * w0 + __uint_as_float(o1[e]) * w1);
          }
          if (!live) continue;
          if (!last) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(po + (size_t)(q * 8 + e) * 512) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            continue;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = present ? __uint_as_float(o[e + i]) * inv : 0.f;
            if (bad && present) add_bad<DH>(a, x.kvh, row, t, lse, q * 32 + e, v, 8);
            *reinterpret_cast<uint4*>(out + q * 32 + e) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          }
        }
        if (live && last) a.lse[(size_t)x.kvh * rows + row] = present ? lse : INFINITY;
        if (live && !last) {
          a.part_m[(size_t)slot * 128 + r] = m;
          a.part_l[(size_t)slot * 128 + r] = l;
        }
      }
      tc_fence_before();
      if (!TWO) mbar_arrive_cta(taken);
    }
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && tree_flagged(fail)) atomicExch(a.err, 1);
  // a wait gave up: one split's rows are final, and none of the CTA's is sure
  if (a.splits == 1 && tree_flagged(fail))
    for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
      const Unit x = unit_of(a, u);
      for (int i = tid; i < kTiles * 128 * DH; i += kThreads) {
        const int row = x.item * kTiles * 128 + i / DH;
        if (row < rows)
          a.out[((size_t)(row / a.G) * a.H + x.kvh * a.G + row % a.G) * DH + i % DH] = __float2bfloat16(NAN);
      }
    }
  if (warp == 0) tmem_dealloc(*tslot, 512);
}

// Weights from scores: thread = key, two blocks of 128 keys per CTA; the
// rows' log-sum-exp from the units' statistics, one row per warp in turn.
SSD_DI void score_weights(const TreeArgs& a, int index) {
  __shared__ float s_lse[kTreeScoreRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = a.T * a.G;
  const int pairs = (a.nb + 1) / 2, kvh = index / pairs;
  const int b = (index - kvh * pairs) * 2 + (threadIdx.x >> 7), k = threadIdx.x & 127;
  const bool bad = *a.err != 0, ctx = b < a.nb_ctx;
  const int key = ctx ? b * kTreeKeys + k : a.n + (b - a.nb_ctx) * kTreeKeys + k;
  const bool live = b < a.nb && key < (ctx ? a.n : a.n + a.T);
  const float* ps = a.part_s + ((size_t)kvh * a.nb + b) * rows * kTreeKeys + k;
  const size_t o = (size_t)kvh * a.max_seq + key;
  // the first rows' scores are on their way meanwhile
  constexpr int kFirst = 8;
  float first[kFirst];
#pragma unroll
  for (int row = 0; row < kFirst; ++row)
    first[row] = live && row < rows ? ps[(size_t)row * kTreeKeys] : 0.f;
  const float before = live && ctx && a.w_in ? a.w_in[o] : 0.f;
  for (int row = warp; row < rows; row += kJoinWarps) {
    const bool present = a.depth[row / a.G] >= 0;
    float lse;
    if (a.splits == 1) {
      lse = a.lse[(size_t)kvh * rows + row];
    } else {
      const size_t s0 = (size_t)kvh * a.splits * 128 + row;
      float m = -INFINITY, l = 0.f;              // of the lane's units, then of all
      for (int i = lane; i < a.splits; i += 32) {
        const float pm = a.part_m[s0 + (size_t)i * 128], pl = a.part_l[s0 + (size_t)i * 128];
        const float mn = fmaxf(m, pm), base = mn == -INFINITY ? 0.f : mn;
        l = l * exp2f(m - base) + pl * exp2f(pm - base);
        m = mn;
      }
      float all = m;
#pragma unroll
      for (int d = 16; d; d >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, d));
      l *= exp2f(m - (all == -INFINITY ? 0.f : all));
#pragma unroll
      for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      lse = l != 0.f && present ? all + log2f(l) : INFINITY;
    }
    if (lane == 0) s_lse[row] = bad ? NAN : lse;
  }
  __syncthreads();
  if (!live) return;
  float sum = 0.f;
  auto add = [&](int row, float score) {
    const float lse = s_lse[row], p = tree_ex2(fmaf(score, a.scale_log2, -lse));
    if (lse != INFINITY) sum += p;               // absent rows take no part
  };
#pragma unroll
  for (int row = 0; row < kFirst; ++row)
    if (row < rows) add(row, first[row]);
#pragma unroll 8
  for (int row = kFirst; row < rows; ++row) add(row, ps[(size_t)row * kTreeKeys]);
  if (isnan(sum) && !ctx && !bad) {
    // a row of NaN has none at the tree's keys that it does not see
    const uint32_t* anc = a.anc + (b - a.nb_ctx) * 4 + (k >> 5);
    sum = 0.f;
    for (int row = 0; row < rows; ++row)
      if ((anc[(size_t)(row / a.G) * a.anc_words] >> (k & 31)) & 1u) add(row, ps[(size_t)row * kTreeKeys]);
  }
  a.w_out[o] = before + sum;
}

// Many slots and few rows: CTA = one 16-byte column of 32 rows; each warp adds
// every eighth slot under the maximum of its own, then the warps' sums are
// added in order.
template <int DH>
SSD_DI void join_column(const TreeArgs& a, int index) {
  __shared__ float4 s_o[kJoinWarps][32];
  __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = a.T * a.G, blocks = (rows + 31) / 32;
  const int c = index % (DH / 4), row0 = (index / (DH / 4)) % blocks * 32;
  const int kvh = index / (DH / 4) / blocks, row = min(row0 + lane, rows - 1);
  const int tile = row >> 7, r = row & 127, t = row / a.G, per = a.two ? a.items * 2 : 1;
  const size_t s0 = (size_t)kvh * a.splits * per + (a.two ? tile : 0);
  const bool present = a.depth[t] >= 0, bad = *a.err != 0;
  const bool marked = any_bad(a, kvh, lane);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // four slots in flight at once, the last ones among them
  constexpr int kBatch = 4;
  for (int i0 = warp; i0 < a.splits; i0 += kBatch * kJoinWarps) {
    float pm[kBatch], pl[kBatch], mn = m;
    float4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kJoinWarps;
      const bool got = i < a.splits;
      const size_t sl = s0 + (size_t)i * per;
      pm[u] = got ? a.part_m[sl * 128 + r] : -INFINITY;
      pl[u] = got ? a.part_l[sl * 128 + r] : 0.f;
      v[u] = got ? *reinterpret_cast<const float4*>(a.part_o + sl * DH * 128 + (size_t)c * 512 + r * 4)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
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
      const float w = exp2f(pm[u] - base);
      l = fmaf(pl[u], w, l);
      o.x = fmaf(v[u].x, w, o.x);
      o.y = fmaf(v[u].y, w, o.y);
      o.z = fmaf(v[u].z, w, o.z);
      o.w = fmaf(v[u].w, w, o.w);
    }
    m = mn;
  }
  s_o[warp][lane] = o;
  s_l[warp][lane] = l;
  s_m[warp][lane] = m;
  __syncthreads();
  if (warp) return;
  for (int i = 1; i < kJoinWarps; ++i) m = fmaxf(m, s_m[i][lane]);
  const float base = m == -INFINITY ? 0.f : m;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < kJoinWarps; ++i) {
    const float4 v = s_o[i][lane];
    const float w = exp2f(s_m[i][lane] - base);
    l = fmaf(s_l[i][lane], w, l);
    o.x = fmaf(v.x, w, o.x);
    o.y = fmaf(v.y, w, o.y);
    o.z = fmaf(v.z, w, o.z);
    o.w = fmaf(v.w, w, o.w);
  }
  const float lse = l != 0.f ? m + log2f(l) : INFINITY, inv = l != 0.f ? 1.f / l : 0.f;
  float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  if (!present)
    v[0] = v[1] = v[2] = v[3] = 0.f;
  else if (marked)
    add_bad<DH>(a, kvh, row, t, lse, c * 4, v, 4);
  if (bad) v[0] = v[1] = v[2] = v[3] = NAN;
  if (row0 + lane < rows)
    *reinterpret_cast<uint2*>(a.out + ((size_t)t * a.H + kvh * a.G + row % a.G) * DH + c * 4) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// After the units: CTAs 0 .. joins - 1 join their partial results, the rest
// sum the weights from stored scores (where there are any).  Both read the
// units' statistics, so that neither waits for the other.
template <int DH, bool COLUMNS>
__global__ void __launch_bounds__(kJoinWarps * 32)
    tree_finish_kernel(const __grid_constant__ TreeArgs a, int joins) {
  pdl_wait();
  if ((int)blockIdx.x >= joins)
    score_weights(a, blockIdx.x - joins);
  else if (COLUMNS)
    join_column<DH>(a, blockIdx.x);
  else
    tree_join_rows<DH>(a, blockIdx.x, threadIdx.x >> 5);
}

template <int DH, bool TWO>
cudaError_t launch(const TreeArgs& a, const TreeMaps& m, cudaStream_t st) {
  const int rows = a.T * a.G;
  const size_t smem = (size_t)kTileSmem + 1024 + 1024 + 512;
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e = cudaFuncSetAttribute(
        tree_attn_tc_kernel<DH, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dv >= 0) ready[dv] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(a.ctas);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&lc, tree_attn_tc_kernel<DH, TWO>, m.k, m.v, m.ws, a);
  if (e != cudaSuccess || (a.splits == 1 && !a.part_s)) return e;
  if (a.w_out && !a.part_s) return e;            // the weights' kernel joins
  const bool columns = a.splits >= 16 && rows <= 128;
  const int joins = a.splits == 1 ? 0 : (rows + 31) / 32 * a.Hkv * (columns ? DH / 4 : 1);
  const int sums = a.part_s ? (a.nb + 1) / 2 * a.Hkv : 0;
  lc.gridDim = dim3(joins + sums);
  lc.blockDim = dim3(kJoinWarps * 32);
  lc.dynamicSmemBytes = 0;
  return columns ? cudaLaunchKernelEx(&lc, tree_finish_kernel<DH, true>, a, joins)
                 : cudaLaunchKernelEx(&lc, tree_finish_kernel<DH, false>, a, joins);
}

}  // namespace

int tree_sms() {
  static int cached[kDeviceSlots] = {0};
  const int dv = device_slot();
  if (dv >= 0 && cached[dv]) return cached[dv];
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    cudaGetLastError();
  else if (dv >= 0)
    cached[dv] = sms;
  return sms;
}

// Splits the key blocks so that the units of all heads and row tiles fill the
// SMs in as few block steps as possible: a wave of units takes as long as its
// longest run of blocks plus about three for the start and the hand-over, and
// more than one split costs the second kernel, about three more.
void tree_split(TreeArgs& a) {
  const int rows = a.T * a.G, sms = tree_sms();
  a.tiles = (rows + 127) / 128;
  a.two = a.tiles > 1;
  a.items = a.two ? (a.tiles + 1) / 2 : 1;
  a.nb_ctx = a.n / kTreeKeys + (a.n % kTreeKeys != 0);
  a.nb = a.nb_ctx + (a.T + kTreeKeys - 1) / kTreeKeys;
  const long long lanes = (long long)a.Hkv * a.items;
  long long best = -1;
  // of the splits that take the same number of waves the most is the best;
  // and one split, whatever it takes
  for (long long waves = 0; waves <= 8; ++waves) {
    long long n = waves ? waves * sms / lanes : 1;
    if (n < 1) continue;
    n = n > a.nb ? a.nb : n > 160 ? 160 : n;
    // a stream takes every other block of a single tile's run
    const long long len = (a.nb + n - 1) / n, steps = a.two ? len : (len + 1) / 2;
    const long long cost = ((lanes * n + sms - 1) / sms) * (steps + 3) + (n > 1 ? 3 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      a.splits = (int)n;
    }
  }
  a.units = (int)(lanes * a.splits);
  a.ctas = a.units < sms ? a.units : sms;
}

int tree_slots(const TreeArgs& a) { return a.Hkv * a.splits * (a.two ? a.items * 2 : 1); }

cudaError_t launch_tree_attn_tc(const TreeArgs& a, const TreeMaps& m, cudaStream_t s) {
  if (a.dh == 128) return a.two ? launch<128, true>(a, m, s) : launch<128, false>(a, m, s);
  return a.two ? launch<64, true>(a, m, s) : launch<64, false>(a, m, s);
}

}  // namespace ssd
