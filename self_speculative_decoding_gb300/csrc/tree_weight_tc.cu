// Attention weight received by each key of a tree attention, on the
// 5th-generation tensor cores:
//   w_out[key] = w_in[key] + sum over the group's rows of 2^(s c - lse_row).
// The scores are computed again, transposed (S^T = K Q^T: one key per tensor
// memory lane, one row per column), so that a key's sum is one thread's sum
// over its columns: no exchange between threads and a fixed order.
//
// A CTA has a run of key blocks, taken in segments of up to 32.  A pass goes
// over a segment with a pair of row tiles (or the only one): their planes (q's
// low and high part) stay in shared memory while the K blocks stream, in turn
// to two streams of four warps, each block against both tiles at once (256
// columns to an instruction: twice the time of 128, which covers what the
// issuing warp does between two groups); the sums of a segment's keys stay
// with their threads until every pair has passed.  Passes zigzag over the
// pairs, so that a new segment starts with the planes that are there.
// Warp 8: TMA copies, warp 9: the products, warps 10 and 11: the join of the
// attention's partial results meanwhile, so that no kernel runs between.
// Waits are bounded; one that gives up makes the CTA's weights NaN.
//
// 64 nodes of 64 / 8 heads over 32768 rows: 52 us (62 with one tile to a
// pass), of which the products of both planes are 36 at the matrix peak; a
// stream's chain of products (2400 cycles for 256 columns) and sums (3100)
// bounds it, with the two streams' products in turn.
#include "tc_dev.cuh"
#include "tree.cuh"
#include "tree_join.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kPolls = 1 << 22;
constexpr int kRegion = 128 * 128;
constexpr int kTileSmem = 224 * 1024;            // Q tiles (hi, lo), then the ring of K blocks
constexpr int kMaxStages = 12;
constexpr int kSegment = 32;                     // key blocks of a segment

// Barriers of the two streams' 256 threads; the second tells whether any of
// them passed true.
SSD_DI void streams_sync() { asm volatile("barrier.cta.sync.aligned 1, 256;" ::: "memory"); }
SSD_DI bool streams_any(bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, 1, 256, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)x)
      : "memory");
  return r != 0;
}

// A CTA's passes in order: every pair of tiles over each segment of its run.
struct Pass {
  int pos, end, kvh, b0, cnt;                    // the segment
  int pairs, done_pairs, back;                   // of tiles; zigzag
  SSD_DI void segment(const TreeArgs& a) {
    kvh = pos / a.nb;
    b0 = pos - kvh * a.nb;
    cnt = min(kSegment, min(a.nb - b0, end - pos));
    done_pairs = 0;
  }
  SSD_DI bool over() const { return pos >= end; }
  SSD_DI int pair() const { return back ? pairs - 1 - done_pairs : done_pairs; }
  SSD_DI bool first() const { return done_pairs == 0; }
  SSD_DI bool last() const { return done_pairs + 1 == pairs; }
  SSD_DI Pass next(const TreeArgs& a) const {
    Pass p = *this;
    if (++p.done_pairs < pairs) return p;
    p.pos += cnt;
    p.back ^= 1;
    if (p.pos < end) p.segment(a);
    return p;
  }
  // whether this pass has other planes than the one before
  SSD_DI bool other(const Pass& before) const { return kvh != before.kvh || pair() != before.pair(); }
};
SSD_DI Pass first_pass(const TreeArgs& a) {
  const long long total = (long long)a.Hkv * a.nb;
  Pass p;
  p.pos = (int)(blockIdx.x * total / gridDim.x);
  p.end = (int)((blockIdx.x + 1) * total / gridDim.x);
  p.pairs = (a.tiles + 1) / 2;
  p.back = 0;
  p.kvh = p.b0 = p.cnt = p.done_pairs = 0;
  if (p.pos < p.end) p.segment(a);
  return p;
}

// Sum over `cols` score columns (rows row0 ..) of a key's 2^(s c - lse), of the
// rows that take part (another one may meet inf or NaN) and, in a tree block
// (word >= 0), that see the key.  Apart from the plain sum: conditions within
// its loop became selections on every column, and 256 columns took 4200 cycles.
__device__ __noinline__ float masked_columns(const TreeArgs& a, uint32_t col, const float* nlse,
                                             int row0, int cols, int word) {
  const int lane = threadIdx.x & 31, rows = a.T * a.G;
  float part = 0.f;
  for (int q = 0; q < cols; q += 32) {
    uint32_t w[32];
    tmem_ld32_nw(col + (uint32_t)q, w);
    // lane e: the ancestor word of row e (a context key is seen by all)
    const int row = row0 + q + lane;
    uint32_t mine = ~0u;
    if (word >= 0)
      mine = row < rows ? a.anc[(size_t)(row / a.G) * a.anc_words + word] : 0u;
    tmem_wait_ld();
    tmem_pin32(w);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t bits = __shfl_sync(0xffffffffu, mine, e);
      const float n = nlse[q + e], p = tree_ex2(fmaf(__uint_as_float(w[e]), a.scale_log2, n));
      if (((bits >> lane) & 1u) && n != -INFINITY) part += p;
    }
  }
  return part;
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
    tree_weight_tc_kernel(const __grid_constant__ CUtensorMap mK,
                          const __grid_constant__ CUtensorMap mW,
                          const __grid_constant__ TreeArgs a) {
  constexpr int kRegs = DH / 64;
  constexpr int kItem = kRegs * kRegion;
  extern __shared__ unsigned char sm_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  float* nlse = reinterpret_cast<float*>(sm + kTileSmem);  // [tile of the pair][128], -lse
  uint64_t* bars = reinterpret_cast<uint64_t*>(nlse + 256);
  uint64_t* qfull = bars;                        // the pass's planes
  uint64_t* qempty = bars + 1;
  uint64_t* sfull = bars + 2;                    // [stream][buffer]
  uint64_t* sfree = sfull + 4;
  uint64_t* mdone = sfull + 8;
  uint64_t* full = sfull + 9;
  uint64_t* empty = full + kMaxStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(empty + kMaxStages);
  int* fail = reinterpret_cast<int*>(tslot + 1);
  const int tid = threadIdx.x, warp = tree_warp(), lane = tid & 31;
  const int rows = a.T * a.G;
  const int polls = (int)blockIdx.x == a.give_up_weights ? 0 : kPolls;
  const int planes = a.tiles > 1 ? 4 : 2;        // of the pass's one or two tiles
  const int stages = min(kMaxStages, kTileSmem / kItem - planes);
  const int bufs = a.tiles > 1 ? 1 : 2;          // of a stream's 256 score columns
  unsigned char* ring = sm + planes * kItem;

  if (tid == 0) {
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sfree[s], 128);
    }
    mbar_init(mdone, 1);
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    *fail = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  if (warp == 8) {
    if (lane == 0) {
      int issued = 0, slot = 0, sent = 0;        // copies, their slot; loads of planes
      uint32_t phase = 0;
      bool ok = true;
      pdl_wait();                                // Q and the tree's K rows
      Pass before = first_pass(a);
      for (Pass x = before; ok && !x.over(); x = x.next(a)) {
        if (!sent || x.other(before)) {
          if (sent) ok = mbar_wait_n(qempty, (uint32_t)((sent - 1) & 1), polls);
          if (!ok) break;
          ++sent;
          mbar_arrive_expect_tx(qfull, (uint32_t)(planes * kItem));
          // [plane][64 columns][row of the pair] (beyond the last: of no use)
          for (int p = 0; p < 2; ++p)
            for (int r = 0; r < kRegs; ++r)
              for (int t = 0; t < planes / 2; ++t)
                tma_load_3d(sm + ((p * kRegs + r) * (planes / 2) + t) * kRegion, &mW, r * 64,
                            ((1 - p) * a.Hkv + x.kvh) * rows + (x.pair() * 2 + t) * 128, 0, qfull);
        }
        before = x;
        for (int j = 0; ok && j < x.cnt; ++j) {
          if (issued >= stages) ok = mbar_wait_n(&empty[slot], phase ^ 1u, polls);
          if (!ok || tree_flagged(fail)) {
            ok = false;
            break;
          }
          const int b = x.b0 + j;
          const bool ctx = b < a.nb_ctx;
          const int row = ctx ? b * kTreeKeys : a.row_kt + x.kvh * a.T + (b - a.nb_ctx) * kTreeKeys;
          mbar_arrive_expect_tx(&full[slot], (uint32_t)kItem);
          for (int r = 0; r < kRegs; ++r)
            tma_load_3d(ring + (size_t)slot * kItem + r * kRegion, ctx ? &mK : &mW, r * 64, row,
                        ctx ? x.kvh : 0, &full[slot]);
          ++issued;
          if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) atomicExch(fail, 1);
      for (int i = max(0, issued - stages); i < issued; ++i)
        mbar_wait_n(&full[i % stages], (uint32_t)((i / stages) & 1), kPolls);
      if (sent) mbar_wait_n(qfull, (uint32_t)((sent - 1) & 1), kPolls);
    }
  } else if (warp == 9) {
    // the warp runs together, one lane issues.  (A CTA may start while the
    // attention still runs, for as long as that takes: bounded waits begin after
    // the wait for it.)
    pdl_wait();
    const uint32_t lead = tree_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t qa = smem_addr(sm), ra = smem_addr(ring);
    const uint32_t qregion = (uint32_t)(planes / 2) * kRegion;
    int slot = 0, loads = 0;
    uint32_t phase = 0;
    int cs[2] = {0, 0};                          // score tiles per stream
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      ok = __all_sync(0xffffffffu, ok && tree_wait(fail, polls, bar, ph));
    };
    Pass before = first_pass(a);
    for (Pass x = before; ok && !x.over();) {
      if (!loads || x.other(before)) {
        wait(qfull, (uint32_t)(loads & 1));
        ++loads;
      }
      before = x;
      const int cols = min(256, rows - x.pair() * 256);
      const uint32_t id = idesc_bf16(128, (cols + 15) / 16 * 16);
      for (int j = 0; ok && j < x.cnt; j += 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || j + s >= x.cnt) continue;
          // the block has landed and the stream's score columns have been read
          const int buf = cs[s] % bufs, use = cs[s] / bufs;
          if (use > 0)
            ok = __all_sync(0xffffffffu, tree_wait(fail, polls, &sfree[s * 2 + buf], (uint32_t)((use - 1) & 1),
                                                   &full[slot], phase));
          else
            wait(&full[slot], phase);
          tc_fence_after();
          if (!ok) continue;
          const uint32_t kb = ra + (uint32_t)slot * kItem;
          const uint32_t acc = tm + (uint32_t)(s * 256 + buf * 128);
#pragma unroll
          for (int p = 0; p < 2; ++p)            // the low part first
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
              const uint32_t rg = (uint32_t)(ks >> 2);
              tree_mma_ss(lead, acc, sw128_desc(kb + rg * kRegion) + 2 * (ks & 3),
                          sw128_desc(qa + (p * kRegs + rg) * qregion) + 2 * (ks & 3), id,
                          (p || ks > 0) ? 1u : 0u);
            }
          tree_commit(lead, &sfull[s * 2 + buf]);
          tree_commit(lead, &empty[slot]);
          ++cs[s];
          if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      x = x.next(a);
      if (x.over() || x.other(before)) tree_commit(lead, qempty);
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
    tree_commit(lead, mdone);
    mbar_wait_n(mdone, 0u, kPolls);
  } else if (warp > 9) {
    pdl_wait();
    if (a.splits > 1)
      for (int i = blockIdx.x + gridDim.x * (warp - 10); i < tree_joins(a) * kJoinWarps;
           i += gridDim.x * (kThreads / 32 - 10))
        tree_join_rows<DH>(a, i / kJoinWarps, i % kJoinWarps);
  } else {
    // one key per thread.  Every thread passes every barrier: a wait that
    // gives up only turns the sums into NaN.
    pdl_wait();
    const int s = warp >> 2, r = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)s * 256;
    const uint64_t sc2 = tree_pack2(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
    const bool bad = *a.err != 0;
    int c = 0;
    bool ok = !bad;
    // -log-sum-exp of a row of a pass's tiles, one per thread; rows that are
    // absent, or beyond the last, take no part
    auto row_lse = [&](const Pass& x) {
      const int row = x.pair() * 256 + tid;
      return row < rows ? -tree_row_lse(a, x.kvh, row) : -INFINITY;
    };
    Pass x = first_pass(a);
    float next = x.over() ? 0.f : row_lse(x);
    float sums[kSegment / 2];                    // of this stream's blocks of the segment
    while (!x.over()) {
      streams_sync();                            // the pass before has been read
      nlse[tid] = next;
      const int cols = min(256, rows - x.pair() * 256);
      const bool some = streams_any(next == -INFINITY && tid < cols);
      const Pass y = x.next(a);
      if (!y.over()) next = row_lse(y);
      for (int j = s; j < x.cnt; j += 2, ++c) {
        const int b = x.b0 + j, buf = c % bufs, use = c / bufs;
        const bool ctx = b < a.nb_ctx;
        // pairs of partial sums
        uint64_t sum[2] = {x.first() ? 0 : (uint64_t)__float_as_uint(sums[j >> 1]), 0};
        ok = ok && tree_wait(fail, polls, &sfull[s * 2 + buf], (uint32_t)(use & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) atomicExch(fail, 1);
          ok = false;
        } else {
          tc_fence_after();
          const uint32_t col = trow + (uint32_t)(buf * 128);
          // columns that all take part, 32 at a time; the others by selection
          const int plain = ctx && !some ? cols & ~31 : 0;
          if (plain) {
            // (a short loop: unrolled over 64 or 128 columns, with the next ones
            // loading meanwhile, it was slower by 2 to 25 us on 64 nodes over
            // 32768 rows)
            auto add = [&](uint32_t(&w)[32], int q) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const ulonglong2 n4 = *reinterpret_cast<const ulonglong2*>(nlse + q + e);
                float p0, p1, p2, p3;
                tree_unpack2(tree_fma2(tree_pack2(w[e], w[e + 1]), sc2, n4.x), p0, p1);
                tree_unpack2(tree_fma2(tree_pack2(w[e + 2], w[e + 3]), sc2, n4.y), p2, p3);
                sum[0] = tree_add2(sum[0], tree_pack2(__float_as_uint(tree_ex2(p0)),
                                                      __float_as_uint(tree_ex2(p1))));
                sum[1] = tree_add2(sum[1], tree_pack2(__float_as_uint(tree_ex2(p2)),
                                                      __float_as_uint(tree_ex2(p3))));
              }
            };
#pragma unroll 1
            for (int q = 0; q < plain; q += 32) {
              uint32_t v0[32];
              tmem_ld32_nw(col + (uint32_t)q, v0);
              tmem_wait_ld();
              tmem_pin32(v0);
              add(v0, q);
            }
          }
          if (plain < cols) {
            const float part =
                masked_columns(a, col + (uint32_t)plain, nlse + plain, x.pair() * 256 + plain,
                               cols - plain, ctx ? -1 : (b - a.nb_ctx) * 4 + (warp & 3));
            sum[0] = tree_add2(sum[0], (uint64_t)__float_as_uint(part));
          }
        }
        tc_fence_before();
        mbar_arrive_cta(&sfree[s * 2 + buf]);
        float s0, s1;
        tree_unpack2(tree_add2(sum[0], sum[1]), s0, s1);
        const float total = s0 + s1;
        sums[j >> 1] = total;
        if (x.last()) {
          const int key = ctx ? b * kTreeKeys + r : a.n + (b - a.nb_ctx) * kTreeKeys + r;
          const size_t o = (size_t)x.kvh * a.max_seq + key;
          if (key < (ctx ? a.n : a.n + a.T))
            a.w_out[o] = !ok ? NAN : ctx && a.w_in ? a.w_in[o] + total : total;
        }
      }
      x = y;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int DH>
cudaError_t launch(const TreeArgs& a, const TreeMaps& m, cudaStream_t st) {
  const int sms = tree_sms();
  const size_t smem = (size_t)kTileSmem + 1024 + 1024 + 512;
  static bool ready[kDeviceSlots] = {};
  const int dv = device_slot();
  if (dv < 0 || !ready[dv]) {
    const cudaError_t e = cudaFuncSetAttribute(
        tree_weight_tc_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dv >= 0) ready[dv] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  const long long blocks = (long long)a.Hkv * a.nb;
  lc.gridDim = dim3((unsigned)(blocks < sms ? blocks : sms));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, tree_weight_tc_kernel<DH>, m.k, m.ws, a);
}

}  // namespace

cudaError_t launch_tree_weight_tc(const TreeArgs& a, const TreeMaps& m, cudaStream_t s) {
  return a.dh == 128 ? launch<128>(a, m, s) : launch<64>(a, m, s);
}

}  // namespace ssd
