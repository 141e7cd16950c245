// Attention weight received by each key of a tree attention, on the
// 5th-generation tensor cores:
//   w_out[key] = w_in[key] + sum over the group's rows of 2^(s c - lse_row).
// The scores are computed again, transposed (S^T = K Q^T: one key per tensor
// memory lane, one row per column), so that a key's sum is one thread's sum
// over its columns: no exchange between threads and a fixed order.
//
// A CTA has a run of key blocks, taken in segments of up to 16.  A pass goes
// over a segment with one tile of 128 rows: the tile's two planes (q's low and
// high part) stay in shared memory while the K blocks stream, in turn to two
// streams of four warps; the sums of a segment's keys stay with their threads
// until every tile has passed.  The next pass's planes load meanwhile; up to
// two tiles stay for all of a head's segments.  (Held the other way round, two
// K blocks with the Q planes streaming, 64 nodes of 64 / 8 heads over 32768
// rows took 61 us.)  The softmax warps first join the attention's partial
// results, so that no kernel runs between.
// Warp 8: TMA copies, warp 9: MMA.  Waits are bounded; one that gives up makes
// the CTA's weights NaN.
#include "tc_dev.cuh"
#include "tree.cuh"
#include "tree_join.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kThreads = 320;
constexpr int kPolls = 1 << 22;
constexpr int kRegion = 128 * 128;
constexpr int kTileSmem = 224 * 1024;            // Q tiles (hi, lo), then the ring of K blocks
constexpr int kMaxStages = 12;
constexpr int kMaxPlanes = 4;
constexpr int kSegment = 16;                     // key blocks of a segment

// Barrier of one stream's 128 threads; true if any of them passed true.
SSD_DI bool stream_any(int s, bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %1, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(s + 1), "r"(128), "r"((int)x)
      : "memory");
  return r != 0;
}

SSD_DI void stream_sync(int s) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(s + 1), "r"(128) : "memory");
}

// A CTA's passes in order: every tile over each segment of its run.
struct Pass {
  int pos, end, kvh, b0, cnt, t;
  SSD_DI void segment(const TreeArgs& a) {
    kvh = pos / a.nb;
    b0 = pos - kvh * a.nb;
    cnt = min(kSegment, min(a.nb - b0, end - pos));
    t = 0;
  }
  SSD_DI bool done() const { return pos >= end; }
  SSD_DI bool last_of_head(const TreeArgs& a) const {
    return t + 1 == a.tiles && (b0 + cnt == a.nb || pos + cnt == end);
  }
  SSD_DI bool first_of_head(int begin) const { return t == 0 && (b0 == 0 || pos == begin); }
  SSD_DI void next(const TreeArgs& a) {
    if (++t < a.tiles) return;
    pos += cnt;
    if (pos < end) segment(a);
  }
};
SSD_DI Pass first_pass(const TreeArgs& a) {
  const long long total = (long long)a.Hkv * a.nb;
  Pass p;
  p.pos = (int)(blockIdx.x * total / gridDim.x);
  p.end = (int)((blockIdx.x + 1) * total / gridDim.x);
  if (p.pos < p.end) p.segment(a);
  return p;
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
  float* nlse = reinterpret_cast<float*>(sm + kTileSmem);  // [stream][128], -lse
  uint64_t* bars = reinterpret_cast<uint64_t*>(nlse + 256);
  uint64_t* qfull = bars;                        // [planes]
  uint64_t* qempty = bars + kMaxPlanes;
  uint64_t* sfull = bars + 2 * kMaxPlanes;       // [stream][buffer]
  uint64_t* sfree = sfull + 4;
  uint64_t* mdone = sfull + 8;
  uint64_t* full = sfull + 9;
  uint64_t* empty = full + kMaxStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(empty + kMaxStages);
  int* fail = reinterpret_cast<int*>(tslot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.T * a.G;
  const bool resident = a.tiles <= 2;            // Q stays for all segments of a head
  const int qslots = resident ? 2 * a.tiles : kMaxPlanes;
  const int stages = min(kMaxStages, kTileSmem / kItem - qslots);
  unsigned char* ring = sm + qslots * kItem;

  if (tid == 0) {
    for (int s = 0; s < kMaxPlanes; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&qempty[s], 1);
    }
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
      const Pass begin = first_pass(a);
      int issued = 0, slot = 0, qsent = 0, heads = 0;  // copies, their slot, passes' and heads' planes
      uint32_t phase = 0;
      bool ok = true;
      auto plane = [&](int sl, bool again, uint32_t ph, int kvh, int tile, int p) {
        if (again && !mbar_wait_n(&qempty[sl], ph, kPolls)) return false;
        mbar_arrive_expect_tx(&qfull[sl], (uint32_t)kItem);
        for (int r = 0; r < kRegs; ++r)
          tma_load_3d(sm + sl * kItem + r * kRegion, &mW, r * 64,
                      (p * a.Hkv + kvh) * rows + tile * 128, 0, &qfull[sl]);
        return true;
      };
      // the planes of a pass (streaming): two slots in turn
      auto send_pass = [&](const Pass& x) {
        const int sl = (qsent & 1) * 2;
        const uint32_t ph = (uint32_t)(((qsent >> 1) - 1) & 1);
        const bool again = qsent >= 2;
        ++qsent;
        return plane(sl, again, ph, x.kvh, x.t, 1) && plane(sl + 1, again, ph, x.kvh, x.t, 0);
      };
      pdl_wait();                                // Q and the tree's K rows
      if (!resident && !begin.done()) ok = send_pass(begin);
      for (Pass x = begin; ok && !x.done(); x.next(a)) {
        if (resident && x.first_of_head(begin.pos)) {
          for (int t = 0; ok && t < a.tiles; ++t)
            for (int p = 1; ok && p >= 0; --p)
              ok = plane(2 * t + 1 - p, heads > 0, (uint32_t)((heads - 1) & 1), x.kvh, t, p);
          ++heads;
        }
        for (int j = 0; ok && j < x.cnt; ++j) {
          if (!resident && j == min(2, x.cnt - 1)) {
            // the next pass's planes: their slots are the pass before's
            Pass y = x;
            y.next(a);
            if (!y.done()) ok = send_pass(y);
          }
          if (ok && issued >= stages) ok = mbar_wait_n(&empty[slot], phase ^ 1u, kPolls);
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
      // the planes sent last (a slot's last use)
      if (resident) {
        for (int i = 0; heads > 0 && i < qslots; ++i)
          mbar_wait_n(&qfull[i], (uint32_t)((heads - 1) & 1), ok ? kPolls : 1 << 16);
      } else {
        for (int q = max(0, qsent - 2); q < qsent; ++q)
          for (int p = 0; p < 2; ++p)
            mbar_wait_n(&qfull[(q & 1) * 2 + p], (uint32_t)((q >> 1) & 1), ok ? kPolls : 1 << 16);
      }
    }
  } else if (warp == 9) {
    // the warp runs together, one lane issues
    const uint32_t lead = tree_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t qa = smem_addr(sm), ra = smem_addr(ring);
    const Pass begin = first_pass(a);
    int slot = 0, passes = 0, heads = 0;
    uint32_t phase = 0;
    int cs[2] = {0, 0};                          // score tiles per stream
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_n(bar, ph, kPolls));
      tc_fence_after();
    };
    for (Pass x = begin; ok && !x.done(); x.next(a), ++passes) {
      if (resident && x.first_of_head(begin.pos)) ++heads;
      const int q0 = resident ? 2 * x.t : (passes & 1) * 2;
      const uint32_t qph = (uint32_t)((resident ? heads - 1 : passes >> 1) & 1);
      wait(&qfull[q0], qph);
      wait(&qfull[q0 + 1], qph);
      const int cols = min(128, (rows - x.t * 128 + 15) / 16 * 16);
      const uint32_t id = idesc_bf16(128, cols);
      const uint32_t qb = qa + (uint32_t)q0 * kItem;
      for (int j = 0; ok && j < x.cnt; j += 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || j + s >= x.cnt) continue;
          const int buf = cs[s] & 1;
          wait(&full[slot], phase);
          if (cs[s] >= 2) wait(&sfree[s * 2 + buf], (uint32_t)((cs[s] / 2 - 1) & 1));
          ok = __all_sync(0xffffffffu, ok && !tree_flagged(fail));
          if (!ok) continue;
          const uint32_t kb = ra + (uint32_t)slot * kItem;
          const uint32_t acc = tm + (uint32_t)(s * 256 + buf * 128);
#pragma unroll
          for (int p = 0; p < 2; ++p)            // the low part first
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
              const uint32_t o = (uint32_t)(ks >> 2) * kRegion;
              tree_mma_ss(lead, acc, sw128_desc(kb + o) + 2 * (ks & 3),
                          sw128_desc(qb + p * kItem + o) + 2 * (ks & 3), id, (p || ks > 0) ? 1u : 0u);
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
      if (!resident) {
        tree_commit(lead, &qempty[q0]);
        tree_commit(lead, &qempty[q0 + 1]);
      } else if (x.last_of_head(a)) {
        for (int i = 0; i < qslots; ++i) tree_commit(lead, &qempty[i]);
      }
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
    tree_commit(lead, mdone);
    mbar_wait_n(mdone, 0u, kPolls);
  } else {
    // one key per thread.  Every thread passes every barrier: a wait that
    // gives up only turns the sums into NaN.
    pdl_wait();
    if (a.splits > 1)
      for (int i = blockIdx.x; i < tree_joins(a); i += gridDim.x) tree_join_rows<DH>(a, i);
    const int s = warp >> 2, r = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)s * 256;
    const float scale = a.scale_log2;
    const bool bad = *a.err != 0;
    float* nl = nlse + s * 128;
    int c = 0;
    bool ok = !bad;
    const Pass begin = first_pass(a);
    // -log-sum-exp of row r of a pass's tile; rows that are absent, or beyond
    // the last, take no part
    auto row_lse = [&](const Pass& x) {
      const int row = x.t * 128 + r;
      return row < rows ? -tree_row_lse(a, x.kvh, row) : -INFINITY;
    };
    float next = begin.done() ? 0.f : row_lse(begin);
    float sums[kSegment / 2];                    // of this stream's blocks of the segment
    for (Pass x = begin; !x.done(); x.next(a)) {
      const float mine = next;
      stream_sync(s);                            // the pass before has been read
      nl[r] = mine;
      const bool some = stream_any(s, mine == -INFINITY);
      Pass y = x;
      y.next(a);
      if (!y.done()) next = row_lse(y);
      const int cols = min(128, rows - x.t * 128);
      for (int j = s; j < x.cnt; j += 2, ++c) {
        const int buf = c & 1, b = x.b0 + j;
        const bool ctx = b < a.nb_ctx;
        ok = ok && !tree_flagged(fail) &&
             mbar_wait_n(&sfull[s * 2 + buf], (uint32_t)((c >> 1) & 1), kPolls);
        float sum[4] = {x.t ? sums[j >> 1] : 0.f, 0.f, 0.f, 0.f};
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) atomicExch(fail, 1);
          ok = false;
        } else {
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < cols; q += 64) {
            uint32_t v[2][32];
            tmem_ld32_nw(trow + (uint32_t)(buf * 128 + q), v[0]);
            if (q + 32 < cols) tmem_ld32_nw(trow + (uint32_t)(buf * 128 + q + 32), v[1]);
            tmem_wait_ld();
            tmem_pin32(v[0]);
            tmem_pin32(v[1]);
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
              if (q + hlf * 32 >= cols) break;
              const int q0 = q + hlf * 32;
              if (some) {
                // a row without part may meet inf or NaN among the keys: its
                // score is made 0, and its 2^(0 - inf) is 0
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float4 n4 = *reinterpret_cast<const float4*>(nl + q0 + e);
                  if (n4.x == -INFINITY) v[hlf][e] = 0u;
                  if (n4.y == -INFINITY) v[hlf][e + 1] = 0u;
                  if (n4.z == -INFINITY) v[hlf][e + 2] = 0u;
                  if (n4.w == -INFINITY) v[hlf][e + 3] = 0u;
                }
              }
              if (ctx) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float4 n4 = *reinterpret_cast<const float4*>(nl + q0 + e);
                  sum[0] += tree_ex2(fmaf(__uint_as_float(v[hlf][e]), scale, n4.x));
                  sum[1] += tree_ex2(fmaf(__uint_as_float(v[hlf][e + 1]), scale, n4.y));
                  sum[2] += tree_ex2(fmaf(__uint_as_float(v[hlf][e + 2]), scale, n4.z));
                  sum[3] += tree_ex2(fmaf(__uint_as_float(v[hlf][e + 3]), scale, n4.w));
                }
              } else {
                // a tree block: lane e holds the ancestor word of row q0 + e
                const int row = min(x.t * 128 + q0 + lane, rows - 1);
                const uint32_t word =
                    a.anc[(size_t)(row / a.G) * a.anc_words + (b - a.nb_ctx) * 4 + (warp & 3)];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const uint32_t w = __shfl_sync(0xffffffffu, word, e);
                  const float p = tree_ex2(fmaf(__uint_as_float(v[hlf][e]), scale, nl[q0 + e]));
                  if ((w >> lane) & 1u) sum[e & 3] += p;
                }
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive_cta(&sfree[s * 2 + buf]);
        const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        sums[j >> 1] = total;
        if (x.t + 1 == a.tiles) {
          const int key = ctx ? b * kTreeKeys + r : a.n + (b - a.nb_ctx) * kTreeKeys + r;
          const size_t o = (size_t)x.kvh * a.max_seq + key;
          if (key < (ctx ? a.n : a.n + a.T))
            a.w_out[o] = !ok ? NAN : ctx && a.w_in ? a.w_in[o] + total : total;
        }
      }
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
