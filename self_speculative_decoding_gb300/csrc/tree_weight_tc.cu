// Attention weight received by each key of a tree attention, on the
// 5th-generation tensor cores:
//   w_out[key] = w_in[key] + sum over the group's rows of 2^(s c - lse_row).
// The scores are computed again, transposed (S^T = K Q^T: one key per tensor
// memory lane, one row per column), so that a key's sum is one thread's sum
// over its columns: no exchange between threads and a fixed order.
//
// Unit = two blocks of 128 keys of one K/V head; warps 0-3 and 4-7 take a
// block each, every tile of 128 rows passes both (a Q tile read from L2
// serves 256 keys), plane by plane (low part, high part).  Up to two Q tiles
// stay in shared memory for all of a CTA's units of a head; more stream
// through three slots of a plane each.  Warp 8: TMA copies, warp 9: MMA.  Waits are bounded;
// one that gives up makes the CTA's weights NaN.
#include "tc_dev.cuh"
#include "tree.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kThreads = 320;
constexpr int kPolls = 1 << 22;
constexpr int kRegion = 128 * 128;
constexpr int kTileSmem = 224 * 1024;            // Q tiles (hi, lo), then the ring of K blocks
constexpr int kMaxStages = 12;
constexpr int kMaxPlanes = 4;

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

struct Range {
  int u0, u1;
};
SSD_DI Range my_units(const TreeArgs& a) {
  const long long total = (long long)a.Hkv * ((a.nb + 1) / 2);
  return {(int)(blockIdx.x * total / gridDim.x), (int)((blockIdx.x + 1) * total / gridDim.x)};
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
  const bool resident = a.tiles <= 2;            // Q stays for all units of a head
  const int qslots = resident ? 2 * a.tiles : 3;
  const int stages = min(kMaxStages, kTileSmem / kItem - qslots);
  unsigned char* ring = sm + qslots * kItem;
  const int pairs = (a.nb + 1) / 2;
  const Range rg = my_units(a);

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
      int issued = 0, qissued = 0;
      bool ok = true;
      auto send_q = [&](int kvh, int tile) {
        for (int p = 1; p >= 0; --p) {
          const int sl = qissued % qslots, use = qissued / qslots;
          if (use > 0 && !mbar_wait_n(&qempty[sl], (uint32_t)((use - 1) & 1), kPolls)) return false;
          mbar_arrive_expect_tx(&qfull[sl], (uint32_t)kItem);
          for (int r = 0; r < kRegs; ++r)
            tma_load_3d(sm + sl * kItem + r * kRegion, &mW, r * 64,
                        (p * a.Hkv + kvh) * rows + tile * 128, 0, &qfull[sl]);
          ++qissued;
        }
        return true;
      };
      for (int u = rg.u0; ok && u < rg.u1; ++u) {
        const int kvh = u / pairs, b0 = (u - kvh * pairs) * 2, nblk = min(2, a.nb - b0);
        if (u == rg.u0) pdl_wait();              // Q and the tree's K rows
        // Q of a new head before its keys: its slots wait for the old head's
        // products only, and these for nothing of this unit
        if (resident && (u == rg.u0 || u % pairs == 0))
          for (int t = 0; ok && t < a.tiles; ++t) ok = send_q(kvh, t);
        for (int s = 0; ok && s < nblk; ++s) {
          const int b = b0 + s, st = issued % stages, use = issued / stages;
          if (use > 0) ok = mbar_wait_n(&empty[st], (uint32_t)((use - 1) & 1), kPolls);
          if (!ok || tree_flagged(fail)) {
            ok = false;
            break;
          }
          const bool ctx = b < a.nb_ctx;
          mbar_arrive_expect_tx(&full[st], (uint32_t)kItem);
          const int row = ctx ? b * kTreeKeys : a.row_kt + kvh * a.T + (b - a.nb_ctx) * kTreeKeys;
          for (int r = 0; r < kRegs; ++r)
            tma_load_3d(ring + (size_t)st * kItem + r * kRegion, ctx ? &mK : &mW, r * 64, row,
                        ctx ? kvh : 0, &full[st]);
          ++issued;
        }
        if (!resident)
          for (int t = 0; ok && t < a.tiles; ++t) ok = !tree_flagged(fail) && send_q(kvh, t);
      }
      if (!ok) atomicExch(fail, 1);
      for (int i = max(0, issued - stages); i < issued; ++i)
        mbar_wait_n(&full[i % stages], (uint32_t)((i / stages) & 1), kPolls);
      for (int i = max(0, qissued - qslots); i < qissued; ++i)
        mbar_wait_n(&qfull[i % qslots], (uint32_t)((i / qslots) & 1), kPolls);
    }
  } else if (warp == 9) {
    // the warp runs together, one lane issues
    const uint32_t lead = tree_elect();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t qa = smem_addr(sm), ra = smem_addr(ring);
    int k0 = 0, kslot[2];                        // K slots of the unit
    uint32_t kphase = 0;
    int qslot = 0;
    uint32_t qphase = 0;
    int cs[2] = {0, 0};                          // score tiles per stream
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_n(bar, phase, kPolls));
      tc_fence_after();
    };
    for (int u = rg.u0; ok && u < rg.u1; ++u) {
      const int kvh = u / pairs, b0 = (u - kvh * pairs) * 2, nblk = min(2, a.nb - b0);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s < nblk) {
          wait(&full[k0], kphase);
          kslot[s] = k0;
          if (++k0 == stages) {
            k0 = 0;
            kphase ^= 1u;
          }
        }
      const int q0 = qslot;
      const uint32_t qp0 = qphase;
      for (int t = 0; ok && t < a.tiles; ++t) {
        const int cols = min(128, (rows - t * 128 + 15) / 16 * 16);
        const uint32_t id = idesc_bf16(128, cols);
#pragma unroll
        for (int p = 1; p >= 0; --p) {           // the low part first
          wait(&qfull[qslot], qphase);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || s >= nblk) continue;
            const int buf = cs[s] & 1;
            if (p && cs[s] >= 2) wait(&sfree[s * 2 + buf], (uint32_t)((cs[s] / 2 - 1) & 1));
            ok = __all_sync(0xffffffffu, ok && !tree_flagged(fail));
            if (!ok) continue;
            const uint32_t kb = ra + (uint32_t)kslot[s] * kItem;
            const uint32_t qb = qa + (uint32_t)qslot * kItem;
            const uint32_t acc = tm + (uint32_t)(s * 256 + buf * 128);
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
              const uint32_t o = (uint32_t)(ks >> 2) * kRegion;
              tree_mma_ss(lead, acc, sw128_desc(kb + o) + 2 * (ks & 3),
                          sw128_desc(qb + o) + 2 * (ks & 3), id, (p == 0 || ks > 0) ? 1u : 0u);
            }
            if (p == 0) {
              tree_commit(lead, &sfull[s * 2 + buf]);
              ++cs[s];
            }
          }
          if (!resident) tree_commit(lead, &qempty[qslot]);
          if (++qslot == qslots) {
            qslot = 0;
            qphase ^= 1u;
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s < nblk) tree_commit(lead, &empty[kslot[s]]);
      if (resident) {
        if ((u + 1) % pairs == 0) {              // the head's last unit
          for (int i = 0; i < 2 * a.tiles; ++i) tree_commit(lead, &qempty[i]);
        } else {                                 // the same planes again
          qslot = q0;
          qphase = qp0;
        }
      }
    }
    if (!ok && lane == 0) atomicExch(fail, 1);
    tree_commit(lead, mdone);
    mbar_wait_n(mdone, 0u, kPolls);
  } else {
    // one key per thread.  Every thread passes every barrier: a wait that
    // gives up only turns the sums into NaN.
    pdl_wait();
    const int s = warp >> 2, r = tid & 127;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)s * 256;
    const float scale = a.scale_log2;
    int c = 0;
    bool ok = true;
    // -lse of row r of a tile; rows that are absent, or beyond the last, take
    // no part
    auto row_lse = [&](int kvh, int t) {
      return t * 128 + r < rows ? -a.lse[(size_t)kvh * rows + t * 128 + r] : -INFINITY;
    };
    float next = rg.u0 < rg.u1 ? row_lse(rg.u0 / pairs, 0) : 0.f;
    for (int u = rg.u0; u < rg.u1; ++u) {
      const int kvh = u / pairs, b = (u - kvh * pairs) * 2 + s;
      if (b >= a.nb) {                           // an odd last block: no second one
        if (u + 1 < rg.u1) next = row_lse((u + 1) / pairs, 0);
        continue;
      }
      const bool ctx = b < a.nb_ctx;
      const int key = ctx ? b * kTreeKeys + r : a.n + (b - a.nb_ctx) * kTreeKeys + r;
      const bool live = key < (ctx ? a.n : a.n + a.T);
      const size_t o = (size_t)kvh * a.max_seq + key;
      const float before = live && ctx && a.w_in ? a.w_in[o] : 0.f;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int t = 0; t < a.tiles; ++t, ++c) {
        const int buf = c & 1, cols = min(128, rows - t * 128);
        float* nl = nlse + s * 128;
        const float x = next;
        stream_sync(s);                          // the tile before has been read
        nl[r] = x;
        const bool some = stream_any(s, x == -INFINITY);
        // the next tile's, or the next unit's first, ahead of its use
        if (t + 1 < a.tiles)
          next = row_lse(kvh, t + 1);
        else if (u + 1 < rg.u1)
          next = row_lse((u + 1) / pairs, 0);
        ok = ok && !tree_flagged(fail) && mbar_wait_n(&sfull[s * 2 + buf], (uint32_t)((c >> 1) & 1), kPolls);
        const bool all_ok = __all_sync(0xffffffffu, ok);
        if (!all_ok) {
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
                const int row = min(t * 128 + q0 + lane, rows - 1);
                const uint32_t mine =
                    a.anc[(size_t)(row / a.G) * a.anc_words + (b - a.nb_ctx) * 4 + (warp & 3)];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const uint32_t w = __shfl_sync(0xffffffffu, mine, e);
                  const float p = tree_ex2(fmaf(__uint_as_float(v[hlf][e]), scale, nl[q0 + e]));
                  if ((w >> lane) & 1u) sum[e & 3] += p;
                }
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive_cta(&sfree[s * 2 + buf]);
      }
      if (live) a.w_out[o] = ok ? before + ((sum[0] + sum[1]) + (sum[2] + sum[3])) : NAN;
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
  const long long units = (long long)a.Hkv * ((a.nb + 1) / 2);
  lc.gridDim = dim3((unsigned)(units < sms ? units : sms));
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
