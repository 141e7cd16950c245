// Norms of the query and key heads, rotation and append (sm_103a).
//
// Token t of sequence b, at position p, for each query and key head:
//   x' = x / sqrt(mean x^2 + eps) * gain            (where there is a gain)
//   (x'_i, x'_{i + dh/2}) turned by the angle p theta^(-2 i / dh),
// q rounded to bf16 into q, k' and v into row (length + t) % rows of the caches.
//
// Angles: a turn is 2^64, so that position * frequency wraps by itself.  The
// frequencies come from 64-bit floats and are good to 2^-54 of a turn (bases of 1 or
// more), which is 2^-22 of a half turn at position 2^31; the product's upper half, as
// fp32 good to 2^-25 of a half turn, gives sine and cosine.
//
// Bound by the bytes: fp32 in, bf16 out, once each.  8064 tokens of 120 heads: 743 MB
// in 114 us, 6.5 TB/s, 97% of a plain copy's; one token: 2.3 us, a launch.  Roundings: q,
// k', v to bf16, which the caches and the products take; all else is fp32.
#include "batch.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

SSD_DI float2 turn_of(int64_t pos, uint64_t frequency) {
  const int32_t x = (int32_t)((uint64_t)pos * frequency >> 32);  // of a turn, -1/2 .. 1/2
  float2 r;
  sincospif((float)x * 0x1p-31f, &r.y, &r.x);
  return r;
}

SSD_DI void load_quads(const float* p, float (&x)[8], int half) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + half);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// A warp takes one token and `kSteps` times as many heads as it holds at once (256
// elements): a lane has four pairs (i, i + dh/2) of a head, and needs their four
// angles once.  No barrier; the next step's loads go out before this one's work.
template <int DH, int kSteps, bool NORMS>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int kLanes = DH / 8, kAtOnce = 32 / kLanes, kHalf = DH / 2;
  const int lane = threadIdx.x & 31, i = 4 * (lane % kLanes);
  const int heads = a.H + 2 * a.Hkv, groups = (heads + kAtOnce * kSteps - 1) / (kAtOnce * kSteps);
  const unsigned w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned token = w / groups;
  if (token >= (unsigned)(a.B * a.T)) return;
  int h = (int)(w - token * groups) * kAtOnce * kSteps + lane / kLanes;
  const int b = (int)(token / (unsigned)a.T), t = (int)(token - (unsigned)b * a.T);
  const float* src = a.qkv + ((size_t)token * heads + h) * DH + i;
  float x[8], next[8] = {};
  pdl_wait();
  pdl_trigger();
  if (h < heads) load_quads(src, next, kHalf);
  const int n = a.lengths[b];
  const bool here = t < batch_count(a.counts, a.lengths, b, a.T);
  const int64_t pos = (int64_t)(a.positions ? a.positions[b] : n) + t;
  float2 r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = turn_of(pos, a.turns[i + e]);
  const size_t row = (size_t)b * a.seq_stride + (size_t)(here ? (n + t) % a.rows : 0) * DH + i;
#pragma unroll 1
  for (int step = 0; step < kSteps; ++step, h += kAtOnce) {
    if (NORMS ? h - lane / kLanes >= heads : h >= heads) break;
    src += kAtOnce * DH;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = next[e];
    if (step + 1 < kSteps && h + kAtOnce < heads) load_quads(src, next, kHalf);
    if (NORMS) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      const float* gain = h < a.H ? a.q_gain : h < a.H + a.Hkv ? a.k_gain : nullptr;
      if (gain) {
        const float scale = rsqrtf(fmaf(ss, 1.f / DH, a.eps));
        float g[8];
        load_quads(gain + i, g, kHalf);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= scale * g[e];
      }
      if (h >= heads) continue;
    }
    if (h < a.H + a.Hkv)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[e] * r[e].x - x[e + 4] * r[e].y;
        x[e + 4] = x[e + 4] * r[e].x + x[e] * r[e].y;
        x[e] = u;
      }
    bf16* to;
    if (h < a.H) {
      to = a.q + ((size_t)token * a.H + h) * DH + i;
      if (!here)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
    } else {
      if (!here) continue;
      to = (h < a.H + a.Hkv ? a.k : a.v) + row + (size_t)(h - a.H - (h < a.H + a.Hkv ? 0 : a.Hkv)) * a.rows * DH;
    }
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    *reinterpret_cast<uint2*>(to + kHalf) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

template <int DH, int kSteps>
cudaError_t launch(const RopeAppendArgs& a, cudaStream_t s) {
  constexpr int kEach = 256 / DH * kSteps;
  const long long warps = (long long)a.B * a.T * ((a.H + 2 * a.Hkv + kEach - 1) / kEach);
  const unsigned ctas = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
  return a.q_gain || a.k_gain ? launch_early(rope_append_kernel<DH, kSteps, true>, ctas, kThreads, 0, s, 0, a)
                              : launch_early(rope_append_kernel<DH, kSteps, false>, ctas, kThreads, 0, s, 0, a);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s) {
  // Few tokens: a warp for every 256 elements; many: the angles serve 8 times that.
  // (48 heads of 128, us: 64 tokens 3.3 and 4.0, 128 tokens 3.8 and 4.0, 192 tokens
  // 4.5 and 4.1, 512 tokens 9.2 and 5.1, 4096 tokens 57 and 28)
  const bool many = (long long)a.B * a.T * (a.H + 2 * a.Hkv) * a.dh >= (long long)1 << 20;
  if (a.dh == 128) return many ? launch<128, 8>(a, s) : launch<128, 1>(a, s);
  return many ? launch<64, 8>(a, s) : launch<64, 1>(a, s);
}

}  // namespace ssd
