// Norms of the query and key heads, rotation and append (sm_103a).
//
// Token t of sequence b, at position p, for each query and key head:
//   x' = x / sqrt(mean x^2 + eps) * gain            (where there is a gain)
//   (x'_i, x'_{i + dh/2}) turned by the angle p theta^(-2 i / dh),
// q rounded to bf16 into q, k' and v into row (length + t) % rows of the caches.
//
// Angles: a turn is 2^64, so that position * frequency wraps by itself and
// keeps 2^-64 of a turn times the position, however far that is; the product's
// upper half, exact to 2^-24 of a half turn as fp32, gives sine and cosine.
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

SSD_DI void load_pair(const float* p, float (&x)[4], int half) {
  const float2 a = *reinterpret_cast<const float2*>(p), b = *reinterpret_cast<const float2*>(p + half);
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

// A warp takes one token and `kHeads` groups of heads; a lane two pairs of
// (i, i + dh/2) of a head, so that a warp holds 128 / dh heads at a time and
// needs no barrier.  The loads of all its heads go out before the first use.
template <int DH, int kHeads>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int kLanes = DH / 4, kAtOnce = 32 / kLanes, kHalf = DH / 2;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, i = 2 * (lane % kLanes);
  const int heads = a.H + 2 * a.Hkv, groups = (heads + kAtOnce * kHeads - 1) / (kAtOnce * kHeads);
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long token = w / groups;
  const int h0 = (int)(w - token * groups) * kAtOnce * kHeads + sub;
  if (token >= (long long)a.B * a.T) return;
  const int b = (int)(token / a.T), t = (int)(token - (long long)b * a.T);
  float x[kHeads][4];
#pragma unroll
  for (int q = 0; q < kHeads; ++q) {
    const int h = h0 + q * kAtOnce;
    if (h < heads) load_pair(a.qkv + (size_t)token * heads * DH + (size_t)h * DH + i, x[q], kHalf);
  }
  const int n = a.lengths[b];
  const bool here = t < batch_count(a.counts, a.lengths, b, a.T);
  const int64_t pos = (int64_t)(a.positions ? a.positions[b] : n) + t;
  const float2 r0 = turn_of(pos, a.turns[i]), r1 = turn_of(pos, a.turns[i + 1]);
  const size_t slot = here ? (size_t)((n + t) % a.rows) : 0;
#pragma unroll
  for (int q = 0; q < kHeads; ++q) {
    const int h = h0 + q * kAtOnce;
    float(&y)[4] = x[q];
    const float* gain = h < a.H ? a.q_gain : h < a.H + a.Hkv ? a.k_gain : nullptr;
    float ss = h < heads ? y[0] * y[0] + y[1] * y[1] + y[2] * y[2] + y[3] * y[3] : 0.f;
    if (a.q_gain || a.k_gain)
#pragma unroll
      for (int d = kLanes / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if (h >= heads) continue;
    if (gain) {
      const float s = 1.f / sqrtf(ss * (1.f / DH) + a.eps);
      float g[4];
      load_pair(gain + i, g, kHalf);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= s * g[e];
    }
    if (h < a.H + a.Hkv) {
      const float u0 = y[0] * r0.x - y[2] * r0.y, u1 = y[1] * r1.x - y[3] * r1.y;
      y[2] = y[2] * r0.x + y[0] * r0.y;
      y[3] = y[3] * r1.x + y[1] * r1.y;
      y[0] = u0;
      y[1] = u1;
    }
    bf16* to;
    if (h < a.H) {
      to = a.q + ((size_t)token * a.H + h) * DH;
      if (!here) y[0] = y[1] = y[2] = y[3] = 0.f;
    } else {
      if (!here) continue;
      const bool is_k = h < a.H + a.Hkv;
      const int kvh = h - a.H - (is_k ? 0 : a.Hkv);
      to = (is_k ? a.k : a.v) + (size_t)b * a.seq_stride + ((size_t)kvh * a.rows + slot) * DH;
    }
    *reinterpret_cast<uint32_t*>(to + i) = pack_bf16x2(y[0], y[1]);
    *reinterpret_cast<uint32_t*>(to + kHalf + i) = pack_bf16x2(y[2], y[3]);
  }
}

template <int DH, int kHeads>
cudaError_t launch(const RopeAppendArgs& a, cudaStream_t s) {
  constexpr int kEach = 128 / DH * kHeads;
  const long long warps = (long long)a.B * a.T * ((a.H + 2 * a.Hkv + kEach - 1) / kEach);
  const long long ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
  rope_append_kernel<DH, kHeads><<<dim3((unsigned)ctas), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendArgs& a, cudaStream_t s) {
  return a.dh == 128 ? launch<128, 4>(a, s) : launch<64, 4>(a, s);
}

}  // namespace ssd
