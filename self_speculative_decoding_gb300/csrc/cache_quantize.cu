// Cache rows to 8 bits (sm_103a).
//
// A block of `block` rows of one head becomes e4m3 values and one scale,
//   scale = 2^e, the smallest with max |x| <= 448 2^e   (e >= -64; 1 for zeros)
//   x8    = e4m3(x / scale), to nearest, ties to even.
// The scale is a power of two: a division by it is exact, so that each value is
// rounded once, and e4m3, being a floating format, has the same relative steps
// wherever the largest value lies in its last binade.  Infinities and NaN become
// NaN and do not enter the scale.
//
// Bound by the bytes: bf16 in, e4m3 out, once each, as a block stays in registers
// between its maximum and its conversion.  128 K rows of 8 heads: 489 MB in 79 us, 6.2
// TB/s, 92% of a plain copy's (the rest is the wait between a block's loads and its
// stores, which eight CTAs of an SM hide from one another); one block each of a
// few sequences: 3.1 us, a launch and three latencies.
#include <cuda_fp8.h>

#include "batch.cuh"
#include "tree.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

// Sequence b's whole blocks that are to be moved: [from, to).
SSD_DI void blocks_of(const QuantizeArgs& a, int b, int& from, int& to) {
  const int held = a.held[b], n = a.lengths[b];
  from = to = 0;
  if (held < 0 || held % a.block || held > a.max_seq || n > a.max_seq || n <= held) return;
  if (n - held > a.rows) return;                 // the ring has lost a row
  from = held / a.block;
  to = n / a.block;
}

SSD_DI uint32_t abs_finite(uint32_t x) {         // of two bf16: |x|'s bits, 0 if not finite
  x &= 0x7fff7fffu;
  if ((x & 0xffffu) >= 0x7f80u) x &= 0xffff0000u;
  if (x >= 0x7f800000u) x &= 0xffffu;
  return x;
}
// Two bf16 times inv as two e4m3; what is not finite as NaN.
SSD_DI uint32_t two_of(uint32_t x, float inv) {
  return __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(x) * inv, bf16_hi(x) * inv), __NV_SATFINITE, __NV_E4M3);
}
SSD_DI uint32_t two_any(uint32_t x, float inv) {
  uint32_t r = two_of(x, inv);
  if ((x & 0x7f80u) == 0x7f80u) r |= 0x7fu;
  if ((x & 0x7f800000u) == 0x7f800000u) r |= 0x7f00u;
  return r;
}
SSD_DI uint32_t largest(uint32_t most) {         // over a warp, of packed pairs
  return __reduce_max_sync(~0u, max(most & 0xffffu, most >> 16));
}

// Items = (sequence, block, head), dealt to the CTAs in turn; a CTA has a block of K
// and of V in registers: one read, one write.
template <int DH, int UNITS>                     // 16-byte units of a block per thread
__global__ void __launch_bounds__(kThreads) cache_quantize_kernel(const __grid_constant__ QuantizeArgs a) {
  __shared__ int first[kBatchMaxSeqs + 1];       // blocks of all sequences before b
  __shared__ uint32_t warp_max[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  for (int b = tid; b < a.B; b += kThreads) {
    int from, to;
    blocks_of(a, b, from, to);
    first[b + 1] = to - from;
    if (blockIdx.x == 0) a.held_out[b] = to > from ? to * a.block : a.held[b];
  }
  if (tid == 0) first[0] = 0;
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int x = b0 + lane < a.B ? first[b0 + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
      }
      if (b0 + lane < a.B) first[b0 + lane + 1] = sum + x;
      sum += __shfl_sync(~0u, x, 31);
    }
  }
  __syncthreads();
  const int total = first[a.B];
  for (long long item = blockIdx.x; item < (long long)total * a.Hkv; item += gridDim.x) {
    const int j = (int)(item / a.Hkv), h = (int)(item - (long long)j * a.Hkv);
    int lo = 0, hi = a.B - 1;                    // the last b with first[b] <= j
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (first[mid] <= j) lo = mid;
      else hi = mid - 1;
    }
    int from, to;
    blocks_of(a, lo, from, to);
    const int block = from + j - first[lo];
    const size_t row0 = (size_t)block * a.block;
    const size_t from_head = (size_t)lo * a.seq_stride + (size_t)h * a.rows * DH;
    const size_t to_head = (size_t)lo * a.seq8_stride + ((size_t)h * a.max_seq + row0) * DH;
    // (a block turns over at the ring's end once at most)
    const int slot0 = (int)((unsigned)row0 % (unsigned)a.rows);
    uint4 x[2][UNITS];                           // of K, of V
#pragma unroll
    for (int q = 0; q < UNITS; ++q) {
      const int e = (tid + q * kThreads) * 8, at = slot0 + e / DH;
      const size_t o = from_head + (size_t)(at < a.rows ? at : at - a.rows) * DH + e % DH;
      x[0][q] = __ldcs(reinterpret_cast<const uint4*>(a.k + o));
      x[1][q] = __ldcs(reinterpret_cast<const uint4*>(a.v + o));
    }
    uint32_t most[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < UNITS; ++q)
        m = __vmaxu2(__vmaxu2(m, __vmaxu2(x[z][q].x & 0x7fff7fffu, x[z][q].y & 0x7fff7fffu)),
                     __vmaxu2(x[z][q].z & 0x7fff7fffu, x[z][q].w & 0x7fff7fffu));
      most[z] = largest(m);
    }
    __syncthreads();                             // (the item before has read)
    if (lane < 2) warp_max[lane][warp] = lane ? most[1] : most[0];
    __syncthreads();
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint32_t m = __reduce_max_sync(~0u, lane < kThreads / 32 ? warp_max[z][lane] : 0u);
      const bool odd = m >= 0x7f80u;             // something is not finite: without it
      if (odd) {
        m = 0;
#pragma unroll
        for (int q = 0; q < UNITS; ++q)
          m = __vmaxu2(__vmaxu2(m, __vmaxu2(abs_finite(x[z][q].x), abs_finite(x[z][q].y))),
                       __vmaxu2(abs_finite(x[z][q].z), abs_finite(x[z][q].w)));
        m = largest(m);
        __syncthreads();
        if (lane == 0) warp_max[z][warp] = m;
        __syncthreads();
        m = __reduce_max_sync(~0u, lane < kThreads / 32 ? warp_max[z][lane] : 0u);
      }
      float scale = 1.f;
      int e = 0;
      if (m) {
        const float part = frexpf(__uint_as_float(m << 16), &e);
        e = max(e - (part > 0.875f ? 8 : 9), -64);
        scale = ldexpf(1.f, e);
      }
      const float inv = ldexpf(1.f, -e);
      uint8_t* dst = (z ? a.v8 : a.k8) + to_head;
#pragma unroll
      for (int q = 0; q < UNITS; ++q) {
        const uint4 w = x[z][q];
        uint2 y;
        if (!odd)
          y = make_uint2(two_of(w.x, inv) | two_of(w.y, inv) << 16, two_of(w.z, inv) | two_of(w.w, inv) << 16);
        else
          y = make_uint2(two_any(w.x, inv) | two_any(w.y, inv) << 16, two_any(w.z, inv) | two_any(w.w, inv) << 16);
        *reinterpret_cast<uint2*>(dst + (size_t)(tid + q * kThreads) * 8) = y;
      }
      if (tid == 0)
        (z ? a.v_scale : a.k_scale)[(size_t)lo * a.scale_stride + (size_t)h * (a.max_seq / a.block) + block] = scale;
    }
  }
}

template <int DH>
cudaError_t launch(const QuantizeArgs& a, unsigned ctas, cudaStream_t s) {
  switch (a.block) {
    case 32: return launch_early(cache_quantize_kernel<DH, 32 * DH / 8 / kThreads>, ctas, kThreads, 0, s, 0, a);
    case 64: return launch_early(cache_quantize_kernel<DH, 64 * DH / 8 / kThreads>, ctas, kThreads, 0, s, 0, a);
    default: return launch_early(cache_quantize_kernel<DH, 128 * DH / 8 / kThreads>, ctas, kThreads, 0, s, 0, a);
  }
}

}  // namespace

cudaError_t launch_cache_quantize(const QuantizeArgs& a, cudaStream_t s) {
  // at most so many items, and eight CTAs for each SM
  const long long most = (long long)a.B * a.Hkv * ((a.rows < a.max_seq ? a.rows : a.max_seq) / a.block + 1);
  const unsigned ctas = (unsigned)(most < 8 * tree_sms() ? most : 8 * tree_sms());
  return a.dh == 128 ? launch<128>(a, ctas, s) : launch<64>(a, ctas, s);
}

}  // namespace ssd
