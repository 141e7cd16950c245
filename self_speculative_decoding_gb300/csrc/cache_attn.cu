// Attention of a few tokens per sequence over a cache of 8-bit and bf16 rows
// (sm_103a), the plain way: a CTA per (sequence, token, head), a warp per row.
#include <cuda_fp8.h>

#include "batch.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;

template <int DH>
__global__ void __launch_bounds__(kWarps * 32) cache_attn_kernel(const __grid_constant__ CacheAttnArgs a) {
  constexpr int E = DH / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][DH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % a.H, t = blockIdx.x / a.H % a.T, b = blockIdx.x / a.H / a.T;
  const int kvh = h / a.G;
  const SeqRange r = seq_range(a, b);
  bf16* out = a.out + (size_t)blockIdx.x * DH;
  if (t >= r.count) {
    for (int i = threadIdx.x; i < DH; i += kWarps * 32) out[i] = __float2bfloat16(r.count < 0 ? NAN : 0.f);
    return;
  }
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[(size_t)blockIdx.x * DH + lane * E + e]);
  const int pos = r.length + t;
  for (int j = warp; j <= pos; j += kWarps) {
    if (a.window && j >= a.sinks && j <= pos - a.window) continue;
    float k[E], v[E];
    if (j < r.held) {
      const size_t at = (size_t)b * a.seq8_stride + ((size_t)kvh * a.max_seq + j) * DH + lane * E;
      const size_t sc = (size_t)b * a.scale_stride + (size_t)kvh * (a.max_seq / a.block) + j / a.block;
      for (int e = 0; e < E; ++e) {
        __nv_fp8_e4m3 x, y;
        x.__x = a.k8[at + e];
        y.__x = a.v8[at + e];
        k[e] = (float)x * a.k_scale[sc];
        v[e] = (float)y * a.v_scale[sc];
      }
    } else {
      const size_t at = (size_t)b * a.seq_stride + ((size_t)kvh * a.rows + j % a.rows) * DH + lane * E;
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(a.k[at + e]);
        v[e] = __bfloat162float(a.v[at + e]);
      }
    }
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float w = exp2f(m - base), p = exp2f(s - base);
    l = l * w + p;
    for (int e = 0; e < E; ++e) o[e] = o[e] * w + p * v[e];
    m = mn;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  float all = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) all = fmaxf(all, s_m[w]);
  if (all == -INFINITY) all = 0.f;
  for (int w = 0; w < kWarps; ++w) sum += s_l[w] * exp2f(s_m[w] - all);
  for (int i = threadIdx.x; i < DH; i += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += s_o[w][i] * exp2f(s_m[w] - all);
    out[i] = __float2bfloat16(sum != 0.f ? x / sum : 0.f);
  }
}

}  // namespace

size_t cache_attn_workspace(CacheAttnArgs&, void*) { return 256; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, cudaStream_t s) {
  const unsigned ctas = (unsigned)(a.B * a.T * a.H);
  if (a.dh == 128) cache_attn_kernel<128><<<ctas, kWarps * 32, 0, s>>>(a);
  else cache_attn_kernel<64><<<ctas, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssd
