// Attention of a tree of drafted tokens over the K/V cache (sm_103a).
//
// T nodes follow n cache rows.  Node t with parent chain t -> p -> ... -> -1
// has depth(t) ancestors; its query and key are rotated to position
// pos0 + depth(t), its K/V rows go to cache rows n + t, and it attends to
// every cache row < n, its ancestors and itself:
//   out_t = sum_j softmax_j(q_t k_j / sqrt(dh)) v_j.
// A row whose chain does not end in -1 is absent.
#include "tree.cuh"

namespace ssd {
namespace {

constexpr int kPrepHeads = 8;      // heads per CTA of the preparation
constexpr int kPrepThreads = 256;

// One CTA per (node, group of heads): the node's ancestor bits and depth,
// the rotated query in two bf16 parts (q = hi + lo to 2^-17: the scores keep
// 32-bit accuracy on bf16 matrix instructions), the K/V rows rounded to bf16
// into the cache and, with inf and NaN of V replaced by 0, into the tree's
// own copy (a matrix product must not meet 0 x inf at masked keys).
// Angles: position * frequency in 64 bits, reduced to one turn, so that far
// positions keep their angle.
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ int par[kTreeMaxNodes];
  __shared__ uint32_t bits[kTreeMaxNodes / 32];
  __shared__ int s_depth;
  __shared__ int bad[kPrepHeads];
  const int t = blockIdx.x, tid = threadIdx.x;
  for (int i = tid; i <= t; i += kPrepThreads) par[i] = a.parents[i];
  for (int i = tid; i < kTreeMaxNodes / 32; i += kPrepThreads) bits[i] = 0u;
  if (tid < kPrepHeads) bad[tid] = 0;
  __syncthreads();
  if (tid == 0) {
    int cur = t, d = 0;
    while (true) {  // parents strictly decrease: at most t + 1 steps
      bits[cur >> 5] |= 1u << (cur & 31);
      const int p = par[cur];
      if (p == -1) break;
      if (p < 0 || p >= cur) {
        d = -1;
        break;
      }
      cur = p;
      ++d;
    }
    s_depth = d;
  }
  __syncthreads();
  const int d = s_depth;
  if (blockIdx.y == 0) {
    for (int w = tid; w < a.anc_words; w += kPrepThreads)
      a.anc[(size_t)t * a.anc_words + w] = d >= 0 ? bits[w] : 0u;
    if (tid == 0) a.depth[t] = d;
  }
  const int half = a.dh >> 1, heads = a.H + 2 * a.Hkv;
  const int h0 = blockIdx.y * kPrepHeads, h1 = min(h0 + kPrepHeads, heads);
  const float* row = a.qkv + (size_t)t * heads * a.dh;
  const size_t qplane = (size_t)a.Hkv * a.T * a.G * a.dh;
  for (int e = tid; e < (h1 - h0) * half; e += kPrepThreads) {
    const int h = h0 + e / half, i = e % half;
    float x = row[(size_t)h * a.dh + i], y = row[(size_t)h * a.dh + half + i];
    if (d < 0) x = y = 0.f;
    if (h < a.H + a.Hkv) {
      double turn = (double)(a.pos0 + max(d, 0)) * a.inv_freq[i];  // angle / pi
      turn -= 2.0 * rint(0.5 * turn);
      float sn, cs;
      sincospif((float)turn, &sn, &cs);
      const float rx = x * cs - y * sn, ry = y * cs + x * sn;
      x = rx;
      y = ry;
    }
    if (h < a.H) {
      const int kvh = h / a.G, g = h - kvh * a.G;
      const size_t o = ((size_t)kvh * a.T * a.G + (size_t)t * a.G + g) * a.dh + i;
      const bf16 xh = __float2bfloat16(x), yh = __float2bfloat16(y);
      a.q[o] = xh;
      a.q[o + half] = yh;
      const float xl = x - __bfloat162float(xh), yl = y - __bfloat162float(yh);
      a.q[qplane + o] = __float2bfloat16(isfinite(xl) ? xl : 0.f);
      a.q[qplane + o + half] = __float2bfloat16(isfinite(yl) ? yl : 0.f);
    } else {
      const bool is_k = h < a.H + a.Hkv;
      const int kvh = is_k ? h - a.H : h - a.H - a.Hkv;
      bf16 b0 = __float2bfloat16(x), b1 = __float2bfloat16(y);
      bf16* c = (is_k ? a.kc : a.vc) + ((size_t)kvh * a.max_seq + a.n + t) * a.dh + i;
      c[0] = b0;
      c[half] = b1;
      if (!is_k) {
        const bool f0 = isfinite(__bfloat162float(b0)), f1 = isfinite(__bfloat162float(b1));
        if (!f0) b0 = __float2bfloat16(0.f);
        if (!f1) b1 = __float2bfloat16(0.f);
        if (!(f0 && f1)) bad[h - h0] = 1;
      }
      bf16* m = (is_k ? a.kt : a.vt) + ((size_t)kvh * a.T + t) * a.dh + i;
      m[0] = b0;
      m[half] = b1;
    }
  }
  __syncthreads();
  for (int h = h0 + tid; h < h1; h += kPrepThreads)
    if (h >= a.H + a.Hkv) a.vbad[(size_t)(h - a.H - a.Hkv) * a.T + t] = (uint8_t)bad[h - h0];
}

SSD_DI bool sees(const TreeArgs& a, int t, int node) {
  return (a.anc[(size_t)t * a.anc_words + (node >> 5)] >> (node & 31)) & 1u;
}

constexpr int kRowsPerCta = 8;
constexpr int kTile = 64;

// One warp per (row, query head), keys in tiles of 64 shared by eight rows of
// a K/V head: each lane scores two keys, the running maximum and sum are
// those of the warp, and each lane sums dh / 32 output columns.
template <int DH>
__global__ void __launch_bounds__(kRowsPerCta * 32)
    tree_attn_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kPad = DH + 2;  // one 4-byte bank further per key
  constexpr int kCols = DH / 32;
  __shared__ bf16 sk[kTile * kPad], sv[kTile * kPad];
  __shared__ float sq[kRowsPerCta][DH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y, rows = a.T * a.G;
  const int r = blockIdx.x * kRowsPerCta + warp;
  const bool live = r < rows;
  const int t = live ? r / a.G : 0;
  const bool present = live && a.depth[t] >= 0;
  const size_t plane = (size_t)a.Hkv * rows * DH;
  if (live) {
    const bf16* q = a.q + ((size_t)kvh * rows + r) * DH;
    for (int i = lane; i < DH; i += 32)
      sq[warp][i] = __bfloat162float(q[i]) + __bfloat162float(q[plane + i]);
  }
  float m = -INFINITY, l = 0.f, o[kCols] = {};
  const int total = a.n + a.T;
  for (int k0 = 0; k0 < total; k0 += kTile) {
    __syncthreads();
    for (int e = threadIdx.x; e < kTile * DH; e += blockDim.x) {
      const int kk = k0 + e / DH, i = e % DH;
      bf16 kx = __float2bfloat16(0.f), vx = kx;
      if (kk < a.n) {
        kx = a.kc[((size_t)kvh * a.max_seq + kk) * DH + i];
        vx = a.vc[((size_t)kvh * a.max_seq + kk) * DH + i];
      } else if (kk < total) {
        kx = a.kt[((size_t)kvh * a.T + kk - a.n) * DH + i];
        vx = a.vt[((size_t)kvh * a.T + kk - a.n) * DH + i];
      }
      sk[(e / DH) * kPad + i] = kx;
      sv[(e / DH) * kPad + i] = vx;
    }
    __syncthreads();
    if (!present) continue;
    float s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = lane + 32 * u, kk = k0 + key;
      float acc = 0.f;
      for (int i = 0; i < DH; ++i) acc = fmaf(sq[warp][i], __bfloat162float(sk[key * kPad + i]), acc);
      const bool vis = kk < a.n || (kk < total && sees(a, t, kk - a.n));
      s[u] = vis ? acc * a.scale_log2 : -INFINITY;
    }
    float bm = fmaxf(s[0], s[1]);
    for (int w = 16; w; w >>= 1) bm = fmaxf(bm, __shfl_xor_sync(~0u, bm, w));
    const float mn = fmaxf(m, bm), base = mn == -INFINITY ? 0.f : mn;
    const float corr = exp2f(m - base);  // m = -inf: 0 times an empty sum
    l *= corr;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] *= corr;
    m = mn;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float p = exp2f(s[u] - base);
      float ps = p;
      for (int w = 16; w; w >>= 1) ps += __shfl_xor_sync(~0u, ps, w);
      l += ps;
      for (int j = 0; j < 32; ++j) {
        const float pj = __shfl_sync(~0u, p, j);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          o[c] = fmaf(pj, __bfloat162float(sv[(u * 32 + j) * kPad + c * 32 + lane]), o[c]);
      }
    }
  }
  if (!live) return;
  const float lse = l > 0.f || isnan(l) ? m + log2f(l) : INFINITY;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] *= inv;
  if (present) {
    // inf and NaN of the V rows that this row sees (left out above)
    for (int j = 0; j <= t; ++j) {
      if (!a.vbad[(size_t)kvh * a.T + j] || !sees(a, t, j)) continue;
      float acc = 0.f;
      for (int i = 0; i < DH; ++i)
        acc = fmaf(sq[warp][i], __bfloat162float(a.kt[((size_t)kvh * a.T + j) * DH + i]), acc);
      const float p = exp2f(acc * a.scale_log2 - lse);
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float v = __bfloat162float(a.vc[((size_t)kvh * a.max_seq + a.n + j) * DH + c * 32 + lane]);
        if (!isfinite(v)) o[c] += p * v;
      }
    }
  }
  const int h = kvh * a.G + r % a.G;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    a.out[((size_t)t * a.H + h) * DH + c * 32 + lane] = __float2bfloat16(o[c]);
  if (lane == 0) a.lse[(size_t)kvh * rows + r] = present ? lse : INFINITY;
}

// Weights: thread = key; w_out = w_in + the sum over the group's rows of
// 2^(score - lse), added in row order (the same bits on every call).
template <int DH>
__global__ void __launch_bounds__(kTreeKeys) tree_weight_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float sq[DH];
  const int kvh = blockIdx.y, kk = blockIdx.x * kTreeKeys + threadIdx.x;
  const int total = a.n + a.T, rows = a.T * a.G;
  const size_t plane = (size_t)a.Hkv * rows * DH;
  float kx[DH];
  if (kk < total) {
    const bf16* k = kk < a.n ? a.kc + ((size_t)kvh * a.max_seq + kk) * DH
                             : a.kt + ((size_t)kvh * a.T + kk - a.n) * DH;
#pragma unroll
    for (int i = 0; i < DH; ++i) kx[i] = __bfloat162float(k[i]);
  }
  float sum = 0.f;
  for (int r = 0; r < rows; ++r) {
    const bf16* q = a.q + ((size_t)kvh * rows + r) * DH;
    __syncthreads();
    for (int i = threadIdx.x; i < DH; i += kTreeKeys)
      sq[i] = __bfloat162float(q[i]) + __bfloat162float(q[plane + i]);
    __syncthreads();
    const float lse = a.lse[(size_t)kvh * rows + r];
    if (kk >= total || (kk >= a.n && !sees(a, r / a.G, kk - a.n))) continue;
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < DH; ++i) acc = fmaf(sq[i], kx[i], acc);
    if (lse != INFINITY) sum += exp2f(acc * a.scale_log2 - lse);
  }
  if (kk < total) {
    const size_t o = (size_t)kvh * a.max_seq + kk;
    a.w_out[o] = kk < a.n && a.w_in ? a.w_in[o] + sum : sum;
  }
}

}  // namespace

size_t tree_workspace(TreeArgs& a, void* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return base ? (void*)((char*)base + at) : nullptr;
  };
  const size_t rows = (size_t)a.T * a.G;
  a.anc_words = tree_anc_words(a.T);
  a.anc = (uint32_t*)take((size_t)a.T * a.anc_words * 4);
  a.depth = (int32_t*)take((size_t)a.T * 4);
  a.vbad = (uint8_t*)take((size_t)a.Hkv * a.T);
  a.q = (bf16*)take(2 * a.Hkv * rows * a.dh * sizeof(bf16));
  a.kt = (bf16*)take((size_t)a.Hkv * a.T * a.dh * sizeof(bf16));
  a.vt = (bf16*)take((size_t)a.Hkv * a.T * a.dh * sizeof(bf16));
  a.lse = (float*)take(a.Hkv * rows * 4);
  return off;
}

cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s) {
  const int heads = a.H + 2 * a.Hkv, rows = a.T * a.G;
  tree_prep_kernel<<<dim3(a.T, (heads + kPrepHeads - 1) / kPrepHeads), kPrepThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((rows + kRowsPerCta - 1) / kRowsPerCta, a.Hkv);
  if (a.dh == 128)
    tree_attn_kernel<128><<<grid, kRowsPerCta * 32, 0, s>>>(a);
  else
    tree_attn_kernel<64><<<grid, kRowsPerCta * 32, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || !a.w_out) return e;
  const dim3 wgrid((a.n + a.T + kTreeKeys - 1) / kTreeKeys, a.Hkv);
  if (a.dh == 128)
    tree_weight_kernel<128><<<wgrid, kTreeKeys, 0, s>>>(a);
  else
    tree_weight_kernel<64><<<wgrid, kTreeKeys, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ssd
