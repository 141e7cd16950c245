// Attention of a tree of drafted tokens over the K/V cache (sm_103a).
//
// T nodes follow n cache rows.  Node t with parent chain t -> p -> ... -> -1
// has depth(t) ancestors; its query and key are rotated to position
// pos0 + depth(t), its K/V rows go to cache rows n + t, and it attends to
// every cache row < n, its ancestors and itself:
//   out_t = sum_j softmax_j(q_t k_j / sqrt(dh)) v_j.
// A row whose chain does not end in -1 is absent.
#include "tc_dev.cuh"
#include "tree.cuh"

namespace ssd {
namespace {

constexpr int kPrepHeads = 8;      // heads per CTA of the preparation
constexpr int kPrepThreads = 256;
constexpr int kWalk = 32;          // ancestors found one by one

// A node deep in its tree: of the nodes up to t, those that a marked one (bits)
// reaches, by jumps of 1, 2, 4, ... nodes (one by one, a chain of 1024 nodes over
// 1000 rows, 8 heads, took 139 us, 55 so).  par becomes the jumps' ends; depth
// -1: absent.
__device__ __noinline__ void far_ancestors(int t, int* par, uint32_t* bits, int& depth) {
  constexpr int kRoot = kTreeMaxNodes, kAbsent = kTreeMaxNodes + 1;
  constexpr int kEach = kTreeMaxNodes / kPrepThreads;
  const int tid = threadIdx.x;
  for (int i = tid; i <= t; i += kPrepThreads) {
    const int p = par[i];
    par[i] = p == -1 ? kRoot : p < 0 || p >= i ? kAbsent : p;
  }
  if (tid < 2) par[kRoot + tid] = kRoot + tid;
  if (tid == 0) depth = 0;
  __syncthreads();
  for (int reach = 1; reach <= t; reach *= 2) {
    int far[kEach];
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      const int i = q * kPrepThreads + tid;
      if (i > t) continue;
      const int p = par[i];
      if ((bits[i >> 5] >> (i & 31)) & 1u) {
        if (p < kRoot) atomicOr(&bits[p >> 5], 1u << (p & 31));
        if (p == kAbsent) depth = -1;
      }
      far[q] = par[p];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kEach; ++q)
      if (q * kPrepThreads + tid <= t) par[q * kPrepThreads + tid] = far[q];
    __syncthreads();
  }
  if (tid < 32) {
    const int n = __reduce_add_sync(~0u, __popc(bits[tid]));
    if (tid == 0 && depth == 0) depth = n - 1;
  }
  __syncthreads();
}

// q = hi + lo to 2^-16 of q (hi alone: 2^-7), so that bf16 matrix instructions
// give scores to 2^-16 of sum |q_i k_i|.  hi is cut towards zero and lo is never
// zero beside a hi that is not (hi 2^-24 for it, an fp32 rounding): both have
// q's sign, so that an infinite element of K makes the score the infinity that
// it is with q, not inf - inf or 0 x inf.  (hi rounded would give 2^-17; a pass
// over scores that are NaN would cost one token over 16385 rows 3 %.)
SSD_DI void two_parts(float q, bf16& hi, bf16& lo) {
  hi = __float2bfloat16_rz(q);
  const float h = __bfloat162float(hi), rest = q - h;  // exact
  lo = __float2bfloat16(rest);
  if (!(rest != 0.f && isfinite(rest))) lo = __float2bfloat16(h * 0x1p-24f);
}

// One CTA per (node, group of heads): the node's ancestor bits and depth,
// the rotated query in two bf16 parts, the K/V rows rounded to bf16
// into the cache and, with inf and NaN of V replaced by 0, into the tree's
// own copy (a matrix product must not meet 0 x inf at masked keys).
// Angles: position * frequency in 64 bits, reduced to one turn, so that far
// positions keep their angle.
// Bound by latency: 4 us for one node, 7 for 61 nodes of 40 heads (4.7 MB
// moved, under 1 us at the memory's rate): launch, parents, ancestor walk,
// angle and stores one behind the other.  The projections load before the walk.
__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ int par[kTreeMaxNodes + 2];
  __shared__ uint32_t bits[kTreeMaxNodes / 32];
  __shared__ int s_depth, s_left;
  __shared__ int bad[kPrepHeads];
  __shared__ float2 turn[kTreeMaxHalf];  // (cos, sin) of the node's position
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x;
  const int half = a.dh >> 1, heads = a.H + 2 * a.Hkv;
  const int h0 = blockIdx.y * kPrepHeads, h1 = min(h0 + kPrepHeads, heads);
  const float* row = a.qkv + (size_t)t * heads * a.dh;
  // the projections load while the ancestors are found
  constexpr int kPairs = kPrepHeads * kTreeMaxHalf / kPrepThreads;
  float px[kPairs], py[kPairs];
#pragma unroll
  for (int q = 0; q < kPairs; ++q) {
    const int e = tid + q * kPrepThreads, h = h0 + e / half, i = e % half;
    px[q] = py[q] = 0.f;
    if (h < h1) {
      px[q] = row[(size_t)h * a.dh + i];
      py[q] = row[(size_t)h * a.dh + half + i];
    }
  }
  if (t == 0 && blockIdx.y == 0 && tid == 0) *a.err = 0;
  for (int i = tid; i <= t; i += kPrepThreads) par[i] = a.parents[i];
  for (int i = tid; i < kTreeMaxNodes / 32; i += kPrepThreads) bits[i] = 0u;
  if (tid < kPrepHeads) bad[tid] = 0;
  __syncthreads();
  if (tid == 0) {
    int cur = t, d = 0, left = -1;
    while (true) {  // parents strictly decrease
      bits[cur >> 5] |= 1u << (cur & 31);
      if (d == kWalk) {
        left = cur;
        break;
      }
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
    s_left = left;
  }
  __syncthreads();
  if (s_left >= 0) far_ancestors(t, par, bits, s_depth);
  const int d = s_depth;
  if (blockIdx.y == 0) {
    for (int w = tid; w < a.anc_words; w += kPrepThreads)
      a.anc[(size_t)t * a.anc_words + w] = d >= 0 ? bits[w] : 0u;
    if (tid == 0) a.depth[t] = d;
  }
  if (tid < (a.dh >> 1)) {
    double x = (double)(a.pos0 + max(d, 0)) * a.inv_freq[tid];  // angle / pi
    x -= 2.0 * rint(0.5 * x);
    sincospif((float)x, &turn[tid].y, &turn[tid].x);
  }
  __syncthreads();
  const size_t qplane = (size_t)a.Hkv * a.T * a.G * a.dh;
#pragma unroll
  for (int q = 0; q < kPairs; ++q) {
    const int e = tid + q * kPrepThreads, h = h0 + e / half, i = e % half;
    if (h >= h1) continue;
    float x = d < 0 ? 0.f : px[q], y = d < 0 ? 0.f : py[q];
    if (h < a.H + a.Hkv) {
      const float cs = turn[i].x, sn = turn[i].y;
      const float rx = x * cs - y * sn, ry = y * cs + x * sn;
      x = rx;
      y = ry;
    }
    if (h < a.H) {
      const int kvh = h / a.G, g = h - kvh * a.G;
      const size_t o = ((size_t)kvh * a.T * a.G + (size_t)t * a.G + g) * a.dh + i;
      two_parts(x, a.q[o], a.q[qplane + o]);
      two_parts(y, a.q[o + half], a.q[qplane + o + half]);
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
    if (h >= a.H + a.Hkv)
      a.vbad[(size_t)(h - a.H - a.Hkv) * tree_vbad_stride(a.T) + t] = (uint8_t)bad[h - h0];
}

// d2 matrices of d1 rows of dh bf16, `stride` bytes apart, in 128-row boxes.
bool tree_map(CUtensorMap* m, const void* base, int dh, int d1, int d2, size_t stride) {
  EncodeTiled enc = tma_encoder();
  const cuuint64_t dims[3] = {(cuuint64_t)dh, (cuuint64_t)d1, (cuuint64_t)d2};
  const cuuint64_t strides[2] = {dh * sizeof(bf16), stride};
  const cuuint32_t box[3] = {64, 128, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  tree_split(a);
  const size_t slots = (size_t)tree_slots(a);
  a.anc_words = tree_anc_words(a.T);
  a.anc = (uint32_t*)take((size_t)a.T * a.anc_words * 4);
  a.depth = (int32_t*)take((size_t)a.T * 4);
  a.vbad = (uint8_t*)take((size_t)a.Hkv * tree_vbad_stride(a.T));
  a.row_kt = (int)(2 * a.Hkv * rows);
  a.row_vt = a.row_kt + a.Hkv * a.T;
  a.q = (bf16*)take((size_t)(a.row_vt + a.Hkv * a.T) * a.dh * sizeof(bf16));
  a.kt = a.q + (size_t)a.row_kt * a.dh;
  a.vt = a.q + (size_t)a.row_vt * a.dh;
  a.lse = (float*)take(a.Hkv * rows * 4);
  if (a.splits > 1) {                            // (one split's results are final)
    a.part_o = (float*)take(slots * a.dh * 128 * 4);
    a.part_m = (float*)take(slots * 128 * 4);
    a.part_l = (float*)take(slots * 128 * 4);
  }
  if (rows <= (size_t)kTreeScoreRows) {
    a.part_s = (float*)take((size_t)a.Hkv * a.nb * rows * kTreeKeys * 4);
    if (!a.w_out) a.part_s = nullptr;
  }
  a.err = (int*)take(4);
  return off;
}

cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s) {
  const int heads = a.H + 2 * a.Hkv;
  tree_prep_kernel<<<dim3(a.T, (heads + kPrepHeads - 1) / kPrepHeads), kPrepThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  TreeMaps m;
  const size_t cache_row = (size_t)a.dh * sizeof(bf16);
  const int n = a.n ? a.n : 1;                   // no context: never read
  if (!tree_map(&m.k, a.kc, a.dh, n, a.Hkv, a.max_seq * cache_row) ||
      !tree_map(&m.v, a.vc, a.dh, n, a.Hkv, a.max_seq * cache_row) ||
      !tree_map(&m.ws, a.q, a.dh, a.row_vt + a.Hkv * a.T, 1, cache_row))
    return cudaErrorInvalidValue;
  if ((e = launch_tree_attn_tc(a, m, s)) != cudaSuccess || !a.w_out || a.part_s) return e;
  return launch_tree_weight_tc(a, m, s);
}

}  // namespace ssd
