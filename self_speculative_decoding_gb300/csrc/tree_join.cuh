// Joining the partial results of a tree attention's units (shared by the
// kernel after the units and the one that sums the weights).
#pragma once

#include "tree.cuh"

namespace ssd {

// Whether any node's V row of this head holds inf or NaN (a warp asks).
SSD_DI bool any_bad(const TreeArgs& a, int kvh, int lane) {
  const uint8_t* flags = a.vbad + kvh * tree_vbad_stride(a.T);
  bool any = false;
  for (int j = lane; j < a.T; j += 32) any |= flags[j] != 0;
  return __any_sync(0xffffffffu, any);
}

// Adds to n columns from c0 on of row (node t) the inf and NaN of the V rows
// that it sees, which the products left out: v += p_j V_j for those values.
template <int DH>
static __device__ __noinline__ void add_bad(const TreeArgs& a, int kvh, int row, int t, float lse,
                                            int c0, float* v, int n) {
  const uint8_t* flags = a.vbad + kvh * tree_vbad_stride(a.T);
  const int rows = a.T * a.G;
  const size_t plane = (size_t)a.Hkv * rows * DH;
  const bf16* q = a.q + ((size_t)kvh * rows + row) * DH;
  for (int j = 0; j <= t; ++j) {
    if (!flags[j] || !((a.anc[(size_t)t * a.anc_words + (j >> 5)] >> (j & 31)) & 1u)) continue;
    const bf16* k = a.kt + ((size_t)kvh * a.T + j) * DH;
    float acc = 0.f;
    for (int i = 0; i < DH; ++i)
      acc = fmaf(__bfloat162float(q[i]) + __bfloat162float(q[plane + i]), __bfloat162float(k[i]), acc);
    const float p = exp2f(acc * a.scale_log2 - lse);
    for (int e = 0; e < n; ++e) {
      const float x = __bfloat162float(a.vc[((size_t)kvh * a.max_seq + a.n + j) * DH + c0 + e]);
      if (!isfinite(x)) v[e] += p * x;
    }
  }
}

// Base-2 log-sum-exp of a row from the units' statistics (one split: as the
// attention wrote it); infinity for an absent row.
SSD_DI float tree_row_lse(const TreeArgs& a, int kvh, int row) {
  if (a.splits == 1) return a.lse[(size_t)kvh * a.T * a.G + row];
  const int per = a.two ? a.items * 2 : 1;
  const size_t s0 = ((size_t)kvh * a.splits * per + (a.two ? row >> 7 : 0)) * 128 + (row & 127);
  const bool present = a.depth[row / a.G] >= 0;
  float m = -INFINITY, l = 0.f;
  // eight units' statistics in flight at once, the last ones' among them
  for (int i0 = 0; i0 < a.splits; i0 += 8) {
    float pm[8], pl[8], mn = m;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool got = i0 + u < a.splits;
      const size_t at = s0 + (size_t)(i0 + u) * per * 128;
      pm[u] = got ? a.part_m[at] : -INFINITY;
      pl[u] = got ? a.part_l[at] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) mn = fmaxf(mn, pm[u]);
    const float base = mn == -INFINITY ? 0.f : mn;
    l *= exp2f(m - base);
#pragma unroll
    for (int u = 0; u < 8; ++u) l = fmaf(pl[u], exp2f(pm[u] - base), l);
    m = mn;
  }
  return l != 0.f && present ? m + log2f(l) : INFINITY;
}

// Joins of 32 rows each by eight parts of a warp: lane = row, each part an
// eighth of the columns (whole 16- or 32-byte sectors per row); the slots are
// added in order.
constexpr int kJoinWarps = 8;
SSD_DI int tree_joins(const TreeArgs& a) { return (a.T * a.G + 31) / 32 * a.Hkv; }

template <int DH>
SSD_DI void tree_join_rows(const TreeArgs& a, int index, int part) {
  constexpr int kChunks = DH / 4 / kJoinWarps;   // 16-byte columns per part
  const int lane = threadIdx.x & 31;
  const int rows = a.T * a.G, blocks = (rows + 31) / 32;
  const int kvh = index / blocks, row0 = (index - kvh * blocks) * 32;
  const int row = min(row0 + lane, rows - 1), c0 = part * kChunks;
  const int tile = row >> 7, r = row & 127, t = row / a.G;
  const int per = a.two ? a.items * 2 : 1;       // slots per (head, split)
  const size_t s0 = (size_t)kvh * a.splits * per + (a.two ? tile : 0);
  const bool present = a.depth[t] >= 0, bad = *a.err != 0;
  const bool marked = any_bad(a, kvh, lane);
  float m = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < a.splits; ++i) m = fmaxf(m, a.part_m[(s0 + (size_t)i * per) * 128 + r]);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o[kChunks];
#pragma unroll
  for (int q = 0; q < kChunks; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  // four slots' values in flight at once, the last ones' among them
  for (int i0 = 0; i0 < a.splits; i0 += 4) {
    float4 v[4][kChunks];
    float pm[4], pl[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool got = i0 + u < a.splits;
      const size_t sl = s0 + (size_t)(i0 + u) * per;
      pm[u] = got ? a.part_m[sl * 128 + r] : -INFINITY;
      pl[u] = got ? a.part_l[sl * 128 + r] : 0.f;
#pragma unroll
      for (int q = 0; q < kChunks; ++q)
        v[u][q] = got ? *reinterpret_cast<const float4*>(a.part_o + sl * DH * 128 +
                                                         (size_t)(c0 + q) * 512 + r * 4)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w = exp2f(pm[u] - base);
      l = fmaf(pl[u], w, l);
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        o[q].x = fmaf(v[u][q].x, w, o[q].x);
        o[q].y = fmaf(v[u][q].y, w, o[q].y);
        o[q].z = fmaf(v[u][q].z, w, o[q].z);
        o[q].w = fmaf(v[u][q].w, w, o[q].w);
      }
    }
  }
  const float lse = l != 0.f ? m + log2f(l) : INFINITY;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  uint32_t packed[2 * kChunks];
#pragma unroll
  for (int q = 0; q < kChunks; ++q) {
    float v[4] = {o[q].x * inv, o[q].y * inv, o[q].z * inv, o[q].w * inv};
    if (!present)
      v[0] = v[1] = v[2] = v[3] = 0.f;
    else if (marked)
      add_bad<DH>(a, kvh, row, t, lse, (c0 + q) * 4, v, 4);
    if (bad) v[0] = v[1] = v[2] = v[3] = NAN;
    packed[2 * q] = pack_bf16x2(v[0], v[1]);
    packed[2 * q + 1] = pack_bf16x2(v[2], v[3]);
  }
  if (row0 + lane >= rows) return;
  bf16* out = a.out + ((size_t)t * a.H + kvh * a.G + row % a.G) * DH + c0 * 4;
#pragma unroll
  for (int q = 0; q < kChunks; q += 2)
    *reinterpret_cast<uint4*>(out + q * 4) =
        make_uint4(packed[2 * q], packed[2 * q + 1], packed[2 * q + 2], packed[2 * q + 3]);
}

}  // namespace ssd
