// Kernel-level C-ABI (ssd_ops.h): each call runs one hot-path kernel on
// caller-provided device buffers, so that every kernel can be checked on
// its own against the CPU oracle.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <string>

#include "../../include/ssd_ops.h"
#include "kernels.cuh"
#include "tree.cuh"

using namespace ssd;

namespace {

thread_local std::string g_op_err;

ssd_status op_fail(ssd_status s, const std::string& m) {
  g_op_err = m;
  return s;
}

bool al16(const void* p) { return p && ((uintptr_t)p & 15u) == 0; }

ssd_status check_linear(const void* W, int R, int K, int M) {
  if (!al16(W)) return op_fail(SSD_ERR_INVALID_ARG, "W must be non-null and 16-byte aligned");
  if (R <= 0 || R % 16) return op_fail(SSD_ERR_INVALID_ARG, "R must be a positive multiple of 16");
  if (K <= 0 || K % 32) return op_fail(SSD_ERR_INVALID_ARG, "K must be a positive multiple of 32");
  if (M < 1 || M > kMaxRows) return op_fail(SSD_ERR_INVALID_ARG, "M must be in 1..16");
  return SSD_OK;
}

ssd_status cu(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return SSD_OK;
  cudaGetLastError();
  return op_fail(e == cudaErrorMemoryAllocation ? SSD_ERR_OOM : SSD_ERR_CUDA,
                 std::string(what) + ": " + cudaGetErrorString(e));
}

// Stream-ordered scratch that is freed on scope exit.
struct Scratch {
  cudaStream_t s;
  void* p = nullptr;
  Scratch(cudaStream_t st) : s(st) {}
  cudaError_t alloc(size_t bytes) { return cudaMallocAsync(&p, bytes, s); }
  ~Scratch() {
    if (p) cudaFreeAsync(p, s);
  }
};

// Scratch for one GEMV launch (zeroed counters).
struct GemvOpScratch {
  Scratch part, cnt, rec, err;
  explicit GemvOpScratch(cudaStream_t s) : part(s), cnt(s), rec(s), err(s) {}
  ssd_status init(int R, int K, int epi, LinearArgs& a, cudaStream_t s) {
    const GemvScratch gs = gemv_scratch(R, K, epi);
    ssd_status r;
    if ((r = cu(part.alloc(gs.part_floats * 4), "scratch")) != SSD_OK) return r;
    if ((r = cu(cnt.alloc(gs.counters * 4), "scratch")) != SSD_OK) return r;
    if ((r = cu(rec.alloc(gs.rec_floats ? gs.rec_floats * 4 : 16), "scratch")) != SSD_OK) return r;
    if ((r = cu(err.alloc(16), "scratch")) != SSD_OK) return r;
    if ((r = cu(cudaMemsetAsync(cnt.p, 0, gs.counters * 4, s), "memset")) != SSD_OK) return r;
    if ((r = cu(cudaMemsetAsync(err.p, 0, 16, s), "memset")) != SSD_OK) return r;
    a.part = (float*)part.p;
    a.counter = (unsigned*)cnt.p;
    a.rec = (float*)rec.p;
    a.err = (int*)err.p;
    return SSD_OK;
  }
};

// A norm-fused projection: when the rows do not fit the GEMV's activation
// stage, a RMSNorm pre-pass writes bf16 rows and the projection reads those
// (the same bits; what the context runtime does for wide passes).
ssd_status launch_norm_fused(int epi, LinearArgs a, cudaStream_t s, Scratch& xn, const char* what) {
  if (a.M_static <= gemv_stage_rows(a.K)) return cu(launch_gemv(IN_NORM, epi, a, s, false), what);
  ssd_status r;
  if ((r = cu(xn.alloc((size_t)a.M_static * a.K * sizeof(bf16)), "scratch")) != SSD_OK) return r;
  if ((r = cu(launch_norm_rows(a.x, a.ss, a.gain, a.eps, a.M_static, nullptr, a.K, (bf16*)xn.p, s,
                               false),
              "rmsnorm")) != SSD_OK)
    return r;
  a.act = (const bf16*)xn.p;
  a.x = nullptr;
  a.ss = nullptr;
  a.gain = nullptr;
  return cu(launch_gemv(IN_BF16, epi, a, s, false), what);
}

bool al4(const void* p) { return p && ((uintptr_t)p & 3u) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y ? x + na > y : y + nb > x;
}

ssd_status check_tree_sizes(int T, int n_ctx, int H, int Hkv, int dh) {
  if (T < 1 || T > kTreeMaxNodes || n_ctx < 0 || n_ctx > INT32_MAX - T || H < 1 || Hkv < 1 || H % Hkv || H > 4096 ||
      (dh != 64 && dh != 128))
    return op_fail(SSD_ERR_INVALID_ARG, "tree_attention sizes");
  return SSD_OK;
}

void tree_sizes(TreeArgs& a, int T, int n_ctx, int H, int Hkv, int dh) {
  a.T = T;
  a.n = n_ctx;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.dh = dh;
}

// What ssd_debug_tree_give_up asked for.
thread_local int t_give_up[2] = {-1, -1};

// theta^(-2 i / dh) / pi.  The table of the thread's last (theta, dh) is kept:
// 64 powers cost a small call several microseconds.
void tree_frequencies(float theta, int dh, double* out) {
  thread_local float last_theta = 0.f;
  thread_local int last_dh = 0;
  thread_local double table[kTreeMaxHalf];
  if (theta != last_theta || dh != last_dh) {
    for (int i = 0; i < dh / 2; ++i)
      table[i] = std::pow((double)theta, -2.0 * i / dh) / 3.14159265358979323846;
    last_theta = theta;
    last_dh = dh;
  }
  std::memcpy(out, table, sizeof(double) * (dh / 2));
}

}  // namespace

extern "C" {

const char* ssd_ops_last_error(void) { return g_op_err.c_str(); }

ssd_status ssd_pack_weight(const void* src, void* dst, int32_t R, int32_t K, void* stream) {
  if (!al16(src) || !al16(dst) || src == dst)
    return op_fail(SSD_ERR_INVALID_ARG, "pack: src / dst must be distinct, 16-byte aligned");
  if (R <= 0 || R % 16 || K <= 0 || K % 32)
    return op_fail(SSD_ERR_INVALID_ARG, "pack: R % 16 == 0 and K % 32 == 0 required");
  const char* lo = (const char*)src;
  const char* hi = (const char*)dst;
  const size_t bytes = (size_t)R * K * 2;
  if ((lo < hi && lo + bytes > hi) || (hi < lo && hi + bytes > lo))
    return op_fail(SSD_ERR_INVALID_ARG, "pack: src and dst overlap");
  return cu(launch_pack((const bf16*)src, (bf16*)dst, R, K, (cudaStream_t)stream), "pack");
}

ssd_status ssd_op_linear(const void* W, int32_t R, int32_t K, const void* act, int32_t M,
                         float* y, void* stream) {
  ssd_status r = check_linear(W, R, K, M);
  if (r != SSD_OK) return r;
  if (!al16(act) || !al16(y)) return op_fail(SSD_ERR_INVALID_ARG, "act / y alignment");
  LinearArgs a;
  a.W0 = (const bf16*)W;
  a.R = R;
  a.K = K;
  a.act = (const bf16*)act;
  a.M_static = M;
  a.y = y;
  GemvOpScratch gs((cudaStream_t)stream);
  if ((r = gs.init(R, K, EPI_STORE, a, (cudaStream_t)stream)) != SSD_OK) return r;
  return cu(launch_gemv(IN_BF16, EPI_STORE, a, (cudaStream_t)stream, false), "linear");
}

ssd_status ssd_op_rmsnorm_linear(const void* W, int32_t R, int32_t K, const float* x,
                                 const float* gain, float eps, int32_t M, float* y, void* stream) {
  ssd_status r = check_linear(W, R, K, M);
  if (r != SSD_OK) return r;
  if (!al16(x) || !al16(gain) || !al16(y) || !(eps > 0.f))
    return op_fail(SSD_ERR_INVALID_ARG, "x / gain / y / eps");
  cudaStream_t s = (cudaStream_t)stream;
  Scratch ss(s);
  if ((r = cu(ss.alloc((size_t)M * (K / kSsGroup) * 4), "scratch")) != SSD_OK) return r;
  if ((r = cu(launch_ss_partials(x, M, K, (float*)ss.p, s), "ss")) != SSD_OK) return r;
  LinearArgs a;
  a.W0 = (const bf16*)W;
  a.R = R;
  a.K = K;
  a.x = x;
  a.ss = (const float*)ss.p;
  a.gain = gain;
  a.eps = eps;
  a.M_static = M;
  a.y = y;
  GemvOpScratch gs(s);
  if ((r = gs.init(R, K, EPI_STORE, a, s)) != SSD_OK) return r;
  Scratch xn(s);
  return launch_norm_fused(EPI_STORE, a, s, xn, "rmsnorm_linear");
}

ssd_status ssd_op_residual_linear(const void* W, int32_t R, int32_t K, const void* act, int32_t M,
                                  float* x, void* stream) {
  ssd_status r = check_linear(W, R, K, M);
  if (r != SSD_OK) return r;
  if (!al16(act) || !al16(x)) return op_fail(SSD_ERR_INVALID_ARG, "act / x alignment");
  cudaStream_t s = (cudaStream_t)stream;
  Scratch ss(s);
  if ((r = cu(ss.alloc((size_t)M * (R / kSsGroup) * 4), "scratch")) != SSD_OK) return r;
  LinearArgs a;
  a.W0 = (const bf16*)W;
  a.R = R;
  a.K = K;
  a.act = (const bf16*)act;
  a.M_static = M;
  a.xres = x;
  a.ss_out = (float*)ss.p;
  GemvOpScratch gs(s);
  if ((r = gs.init(R, K, EPI_RESID, a, s)) != SSD_OK) return r;
  return cu(launch_gemv(IN_BF16, EPI_RESID, a, s, false), "residual_linear");
}

ssd_status ssd_op_swiglu(const void* Wg, const void* Wu, int32_t F, int32_t K, const float* x,
                         const float* gain, float eps, int32_t M, void* u, void* stream) {
  ssd_status r = check_linear(Wg, F, K, M);
  if (r != SSD_OK) return r;
  if (!al16(Wu) || !al16(x) || !al16(gain) || !al16(u) || !(eps > 0.f))
    return op_fail(SSD_ERR_INVALID_ARG, "Wu / x / gain / u / eps");
  cudaStream_t s = (cudaStream_t)stream;
  Scratch ss(s);
  if ((r = cu(ss.alloc((size_t)M * (K / kSsGroup) * 4), "scratch")) != SSD_OK) return r;
  if ((r = cu(launch_ss_partials(x, M, K, (float*)ss.p, s), "ss")) != SSD_OK) return r;
  LinearArgs a;
  a.W0 = (const bf16*)Wg;
  a.W1 = (const bf16*)Wu;
  a.R = F;
  a.K = K;
  a.x = x;
  a.ss = (const float*)ss.p;
  a.gain = gain;
  a.eps = eps;
  a.M_static = M;
  a.u = (bf16*)u;
  GemvOpScratch gs(s);
  if ((r = gs.init(F, K, EPI_SWIGLU, a, s)) != SSD_OK) return r;
  Scratch xn(s);
  return launch_norm_fused(EPI_SWIGLU, a, s, xn, "swiglu");
}

ssd_status ssd_op_attention(const float* qkv, int32_t M, int32_t pos0, void* k_cache,
                            void* v_cache, int32_t max_seq, int32_t H, int32_t Hkv, int32_t dh,
                            float theta, void* out, void* stream) {
  if (M < 1 || M > kMaxRows || pos0 < 0 || H <= 0 || Hkv <= 0 || H % Hkv || H / Hkv > 8 ||
      (dh != 64 && dh != 128) || max_seq <= 0 || max_seq % kAttnChunk || pos0 + M > max_seq ||
      !(theta > 0.f))
    return op_fail(SSD_ERR_INVALID_ARG, "attention sizes");
  if (!al16(qkv) || !al16(k_cache) || !al16(v_cache) || !al16(out))
    return op_fail(SSD_ERR_INVALID_ARG, "attention pointers");
  cudaStream_t s = (cudaStream_t)stream;
  ssd_status r;
  Scratch rope(s), part(s), cnt(s), err(s);
  const int half = dh / 2;
  if ((r = cu(rope.alloc((size_t)max_seq * half * sizeof(float2)), "scratch")) != SSD_OK) return r;
  if ((r = cu(part.alloc(attn_part_floats(Hkv, H, dh, max_seq) * 4), "scratch")) != SSD_OK) return r;
  if ((r = cu(cnt.alloc((size_t)Hkv * 4), "scratch")) != SSD_OK) return r;
  if ((r = cu(err.alloc(4), "scratch")) != SSD_OK) return r;
  if ((r = cu(cudaMemsetAsync(cnt.p, 0, (size_t)Hkv * 4, s), "memset")) != SSD_OK) return r;
  if ((r = cu(cudaMemsetAsync(err.p, 0, 4, s), "memset")) != SSD_OK) return r;
  if ((r = cu(launch_rope_table((float2*)rope.p, max_seq, half, (double)theta, s), "rope")) != SSD_OK)
    return r;
  AttnArgs a;
  a.qkv = qkv;
  a.ld_qkv = (H + 2 * Hkv) * dh;
  a.M_static = M;
  a.pos0_static = pos0;
  a.kc = (bf16*)k_cache;
  a.vc = (bf16*)v_cache;
  a.max_seq = max_seq;
  a.H = H;
  a.Hkv = Hkv;
  a.dh = dh;
  a.rope = (const float2*)rope.p;
  a.out = (bf16*)out;
  a.part = (float*)part.p;
  a.counters = (unsigned*)cnt.p;
  a.err = (int*)err.p;
  a.scale = (float)(1.0 / std::sqrt((double)dh));
  if ((r = cu(attn_prepare(a), "attn_prepare")) != SSD_OK) return r;
  return cu(launch_attention(a, s, false), "attention");
}

ssd_status ssd_op_lm_head(const void* W, int32_t V, int32_t D, const float* x, const float* gain,
                          float eps, int32_t M, float temperature, uint64_t seed, int32_t round,
                          int32_t stream_id, int32_t pos0, float* logits, ssd_row_stats* stats,
                          void* stream) {
  ssd_status r = check_linear(W, V, D, M);
  if (r != SSD_OK) return r;
  if (!al16(x) || !al16(gain) || !al16(stats) || (logits && !al16(logits)) || !(eps > 0.f) ||
      !(temperature >= 0.f))
    return op_fail(SSD_ERR_INVALID_ARG, "lm_head pointers / eps / temperature");
  cudaStream_t s = (cudaStream_t)stream;
  Scratch ss(s);
  if ((r = cu(ss.alloc((size_t)M * (D / kSsGroup) * 4), "scratch")) != SSD_OK) return r;
  if ((r = cu(launch_ss_partials(x, M, D, (float*)ss.p, s), "ss")) != SSD_OK) return r;
  LinearArgs a;
  a.W0 = (const bf16*)W;
  a.R = V;
  a.K = D;
  a.x = x;
  a.ss = (const float*)ss.p;
  a.gain = gain;
  a.eps = eps;
  a.M_static = M;
  a.logits = logits;
  a.stats = (RowStats*)stats;
  GemvOpScratch gs(s);
  if ((r = gs.init(V, D, EPI_LMHEAD, a, s)) != SSD_OK) return r;
  a.temperature = temperature;
  a.sample = temperature > 0.f ? 1 : 0;
  a.seed = seed;
  a.round_static = round;
  a.sample_stream = stream_id;
  a.pos0_static = pos0;
  Scratch xn(s);
  return launch_norm_fused(EPI_LMHEAD, a, s, xn, "lm_head");
}

ssd_status ssd_op_accept_stochastic(const float* P, const float* Q, const int32_t* drafts,
                                    int32_t d, int32_t V, float temperature, uint64_t seed,
                                    int32_t round, int32_t n, int32_t* emitted,
                                    int32_t* n_emitted, void* stream) {
  if (!P || (d > 0 && (!Q || !drafts)) || !emitted || !n_emitted || d < 0 || d > kMaxRows - 1 ||
      V <= 0 || !(temperature > 0.f) || n < 0)
    return op_fail(SSD_ERR_INVALID_ARG, "accept arguments");
  AcceptArgs a;
  a.P = P;
  a.Q = Q;
  a.drafts = drafts;
  a.d_static = d;
  a.V = V;
  a.temperature = temperature;
  a.seed = seed;
  a.round_static = round;
  a.n_static = n;
  a.emitted = emitted;
  a.n_emitted = n_emitted;
  return cu(launch_accept_stochastic(a, (cudaStream_t)stream, false), "accept");
}

ssd_status ssd_op_wait_selftest(int32_t polls, int32_t* code_out, void* stream) {
  if (polls < 1 || polls > (1 << 20) || !code_out)
    return op_fail(SSD_ERR_INVALID_ARG, "polls in 1..2^20 and code_out required");
  cudaStream_t s = (cudaStream_t)stream;
  Scratch never(s), code(s);
  ssd_status r;
  if ((r = cu(never.alloc(16), "scratch")) != SSD_OK) return r;
  if ((r = cu(code.alloc(16), "scratch")) != SSD_OK) return r;
  if ((r = cu(cudaMemsetAsync(never.p, 0, 16, s), "memset")) != SSD_OK) return r;
  if ((r = cu(cudaMemsetAsync(code.p, 0xff, 16, s), "memset")) != SSD_OK) return r;
  if ((r = cu(launch_wait_selftest((const unsigned*)never.p, polls, (int32_t*)code.p, s),
              "selftest")) != SSD_OK)
    return r;
  if ((r = cu(cudaMemcpyAsync(code_out, code.p, 4, cudaMemcpyDeviceToHost, s), "copy")) != SSD_OK)
    return r;
  return cu(cudaStreamSynchronize(s), "synchronize");
}

ssd_status ssd_op_philox(const uint32_t* ctr, int32_t count, uint64_t key, uint32_t* out,
                         void* stream) {
  if (count < 0 || (count > 0 && (!al16(ctr) || !al16(out))))
    return op_fail(SSD_ERR_INVALID_ARG, "philox arguments");
  return cu(launch_philox(ctr, count, key, out, (cudaStream_t)stream), "philox");
}

ssd_status ssd_op_linear_rows(const void* W, const void* W1, int32_t R, int32_t K,
                              const void* act, int32_t T, int32_t epi, void* out,
                              const int32_t* map, void* stream) {
  const bool act_packed = (epi & SSD_ROWS_ACT_PACKED) != 0;
  epi &= ~SSD_ROWS_ACT_PACKED;
  if (!al16(W) || (epi == GEMM_SWIGLU && !al16(W1)) || R <= 0 || R % 16 || K <= 0 || K % 32 ||
      T < 1 || !al16(act) || !al16(out) || epi < GEMM_STORE || epi > GEMM_ARGMAX)
    return op_fail(SSD_ERR_INVALID_ARG, "linear_rows arguments");
  cudaStream_t s = (cudaStream_t)stream;
  GemmArgs a;
  a.W0 = (const bf16*)W;
  a.W1 = (const bf16*)W1;
  a.R = R;
  a.K = K;
  a.T = T;
  a.act = (const bf16*)act;
  a.epi = epi;
  Scratch best(s), err(s), packed(s);
  ssd_status r;
  if ((r = cu(err.alloc(16), "scratch")) != SSD_OK) return r;
  if ((r = cu(cudaMemsetAsync(err.p, 0, 16, s), "memset")) != SSD_OK) return r;
  a.err = (int*)err.p;
  // the projection reads its activations in the packed unit layout
  if (!act_packed) {
    const size_t Tp = ((size_t)T + 15) / 16 * 16;
    if ((r = cu(packed.alloc(Tp * K * sizeof(bf16)), "scratch")) != SSD_OK) return r;
    if ((r = cu(launch_pack_act((const bf16*)act, T, K, (bf16*)packed.p, s), "pack_act")) !=
        SSD_OK)
      return r;
    a.act = (const bf16*)packed.p;
  }
  if (epi == GEMM_STORE) a.y = (float*)out;
  if (epi == GEMM_RESID) {
    a.x = (float*)out;
    a.rowmap = map;
  }
  if (epi == GEMM_SWIGLU) a.u = (bf16*)out;
  if (epi == GEMM_ARGMAX) {
    if ((r = cu(best.alloc((size_t)T * 8), "scratch")) != SSD_OK) return r;
    if ((r = cu(cudaMemsetAsync(best.p, 0, (size_t)T * 8, s), "memset")) != SSD_OK) return r;
    a.best = (unsigned long long*)best.p;
  }
  if ((r = cu(launch_gemm_rows(a, s), "linear_rows")) != SSD_OK) return r;
  if (epi == GEMM_ARGMAX)
    return cu(launch_argmax_index(a.best, T, (int32_t*)out, s), "argmax_index");
  return SSD_OK;
}

ssd_status ssd_op_score_attention(const void* q, const int32_t* cand, int32_t n_cand, int32_t N,
                                  int32_t split, const void* k_cache, const void* v_cache,
                                  int32_t max_seq, const void* wk, const void* wv, int32_t w_rows,
                                  int32_t H, int32_t Hkv, int32_t dh, void* out, void* stream) {
  if (!al16(q) || !cand || n_cand < 1 || N < 1 || split < 1 || split > max_seq || w_rows < N ||
      !al16(k_cache) || !al16(v_cache) || !al16(wk) || !al16(wv) || !al16(out) || H < 1 ||
      Hkv < 1 || H % Hkv || (dh != 64 && dh != 128))
    return op_fail(SSD_ERR_INVALID_ARG, "score_attention arguments");
  ScoreAttnArgs a;
  a.q = (const bf16*)q;
  a.kc = (const bf16*)k_cache;
  a.vc = (const bf16*)v_cache;
  a.sk = (const bf16*)wk;
  a.sv = (const bf16*)wv;
  a.cand = cand;
  a.N = N;
  a.split = split;
  a.max_seq = max_seq;
  a.H = H;
  a.Hkv = Hkv;
  a.dh = dh;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)dh));
  a.out = (bf16*)out;
  a.w_rows = w_rows;
  return cu(launch_score_attn(a, n_cand, (cudaStream_t)stream), "score_attention");
}

size_t ssd_op_tree_attention_workspace(int32_t T, int32_t n_ctx, int32_t H, int32_t Hkv,
                                       int32_t dh) {
  if (check_tree_sizes(T, n_ctx, H, Hkv, dh) != SSD_OK) return 0;
  TreeArgs a;
  tree_sizes(a, T, n_ctx, H, Hkv, dh);
  return tree_workspace(a, nullptr);
}

ssd_status ssd_op_tree_attention(const float* qkv, const int32_t* parents, int32_t T,
                                 int32_t n_ctx, int32_t pos0, void* k_cache, void* v_cache,
                                 int32_t max_seq, int32_t H, int32_t Hkv, int32_t dh, float theta,
                                 const float* weight_in, float* weight_out, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  ssd_status r = check_tree_sizes(T, n_ctx, H, Hkv, dh);
  if (r != SSD_OK) return r;
  if (max_seq <= 0 || n_ctx > max_seq - T || pos0 < 0 || pos0 > INT32_MAX - T || !(theta > 0.f) ||
      !std::isfinite(theta))
    return op_fail(SSD_ERR_INVALID_ARG, "tree_attention: max_seq / pos0 / theta");
  if (!al16(qkv) || !al4(parents) || !al16(k_cache) || !al16(v_cache) || !al16(out) ||
      ((uintptr_t)workspace & 255u) || !workspace)
    return op_fail(SSD_ERR_INVALID_ARG, "tree_attention pointers");
  if ((weight_in && (!weight_out || !al4(weight_in))) || (weight_out && !al4(weight_out)))
    return op_fail(SSD_ERR_INVALID_ARG, "tree_attention: weight_in needs weight_out");
  const size_t per_key = (size_t)4 * Hkv * max_seq, cache = per_key / 2 * dh;
  if (overlap(k_cache, cache, v_cache, cache) ||
      (weight_in && weight_in != weight_out && overlap(weight_in, per_key, weight_out, per_key)))
    return op_fail(SSD_ERR_INVALID_ARG, "tree_attention: buffers overlap");
  TreeArgs a;
  tree_sizes(a, T, n_ctx, H, Hkv, dh);
  a.w_out = weight_out;
  if (tree_workspace(a, workspace) > workspace_bytes)
    return op_fail(SSD_ERR_CAPACITY, "tree_attention: workspace too small");
  a.qkv = qkv;
  a.parents = parents;
  a.pos0 = pos0;
  a.max_seq = max_seq;
  a.kc = (bf16*)k_cache;
  a.vc = (bf16*)v_cache;
  a.w_in = weight_in;
  a.out = (bf16*)out;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)dh));
  tree_frequencies(theta, dh, a.inv_freq);
  a.give_up = t_give_up[0];
  a.give_up_weights = t_give_up[1];
  return cu(launch_tree_attention(a, (cudaStream_t)stream), "tree_attention");
}

ssd_status ssd_debug_tree_give_up(int32_t attention, int32_t weights) {
  if (attention < -1 || weights < -1) return op_fail(SSD_ERR_INVALID_ARG, "tree_give_up: a CTA, or -1");
  t_give_up[0] = attention;
  t_give_up[1] = weights;
  return SSD_OK;
}

ssd_status ssd_op_cache_evict(const void* k, const void* v, const float* weight, int32_t n,
                              int32_t keep, int32_t sinks, int32_t recent, int32_t max_seq,
                              int32_t Hkv, int32_t dh, int32_t dtype, void* k_out, void* v_out,
                              float* weight_out, int32_t max_out, int32_t* kept, void* stream) {
  if (n < 1 || n > max_seq || keep < 1 || keep > n || keep > max_out || sinks < 0 || recent < 0 ||
      sinks > keep || recent > keep - sinks || Hkv < 1 || Hkv > 65535 || dh < 1 || dh > 65536 ||
      (dtype != SSD_DTYPE_BF16 && dtype != SSD_DTYPE_FP32))
    return op_fail(SSD_ERR_INVALID_ARG, "cache_evict sizes");
  const size_t row = (size_t)dh * (dtype == SSD_DTYPE_BF16 ? 2 : 4);
  if (row % 16) return op_fail(SSD_ERR_INVALID_ARG, "cache_evict: a row's bytes must be a multiple of 16");
  if (!al16(k) || !al16(v) || !al4(weight) || !al16(k_out) || !al16(v_out) || !al4(kept) ||
      (weight_out && !al4(weight_out)))
    return op_fail(SSD_ERR_INVALID_ARG, "cache_evict pointers");
  const size_t in = row * Hkv * max_seq, o = row * Hkv * max_out;
  const size_t win = (size_t)4 * Hkv * max_seq, wo = (size_t)4 * Hkv * max_out;
  if (overlap(k, in, k_out, o) || overlap(k, in, v_out, o) || overlap(v, in, k_out, o) ||
      overlap(v, in, v_out, o) || overlap(k_out, o, v_out, o) ||
      (weight_out && overlap(weight, win, weight_out, wo)))
    return op_fail(SSD_ERR_INVALID_ARG, "cache_evict: outputs overlap");
  EvictArgs a;
  a.k = (const uint4*)k;
  a.v = (const uint4*)v;
  a.weight = weight;
  a.k_out = (uint4*)k_out;
  a.v_out = (uint4*)v_out;
  a.weight_out = weight_out;
  a.kept = kept;
  a.n = n;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  a.max_seq = max_seq;
  a.max_out = max_out;
  a.Hkv = Hkv;
  a.units = (int)(row / 16);
  return cu(launch_cache_evict(a, (cudaStream_t)stream), "cache_evict");
}

size_t ssd_op_beam_select_workspace(int32_t B, int32_t V, int32_t W) {
  if (B < 1 || B > 256 || W < 1 || W > 256 || V < 1) return 0;
  return beam_select_workspace(B, V, W);
}

ssd_status ssd_op_beam_select(const float* logits, int32_t B, int32_t V, const float* lse,
                              int32_t lse_stride, const float* scores, const int32_t* done,
                              int32_t end_id, int32_t W, int32_t* tokens, int32_t* parents,
                              float* scores_out, int32_t* done_out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (B < 1 || B > 256 || W < 1 || W > 256 || V < 1 || end_id < -1 || end_id >= V ||
      (done && end_id < 0) || (lse && lse_stride < 1))
    return op_fail(SSD_ERR_INVALID_ARG, "beam_select sizes");
  if (!al4(logits) || !al4(scores) || (lse && !al4(lse)) || (done && !al4(done)) ||
      !al4(tokens) || !al4(parents) || !al4(scores_out) || (done_out && !al4(done_out)) ||
      ((uintptr_t)workspace & 255u))
    return op_fail(SSD_ERR_INVALID_ARG, "beam_select pointers");
  const size_t need = beam_select_workspace(B, V, W);
  if (need && !workspace) return op_fail(SSD_ERR_INVALID_ARG, "beam_select pointers");
  if (workspace_bytes < need)
    return op_fail(SSD_ERR_CAPACITY, "beam_select: workspace too small");
  BeamArgs a;
  a.logits = logits;
  a.lse = lse;
  a.lse_stride = lse_stride;
  a.scores = scores;
  a.done = done;
  a.B = B;
  a.V = V;
  a.W = W;
  a.end_id = end_id;
  a.lists = (uint64_t*)workspace;
  a.tokens = tokens;
  a.parents = parents;
  a.scores_out = scores_out;
  a.done_out = done_out;
  return cu(launch_beam_select(a, (cudaStream_t)stream), "beam_select");
}

ssd_status ssd_op_beam_reorder(const void* k, const void* v, const int32_t* parents, int32_t B,
                               int32_t W, int32_t groups, int32_t max_seq, int32_t start,
                               int32_t stop, int32_t row_bytes, void* k_out, void* v_out,
                               void* stream) {
  if (B < 1 || W < 1 || groups < 1 || max_seq < 1 || start < 0 || stop < start || stop > max_seq ||
      row_bytes < 16 || row_bytes % 16)
    return op_fail(SSD_ERR_INVALID_ARG, "beam_reorder sizes");
  if (!al16(k) || !al16(k_out) || !al4(parents) || (!v) != (!v_out) || (v && (!al16(v) || !al16(v_out))))
    return op_fail(SSD_ERR_INVALID_ARG, "beam_reorder pointers");
  const size_t state = (size_t)groups * max_seq * row_bytes, in = state * B, o = state * W;
  if (overlap(k, in, k_out, o) ||
      (v && (overlap(k, in, v_out, o) || overlap(v, in, k_out, o) || overlap(v, in, v_out, o) ||
             overlap(k_out, o, v_out, o))))
    return op_fail(SSD_ERR_INVALID_ARG, "beam_reorder: outputs overlap");
  if (start == stop) return SSD_OK;
  ReorderArgs a;
  a.k = (const uint4*)k;
  a.v = (const uint4*)v;
  a.parents = parents;
  a.k_out = (uint4*)k_out;
  a.v_out = (uint4*)v_out;
  a.B = B;
  a.W = W;
  a.groups = groups;
  a.max_seq = max_seq;
  a.start = start;
  a.stop = stop;
  a.units = row_bytes / 16;
  return cu(launch_beam_reorder(a, (cudaStream_t)stream), "beam_reorder");
}

}  // extern "C"
