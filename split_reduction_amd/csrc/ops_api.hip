// C ABI of the operators around the layers and the head: argument checks,
// their workspace and kernel dispatch. Declarations and contracts:
// include/skgemm.h.

#include <math.h>

#include <map>
#include <mutex>

#include "ops_internal.h"
#include "skgemm.h"
#include "skgemm_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

// ---- workspace: one of a fixed size per (device, stream), skg::StreamKey ----

std::mutex g_mu;
std::map<skg::StreamKey, uint8_t*> g_work;

static_assert(skg::kOpsPartBytes + (size_t)skg::kOpsCounters * skg::kOpsCounterStride * 4 <= SKGEMM_OPS_WORKSPACE_BYTES,
              "partial results and counters fit");

// The stream's workspace, allocated and its counters zeroed on the first call,
// which waits for that: a graph captured on this stream may be replayed on
// another. It never grows or moves, so graphs captured with it stay valid until
// skgemm_release. Under capture nothing can be allocated.
int ops_workspace(hipStream_t stream, uint8_t** out) {
  skg::StreamKey key;
  hipError_t e = skg::stream_key(stream, &key);
  if (e != hipSuccess) return skg::hip_fail(e);
  std::lock_guard<std::mutex> lock(g_mu);
  auto it = g_work.find(key);
  if (it != g_work.end()) {
    *out = it->second;
    return SKGEMM_OK;
  }
  hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
  e = hipStreamIsCapturing(stream, &st);
  if (e != hipSuccess) return skg::hip_fail(e);
  if (st != hipStreamCaptureStatusNone) return SKGEMM_ENOMEM;
  void* p = nullptr;
  if (hipMalloc(&p, SKGEMM_OPS_WORKSPACE_BYTES) != hipSuccess) {
    (void)hipGetLastError();  // reported by the return code
    return SKGEMM_ENOMEM;
  }
  e = hipMemsetAsync(static_cast<uint8_t*>(p) + skg::kOpsPartBytes, 0, (size_t)skg::kOpsCounters * skg::kOpsCounterStride * 4,
                     stream);
  if (e == hipSuccess) e = hipStreamSynchronize(stream);
  if (e != hipSuccess) {
    (void)hipFree(p);
    return skg::hip_fail(e);
  }
  try {
    g_work[key] = static_cast<uint8_t*>(p);
  } catch (...) {  // no exception leaves a C entry
    (void)hipFree(p);
    return SKGEMM_ENOMEM;
  }
  *out = static_cast<uint8_t*>(p);
  return SKGEMM_OK;
}

// The kernels work with scale / log 2.
static_assert(SKGEMM_MAX_SCALE * 1.4426950408889634 < 3.4e38, "in FP32's range");

// The logits' (or their gradient's) own arguments.
int check_logits(const void* logits, int T, int V, float scale, int format, size_t stride) {
  if (T < 0 || V < 0 || (format != SKGEMM_BF16 && format != SKGEMM_F32)) return SKGEMM_EINVAL;
  if (!(scale > 0.0f) || !(scale <= SKGEMM_MAX_SCALE)) return SKGEMM_EINVAL;
  if (V > SKGEMM_MAX_V || T > SKGEMM_MAX_ROWS) return SKGEMM_ESHAPE;
  if (T == 0 || V == 0) return SKGEMM_OK;
  if (logits == nullptr) return SKGEMM_EINVAL;
  const size_t size = format == SKGEMM_F32 ? 4 : 2;
  if (!aligned(logits, 16) || (T > 1 && stride % size != 0)) return SKGEMM_EALIGN;
  if (T > 1 && stride < size * (size_t)V) return SKGEMM_EINVAL;
  return SKGEMM_OK;
}

// Rows of heads: `needed` and, with more than one row, their stride.
int check_heads(const void* a, int T, size_t row, size_t stride, bool written) {
  if (a == nullptr) return SKGEMM_EINVAL;
  if (!aligned(a, 16) || (T > 1 && stride % 16 != 0)) return SKGEMM_EALIGN;
  return written && T > 1 && stride < row ? SKGEMM_EINVAL : SKGEMM_OK;
}

// The rotation's and the norm's own arguments.
int check_turn(int D, int rot, int layout, bool norm, float eps, float amplitude) {
  if (layout != SKGEMM_ROPE_HALF && layout != SKGEMM_ROPE_INTERLEAVED) return SKGEMM_EINVAL;
  if (rot < 0 || D < 0 || !(amplitude > -INFINITY) || !(amplitude < INFINITY)) return SKGEMM_EINVAL;
  if (norm && (!(eps >= 1e-30f) || !(eps < INFINITY))) return SKGEMM_EINVAL;
  if (D % 16 != 0 || D < 16 || D > 256 || rot % 16 != 0 || rot > D) return SKGEMM_ESHAPE;
  return SKGEMM_OK;
}

// A paged cache's own arguments.
int check_cache(const void* K, const void* V, int Hkv, int D, int n_pages, int page_size, int format, float k_scale,
                float v_scale, size_t page_stride, size_t slot_stride, size_t head_stride, bool written) {
  if (format != SKGEMM_BF16 && format != SKGEMM_E4M3) return SKGEMM_EINVAL;
  if (!(k_scale >= 1e-30f) || !(k_scale <= 1e30f) || !(v_scale >= 1e-30f) || !(v_scale <= 1e30f)) return SKGEMM_EINVAL;
  if (format == SKGEMM_BF16 && (k_scale != 1.0f || v_scale != 1.0f)) return SKGEMM_EINVAL;
  if (n_pages < 1 || page_size < 1 || K == nullptr || V == nullptr) return SKGEMM_EINVAL;
  if ((page_size & (page_size - 1)) != 0 || page_size > SKGEMM_MAX_PAGE) return SKGEMM_ESHAPE;
  if (!aligned(K, 16) || !aligned(V, 16)) return SKGEMM_EALIGN;
  // (count, stride) of the axes that have more than one place.
  struct Axis {
    size_t count, stride;
  } axes[3];
  int n = 0;
  const Axis all[3] = {{(size_t)n_pages, page_stride}, {(size_t)page_size, slot_stride}, {(size_t)Hkv, head_stride}};
  for (const Axis& a : all) {
    if (a.count < 2) continue;
    if (a.stride % 16 != 0) return SKGEMM_EALIGN;
    axes[n++] = a;
  }
  const size_t row = (size_t)D * (format == SKGEMM_BF16 ? 2 : 1);
  const size_t limit = (size_t)1 << 32;
  if ((page_size > 1 && slot_stride >= limit) || (Hkv > 1 && head_stride >= limit) ||
      (n_pages > 1 && page_stride >= limit))
    return SKGEMM_ESHAPE;
  if ((page_size > 1 ? (size_t)(page_size - 1) * slot_stride : 0) + (Hkv > 1 ? (size_t)(Hkv - 1) * head_stride : 0) + row >= limit)
    return SKGEMM_ESHAPE;
  if (!written) return SKGEMM_OK;
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && axes[j].stride < axes[j - 1].stride; --j) {
      const Axis a = axes[j];
      axes[j] = axes[j - 1];
      axes[j - 1] = a;
    }
  size_t span = row;
  for (int i = 0; i < n; ++i) {
    if (axes[i].stride < span) return SKGEMM_EINVAL;
    span += (axes[i].count - 1) * axes[i].stride;
  }
  return SKGEMM_OK;
}

skg::CodeScale code_scale(float scale) {
  int e = 0;
  const float b = 2.0f * frexpf(scale, &e);
  return {ldexpf(1.0f, 1 - e), b, 1.0f / b, 448.0f * b};
}

int log2_of(int v) { return __builtin_ctz((unsigned)v); }

}  // namespace

int skg::release_ops_workspaces() {
  std::lock_guard<std::mutex> lock(g_mu);
  int rc = SKGEMM_OK, caller_dev = -1;
  if (hipGetDevice(&caller_dev) != hipSuccess) caller_dev = -1;
  for (auto& kv : g_work) {
    hipError_t e = hipSetDevice(std::get<0>(kv.first));
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e != hipSuccess) rc = hip_fail(e);
    (void)hipFree(kv.second);
  }
  const bool any = !g_work.empty();
  g_work.clear();
  if (any && caller_dev >= 0) {
    const hipError_t e = hipSetDevice(caller_dev);
    if (e != hipSuccess && rc == SKGEMM_OK) rc = hip_fail(e);
  }
  return rc;
}

extern "C" {

SKGEMM_API int skgemm_reserve_ops(hipStream_t stream) {
  uint8_t* w = nullptr;
  return ops_workspace(stream, &w);
}

SKGEMM_API int skgemm_rmsnorm(const void* X, const void* R, const void* G, void* R_out, void* Y,
                              float* y_scale, int T, int H, float eps, int out_format,
                              size_t x_stride, size_t r_stride, size_t r_out_stride,
                              size_t y_stride, hipStream_t stream) {
  if (T < 0 || H < 0) return SKGEMM_EINVAL;
  if (out_format != SKGEMM_BF16 && out_format != SKGEMM_I8 && out_format != SKGEMM_E4M3) return SKGEMM_EINVAL;
  if (!(eps >= 1e-30f) || !(eps < INFINITY)) return SKGEMM_EINVAL;
  if (H % 8 != 0 || H > SKGEMM_MAX_H || T > SKGEMM_MAX_ROWS) return SKGEMM_ESHAPE;
  if (T == 0 || H == 0) return SKGEMM_OK;
  const bool codes = out_format != SKGEMM_BF16;
  if (X == nullptr || Y == nullptr || (codes && y_scale == nullptr)) return SKGEMM_EINVAL;
  if (!aligned(X, 16) || !aligned(R, 16) || !aligned(G, 16) || !aligned(R_out, 16) || !aligned(Y, 16) ||
      !aligned(y_scale, 4))
    return SKGEMM_EALIGN;
  if (T > 1) {  // one row's stride is never used
    const size_t row = 2 * (size_t)H, y_row = codes ? (size_t)H : row;
    if (x_stride % 16 != 0 || (R != nullptr && r_stride % 16 != 0) || (R_out != nullptr && r_out_stride % 16 != 0) ||
        y_stride % (codes ? 8 : 16) != 0)
      return SKGEMM_EALIGN;
    // Inputs may share rows (stride 0); outputs must not overlap.
    if (y_stride < y_row || (R_out != nullptr && r_out_stride < row)) return SKGEMM_EINVAL;
    // On top of an input, another stride would overwrite rows that other workgroups read.
    if (R_out != nullptr && ((R_out == X && r_out_stride != x_stride) || (R_out == R && r_out_stride != r_stride)))
      return SKGEMM_EINVAL;
  }
  skg::NormParams p{};
  p.x = static_cast<const uint8_t*>(X);
  p.r = static_cast<const uint8_t*>(R);
  p.g = static_cast<const uint8_t*>(G);
  p.r_out = static_cast<uint8_t*>(R_out);
  p.y = static_cast<uint8_t*>(Y);
  p.y_scale = y_scale;
  p.x_stride = x_stride;
  p.r_stride = r_stride;
  p.r_out_stride = r_out_stride;
  p.y_stride = y_stride;
  p.T = T;
  p.H = H;
  p.eps = eps;
  const hipError_t e = skg::launch_rmsnorm(p, out_format, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

SKGEMM_API int skgemm_i8(const void* Wq, const float* w_scale, const void* Xq, const float* x_scale,
                         void* C, int T, int N, int K, int out_format, size_t w_stride,
                         size_t x_stride, size_t c_stride, hipStream_t stream) {
  if (T < 0 || N < 0 || K < 0) return SKGEMM_EINVAL;
  if (out_format != SKGEMM_BF16 && out_format != SKGEMM_F32) return SKGEMM_EINVAL;
  if (K % 16 != 0 || K > SKGEMM_MAX_K_I8 || N > SKGEMM_MAX_N || T > SKGEMM_MAX_ROWS) return SKGEMM_ESHAPE;
  if (T == 0 || N == 0) return SKGEMM_OK;
  if (C == nullptr || w_scale == nullptr || x_scale == nullptr) return SKGEMM_EINVAL;
  if (K > 0 && (Wq == nullptr || Xq == nullptr)) return SKGEMM_EINVAL;
  if (!aligned(Wq, 16) || !aligned(Xq, 16) || !aligned(C, 16) || !aligned(w_scale, 4) || !aligned(x_scale, 4))
    return SKGEMM_EALIGN;
  const size_t size = out_format == SKGEMM_F32 ? 4 : 2;
  if (w_stride % 16 != 0 || x_stride % 16 != 0 || c_stride % size != 0) return SKGEMM_EALIGN;
  if (w_stride > SKGEMM_MAX_ROW_STRIDE || x_stride > SKGEMM_MAX_ROW_STRIDE) return SKGEMM_ESHAPE;
  if (w_stride < (size_t)K || x_stride < (size_t)K || c_stride < size * (size_t)N) return SKGEMM_EINVAL;
  skg::I8Params p{};
  p.w = static_cast<const uint8_t*>(Wq);
  p.x = static_cast<const uint8_t*>(Xq);
  p.w_scale = w_scale;
  p.x_scale = x_scale;
  p.c = static_cast<uint8_t*>(C);
  p.w_stride = w_stride;
  p.x_stride = x_stride;
  p.c_stride = c_stride;
  p.T = T;
  p.N = N;
  p.K = K;
  p.out_f32 = out_format == SKGEMM_F32;
  const skg::I8Tactic tac = skg::pick_i8(T, N, K);
  if (tac.S > 1) {
    uint8_t* w = nullptr;
    const int rc = ops_workspace(stream, &w);
    if (rc != SKGEMM_OK) return rc;
    p.part = w;
    p.cnt = reinterpret_cast<uint32_t*>(w + skg::kOpsPartBytes);
  }
  const hipError_t e = skg::launch_i8(p, tac, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

SKGEMM_API int skgemm_logprobs(const void* logits, const int64_t* tokens, float* logprob,
                               float* entropy, float* lse, float* top_logprob, int64_t* top_ids,
                               int T, int V, int top_k, float scale, int logits_format,
                               size_t stride, hipStream_t stream) {
  int rc = check_logits(logits, T, V, scale, logits_format, stride);
  if (rc != SKGEMM_OK) return rc;
  if (top_k < 0) return SKGEMM_EINVAL;
  if (top_k > SKGEMM_MAX_TOP) return SKGEMM_ESHAPE;
  if (T == 0 || V == 0) return SKGEMM_OK;
  if (top_k > V || (logprob != nullptr && tokens == nullptr)) return SKGEMM_EINVAL;
  if (top_k > 0 && (top_logprob == nullptr || top_ids == nullptr)) return SKGEMM_EINVAL;
  if (!aligned(tokens, 8) || !aligned(top_ids, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
      !aligned(top_logprob, 4))
    return SKGEMM_EALIGN;
  skg::LogprobParams p{};
  p.logits = static_cast<const uint8_t*>(logits);
  p.tokens = tokens;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_logprob = top_logprob;
  p.top_ids = top_ids;
  p.stride = stride;
  p.T = T;
  p.V = V;
  p.k = top_k;
  p.scale = scale;
  p.parts = skg::logprob_parts(T, V, logits_format == SKGEMM_F32, &p.per);
  if (p.parts > 1) {  // then T <= 512: at most 1024 runs
    uint8_t* w = nullptr;
    rc = ops_workspace(stream, &w);
    if (rc != SKGEMM_OK) return rc;
    p.part = w;
    p.cnt = reinterpret_cast<uint32_t*>(w + skg::kOpsPartBytes);
  }
  const hipError_t e = skg::launch_logprobs(p, logits_format == SKGEMM_F32, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

SKGEMM_API int skgemm_logprobs_grad(const void* logits, const int64_t* tokens, const float* lse,
                                    const float* entropy, const float* g_logprob,
                                    const float* g_entropy, void* d_logits, int T, int V,
                                    float scale, int logits_format, size_t stride, size_t d_stride,
                                    hipStream_t stream) {
  int rc = check_logits(logits, T, V, scale, logits_format, stride);
  if (rc != SKGEMM_OK) return rc;
  if (T == 0 || V == 0) return SKGEMM_OK;
  if (d_logits == nullptr || lse == nullptr) return SKGEMM_EINVAL;
  if ((g_logprob != nullptr && tokens == nullptr) || (g_entropy != nullptr && entropy == nullptr)) return SKGEMM_EINVAL;
  rc = check_logits(d_logits, T, V, scale, logits_format, d_stride);
  if (rc != SKGEMM_OK) return rc;
  if (d_logits == logits && T > 1 && d_stride != stride) return SKGEMM_EINVAL;
  if (!aligned(tokens, 8) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(g_logprob, 4) || !aligned(g_entropy, 4))
    return SKGEMM_EALIGN;
  skg::LogprobGradParams p{};
  p.logits = static_cast<const uint8_t*>(logits);
  p.tokens = tokens;
  p.lse = lse;
  p.entropy = entropy;
  p.g_logprob = g_logprob;
  p.g_entropy = g_entropy;
  p.d_logits = static_cast<uint8_t*>(d_logits);
  p.stride = stride;
  p.d_stride = d_stride;
  p.T = T;
  p.V = V;
  p.scale = scale;
  const hipError_t e = skg::launch_logprobs_grad(p, logits_format == SKGEMM_F32, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

SKGEMM_API int skgemm_rope(const void* X, const void* G, const float* inv_freq,
                           const int64_t* positions, void* Y, int T, int H, int D, int rot,
                           int layout, float eps, float amplitude, size_t x_stride,
                           size_t y_stride, hipStream_t stream) {
  if (T < 0 || H < 0) return SKGEMM_EINVAL;
  int rc = check_turn(D, rot, layout, G != nullptr, eps, amplitude);
  if (rc != SKGEMM_OK) return rc;
  if (T > SKGEMM_MAX_ROWS || H > SKGEMM_MAX_HEADS) return SKGEMM_ESHAPE;
  if (T == 0 || H == 0) return SKGEMM_OK;
  const size_t row = (size_t)H * D * 2;
  if ((rc = check_heads(X, T, row, x_stride, false)) != SKGEMM_OK) return rc;
  if ((rc = check_heads(Y, T, row, y_stride, true)) != SKGEMM_OK) return rc;
  if (rot > 0 && (inv_freq == nullptr || positions == nullptr)) return SKGEMM_EINVAL;
  if (!aligned(G, 16) || !aligned(inv_freq, 4) || !aligned(positions, 8)) return SKGEMM_EALIGN;
  if (Y == X && T > 1 && x_stride != y_stride) return SKGEMM_EINVAL;
  skg::RopeParams p{};
  p.q = static_cast<const uint8_t*>(X);
  p.gq = static_cast<const uint8_t*>(G);
  p.freq = inv_freq;
  p.pos = positions;
  p.q_out = static_cast<uint8_t*>(Y);
  p.q_stride = x_stride;
  p.q_out_stride = y_stride;
  p.T = T;
  p.Hq = H;
  p.D = D;
  p.rot = rot;
  p.eps = eps;
  p.amplitude = amplitude;
  const hipError_t e = skg::launch_rope(p, layout == SKGEMM_ROPE_INTERLEAVED, false, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

SKGEMM_API int skgemm_rope_append(const void* Q, const void* K, const void* V, const void* Gq,
                                  const void* Gk, const float* inv_freq,
                                  const int64_t* positions, const int64_t* slots, void* Q_out,
                                  void* K_cache, void* V_cache, int T, int Hq, int Hkv, int D,
                                  int n_pages, int page_size, int rot, int layout, float eps,
                                  float amplitude, int cache_format, float k_scale, float v_scale,
                                  size_t q_stride, size_t k_stride, size_t v_stride,
                                  size_t q_out_stride, size_t page_stride, size_t slot_stride,
                                  size_t head_stride, hipStream_t stream) {
  if (T < 0 || Hq < 0 || Hkv < 0) return SKGEMM_EINVAL;
  int rc = check_turn(D, rot, layout, (Gq != nullptr && Hq > 0) || (Gk != nullptr && Hkv > 0), eps, amplitude);
  if (rc != SKGEMM_OK) return rc;
  if (T > SKGEMM_MAX_ROWS || Hq > SKGEMM_MAX_HEADS || Hkv > SKGEMM_MAX_HEADS) return SKGEMM_ESHAPE;
  if (T == 0 || (Hq == 0 && Hkv == 0)) return SKGEMM_OK;
  if (Hq > 0) {
    const size_t row = (size_t)Hq * D * 2;
    if ((rc = check_heads(Q, T, row, q_stride, false)) != SKGEMM_OK) return rc;
    if ((rc = check_heads(Q_out, T, row, q_out_stride, true)) != SKGEMM_OK) return rc;
    if (Q_out == Q && T > 1 && q_stride != q_out_stride) return SKGEMM_EINVAL;
  }
  if (Hkv > 0) {
    const size_t row = (size_t)Hkv * D * 2;
    if ((rc = check_heads(K, T, row, k_stride, false)) != SKGEMM_OK) return rc;
    if ((rc = check_heads(V, T, row, v_stride, false)) != SKGEMM_OK) return rc;
    rc = check_cache(K_cache, V_cache, Hkv, D, n_pages, page_size, cache_format, k_scale, v_scale, page_stride, slot_stride,
                     head_stride, true);
    if (rc != SKGEMM_OK) return rc;
    if (slots == nullptr || K_cache == V_cache) return SKGEMM_EINVAL;
  }
  if (rot > 0 && (inv_freq == nullptr || positions == nullptr)) return SKGEMM_EINVAL;
  if (!aligned(Gq, 16) || !aligned(Gk, 16) || !aligned(inv_freq, 4) || !aligned(positions, 8) || !aligned(slots, 8))
    return SKGEMM_EALIGN;
  skg::RopeParams p{};
  p.q = static_cast<const uint8_t*>(Q);
  p.k = static_cast<const uint8_t*>(K);
  p.v = static_cast<const uint8_t*>(V);
  p.gq = static_cast<const uint8_t*>(Gq);
  p.gk = static_cast<const uint8_t*>(Gk);
  p.freq = inv_freq;
  p.pos = positions;
  p.slots = slots;
  p.q_out = static_cast<uint8_t*>(Q_out);
  p.kc = static_cast<uint8_t*>(K_cache);
  p.vc = static_cast<uint8_t*>(V_cache);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.page_stride = page_stride;
  p.slot_stride = slot_stride;
  p.head_stride = head_stride;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.rot = rot;
  p.eps = eps;
  p.amplitude = amplitude;
  if (Hkv > 0) {
    p.n_slots = (int64_t)n_pages * page_size;
    p.page_shift = log2_of(page_size);
    p.k_by = code_scale(k_scale);
    p.v_by = code_scale(v_scale);
  }
  const hipError_t e = skg::launch_rope(p, layout == SKGEMM_ROPE_INTERLEAVED, Hkv > 0 && cache_format == SKGEMM_E4M3, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

SKGEMM_API int skgemm_paged_attention(const void* Q, const void* K_cache, const void* V_cache,
                                      const int32_t* page_table, const int32_t* kv_len,
                                      const int32_t* q_start, void* O, float* lse, int T, int B,
                                      int max_q, int Hq, int Hkv, int D, int n_pages,
                                      int page_size, int max_pages, float scale, int window,
                                      int cache_format, float k_scale, float v_scale,
                                      size_t q_stride, size_t o_stride, size_t table_stride,
                                      size_t page_stride, size_t slot_stride, size_t head_stride,
                                      hipStream_t stream) {
  if (T < 0 || B < 0 || max_q < 0 || Hq < 0 || Hkv < 0 || D < 0 || n_pages < 0 || max_pages < 0 || window < 0) return SKGEMM_EINVAL;
  if (!(scale > 0.0f) || !(scale <= SKGEMM_MAX_SCALE)) return SKGEMM_EINVAL;
  if (D != 64 && D != 128 && D != 256) return SKGEMM_ESHAPE;
  if (T == 0 || B == 0 || max_q == 0 || Hq == 0) return SKGEMM_OK;
  if (Hkv == 0 || Hq % Hkv != 0 || Hq > SKGEMM_MAX_HEADS || T > SKGEMM_MAX_ROWS || B > (1 << 20)) return SKGEMM_ESHAPE;
  int rc = check_cache(K_cache, V_cache, Hkv, D, n_pages, page_size, cache_format, k_scale, v_scale, page_stride, slot_stride,
                       head_stride, false);
  if (rc != SKGEMM_OK) return rc;
  const int64_t most = (int64_t)1 << 31, G = Hq / Hkv, len = (int64_t)max_pages * page_size;
  if (len > SKGEMM_MAX_LEN || T * G > ((int64_t)1 << 30) || B * (int64_t)Hkv * (len / 64 + 8) >= most ||
      skg::attention_tiles(T, B, max_q < T ? max_q : T, (int)G) * Hkv >= skg::kMostTiles)
    return SKGEMM_ESHAPE;
  const float c = scale * k_scale;
  if (!(c >= 1e-37f) || !(c <= SKGEMM_MAX_SCALE)) return SKGEMM_EINVAL;
  const size_t row = (size_t)Hq * D * 2;
  if ((rc = check_heads(Q, T, row, q_stride, false)) != SKGEMM_OK) return rc;
  if ((rc = check_heads(O, T, row, o_stride, true)) != SKGEMM_OK) return rc;
  if (O == Q && T > 1 && q_stride != o_stride) return SKGEMM_EINVAL;
  if (kv_len == nullptr || q_start == nullptr || (page_table == nullptr && max_pages > 0)) return SKGEMM_EINVAL;
  if (!aligned(page_table, 4) || !aligned(kv_len, 4) || !aligned(q_start, 4) || !aligned(lse, 4) || (B > 1 && table_stride % 4 != 0))
    return SKGEMM_EALIGN;
  skg::AttnParams p{};
  p.q = static_cast<const uint8_t*>(Q);
  p.kc = static_cast<const uint8_t*>(K_cache);
  p.vc = static_cast<const uint8_t*>(V_cache);
  p.table = page_table;
  p.kv_len = kv_len;
  p.q_start = q_start;
  p.o = static_cast<uint8_t*>(O);
  p.lse = lse;
  p.q_stride = q_stride;
  p.o_stride = o_stride;
  p.table_stride = table_stride;
  p.page_stride = (uint32_t)page_stride;
  p.slot_stride = (uint32_t)slot_stride;
  p.head_stride = (uint32_t)head_stride;
  p.T = T;
  p.B = B;
  p.max_q = max_q < T ? max_q : T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = (int)G;
  p.n_pages = n_pages;
  p.page_shift = log2_of(page_size);
  p.max_len = (int)len;
  // One that no sequence is longer than hides nothing, and differences to a token's
  // place stay inside 32 bits without it (place >= 1 - T).
  p.window = window < len ? window : 0;
  p.c = c * 1.4426950408889634f;
  p.v_scale = v_scale;
  uint8_t* w = nullptr;
  rc = ops_workspace(stream, &w);
  if (rc != SKGEMM_OK) return rc;
  p.part = w;
  p.cnt = reinterpret_cast<uint32_t*>(w + skg::kOpsPartBytes);
  const hipError_t e = skg::launch_attention(p, D, cache_format == SKGEMM_E4M3, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

}  // extern "C"
