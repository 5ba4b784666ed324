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

}  // extern "C"
