// C ABI of the operators around the layers and the head: argument checks,
// their workspace and kernel dispatch. Declarations and contracts:
// include/skgemm.h.

#include <math.h>

#include "ops_internal.h"
#include "skgemm.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (uintptr_t)p % n == 0; }

}  // namespace

extern "C" {

SKGEMM_API int skgemm_rmsnorm(const void* X, const void* R, const void* G, void* R_out, void* Y,
                              float* y_scale, int T, int H, float eps, int out_format,
                              size_t x_stride, size_t r_stride, size_t r_out_stride,
                              size_t y_stride, hipStream_t stream) {
  if (T < 0 || H < 0) return SKGEMM_EINVAL;
  if (out_format != SKGEMM_BF16 && out_format != SKGEMM_I8 && out_format != SKGEMM_E4M3) return SKGEMM_EINVAL;
  if (!(eps >= 1e-30f) || !(eps < INFINITY)) return SKGEMM_EINVAL;
  if (H % 8 != 0 || H > SKGEMM_MAX_H) return SKGEMM_ESHAPE;
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
  if (K % 16 != 0 || K > SKGEMM_MAX_K_I8 || N > SKGEMM_MAX_N) return SKGEMM_ESHAPE;
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
  const hipError_t e = skg::launch_i8(p, stream);
  return e == hipSuccess ? SKGEMM_OK : skg::hip_fail(e);
}

}  // extern "C"
