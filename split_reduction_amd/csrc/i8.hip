// Product of 8-bit integers with a scale for each token and each output
// channel (skgemm_i8):
//   C[t, n] = x_scale[t] * w_scale[n] * sum_k Xq[t, k] Wq[n, k].
//
// v_mfma_i32_16x16x64_i8 with A = weights (rows = output features) and
// B = activations (columns = tokens): lane l = 16 g + i holds the 16 bytes of
// row (column) i at K block g, and D's rows 4g..4g+3 of column i. Sums of
// 32-bit integers are exact and commute, so K is split over waves freely.

#include "device/block.h"
#include "device/pack.h"
#include "ops_internal.h"
#include "skgemm.h"

namespace skg {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Outputs n .. n+3 of token t from their integer sums. The sum is rounded to
// FP32, both products are FP32, and bf16 rounds once more.
__device__ __forceinline__ void store_sums(const I8Params& p, int t, int n, i32x4 s, float xs) {
  if (t >= p.T) return;
  uint8_t* row = p.c + (size_t)t * p.c_stride;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    const float v = (float)s[e] * xs * p.w_scale[n + e];
    if (p.out_f32)
      reinterpret_cast<float*>(row)[n + e] = v;
    else
      reinterpret_cast<uint16_t*>(row)[n + e] = (uint16_t)bf16_rne(v);
  }
}

// Four waves a workgroup split K over a tile of 16 features x 16 NT tokens,
// operands straight from memory into registers, sums joined in LDS.
template <int NT>
__global__ __launch_bounds__(256) void i8_rows_kernel(I8Params p) {
  __shared__ i32x4 part[4][NT][64];
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * 16, t0 = (int)blockIdx.y * 16 * NT;
  const int rows = min(16, p.N - n0), tokens = min(16 * NT, p.T - t0);
  // Resources end with the tile's last row: a row past it reads zeros, and so
  // does K past a row's end by an out-of-range offset.
  const rsrc_t w = make_rsrc(p.w + (size_t)n0 * p.w_stride, (uint32_t)((rows - 1) * p.w_stride + p.K));
  const rsrc_t x = make_rsrc(p.x + (size_t)t0 * p.x_stride, (uint32_t)((tokens - 1) * p.x_stride + p.K));
  i32x4 acc[NT] = {};
  for (int k = wave * 64; k < p.K; k += 256) {
    const int kk = k + 16 * g;
    const bool ok = kk < p.K;
    const u32x4 a = ld16_if(ok && i < rows, w, (uint32_t)(i * p.w_stride + kk));
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const u32x4 b = ld16_if(ok && 16 * j + i < tokens, x, (uint32_t)((16 * j + i) * p.x_stride + kk));
      acc[j] = mfma_i8(a, b, acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  for (int j = wave; j < NT; j += 4) {
    i32x4 s = part[0][j][lane];
#pragma unroll
    for (int v = 1; v < 4; ++v) s += part[v][j][lane];
    const int t = t0 + 16 * j + i;
    store_sums(p, t, n0 + 4 * g, s, t < p.T ? p.x_scale[t] : 0.0f);
  }
}

}  // namespace

hipError_t launch_i8(const I8Params& p, hipStream_t s) {
  const unsigned tiles = (unsigned)((p.N + 15) / 16);
  if (p.T <= 16)
    hipLaunchKernelGGL(i8_rows_kernel<1>, dim3(tiles, (unsigned)((p.T + 15) / 16)), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL(i8_rows_kernel<4>, dim3(tiles, (unsigned)((p.T + 63) / 64)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace skg
