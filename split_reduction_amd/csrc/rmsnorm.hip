// Root-mean-square norm with the residual's addition and a bf16 or 8-bit
// output (skgemm_rmsnorm).
//
//   h = x + r,  y = h * rstd * g,  rstd = 1 / sqrt(mean(h^2) + eps)
//
// One pass: a row stays in the registers of one workgroup between its loads
// and its stores, so each input is read once and each output written once.
// The codes need max|y|, which would be a second reduction after rstd; but
// rstd > 0 is common to the row, so max|y| = rstd * max|h g| and the codes are
//   y / (max|y| / 127) = h g * (127 / max|h g|),
// free of rstd: sum(h^2) and max|h g| meet in one reduction behind one barrier.
//
// Bound by memory: 7 bytes an element (x, r, R_out, codes) and about 10 vector
// operations. T=8192 H=7168 with a residual and E4M3 codes: 70.8 us, 5.8 TB/s (a
// large copy reaches 5.1); T=1: 3.5 us.

#include "device/block.h"
#include "device/pack.h"
#include "ops_internal.h"
#include "skgemm.h"
#include "skgemm_internal.h"

namespace skg {

namespace {

// The low byte of x + 1.5 * 2^23 is x rounded to the nearest even integer in
// two's complement (|x| < 2^22): one addition, no conversion.
__device__ __forceinline__ uint32_t i8_pack4(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b + kMagic), __float_as_uint(a + kMagic), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d + kMagic), __float_as_uint(c + kMagic), 0x0C0C0400u);
  return lo | (hi << 16);
}

template <int OUT>
constexpr float top_code() {
  return OUT == SKGEMM_I8 ? 127.0f : 448.0f;
}

template <bool STREAM>
__device__ __forceinline__ u32x4 load16(const u32x4* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  return *p;
}

// STREAM: x and r are loaded non-temporally.
// VPT: vectors of 8 elements a thread holds; thread i takes vectors i,
// i + blockDim, ... so that a wave's loads and stores are contiguous.
template <int VPT, int OUT, bool STREAM>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormParams p) {
  __shared__ float part[32];
  const size_t t = blockIdx.x;
  const int nv = p.H >> 3;
  const u32x4* x = reinterpret_cast<const u32x4*>(p.x + t * p.x_stride);
  const u32x4* r = p.r != nullptr ? reinterpret_cast<const u32x4*>(p.r + t * p.r_stride) : nullptr;
  const u32x4* g = reinterpret_cast<const u32x4*>(p.g);
  u32x4* ro = p.r_out != nullptr ? reinterpret_cast<u32x4*>(p.r_out + t * p.r_out_stride) : nullptr;

  u32x4 xv[VPT], rv[VPT], gv[VPT];
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = (int)threadIdx.x + i * (int)blockDim.x;
    const bool ok = v < nv;
    xv[i] = ok ? load16<STREAM>(x + v) : u32x4{0, 0, 0, 0};
    rv[i] = (ok && r != nullptr) ? load16<STREAM>(r + v) : u32x4{0, 0, 0, 0};
    gv[i] = (ok && g != nullptr) ? g[v] : ones;
  }
  float h[VPT * 8], hg[VPT * 8];
  float ss = 0.0f, top = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // No residual: zeros are added, which changes nothing but -0.
      const float a = bf16_lo(xv[i][e]) + bf16_lo(rv[i][e]), b = bf16_hi(xv[i][e]) + bf16_hi(rv[i][e]);
      h[8 * i + 2 * e] = a;
      h[8 * i + 2 * e + 1] = b;
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
    }
    if (ro != nullptr) {
      const int v = (int)threadIdx.x + i * (int)blockDim.x;
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = bf16_pair(h[8 * i + 2 * e], h[8 * i + 2 * e + 1]);
      if (v < nv) ro[v] = w;
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hg[8 * i + 2 * e] = h[8 * i + 2 * e] * bf16_lo(gv[i][e]);
      hg[8 * i + 2 * e + 1] = h[8 * i + 2 * e + 1] * bf16_hi(gv[i][e]);
      // NaN counts: a NaN in G (h's own are in ss) must not leave a finite scale.
      top = max_or_nan(top, max_or_nan(fabsf(hg[8 * i + 2 * e]), fabsf(hg[8 * i + 2 * e + 1])));
    }
  block_sum_max(ss, top, part);
  float eps = p.eps;
  constexpr float kInf = __builtin_inff();
  // ss or top out of FP32's range though h may be finite: take the row by a
  // power of two and reduce again (uniform over the workgroup, rare).
  // A NaN in ss stays: the row holds one.
  if (ss == kInf || (top == kInf && ss == ss)) {
    float m = 0.0f, none = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT * 8; ++i) m = fmaxf(m, fabsf(h[i]));
    __syncthreads();
    block_sum_max(none, m, part);
    if (m == kInf) {
      ss = __builtin_nanf("");
    } else {
      // m * f / 4 lies in 1/2..1, so that the products with G stay in range; f
      // alone does for every finite m, f / 4 would pass below FP32's normals.
      const float f = __uint_as_float((255u - (__float_as_uint(m) >> 23)) << 23);
      eps = eps * f * f * 0.0625f;
      ss = 0.0f;
      top = 0.0f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = h[8 * i + e] * f * 0.25f;
          const uint32_t w = gv[i][e >> 1];
          hg[8 * i + e] = a * ((e & 1) ? bf16_hi(w) : bf16_lo(w));
          ss = fmaf(a, a, ss);
          top = max_or_nan(top, fabsf(hg[8 * i + e]));
        }
      __syncthreads();
      block_sum_max(ss, top, part);
    }
  }
  const float rstd = 1.0f / sqrtf(ss / (float)p.H + eps);  // NaN where the row holds a NaN or infinity
  float mul = rstd;
  if constexpr (OUT != SKGEMM_BF16) {
    // The product first, as top alone may be near FP32's smallest; last where it
    // would pass FP32's range and the scale does not.
    float scale = rstd * top;
    scale = scale < kInf ? scale / top_code<OUT>() : rstd * (top / top_code<OUT>());
    if (threadIdx.x == 0) p.y_scale[t] = scale;
    // 127 / top would pass FP32's range for a tiny top: such a row is lifted
    // by a power of two first (exact). Zero rows get zero codes.
    if (top < 1e-30f) {
#pragma unroll
      for (int i = 0; i < VPT * 8; ++i) hg[i] *= 0x1p96f;
      top *= 0x1p96f;
    }
    mul = top > 0.0f && scale == scale ? top_code<OUT>() / top : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = (int)threadIdx.x + i * (int)blockDim.x;
    float* y = hg + 8 * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= mul;
    if (v >= nv) continue;
    if constexpr (OUT == SKGEMM_BF16) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = bf16_pair(y[2 * e], y[2 * e + 1]);
      reinterpret_cast<u32x4*>(p.y + t * p.y_stride)[v] = w;
    } else {
      u32x2 w;
      if constexpr (OUT == SKGEMM_I8) {
        w.x = i8_pack4(y[0], y[1], y[2], y[3]);
        w.y = i8_pack4(y[4], y[5], y[6], y[7]);
      } else {
        w.x = e4m3_pack4(y[0], y[1], y[2], y[3]);
        w.y = e4m3_pack4(y[4], y[5], y[6], y[7]);
      }
      reinterpret_cast<u32x2*>(p.y + t * p.y_stride)[v] = w;
    }
  }
}

template <int VPT, bool STREAM>
hipError_t launch_vpt(const NormParams& p, int out_format, hipStream_t s) {
  const int nv = p.H / 8;
  const dim3 grid((unsigned)p.T), block((unsigned)((((nv + VPT - 1) / VPT) + 63) / 64 * 64));
  if (out_format == SKGEMM_BF16) return launch(rmsnorm_kernel<VPT, SKGEMM_BF16, STREAM>, grid, block, 0, s, p);
  if (out_format == SKGEMM_I8) return launch(rmsnorm_kernel<VPT, SKGEMM_I8, STREAM>, grid, block, 0, s, p);
  return launch(rmsnorm_kernel<VPT, SKGEMM_E4M3, STREAM>, grid, block, 0, s, p);
}

}  // namespace

// Few rows: as many threads as a row has vectors, up to 1024, so that all loads
// go out at once. Many rows of more than 512 vectors: four vectors a thread, so
// that more rows share a CU (T=8192 H=7168: 101 us with one, 77 with two, 75 with
// four; T=8192 H=1024 12.4 / 13.1 us, left at one). Inputs past the 256 MB that
// the last cache holds are loaded non-temporally (T=4096 H=16384: 84 against 76
// us; T=8192 H=1024, which it holds, 12.4 against 13.8).
hipError_t launch_rmsnorm(const NormParams& p, int out_format, hipStream_t s) {
  const int nv = p.H / 8;  // at most 4096
  const bool stream = (size_t)p.T * (size_t)p.H * 7 > ((size_t)256 << 20);
  const int vpt = nv > 2048 || (nv > 512 && p.T > 1024) ? 4 : nv > 1024 ? 2 : 1;
  if (vpt == 4) return stream ? launch_vpt<4, true>(p, out_format, s) : launch_vpt<4, false>(p, out_format, s);
  if (vpt == 2) return launch_vpt<2, false>(p, out_format, s);  // T <= 1024: below 256 MB
  return stream ? launch_vpt<1, true>(p, out_format, s) : launch_vpt<1, false>(p, out_format, s);
}

}  // namespace skg
