// Norm of each head and rotation by position, into rows (skgemm_rope) or on the
// way into a paged cache (skgemm_rope_append).
//
//   y = x / sqrt(mean(x^2) + eps) * g over the D values of a head (with a gain),
//   (a, b) -> A (a cos w - b sin w, b cos w + a sin w), w = position * inv_freq[i],
//   for the rot / 2 pairs of its first rot values.
//
// A head belongs to L = D / 16 neighbouring lanes (rounded up to a power of two)
// that hold two 16-byte vectors each: vectors u and u + rot / 16 of the half
// layout, 2u and 2u + 1 of the interleaved one, so that in both the lane has both
// values of its eight pairs 8u .. 8u + 7 and a head is read and written once. The
// squares meet by exchanges between the head's lanes.
//
// The angles are a token's, not a head's: a workgroup takes whole tokens (or a
// run of one token's heads where tokens are few) and computes each cosine once,
// into LDS, while its first heads are on their way. The angle is a product in
// FP64, reduced to part of a turn there: FP32 has lost a position of 2^20 to 0.06
// radians.
//
// Bound by memory (4 bytes an element of the queries, 6 or 8 of keys and values)
// and below that by the launch. Other inputs in every call: T=8192 of 64 heads of 128, half
// of each turned, 52 us, 5.2 TB/s (as a large copy), with 8 key heads into E4M3 60; T=1 of
// 16: 2.4 us. Non-temporal loads: between 3 % faster and 5 % slower at 100 MB to 1 GB.

#include "device/pack.h"
#include "device/wave.h"
#include "ops_internal.h"
#include "skgemm.h"
#include "skgemm_internal.h"

namespace skg {

namespace {

constexpr int kThreads = 256;

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v = xred_add<1>(v);
  if constexpr (L >= 4) v = xred_add<2>(v);
  if constexpr (L >= 8) v = xred_add<4>(v);
  if constexpr (L >= 16) v = xred_add<8>(v);
  return v;
}
// v / scale on its way to an E4M3 code: saturated, NaN kept. The quotient by the rounded
// reciprocal is up to 1.5 steps off, which takes values beside a border between two codes
// to the other side; one correction by its remainder makes it one of the two nearest
// floats, so that the next remainder is exact and the second correction gives the
// quotient as it is rounded to nearest (Markstein). All in the range of b, where nothing
// underflows that is not 0 as a code. Product with the reciprocal / this / the division
// operator: T=8192 of 64 + 8 heads 60.6 / 61.3 / 61.6 us, T=2048 of 32 + 32 20.7 / 21.5 /
// 23.8, T=16384 of 8 + 8 41.1 / 42.1 / 45.1.
__device__ __forceinline__ float to_code_range(float v, const CodeScale& s) {
  v = __builtin_elementwise_minimum(__builtin_elementwise_maximum(v * s.up, -s.most), s.most);
  float q = v * s.inv;
  q = fmaf(fmaf(-q, s.b, v), s.inv, q);
  return fmaf(fmaf(-q, s.b, v), s.inv, q);
}

// ONE: a workgroup has heads of one token, so that what goes by the token is the same
// in all lanes.
template <int L, bool INTER, bool CODES, bool ONE>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p) {
  constexpr int kSlots = kThreads / L;  // heads at once
  extern __shared__ float2 turn[];      // [tokens of the workgroup][rot / 2]: cos, sin
  const int u = (int)threadIdx.x % L, slot = (int)threadIdx.x / L;
  const int heads = p.Hq + 2 * p.Hkv, half = p.rot >> 1;
  const int t0 = ONE ? (int)blockIdx.x : (int)blockIdx.x * p.tokens, nt = ONE ? 1 : min(p.tokens, p.T - t0);
  const int first = (int)blockIdx.y * p.per, last = min(nt * heads, first + p.per);
  const bool in_head = u < (p.D >> 4), turns = u < (p.rot >> 4);
  // This lane's two vectors: past the rotated ones, neighbours in both layouts.
  const int va = INTER ? 2 * u : turns ? u : 2 * u;
  const int vb = INTER || !turns ? 2 * u + 1 : u + (p.rot >> 4);

  struct Item {
    u32x4 a, b;
    int t, h;
  };
  auto load = [&](int i) {
    Item it{};
    if (i >= last) return it;
    const int tl = ONE ? 0 : i / heads;
    it.h = i - tl * heads;
    if constexpr (!ONE) it.t = t0 + tl;
    const int t = ONE ? t0 : it.t;
    if (!in_head) return it;
    const uint8_t* row;
    if (it.h < p.Hq)
      row = p.q + (size_t)t * p.q_stride + (uint32_t)(it.h * p.D * 2);
    else if (it.h < p.Hq + p.Hkv)
      row = p.k + (size_t)t * p.k_stride + (uint32_t)((it.h - p.Hq) * p.D * 2);
    else
      row = p.v + (size_t)t * p.v_stride + (uint32_t)((it.h - p.Hq - p.Hkv) * p.D * 2);
    const u32x4* const vectors = reinterpret_cast<const u32x4*>(row);
    it.a = vectors[va];
    it.b = vectors[vb];
    return it;
  };

  int i = first + slot;
  Item now = load(i);
  u32x4 gain[2][2] = {};  // the queries' and the keys'
  if (in_head) {
    if (p.gq != nullptr) gain[0][0] = reinterpret_cast<const u32x4*>(p.gq)[va], gain[0][1] = reinterpret_cast<const u32x4*>(p.gq)[vb];
    if (p.gk != nullptr) gain[1][0] = reinterpret_cast<const u32x4*>(p.gk)[va], gain[1][1] = reinterpret_cast<const u32x4*>(p.gk)[vb];
  }
  for (int w = (int)threadIdx.x; w < nt * half; w += kThreads) {
    const int tl = ONE ? 0 : w / half;
    const double in_turns = (double)p.pos[t0 + tl] * (double)p.freq[w - tl * half] * 0.15915494309189533577;  // / 2 pi
    float s, c;
    sincospif(2.0f * (float)(in_turns - rint(in_turns)), &s, &c);
    turn[w] = float2{c * p.amplitude, s * p.amplitude};
  }
  if (half > 0) __syncthreads();

  for (; i < last; i += kSlots) {
    const Item it = now;
    now = load(i + kSlots);
    float a[8], b[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[2 * e] = bf16_lo(it.a[e]);
      a[2 * e + 1] = bf16_hi(it.a[e]);
      b[2 * e] = bf16_lo(it.b[e]);
      b[2 * e + 1] = bf16_hi(it.b[e]);
    }
    const int part = it.h < p.Hq ? 0 : it.h < p.Hq + p.Hkv ? 1 : 2;
    if ((part == 0 && p.gq != nullptr) || (part == 1 && p.gk != nullptr)) {
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
      ss = lanes_sum<L>(ss);
      float eps = p.eps;
      constexpr float kInf = __builtin_inff();
      if (ss == kInf) {  // the squares pass FP32's range (the head's lanes agree): eps is nothing beside them
        eps = ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] *= 0x1p-100f;
          b[e] *= 0x1p-100f;
          ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
        }
        ss = lanes_sum<L>(ss);
        if (ss == kInf) ss = __builtin_nanf("");  // the head holds an infinity
      }
      const float rstd = __builtin_amdgcn_rsqf(ss * p.by_d + eps);
      u32x4 ga, gb;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // by element: an index into the registers would cost 15 times this
        ga[e] = part == 0 ? gain[0][0][e] : gain[1][0][e];
        gb[e] = part == 0 ? gain[0][1][e] : gain[1][1][e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t wa = ga[e >> 1], wb = gb[e >> 1];
        a[e] = a[e] * rstd * ((e & 1) ? bf16_hi(wa) : bf16_lo(wa));
        b[e] = b[e] * rstd * ((e & 1) ? bf16_hi(wb) : bf16_lo(wb));
      }
    }
    if (part != 2 && turns) {
      const float2* const cs = turn + (ONE ? 0 : it.t - t0) * half + 8 * u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = cs[e];
        float &x = INTER ? (e < 4 ? a[2 * e] : b[2 * e - 8]) : a[e], &y = INTER ? (e < 4 ? a[2 * e + 1] : b[2 * e - 7]) : b[e];
        const float x0 = x, y0 = y;
        x = x0 * w.x - y0 * w.y;
        y = y0 * w.x + x0 * w.y;
      }
    }
    if (!in_head) continue;
    const int t = ONE ? t0 : it.t;
    uint8_t* out;
    bool codes = false;
    if (part == 0) {
      out = p.q_out + (size_t)t * p.q_out_stride + (uint32_t)(it.h * p.D * 2);
    } else {
      const int64_t at = p.slots[t];
      if (at < 0 || at >= p.n_slots) continue;  // padding, or past the cache
      const int h = it.h - p.Hq - (part == 2 ? p.Hkv : 0);
      out = (part == 1 ? p.kc : p.vc) + (size_t)(at >> p.page_shift) * p.page_stride +
            (size_t)(at & ((1 << p.page_shift) - 1)) * p.slot_stride + (size_t)h * p.head_stride;
      codes = CODES;
    }
    if (codes) {
      const CodeScale by = part == 1 ? p.k_by : p.v_by;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = to_code_range(a[e], by);
        b[e] = to_code_range(b[e], by);
      }
      reinterpret_cast<u32x2*>(out)[va] = u32x2{e4m3_pack4(a[0], a[1], a[2], a[3]), e4m3_pack4(a[4], a[5], a[6], a[7])};
      reinterpret_cast<u32x2*>(out)[vb] = u32x2{e4m3_pack4(b[0], b[1], b[2], b[3]), e4m3_pack4(b[4], b[5], b[6], b[7])};
    } else {
      u32x4 wa, wb;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wa[e] = bf16_pair_hw(a[2 * e], a[2 * e + 1]);
        wb[e] = bf16_pair_hw(b[2 * e], b[2 * e + 1]);
      }
      reinterpret_cast<u32x4*>(out)[va] = wa;
      reinterpret_cast<u32x4*>(out)[vb] = wb;
    }
  }
}

template <int L, bool ONE>
hipError_t launch_kind(const RopeParams& p, bool inter, bool codes, dim3 grid, size_t lds, hipStream_t s) {
  const dim3 block(kThreads);
  if (inter) {
    if (codes) return launch(rope_kernel<L, true, true, ONE>, grid, block, lds, s, p);
    return launch(rope_kernel<L, true, false, ONE>, grid, block, lds, s, p);
  }
  if (codes) return launch(rope_kernel<L, false, true, ONE>, grid, block, lds, s, p);
  return launch(rope_kernel<L, false, false, ONE>, grid, block, lds, s, p);
}

template <int L>
hipError_t launch_lanes(RopeParams p, bool inter, bool codes, hipStream_t s) {
  constexpr int kSlots = kThreads / L;
  const int heads = p.Hq + 2 * p.Hkv;
  // Few heads: several tokens to a workgroup, one head a slot. Few tokens: a
  // token's heads over several workgroups.
  p.tokens = heads >= kSlots ? 1 : kSlots / heads;
  p.per = p.tokens * heads;
  unsigned gx = (unsigned)((p.T + p.tokens - 1) / p.tokens), gy = 1;
  if (p.tokens == 1 && gx < 1024) {
    p.per = kSlots;
    gy = (unsigned)((heads + kSlots - 1) / kSlots);
  }
  const size_t lds = (size_t)p.tokens * (size_t)(p.rot / 2) * sizeof(float2);  // at most 16 KB
  const dim3 grid(gx, gy);
  p.by_d = 1.0f / (float)p.D;
  return p.tokens == 1 ? launch_kind<L, true>(p, inter, codes, grid, lds, s) : launch_kind<L, false>(p, inter, codes, grid, lds, s);
}

}  // namespace

hipError_t launch_rope(const RopeParams& p, bool inter, bool codes, hipStream_t s) {
  if (p.D <= 64) return launch_lanes<4>(p, inter, codes, s);
  if (p.D <= 128) return launch_lanes<8>(p, inter, codes, s);
  return launch_lanes<16>(p, inter, codes, s);
}

}  // namespace skg
