// Attention of new tokens over a paged cache (skgemm_paged_attention).
//
// Row (i, g) of a sequence's key head is the i-th new token and the g-th of the G
// = Hq / Hkv queries that share the head; it sits at p = L - n + i and sees the
// keys lo <= j < hi with hi = p + 1, lo = p + 1 - window:
//   s_j = scale q.k_j, o = sum_j exp(s_j - lse) v_j, lse = log sum_j exp(s_j).
// All rows of a key head read the same keys, so they are one matrix: tiles of 32
// rows, whichever token and query they are.
//
// Both products are v_mfma_f32_32x32x16_bf16 with the rows as columns:
//   S^T [32 keys x 32 rows] = K Q^T,  O^T [32 values x 32 rows] += V^T P^T.
// Lane l = 32 h + r of a result then holds row r alone, keys 8 a + 4 h + b in
// element 4 a + b, so a row's maximum and sum are taken inside two lanes, the
// rescaling of O is one factor a lane, and P goes into the second product from
// where it lies: slot 8 h + e of the product's K axis stands for key 8 (e / 4) +
// 4 h + e % 4 of its 16, which V^T follows. V lies in LDS by keys;
// ds_read_b64_tr_b16 (16 lanes read 4 rows x 16 columns and get 4 rows of a column
// each) turns it on the way to the registers, ds_read_b64_tr_b8 does for E4M3.
//
// The softmax runs in one pass with the running maximum m (in powers of two) and
// sum l in FP32; O and l are rescaled only where a maximum grows by more than 2^8
// (P stays below 2^8, bf16 has the same relative step there). An exponent is taken as
// s c - m, one fused operation; m is rounded, so past 2^24 that is off by more than
// half a power of two, and the score's own difference to the row's largest is taken
// (a branch that only a grown maximum can turn on). P is rounded to bf16
// for the second product, 2^-9 of each probability; l sums the unrounded ones. The
// product takes both operands in one type and V is bf16; P as the sum of two would cost
// prompts a third (8192 tokens of 32 heads 546 -> 730 us, single tokens up to 5 %) to bring
// the outputs' error from 0.0022 of their size to the 0.0016 of their own rounding.
//
// Keys and values come straight from memory into LDS, 16 bytes a lane, each row
// by its page's id; the ids themselves take the same way two tiles ahead, so that
// no register load is waited for in the loop. 16-byte chunks change places inside
// a row so that the rows of one LDS access meet different banks.

#include "device/mfma.h"
#include "device/pack.h"
#include "device/wave.h"
#include "device/wfmt.h"
#include "ops_internal.h"
#include "skgemm.h"
#include "skgemm_internal.h"

namespace skg {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
#define SKG_LDS __attribute__((address_space(3)))

constexpr float kFloor = -3.402823466e38f;  // maximum of a row that has seen no key: FP32's lowest
constexpr float kGrowth = 8.0f;    // powers of two that P may reach
constexpr float kFar = 0x1p24f;    // maxima whose rounding shows in P
constexpr float kLog2 = 0.69314718055994531f;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16 (4) bytes a lane from each lane's address into LDS at `lds` + 16 (4) l; see
// ld16_to_lds for why in asm and who waits.
template <bool STREAM>
__device__ __forceinline__ void global16_to_lds(const uint8_t* p, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
  if constexpr (STREAM)  // non-temporal
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(lds), "v"(p) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
#endif
}
__device__ __forceinline__ void global4_to_lds(const uint8_t* p, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
#endif
}
// Until at most N vector memory operations of this wave are under way.
template <int N>
__device__ __forceinline__ void wait_vmem() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
#endif
}

__device__ __forceinline__ float swap_max(float v) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_int(v), __float_as_int(v), false, false);
  return fmaxf(__int_as_float(p[0]), __int_as_float(p[1]));
}

// ---- how keys and values lie in LDS ----

template <int D, bool F8>
struct Cache {
  static constexpr int kRow = D * (F8 ? 1 : 2);  // bytes
  static constexpr int kChunks = kRow / 16;
  static constexpr int kRows = 64 / kChunks;     // rows of one wave's load
  // What a row's chunk numbers are exchanged with. Keys are read by 32 rows, the
  // same chunk of each: 8 neighbouring rows (16 of 256 bytes and more) take theirs apart.
  __device__ static __forceinline__ int key_swizzle(int row) {
    return kRow >= 256 ? row & 15 : kRow >= 128 ? row & 7 : (row >> 1) & 3;
  }
  // Values are read by 4 rows x 32 bytes (bf16), or rows 0..3 and 8..11 of 16 x 16
  // bytes (E4M3).
  __device__ static __forceinline__ int value_swizzle(int row) {
    if constexpr (!F8) return kRow >= 256 ? (row & 3) << 2 : (row & 3) << 1;
    return kRow >= 128 ? (row & 3) | ((row >> 1) & 4) : ((row >> 1) & 1) | ((row >> 2) & 2);
  }
};

// One key head's pages and a sequence's table.
struct Pages {
  const uint8_t *k, *v, *ids;
  uint32_t page_stride, slot_stride;
  int n_pages, shift;
};

// The ids of the pages of keys base .. base + KEYS - 1 (none past `last`) on
// their way into 64 words of LDS.
template <int KEYS>
__device__ __forceinline__ void issue_ids(const Pages& c, int base, int last, uint32_t lds, int lane) {
  const int key = min(base + lane % KEYS, last);
  global4_to_lds(c.ids + 4 * (size_t)(uint32_t)(key >> c.shift), lds);
}

// This lane's part of keys base .. base + KEYS - 1, its wave's share of WAVES. Past
// `last` that key is taken again. A page that does not exist is not read (page 0 is)
// and reported.
template <int D, bool F8, int KEYS, int WAVES>
struct Share {
  typedef Cache<D, F8> L;
  static constexpr int kLoads = KEYS / L::kRows / WAVES;
  static_assert(kLoads >= 1, "every wave has a share");
  uint32_t page[kLoads];
  int base, last;

  __device__ __forceinline__ bool find(const Pages& c, int first, int end, const uint32_t* ids, int wave, int lane) {
    bool bad = false;
    base = first;
    last = end;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      page[q] = ids[(wave * kLoads + q) * L::kRows + lane / L::kChunks];
      if (page[q] >= (uint32_t)c.n_pages) {
        page[q] = 0;
        bad = true;
      }
    }
    return bad;
  }
  // VALUES: the values, else the keys, to KEYS rows at `lds`, non-temporally: nobody
  // else reads them (64 tokens over 213k cached: 214 -> 194 us).
  template <bool VALUES>
  __device__ __forceinline__ void issue(const Pages& c, uint32_t lds, int wave, int lane) const {
    // What follows from the lane is the same for every tile; kept from one to the next
    // it would take more registers than there are (D = 256: spills).
    asm volatile("" : "+v"(lane));
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int row = (wave * kLoads + q) * L::kRows + lane / L::kChunks, at = lane % L::kChunks;
      const int chunk = at ^ (VALUES ? L::value_swizzle(row) : L::key_swizzle(row));
      global16_to_lds<true>((VALUES ? c.v : c.k) + place(c, q, row) + 16 * chunk, lds + (uint32_t)(wave * kLoads + q) * 1024u);
    }
  }
  // Both, for a key head that other workgroups read as well.
  __device__ __forceinline__ void issue_both(const Pages& c, uint32_t keys, uint32_t values, int wave, int lane) const {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int row = (wave * kLoads + q) * L::kRows + lane / L::kChunks, at = lane % L::kChunks;
      const size_t off = place(c, q, row);
      const uint32_t to = (uint32_t)(wave * kLoads + q) * 1024u;
      global16_to_lds<false>(c.k + 16 * (at ^ L::key_swizzle(row)) + off, keys + to);
      global16_to_lds<false>(c.v + 16 * (at ^ L::value_swizzle(row)) + off, values + to);
    }
  }
  __device__ __forceinline__ size_t place(const Pages& c, int q, int row) const {
    const uint32_t in_page = (uint32_t)(min(base + row, last) & ((1 << c.shift) - 1)) * c.slot_stride;
    return (size_t)page[q] * c.page_stride + in_page;
  }
};

// ---- a wave's rows ----

__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

template <int D, bool F8, int RT, int KB>
struct Rows {
  typedef Cache<D, F8> L;
  static constexpr int kDT = D / 32;
  bf16x8 q[RT][D / 16];
  f32x16 o[RT][kDT];
  float m[RT], l[RT];
  float largest[RT];   // the score that m is of, as the product leaves it; 0: none yet
  bool far[RT];        // some row of the wave has |m| >= kFar
  int lo[RT], hi[RT];  // keys that this lane's row sees
  uint32_t lost[RT][kDT / 2];  // bit 16 (d % 2) + e: element e of o[t][d] is NaN

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kFloor;
      l[t] = 0.0f;
      largest[t] = 0.0f;
      far[t] = false;
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        o[t][d] = f32x16{};
        lost[t][d / 2] = 0;
      }
    }
  }

  // The row's query as the product takes it: step k, half h. With E4M3 keys a lane
  // reads 16 of them at once and uses them in two steps.
  __device__ __forceinline__ void load_query(int t, const uint8_t* row, bool ok, int h) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const int d = F8 ? 32 * (k >> 1) + 16 * h + 8 * (k & 1) : 16 * k + 8 * h;
      const u32x4 w = ok ? *reinterpret_cast<const u32x4*>(row + 2 * d) : u32x4{0, 0, 0, 0};
      q[t][k] = as_bf16x8(w);
    }
  }

  // The steps of a product go in groups of two or four operands: a group is read from LDS
  // while the one before is multiplied, and no further ahead (the compiler would
  // read everything at once and spill).
  static __device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

  // Where a lane reads: 16 bytes of chunk 2 k + h of key r lie at key_place ^ 32 k, 32
  // keys on is 32 rows on. The swizzle only exchanges chunks inside a row, and tiles lie
  // at multiples of 1024, so one register and an exclusive or a step do.
  static __device__ __forceinline__ uint32_t key_place(int lane) {
    const int r = lane & 31, h = lane >> 5;
    return (uint32_t)(r * L::kRow + 16 * (h ^ L::key_swizzle(r)));
  }
  static __device__ __forceinline__ u32x4 read_key(uint32_t place, int k, int kb) {
    return *(SKG_LDS const u32x4*)((place ^ (32u * (uint32_t)k)) + (uint32_t)(32 * kb * L::kRow));
  }

  __device__ __forceinline__ void scores(f32x16 (&s)[RT][KB], uint32_t keys, int lane) const {
    constexpr int kSteps = D / (F8 ? 32 : 16), kGroup = F8 || D == 256 ? 2 : 4, kGroups = KB * kSteps / kGroup;
    const uint32_t place = keys + key_place(lane);
    u32x4 w[2][kGroup];
    auto read = [&](int g) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i)  // neighbours do not wait for each other's sums
        w[g & 1][i] = read_key(place, (g * kGroup + i) / KB, (g * kGroup + i) % KB);
    };
    read(0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) read(g + 1);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int kb = (g * kGroup + i) % KB, k = (g * kGroup + i) / KB;
        const u32x4 x = w[g & 1][i];
        if constexpr (F8) {
          const bf16x8 a = fp8x8_bf16(x[0], x[1], 1.0f), b = fp8x8_bf16(x[2], x[3], 1.0f);
#pragma unroll
          for (int t = 0; t < RT; ++t) s[t][kb] = mfma32(a, q[t][2 * k], k == 0 ? f32x16{} : s[t][kb]);
#pragma unroll
          for (int t = 0; t < RT; ++t) s[t][kb] = mfma32(b, q[t][2 * k + 1], s[t][kb]);
        } else {
#pragma unroll
          for (int t = 0; t < RT; ++t) s[t][kb] = mfma32(as_bf16x8(x), q[t][k], k == 0 ? f32x16{} : s[t][kb]);
        }
      }
      fence();
    }
  }

  // Values 32 d .. 32 d + 31 of the 16 keys of a step, as they lie in LDS and as the
  // product takes them: at value_place ^ (32 values of a row), 16 keys on 16 rows on.
  static __device__ __forceinline__ uint32_t value_place(int lane) {
    const int i = lane & 15, side = (lane >> 4) & 1, h = lane >> 5;
    const int row = F8 ? 4 * h + ((i >> 1) & 3) + 8 * (i >> 3) : 4 * h + (i >> 2);
    const int chunk = F8 ? side : 2 * side + ((i >> 1) & 1);
    return (uint32_t)(row * L::kRow + 16 * (chunk ^ L::value_swizzle(row)) + 8 * (i & 1));
  }
  static __device__ __forceinline__ u32x4 read_values(uint32_t place, int step, int d) {
    const uint32_t at = (place ^ (uint32_t)(d * (F8 ? 32 : 64))) + (uint32_t)(16 * step * L::kRow);
    if constexpr (F8) {
      const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((SKG_LDS i32x2*)at);
      return u32x4{(uint32_t)w[0], (uint32_t)w[1], 0, 0};
    } else {
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SKG_LDS s16x4*)at);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SKG_LDS s16x4*)(at + 8 * L::kRow));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  static __device__ __forceinline__ bf16x8 value_operand(u32x4 w) {
    if constexpr (F8)
      return fp8x8_bf16(w[0], w[1], 1.0f);
    else
      return as_bf16x8(w);
  }

  // A tile of 32 KB keys from `base` of which some row does not see all: what it does
  // not see has score -inf (hide) and probability 0. A value that is no number would
  // still make a NaN of that 0. Such values are taken out of the tile, and the
  // outputs of rows that do see one are noted in `lost`. SHARE waves share the tile.
  template <int SHARE>
  __device__ __forceinline__ void clean_values(uint32_t values, int base, int wave, int lane) {
    if (any_not_finite(values, lane)) {  // the same in all waves that share the tile
      note_lost(values, base, lane);
      if constexpr (SHARE > 1) __syncthreads();
      take_out(values, wave, SHARE, lane);
      if constexpr (SHARE > 1) __syncthreads();
    }
  }

  __device__ __forceinline__ void hide(f32x16 (&s)[RT][KB], int base, int lane) const {
    asm volatile("" : "+v"(lane));  // or the compiler does this for every tile and selects
    const int h = lane >> 5;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = base + 32 * kb + 8 * (e >> 2) + 4 * h + (e & 3);
          s[t][kb][e] = key >= lo[t] && key < hi[t] ? s[t][kb][e] : -__builtin_inff();
        }
  }

  __device__ __forceinline__ bool is_far(int t) const { return largest[t] != 0.0f && fabsf(m[t]) >= kFar; }
  // Scores to probabilities: maximum, sum and O rescaled where it grows.
  __device__ __forceinline__ void softmax(f32x16 (&s)[RT][KB], bf16x8 (&p)[RT][KB][2], float c) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float top = -__builtin_inff();
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][kb][e]);
      const float score = swap_max(top);
      top = score * c;
      if (D == 256 || __any(top > m[t] + kGrowth)) {
        // Each row by its own need: what it rounds does not hang on its neighbours.
        const bool grows = top > m[t] + kGrowth;
        const float now = grows ? top : m[t], by = __builtin_amdgcn_exp2f(m[t] - now);
        m[t] = now;
        if (grows) largest[t] = score;
        if (D < 256 || __any(grows)) far[t] = __any(is_far(t));
        l[t] *= by;
#pragma unroll
        for (int d = 0; d < kDT; ++d) o[t][d] *= by;
      }
      float minus = m[t];
      // The branch alone costs wide heads 3 % (8192 tokens of 16 heads of 256: 807 -> 835
      // us; as 32 subtractions in every tile 832), many short single tokens 1 % (2048 over
      // 500 956 -> 969), others nothing.
      if (__builtin_expect(far[t], false)) {
        const float from = is_far(t) ? largest[t] : 0.0f;
        if (is_far(t)) minus = 0.0f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[t][kb][e] -= from;
      }
      float sum = 0.0f;  // the tile's, so that long rows add few numbers of unlike size
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          s[t][kb][e] = __builtin_amdgcn_exp2f(fmaf(s[t][kb][e], c, -minus));
          sum += s[t][kb][e];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = bf16_pair_hw(s[t][kb][8 * x + 2 * e], s[t][kb][8 * x + 2 * e + 1]);
          p[t][kb][x] = as_bf16x8(w);
        }
      }
      l[t] += sum;
    }
  }

  static constexpr int kTileLoads = 32 * KB * L::kRow / 1024;  // of 16 bytes a lane

  __device__ __forceinline__ bool any_not_finite(uint32_t values, int lane) const {
    asm volatile("" : "+v"(lane));  // as in hide
    bool is = false;
#pragma unroll
    for (int i = 0; i < kTileLoads; ++i) {
      const u32x4 w = *(SKG_LDS const u32x4*)(values + 1024u * i + 16u * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) is |= F8 ? (((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0 : not_finite(w[e]);
    }
    return __any(is);
  }

  // Zeros for values that are no number, this wave's share.
  static __device__ __forceinline__ void take_out(uint32_t values, int wave, int waves, int lane) {
    for (int i = wave; i < kTileLoads; i += waves) {
      SKG_LDS u32x4* const at = (SKG_LDS u32x4*)(values + 1024u * i + 16u * lane);
      u32x4 w = *at;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F8) {
          const uint32_t top = ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          w[e] &= ~((top >> 7) * 0xFFu);
        } else {
          if ((w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u;
          if ((w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu;
        }
      }
      *at = w;
    }
  }

  // A product of ones: where a value is no number, and where a row sees a key. An
  // output is lost where it is not zero.
  __device__ __forceinline__ void note_lost(uint32_t values, int base, int lane) {
    const int h = lane >> 5;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll 1
      for (int step = 0; step < 2 * KB; ++step) {
        u32x4 sees = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = base + 16 * step + 8 * (e >> 2) + 4 * h + (e & 3);
          if (key >= lo[t] && key < hi[t]) sees[e >> 1] |= (e & 1) ? 0x3F800000u : 0x3F80u;
        }
#pragma unroll
        for (int d = 0; d < kDT; ++d) {
          u32x4 w = __builtin_bit_cast(u32x4, value_operand(read_values(values + value_place(lane), step, d)));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = ((w[e] & 0x7F80u) == 0x7F80u ? 0x3F80u : 0u) | ((w[e] & 0x7F800000u) == 0x7F800000u ? 0x3F800000u : 0u);
          const f32x16 n = mfma32(as_bf16x8(w), as_bf16x8(sees), f32x16{});
#pragma unroll
          for (int e = 0; e < 16; ++e) lost[t][d / 2] |= n[e] > 0.0f ? 1u << (16 * (d & 1) + e) : 0u;
          fence();
        }
      }
  }
  // Makes NaNs of what was noted.
  __device__ __forceinline__ void lose() {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (lost[t][d / 2] >> (16 * (d & 1) + e) & 1) o[t][d][e] = __builtin_nanf("");
  }

  // O += V^T P^T.
  __device__ __forceinline__ void add_values(const bf16x8 (&p)[RT][KB][2], uint32_t values, int lane) {
    constexpr int kGroup = D == 128 ? 4 : 2, kGroups = 2 * KB * kDT / kGroup;
    const uint32_t place = values + value_place(lane);
    bf16x8 v[2][kGroup];
    auto read = [&](int g) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int at = g * kGroup + i;
        v[g & 1][i] = value_operand(read_values(place, at / kDT, at % kDT));
      }
    };
    read(0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) read(g + 1);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int at = g * kGroup + i, step = at / kDT, d = at % kDT;
#pragma unroll
        for (int t = 0; t < RT; ++t) o[t][d] = mfma32(v[g & 1][i], p[t][step / 2][step % 2], o[t][d]);
      }
      fence();
    }
  }
};

// ---- sequences ----

struct Seq {
  int first, n, L;  // its first row of Q, new tokens, tokens up to the last of them
};
// Whatever the arrays hold, rows stay inside Q and keys inside the table.
__device__ __forceinline__ Seq sequence(const AttnParams& p, int b) {
  Seq s;
  s.first = min(max(p.q_start[b], 0), p.T);
  const int all = min(max(p.q_start[b + 1], s.first), p.T) - s.first;
  s.n = min(all, p.max_q);
  s.L = min(max(p.kv_len[b], 0), p.max_len) - (all - s.n);
  return s;
}

__device__ __forceinline__ int wave_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off);
    if (lane >= off) v += o;
  }
  return v;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ Pages pages_of(const AttnParams& p, int b, int kvh) {
  Pages c;
  const size_t head = (size_t)kvh * p.head_stride;
  c.k = p.kc + head;
  c.v = p.vc + head;
  c.ids = reinterpret_cast<const uint8_t*>(p.table) + (size_t)b * p.table_stride;
  c.page_stride = p.page_stride;
  c.slot_stride = p.slot_stride;
  c.n_pages = p.n_pages;
  c.shift = p.page_shift;
  return c;
}

// The outputs of one row's values 32 d .. 32 d + 31 (this lane's half), and lse.
__device__ __forceinline__ void store_values(uint8_t* row, int d, int h, const f32x16& o, float by) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
    *reinterpret_cast<u32x2*>(row + 2 * (32 * d + 8 * a + 4 * h)) =
        u32x2{bf16_pair_hw(o[4 * a] * by, o[4 * a + 1] * by), bf16_pair_hw(o[4 * a + 2] * by, o[4 * a + 3] * by)};
}
__device__ __forceinline__ float over_sum(float v_scale, float l) { return l == 0.0f ? 0.0f : v_scale / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLog2;
}

__device__ __forceinline__ float coherent_load(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void coherent_store(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Counts this workgroup's arrival; true in the last of `all`, which leaves the
// counter at zero. Every thread's stores before it are visible to that one.
__device__ __forceinline__ bool arrive_last(uint32_t* cnt, uint32_t all, uint32_t* shared) {
  wait_vmem_all();
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t a = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (a + 1 == all) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared = a;
  }
  __syncthreads();
  const bool mine = *shared + 1 == all;
  handoff_order();
  return mine;
}

// ---- many rows: a workgroup takes 128 or 256 rows of a key head ----
//
// Four or eight waves of 32 rows share tiles of 64 keys, two buffers: the next
// tile is on its way while one is multiplied. The matrix units bound it, with the
// softmax's vector instructions beside them (about 180, 32 exponentials among them, for 32
// matrix instructions): 8192 tokens of 32 heads of 128 take 540 to 560 us, 1.0 PFLOP/s of visible
// pairs, where a large library product reaches 1.22. Two waves of a SIMD in turns,
// one multiplying while the other has the softmax, with two barriers a tile: 610
// against 567 us; operands read six to nine ahead instead of four: no gain.

constexpr int kRowsKeys = 64;
constexpr int kFewRows = 32;  // of a sequence's key head, at most, for the other form: the columns of its products

// The workspace: the few rows' slots and counters first, then these.
constexpr int kFewCounters = 2 * kChipCUs;
template <int D>
constexpr size_t few_slot() {
  return (size_t)kFewRows * (D + 2) * 4;
}
template <int D>
constexpr size_t few_part() {
  return (size_t)2 * kFewCounters * few_slot<D>();
}

// Waves of the larger form; each has a 64th of a tile's bytes to load at least.
template <int D, bool F8>
constexpr int rows_waves() {
  return D == 256 || (D == 64 && F8) ? 4 : 8;
}
template <int D>
constexpr size_t rows_part(int waves) {  // bytes of a workgroup's results
  return (size_t)64 * waves * 4 * (D / 32 * 16 + 2);
}

template <int D, bool F8, int W>
constexpr int rows_lds() {
  return 4 * kRowsKeys * Cache<D, F8>::kRow + W * 2 * 64 * 4 + 16;
}

// Workgroup `block` of these.
template <int D, bool F8, int W>
__device__ __forceinline__ void rows_body(const AttnParams& p, int block, uint8_t* lds) {
  typedef Cache<D, F8> L;
  constexpr int RT = 1;
  typedef Rows<D, F8, RT, 2> R;
  constexpr int BM = 32 * W, kHalf = kRowsKeys * L::kRow;  // bytes of a tile's keys
  constexpr int kBuffers = 2;                              // of keys, then as many of values
  uint32_t(*const ids)[2][64] = reinterpret_cast<uint32_t(*)[2][64]>(lds + 2 * kBuffers * kHalf);
  uint32_t* const arrived = reinterpret_cast<uint32_t*>(ids + W);
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), h = lane >> 5;

  int rest = block;
  const int kvh = rest % p.Hkv;
  rest /= p.Hkv;
  const int split = rest % p.S, flat = rest / p.S;
  // The sequence and the tile of its rows, from its last ones on, which see most.
  int b = -1, tile = 0, before = 0;
  for (int at = 0; at < p.B; at += 64) {
    int tiles = 0;
    if (at + lane < p.B) {
      const int rows = sequence(p, at + lane).n * p.G;
      tiles = rows <= p.few ? 0 : (rows + BM - 1) / BM;
    }
    const int end = before + wave_scan(tiles, lane);
    const uint64_t past = __ballot(end > flat);
    if (past != 0) {
      const int who = __builtin_ctzll(past);
      b = at + who;
      tile = uniform(__shfl(end, who)) - 1 - flat;
      break;
    }
    before = uniform(__shfl(end, 63));
  }
  b = uniform(b);
  if (b < 0) return;
  const Seq seq = sequence(p, b);
  const int rows = seq.n * p.G, r0 = tile * BM;
  const int tok0 = r0 / p.G, tok1 = min(seq.n - 1, (r0 + BM - 1) / p.G);
  const int place = seq.L - seq.n + 1;  // keys before and at token 0
  const int khi = max(0, place + tok1), see_min = place + tok0;
  const int klo = p.window > 0 ? max(0, place + tok0 - p.window) : 0, lo_max = p.window > 0 ? place + tok1 - p.window : 0;
  // Tiles of keys from klo on, not from a multiple of their size: a page that no row
  // sees may have been given back, so its id is not looked up.
  const int nk = khi > klo ? (khi - klo + kRowsKeys - 1) / kRowsKeys : 0;
  const int j0 = (int)((int64_t)nk * split / p.S), j1 = (int)((int64_t)nk * (split + 1) / p.S);

  R w;
  w.clear();
  int tok[RT], head[RT];
  bool ok[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = r0 + 32 * RT * wave + 32 * t + (lane & 31);
    ok[t] = r < rows;
    const int i = r / p.G;
    tok[t] = seq.first + i;
    head[t] = kvh * p.G + (r - i * p.G);
    w.hi[t] = ok[t] ? place + i : 0;
    w.lo[t] = p.window > 0 ? place + i - p.window : 0;
    w.load_query(t, p.q + (size_t)tok[t] * p.q_stride + (size_t)head[t] * D * 2, ok[t], h);
  }

  const Pages c = pages_of(p, b, kvh);
  const uint32_t k_lds = lds_offset(lds), v_lds = k_lds + kBuffers * kHalf, id_lds = lds_offset(&ids[wave][0][0]);
  bool bad = false;
  const int last = khi - 1;
  Share<D, F8, 64, W> share;

  if (j0 < j1) {
    issue_ids<64>(c, klo + 64 * j0, last, id_lds, lane);
    issue_ids<64>(c, klo + 64 * (j0 + 1), last, id_lds + 256, lane);
    wait_vmem<0>();
    bad = share.find(c, klo + 64 * j0, last, ids[wave][0], wave, lane);
    share.issue_both(c, k_lds, v_lds, wave, lane);
    issue_ids<64>(c, klo + 64 * (j0 + 2), last, id_lds, lane);
  }
  for (int j = j0; j < j1; ++j) {
    const int at = (j - j0) & 1, base = klo + 64 * j;
    wait_vmem<1>();  // this wave's share of tile j; the ids of j + 2 may be under way
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const uint32_t values = v_lds + (uint32_t)at * kHalf;
    f32x16 s[1][2];
    bf16x8 prob[1][2][2];
    w.scores(s, k_lds + (uint32_t)at * kHalf, lane);
    if (j + 1 < j1) {  // behind the product, so that a SIMD's other wave can multiply meanwhile
      const uint32_t next = (uint32_t)(at ^ 1);
      bad |= share.find(c, base + 64, last, ids[wave][next], wave, lane);
      share.issue_both(c, k_lds + next * kHalf, v_lds + next * kHalf, wave, lane);
      issue_ids<64>(c, base + 192, last, id_lds + next * 256, lane);
    }
    if (base + 64 > see_min || base < lo_max) {
      w.hide(s, base, lane);
      w.template clean_values<W>(values, base, wave, lane);
    }
    w.softmax(s, prob, p.c);
    w.add_values(prob, values, lane);
  }
  wait_vmem<0>();
  w.lose();
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    w.l[t] = xred_add<32>(w.l[t]);
    if (bad) w.l[t] = __builtin_nanf("");
  }

  if (p.S > 1) {
    constexpr int kQuads = RT * R::kDT * 4;
    const int group = flat * p.Hkv + kvh;
    const uint32_t one = (uint32_t)rows_part<D>(W);
    uint8_t* const base = p.part + few_part<D>() + (size_t)group * p.S * one;
    const rsrc_t part = make_rsrc(base, (uint32_t)p.S * one);
    const uint32_t mine = (uint32_t)split * one, at = threadIdx.x * 16u;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const f32x16& o = w.o[k / (4 * R::kDT)][k / 4 % R::kDT];
      const int e = 4 * (k % 4);
      st16_coherent_if(true, __builtin_bit_cast(u32x4, f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]}), part, mine + k * 1024u * W + at);
    }
    float* const sums = reinterpret_cast<float*>(base + kQuads * 1024u * W) + threadIdx.x;
    const size_t step = one / 4;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      coherent_store(sums + split * step + 128 * W * t, w.m[t]);
      coherent_store(sums + split * step + 128 * W * t + 64 * W, w.l[t]);
    }
    if (!arrive_last(p.cnt + (size_t)(kFewCounters + group) * kOpsCounterStride, (uint32_t)p.S, arrived)) return;
    float top[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      top[t] = kFloor;
      for (int s = 0; s < p.S; ++s) top[t] = fmaxf(top[t], coherent_load(sums + s * step + 128 * W * t));
    }
    w.clear();
    for (int s = 0; s < p.S; ++s) {
      float by[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        by[t] = __builtin_amdgcn_exp2f(coherent_load(sums + s * step + 128 * W * t) - top[t]);
        w.l[t] += by[t] * coherent_load(sums + s * step + 128 * W * t + 64 * W);
      }
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const f32x4 v = __builtin_bit_cast(f32x4, ld16_coherent_if(true, part, (uint32_t)s * one + k * 1024u * W + at));
        f32x16& o = w.o[k / (4 * R::kDT)][k / 4 % R::kDT];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * (k % 4) + e] = fmaf(v[e], by[k / (4 * R::kDT)], o[4 * (k % 4) + e]);
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) w.m[t] = top[t];
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (!ok[t]) continue;
    uint8_t* const row = p.o + (size_t)tok[t] * p.o_stride + (size_t)head[t] * D * 2;
    const float by = over_sum(p.v_scale, w.l[t]);
#pragma unroll
    for (int d = 0; d < R::kDT; ++d) store_values(row, d, h, w.o[t][d], by);
    if (p.lse != nullptr && h == 0) p.lse[(size_t)tok[t] * p.Hq + head[t]] = lse_of(w.m[t], w.l[t]);
  }
}

// ---- few rows: at most 32 of a key head, the waves split the keys ----
//
// What counts is the cache's stream. Every sequence and key head is cut into units
// of 32 keys a wave, and some more for what a head costs beside its keys; the units
// of the whole call, one sequence after another, are dealt out in equal runs to a
// fixed number of workgroups, whatever the lengths are. A workgroup goes through
// its run head by head; its waves take the unit's keys by 32, each through
// buffers of its own with no barrier, and meet at the head's end. The loads run as many
// tiles ahead of the products as there are buffers, into the next head where one ends. A head that was
// cut between workgroups is joined by the last to arrive, from slots in the
// workspace, in the order of its keys.
//
// Bound by the cache's stream: 64 tokens over 213k cached of 8 key heads of 128, 873
// MB, take 145 us, 6.0 TB/s (a read alone reaches 7.0); below about 30 MB by the chain
// of loads (lengths, page ids, keys) and one joining, 13 us.

// Buffers of keys and of values of a wave: two, or where 160 KB hold only one.
template <int D, bool F8>
constexpr int few_buffers() {
  return D == 256 && !F8 ? 1 : 2;
}
constexpr int kFewWaves = 4;
// What a head costs beside its keys, in units (that batch: 207 us with 1, 153 with 2,
// 145 with 3 and 4), and the units of a workgroup at least (one token over 1000 of 2 key
// heads: 16.4 us with 4, 19.0 with 6, 23.7 with 8; over 257 13.1, 12.8, 13.0).
constexpr uint32_t kHeadUnits = 3;
constexpr uint32_t kFewShare = 4;

// Units of keys of a sequence for each key head, and the first key: the first that a
// row sees, as in rows_body.
__device__ __forceinline__ uint32_t few_units(const AttnParams& p, const Seq& s, int unit, int* first) {
  *first = 0;
  if (s.n == 0 || s.n * p.G > p.few) return 0;
  const int lo = p.window > 0 ? max(0, s.L - s.n + 1 - p.window) : 0;
  *first = lo;
  return s.L > lo ? (uint32_t)(s.L - lo + unit - 1) / (uint32_t)unit : 1;  // a row that sees no key is written too
}
__device__ __forceinline__ uint32_t few_cost(uint32_t units) { return units == 0 ? 0 : units + kHeadUnits; }

// Part of a head that a workgroup does: all lanes hold the same.
struct FewPart {
  int b, kvh;
  uint32_t start, units;  // cost before the head's first unit of keys; its units
  int k0, nu;             // of these, the workgroup's
  int first;              // key of unit 0
  Seq seq;
};

// A workgroup's way through its run.
template <int KUNIT>
struct FewCursor {
  uint32_t u, ue;         // where it is, the run's end
  int chunk = -64;        // 64 sequences that are looked at, one a lane:
  uint32_t end = 0;       // the cost up to each one's end
  uint32_t units = 0;
  int4* seqs;             // LDS: the first 64 sequences and their first keys

  // To the next 64; the cost up to their end.
  __device__ __forceinline__ uint32_t more(const AttnParams& p, int lane, uint32_t before) {
    chunk += 64;
    units = 0;
    if (chunk + lane < p.B) {
      const Seq s = sequence(p, chunk + lane);
      int lo;
      units = few_units(p, s, KUNIT, &lo);
      if (chunk == 0) seqs[lane] = int4{s.first, s.n, s.L, lo};  // every wave writes, and reads back, the same
    }
    end = before + (uint32_t)wave_scan((int)few_cost(units), lane) * (uint32_t)p.Hkv;
    return (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
  }

  // To the next part of a head that has keys to do; false at the run's end.
  __device__ __forceinline__ bool next(const AttnParams& p, int lane, FewPart* part) {
    while (u < ue) {
      const uint64_t past = __ballot(end > u);
      if (past == 0) {
        if (chunk + 64 >= p.B) return false;  // only where the lengths change under the kernel
        more(p, lane, (uint32_t)__builtin_amdgcn_readlane((int)end, 63));
        continue;
      }
      const int who = __builtin_ctzll(past);
      FewPart& x = *part;
      x.units = (uint32_t)__builtin_amdgcn_readlane((int)units, who);
      const uint32_t cost = x.units + kHeadUnits;
      const uint32_t before = (uint32_t)__builtin_amdgcn_readlane((int)end, who) - cost * (uint32_t)p.Hkv;
      x.kvh = (int)((u - before) / cost);
      x.start = before + (uint32_t)x.kvh * cost + kHeadUnits;
      const uint32_t from = max(u, x.start), to = min(ue, x.start + x.units);
      if (from >= to) return false;  // the run ends before the head's first keys
      u = to;
      x.b = chunk + who;
      x.k0 = (int)(from - x.start);
      x.nu = (int)(to - from);
      if (x.b < 64) {
        const int4 s = seqs[x.b];
        x.seq = Seq{uniform(s.x), uniform(s.y), uniform(s.z)};
        x.first = uniform(s.w);
      } else {
        x.seq = sequence(p, x.b);
        few_units(p, x.seq, KUNIT, &x.first);
      }
      return true;
    }
    return false;
  }
};

// Tiles of one wave of a part, and the first one's first key.
template <int KUNIT>
__device__ __forceinline__ int few_tiles(const FewPart& x, int wave, int* key) {
  *key = x.first + x.k0 * KUNIT + 32 * wave;
  return x.seq.L > *key ? min(x.nu, (x.seq.L - *key + KUNIT - 1) / KUNIT) : 0;
}

// What the few rows' workgroups keep in LDS beside their ring of NB buffers.
template <int D, bool F8, int NB>
struct FewLds {
  static constexpr int kRing = 2 * NB * kFewWaves * 32 * Cache<D, F8>::kRow;
  // Where the waves meet, as much as leaves two workgroups to a CU or is left of one.
  static constexpr int kMeet = kRing > 65536 ? 16384 : 8192;
  uint8_t ring[kRing];
  uint8_t meet[kMeet];
  uint32_t ids[kFewWaves][4][64];
  float m[kFewWaves][64], l[kFewWaves][64];
  int4 seqs[64];
  uint32_t arrived;
};

// Workgroup `block` of `blocks`.
template <int D, bool F8, int NB>
__device__ __forceinline__ void few_body(const AttnParams& p, uint32_t block, uint32_t blocks, uint8_t* lds_bytes) {
  typedef Cache<D, F8> L;
  typedef Rows<D, F8, 1, 1> R;
  typedef Share<D, F8, 32, 1> S;
  typedef FewLds<D, F8, NB> M;
  M& mem = *reinterpret_cast<M*>(lds_bytes);
  constexpr int W = kFewWaves;
  constexpr int kTile = 32 * L::kRow, kUnit = 32 * W, kLoads = S::kLoads, kThreads = 64 * W, kMeet = M::kMeet;
  constexpr uint32_t kPairs = kMeet / sizeof(float2);  // maxima and sums of parts that are joined at once
  uint8_t* const meet_lds = mem.meet;
  auto& ids = mem.ids;
  auto& meet_m = mem.m;
  auto& meet_l = mem.l;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), h = lane >> 5, r = lane & 31;

  FewCursor<kUnit> at_head;
  at_head.seqs = mem.seqs;
  uint32_t total = at_head.more(p, lane, 0);
  if (p.B > 64) {
    FewCursor<kUnit> rest = at_head;
    while (rest.chunk + 64 < p.B) total = rest.more(p, lane, total);
  }
  const uint32_t share = max((total + blocks - 1) / blocks, kFewShare);
  at_head.u = min(total, block * share);
  at_head.ue = min(total, at_head.u + share);
  if (at_head.u >= at_head.ue) return;
  FewCursor<kUnit> ahead = at_head;  // where the loads are

  // This wave's ring: NB buffers of keys, as many of values.
  const uint32_t k_lds = lds_offset(mem.ring) + (uint32_t)wave * 2 * NB * kTile, v_lds = k_lds + NB * kTile;
  const uint32_t id_lds = lds_offset(&ids[wave][0][0]);
  S at_keys;     // of the tile that is loaded
  FewPart coming{};
  Pages from{};
  int left = 0, key = 0, slot_of = 0;  // its head's tiles left, its first key, its ids' place
  bool bad_page = false, bad_tile[2] = {false, false};  // of the tile found; of the next two to multiply
  // To the next tile of this wave, if there is one: its ids are there, those of the
  // tile after the next are sent for.
  auto find = [&]() {
    while (left == 0) {
      if (!ahead.next(p, lane, &coming)) return false;
      left = few_tiles<kUnit>(coming, wave, &key);
      if (left == 0) continue;
      from = pages_of(p, coming.b, coming.kvh);
      slot_of = 0;
      issue_ids<32>(from, key, coming.seq.L - 1, id_lds, lane);
      issue_ids<32>(from, key + kUnit, coming.seq.L - 1, id_lds + 256, lane);
      wait_vmem<0>();
    }
    bad_page = at_keys.find(from, key, coming.seq.L - 1, ids[wave][slot_of], 0, lane);
    issue_ids<32>(from, key + 2 * kUnit, coming.seq.L - 1, id_lds + 256 * (uint32_t)((slot_of + 2) & 3), lane);
    slot_of = (slot_of + 1) & 3;
    key += kUnit;
    --left;
    return true;
  };
  R w;
  FewPart now, then;
  // The rows of a part's head, on their way while the waves meet over the last one's.
  auto take_rows = [&](const FewPart& x) {
    const int i = r / p.G, head = x.kvh * p.G + (r - i * p.G), place = x.seq.L - x.seq.n + 1;
    const bool ok = r < x.seq.n * p.G;
    w.hi[0] = ok ? place + i : 0;
    w.lo[0] = p.window > 0 ? place + i - p.window : 0;
    w.load_query(0, p.q + (size_t)(x.seq.first + i) * p.q_stride + (size_t)head * D * 2, ok, h);
  };
  constexpr bool kEarly = D < 256;  // there are no registers for it beside wide heads
  bool any = at_head.next(p, lane, &now);
  if (kEarly && any) take_rows(now);
  int sent = 0;  // tiles on their way or there, not multiplied yet
  uint32_t ring = 0;
  while (sent < NB && find()) {
    at_keys.template issue<false>(from, k_lds + sent * kTile, 0, lane);
    at_keys.template issue<true>(from, v_lds + sent * kTile, 0, lane);
    bad_tile[sent] = bad_page;
    ++sent;
  }
  while (any) {
    if (!kEarly) take_rows(now);
    const Seq seq = now.seq;
    const int rows = seq.n * p.G, place = seq.L - seq.n + 1, kvh = now.kvh;
    const int lo_max = p.window > 0 ? seq.L - p.window : 0;
    int base;
    const int nt = few_tiles<kUnit>(now, wave, &base);
    w.clear();
    bool bad = false;
    // In order of issue: .., K(t) V(t), K(t+1) V(t+1), .. with ids between; loads
    // that come after what is waited for may stay under way.
    for (int j = 0; j < nt; ++j, base += kUnit) {
      const uint32_t at = (ring & (NB - 1)) * kTile;
      bad |= bad_tile[0];
      bad_tile[0] = bad_tile[1];
      if (sent == NB)
        wait_vmem<(2 * NB - 1) * kLoads>();  // K(t)
      else
        wait_vmem<kLoads>();
      f32x16 s[1][1];
      bf16x8 prob[1][1][2];
      w.scores(s, k_lds + at, lane);
      bool more = false;
      if (sent == NB) {
        more = find();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // K(t) is read before K(t+NB) lands there
        if (more) {
          at_keys.template issue<false>(from, k_lds + at, 0, lane);
          bad_tile[NB - 1] = bad_page;
          wait_vmem<(2 * NB - 1) * kLoads>();  // V(t)
        } else {
          wait_vmem<(2 * NB - 2) * kLoads>();
        }
      } else {
        wait_vmem<0>();
      }
      if (base + 32 > place || base < lo_max) {
        w.hide(s, base, lane);
        w.template clean_values<1>(v_lds + at, base, 0, lane);
      }
      w.softmax(s, prob, p.c);
      w.add_values(prob, v_lds + at, lane);
      if (more) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // V(t) is read before V(t+NB) lands there
        at_keys.template issue<true>(from, v_lds + at, 0, lane);
      } else {
        --sent;
      }
      ++ring;
    }
    w.lose();
    const float own_l = xred_add<32>(w.l[0]);
    meet_m[wave][lane] = w.m[0];
    meet_l[wave][lane] = __any(bad) ? __builtin_nanf("") : own_l;
    if constexpr (kEarly) {
      any = at_head.next(p, lane, &then);
      if (any) take_rows(then);
    }

    const bool whole = (uint32_t)now.nu == now.units;
    const uint32_t wg0 = now.start / share, parts = (now.start + now.units - 1) / share - wg0 + 1;
    constexpr size_t kSlot = few_slot<D>();
    auto slot = [&](uint32_t k) { return p.part + (size_t)(2 * (wg0 + k) + (k == 0 ? 1 : 0)) * kSlot; };
    // Four values 4 c4 .. of a row.
    auto put = [&](int row, int c4, f32x4 o, float m, float l) {
      const int i = row / p.G, head = kvh * p.G + (row - i * p.G);
      const float f = over_sum(p.v_scale, l);
      *reinterpret_cast<u32x2*>(p.o + (size_t)(seq.first + i) * p.o_stride + (size_t)head * D * 2 + 8 * c4) =
          u32x2{bf16_pair_hw(o[0] * f, o[1] * f), bf16_pair_hw(o[2] * f, o[3] * f)};
      if (c4 == 0 && p.lse != nullptr) p.lse[(size_t)(seq.first + i) * p.Hq + head] = lse_of(m, l);
    };
    // The waves meet over as many times 16 values of the rows as fit, a power of two;
    // a thread takes four of a row.
    f32x4* const meet = reinterpret_cast<f32x4*>(meet_lds);  // [wave][16 values][quad][half][row]
    int pass_log = 31 - __builtin_clz(kMeet / (W * 64 * rows));
    if (pass_log > 2 + (D == 128) + 2 * (D == 256)) pass_log = 2 + (D == 128) + 2 * (D == 256);
    const int pass = 1 << pass_log;
#pragma unroll
    for (int d = 0; d < 2 * R::kDT; ++d) {
      if (r < rows) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const f32x16& o = w.o[0][d >> 1];
          const int x = 8 * (d & 1) + 4 * e;
          meet[(((wave << pass_log) + (d & (pass - 1))) * 4 + 2 * e + h) * rows + r] = f32x4{o[x], o[x + 1], o[x + 2], o[x + 3]};
        }
      }
      if ((d & (pass - 1)) != pass - 1) continue;
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the tiles on their way are not waited for
      const int d0 = d - (pass - 1);
      for (int v = tid; v < rows * 4 * pass; v += kThreads) {
        const int row = v >> (2 + pass_log), c4 = v & (4 * pass - 1);  // quad 4 d0 + c4 of the row
        float m = meet_m[0][row], l = 0.0f;
#pragma unroll
        for (int x = 1; x < W; ++x) m = fmaxf(m, meet_m[x][row]);
        f32x4 o = {};
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const float by = __builtin_amdgcn_exp2f(meet_m[x][row] - m);
          l += by * meet_l[x][row];
          o += by * meet[((x << pass_log) * 4 + c4) * rows + row];
        }
        if (whole) {
          put(row, 4 * d0 + c4, o, m, l);
        } else {
          uint8_t* const to = slot(block - wg0);
          st16_coherent_if(true, __builtin_bit_cast(u32x4, o), make_rsrc(to, (uint32_t)kSlot),
                           16u * (uint32_t)(row * (D / 4) + 4 * d0 + c4));
          if (d0 == 0 && c4 == 0) {
            float* const ml = reinterpret_cast<float*>(to) + rows * D + 2 * row;
            coherent_store(ml, m);
            coherent_store(ml + 1, l);
          }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    if (!whole && arrive_last(p.cnt + (size_t)wg0 * kOpsCounterStride, parts, &mem.arrived)) {
      // Maxima and sums of `some` parts at once through LDS; values as they come.
      float2* const join_ml = reinterpret_cast<float2*>(meet_lds);
      const uint32_t some = kPairs / (uint32_t)rows;
      const int quads = rows * (D / 4);
      for (int v0 = 0; v0 < quads; v0 += kThreads) {
        const int v = v0 + tid, row = min(v, quads - 1) / (D / 4), c4 = v % (D / 4);
        float m = kFloor, l = 0.0f;
        f32x4 o = {};
        for (uint32_t k0 = 0; k0 < parts; k0 += some) {
          const uint32_t here = min(some, parts - k0);
          if (v0 == 0 || parts > some) {
            __syncthreads();
            for (uint32_t x = (uint32_t)tid; x < here * (uint32_t)rows; x += kThreads) {
              const float* const ml = reinterpret_cast<const float*>(slot(k0 + x / (uint32_t)rows)) + rows * D + 2 * (x % (uint32_t)rows);
              join_ml[x] = float2{coherent_load(ml), coherent_load(ml + 1)};
            }
            __syncthreads();
          }
          float top = m;
          for (uint32_t k = 0; k < here; ++k) top = fmaxf(top, join_ml[k * rows + row].x);
          const float by = __builtin_amdgcn_exp2f(m - top);
          m = top;
          l *= by;
          o *= by;
          if (v < quads) {
#pragma unroll 8
            for (uint32_t k = 0; k < here; ++k) {
              const f32x4 x = __builtin_bit_cast(f32x4, ld16_coherent_if(true, make_rsrc(slot(k0 + k), (uint32_t)kSlot), 16u * (uint32_t)v));
              const float2 ml = join_ml[k * rows + row];
              const float f = __builtin_amdgcn_exp2f(ml.x - m);
              l = fmaf(f, ml.y, l);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = fmaf(f, x[e], o[e]);
            }
          }
        }
        if (v < quads) put(row, c4, o, m, l);
      }
      __syncthreads();
    }
    if constexpr (kEarly)
      now = then;
    else
      any = at_head.next(p, lane, &now);
  }
}

template <int D, bool F8, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attn_rows_kernel(AttnParams p) {
  __shared__ __align__(1024) uint8_t lds[rows_lds<D, F8, W>()];
  rows_body<D, F8, W>(p, (int)blockIdx.x, lds);
}

template <int D, bool F8>
__global__ __launch_bounds__(64 * kFewWaves, D == 256 ? 1 : 2) void attn_few_kernel(AttnParams p) {
  constexpr int NB = few_buffers<D, F8>();
  __shared__ __align__(1024) uint8_t lds[sizeof(FewLds<D, F8, NB>)];
  few_body<D, F8, NB>(p, blockIdx.x, gridDim.x, lds);
}

// Both at once, for batches that may hold sequences of either kind: the first
// few_blocks workgroups take those of few rows. The short work of one kind hides
// under the other's: a mixed batch of 37 takes 32.5 us against 41.5 with two launches, 16
// prompts of up to 500 tokens 27 against 37, 4 x 2048 of 16 heads 106 against 106. Heads of 128
// have one buffer less than on their own, so that two workgroups fit a CU.
template <int D, bool F8>
constexpr int mixed_buffers() {
  return D == 256 ? few_buffers<D, F8>() : D == 128 && !F8 ? 1 : 2;
}
template <int D, bool F8>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_mixed_kernel(AttnParams p, int few_blocks) {
  constexpr int NB = mixed_buffers<D, F8>();
  constexpr int kRows = rows_lds<D, F8, 4>(), kFew = (int)sizeof(FewLds<D, F8, NB>);
  __shared__ __align__(1024) uint8_t lds[kRows > kFew ? kRows : kFew];
  if ((int)blockIdx.x < few_blocks)
    few_body<D, F8, NB>(p, blockIdx.x, (uint32_t)few_blocks, lds);
  else
    rows_body<D, F8, 4>(p, (int)blockIdx.x - few_blocks, lds);
}

// Tiles of BM rows at most: the rows kernel has a workgroup for each, and those past
// what the lengths give end at once.
int64_t most_tiles(int T, int B, int max_q, int G, int BM) {
  const int64_t by_rows = (int64_t)T * G / BM + B;
  const int64_t by_seq = (int64_t)B * (((int64_t)max_q * G + BM - 1) / BM);
  return by_rows < by_seq ? by_rows : by_seq;
}
int64_t tiles_bound(const AttnParams& p, int waves) { return most_tiles(p.T, p.B, p.max_q, p.G, 32 * waves); }

// Workgroups that split the keys of each tile where the tiles alone leave CUs idle:
// rounds of one workgroup a CU, S that leaves the fewest idle, the smallest of equal
// ones; not below 512 keys a workgroup. A kernel of less waves takes the same S as one
// of `most_waves`, which fills the chip with one workgroup a CU.
template <int D>
int rows_splits(const AttnParams& p, int waves, int most_waves) {
  const int64_t slots = tiles_bound(p, waves) * p.Hkv, groups = tiles_bound(p, most_waves) * p.Hkv;
  if (groups <= 0 || slots > kOpsCounters - kFewCounters) return 1;
  const int64_t keys = p.window > 0 && p.window + 32 * waves < p.max_len ? p.window + 32 * waves : p.max_len;
  int64_t most = (keys + kRowsKeys - 1) / kRowsKeys / 8;
  const int64_t room = (int64_t)((kOpsPartBytes - few_part<D>()) / rows_part<D>(waves)) / slots;
  if (most > room) most = room;
  int best = 1;
  auto rounds = [&](int64_t s) { return (groups * s + kChipCUs - 1) / kChipCUs; };
  for (int s = 2; s <= most && s <= 64; ++s)
    if (rounds(s) * best < rounds(best) * s) best = s;
  return best;
}

// Workgroups of the few kernel: as many as the chip holds at once.
template <int D, bool F8>
constexpr int few_grid() {
  return D * (F8 ? 1 : 2) >= 256 ? kChipCUs : 2 * kChipCUs;
}

template <int D, bool F8>
hipError_t launch_format(AttnParams p, hipStream_t s) {
  static_assert(few_grid<D, F8>() <= kFewCounters && few_part<D>() < kOpsPartBytes && kFewCounters < kOpsCounters, "slots fit");
  // A batch may hold sequences of both kinds; a single sequence goes by its bound.
  const bool many = (int64_t)p.max_q * p.G > kFewRows, few = !many || p.B > 1;
  p.few = few ? kFewRows : 0;
  constexpr int kUnit = 32 * kFewWaves;
  const int64_t units = (int64_t)p.B * p.Hkv * (p.max_len / kUnit + 2);
  const unsigned few_blocks = !few ? 0 : (unsigned)(units < few_grid<D, F8>() ? units : few_grid<D, F8>());
  if (many) {
    // Eight waves of a workgroup share a tile's keys, which halves what comes from the
    // L2; two workgroups of four fill a CU as well, go at their own pace and waste
    // less on short work and at the end. A single sequence takes eight where its
    // keys are split (512 over 32768 cached: 279 us against 300 with four), or where they
    // are many and its tiles last more than three rounds of the CUs. Eight / four waves (a
    // pair is of one run) by rounds, 32 heads: 6000 tokens 2.9 329 / 319, 7000 3.4 421 / 428, 8192 4 551 / 568,
    // 16384 8 2092 / 2189 (just 2 rounds, 4096, would take 154 / 168); by keys, at more than
    // three rounds: 2048 193 / 191 and 385 / 375, 2500 285 / 277, 3500 260 / 264, 4096 340 / 345,
    // 6000 695 / 715. Heads of 64 360 / 342, a window of 1024 199 / 183.
    // A batch stays with four, beside the few kernel; eight would be a launch before it: 16 x 512 tokens of
    // 64 heads 170 / 153, 64 of up to 300 over up to 1300 139 / 111, 24 of up to 2000 368 / 348,
    // but 4 x 4096 605 / 620, 16 x 512 over 4000 1027 / 1074; with keys split 12 of up to 64 over
    // up to 8000 88 / 42, 4 of up to 500 over 30000 405 / 335, but 8 x 64 over 16384 173 / 183,
    // 2 of up to 1000 over 60000 333 / 360.
    constexpr int kMost = rows_waves<D, F8>();
    const bool long_rounds = D == 128 && p.window == 0 && p.max_len >= 3000 && tiles_bound(p, 8) * p.Hkv > 3 * kChipCUs;
    p.S = rows_splits<D>(p, few ? 4 : kMost, kMost);  // for the waves that are launched, or 1
    const bool eight = kMost == 8 && !few && (long_rounds || p.S > 1);
    const unsigned grid = (unsigned)(tiles_bound(p, eight ? 8 : 4) * p.Hkv * p.S);
    if (few) return launch(attn_mixed_kernel<D, F8>, dim3(few_blocks + grid), dim3(256), 0, s, p, (int)few_blocks);
    if constexpr (kMost == 8) {
      if (eight) return launch(attn_rows_kernel<D, F8, 8>, dim3(grid), dim3(512), 0, s, p);
    }
    return launch(attn_rows_kernel<D, F8, 4>, dim3(grid), dim3(256), 0, s, p);
  }
  return launch(attn_few_kernel<D, F8>, dim3(few_blocks), dim3(64 * kFewWaves), 0, s, p);
}

}  // namespace

int64_t attention_tiles(int T, int B, int max_q, int G) {
  return (int64_t)max_q * G > kFewRows ? most_tiles(T, B, max_q, G, 128) : 0;
}

hipError_t launch_attention(const AttnParams& p, int D, bool codes, hipStream_t s) {
  switch (D) {
    case 64: return codes ? launch_format<64, true>(p, s) : launch_format<64, false>(p, s);
    case 128: return codes ? launch_format<128, true>(p, s) : launch_format<128, false>(p, s);
    default: return codes ? launch_format<256, true>(p, s) : launch_format<256, false>(p, s);
  }
}

}  // namespace skg
