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
// (P stays below 2^8, bf16 has the same relative step there). P is rounded to bf16
// for the second product, 2^-9 of each probability; l sums the unrounded ones.
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

constexpr float kFloor = -1e30f;   // maximum of a row that has seen no key
constexpr float kGrowth = 8.0f;    // powers of two that P may reach
constexpr float kLog2 = 0.69314718055994531f;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16 (4) bytes a lane from each lane's address into LDS at `lds` + 16 (4) l; see
// ld16_to_lds for why in asm and who waits.
__device__ __forceinline__ void global16_to_lds(const uint8_t* p, uint32_t lds) {
#ifdef __HIP_DEVICE_COMPILE__
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
  // same chunk of 8 neighbouring rows at once.
  __device__ static __forceinline__ int key_swizzle(int row) {
    return kRow >= 128 ? row & 7 : (row >> 1) & 3;
  }
  // Values are read by 4 rows x 32 bytes (bf16), or rows 0..3 and 8..11 of 16 x 16
  // bytes (E4M3).
  __device__ static __forceinline__ int value_swizzle(int row) {
    if constexpr (!F8) return (row & 3) << 1;
    return kRow >= 128 ? (row & 3) | ((row >> 1) & 4) : ((row >> 1) & 1) | ((row >> 2) & 2);
  }
};

// One key head's pages and a sequence's table.
struct Pages {
  const uint8_t *k, *v, *ids;
  size_t page_stride;
  uint32_t slot_stride;
  int n_pages, shift;
};

// The ids of the pages of keys base .. base + KEYS - 1 (none past `last`) on
// their way into 64 words of LDS.
template <int KEYS>
__device__ __forceinline__ void issue_ids(const Pages& c, int base, int last, uint32_t lds, int lane) {
  const int key = min(base + lane % KEYS, last);
  global4_to_lds(c.ids + 4 * (size_t)(uint32_t)(key >> c.shift), lds);
}

// Keys base .. base + KEYS - 1 and their values on their way into LDS, this wave's
// share of WAVES. Past `last` that key is taken again. A page that does not exist
// is not read (page 0 is) and reported.
template <int D, bool F8, int KEYS, int WAVES>
__device__ __forceinline__ bool issue_tile(const Pages& c, int base, int last, const uint32_t* ids, uint32_t lds, int wave, int lane) {
  typedef Cache<D, F8> L;
  constexpr int kLoads = KEYS / L::kRows / WAVES;
  static_assert(kLoads >= 1, "every wave has a share");
  // The offsets below are the same for every tile; kept from one to the next they
  // would take more registers than there are (D = 256: spills).
  asm volatile("" : "+v"(lane));
  bool bad = false;
#pragma unroll
  for (int q = 0; q < kLoads; ++q) {
    const int row = (wave * kLoads + q) * L::kRows + lane / L::kChunks, at = lane % L::kChunks;
    const int key = min(base + row, last);
    uint32_t id = ids[row];
    if (id >= (uint32_t)c.n_pages) {
      id = 0;
      bad = true;
    }
    const size_t off = (size_t)id * c.page_stride + (size_t)((uint32_t)(key & ((1 << c.shift) - 1)) * c.slot_stride);
    const uint32_t to = lds + (uint32_t)(wave * kLoads + q) * 1024u;
    global16_to_lds(c.k + off + 16 * (at ^ L::key_swizzle(row)), to);
    global16_to_lds(c.v + off + 16 * (at ^ L::value_swizzle(row)), to + KEYS * L::kRow);
  }
  return bad;
}

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
  int lo[RT], hi[RT];  // keys that this lane's row sees
  uint32_t lost[RT][kDT / 2];  // bit 16 (d % 2) + e: element e of o[t][d] is NaN

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kFloor;
      l[t] = 0.0f;
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

  // The steps of a product go in groups of four operands: a group is read from LDS
  // while the one before is multiplied, and no further ahead (the compiler would
  // read everything at once and spill).
  static __device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

  __device__ __forceinline__ void scores(f32x16 (&s)[RT][KB], const uint8_t* keys, int lane) const {
    constexpr int kSteps = D / (F8 ? 32 : 16), kGroup = F8 ? 2 : 4, kGroups = KB * kSteps / kGroup;
    const int r = lane & 31, h = lane >> 5, swz = L::key_swizzle(r);
    u32x4 w[2][kGroup];
    auto read = [&](int g) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int kb = (g * kGroup + i) / kSteps, k = (g * kGroup + i) % kSteps;
        w[g & 1][i] = *reinterpret_cast<const u32x4*>(keys + (32 * kb + r) * L::kRow + 16 * ((2 * k + h) ^ swz));
      }
    };
    read(0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (g + 1 < kGroups) read(g + 1);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int kb = (g * kGroup + i) / kSteps, k = (g * kGroup + i) % kSteps;
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

  // Values 32 d .. 32 d + 31 of the 16 keys from `key`, as the product takes them.
  __device__ __forceinline__ bf16x8 value_operand(uint32_t values, int key, int d, int lane) const {
    const int i = lane & 15, side = (lane >> 4) & 1, h = lane >> 5;
    if constexpr (F8) {
      const int row = key + 4 * h + ((i >> 1) & 3) + 8 * (i >> 3);
      const uint32_t at = values + row * L::kRow + 16 * ((2 * d + side) ^ L::value_swizzle(row)) + 8 * (i & 1);
      const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((SKG_LDS i32x2*)at);
      return fp8x8_bf16((uint32_t)w[0], (uint32_t)w[1], 1.0f);
    } else {
      const int row = key + 4 * h + (i >> 2);
      const uint32_t at = values + row * L::kRow + 16 * ((4 * d + 2 * side + ((i >> 1) & 1)) ^ L::value_swizzle(row)) + 8 * (i & 1);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SKG_LDS s16x4*)at);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SKG_LDS s16x4*)(at + 8 * L::kRow));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }

  // A tile of 32 KB keys from `base`. mask: some row does not see all of them. What
  // it does not see has score -inf and probability 0; a value that is no number
  // would still make a NaN of that 0. Such values are taken out of the tile, and the
  // outputs of rows that do see one are noted in `lost`. SHARE waves share the tile.
  template <int SHARE>
  __device__ __forceinline__ void tile(const uint8_t* keys, uint32_t values, int base, bool mask, float c, int wave, int lane) {
    const int h = lane >> 5;
    f32x16 s[RT][KB];
    scores(s, keys, lane);
    if (mask) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int key = base + 32 * kb + 8 * (e >> 2) + 4 * h + (e & 3);
            s[t][kb][e] = key >= lo[t] && key < hi[t] ? s[t][kb][e] : -__builtin_inff();
          }
      if (any_not_finite(values, lane)) {  // the same in all waves that share the tile
        note_lost(values, base, lane);
        if constexpr (SHARE > 1) __syncthreads();
        take_out(values, wave, SHARE, lane);
        if constexpr (SHARE > 1) __syncthreads();
      }
    }
    bf16x8 p[RT][KB][2];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float top = -__builtin_inff();
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][kb][e]);
      top = swap_max(top) * c;
      if (D == 256 || __any(top > m[t] + kGrowth)) {
        // Each row by its own need: what it rounds does not hang on its neighbours.
        const float now = top > m[t] + kGrowth ? top : m[t], by = __builtin_amdgcn_exp2f(m[t] - now);
        m[t] = now;
        l[t] *= by;
#pragma unroll
        for (int d = 0; d < kDT; ++d) o[t][d] *= by;
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          s[t][kb][e] = __builtin_amdgcn_exp2f(fmaf(s[t][kb][e], c, -m[t]));
          l[t] += s[t][kb][e];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = bf16_pair_hw(s[t][kb][8 * x + 2 * e], s[t][kb][8 * x + 2 * e + 1]);
          p[t][kb][x] = as_bf16x8(w);
        }
      }
    }
    add_values(p, values, lane);
  }

  static constexpr int kTileLoads = 32 * KB * L::kRow / 1024;  // of 16 bytes a lane

  __device__ __forceinline__ bool any_not_finite(uint32_t values, int lane) const {
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
          u32x4 w = __builtin_bit_cast(u32x4, value_operand(values, 16 * step, d, lane));
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
    constexpr int kGroup = kDT < 4 ? kDT : 4, kGroups = 2 * KB * kDT / kGroup;
    bf16x8 v[2][kGroup];
    auto read = [&](int g) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int at = g * kGroup + i;
        v[g & 1][i] = value_operand(values, 16 * (at / kDT), at % kDT, lane);
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
  int first, n, L;  // its first row of Q, new tokens, tokens in all
};
// Whatever the arrays hold, rows stay inside Q and keys inside the table.
__device__ __forceinline__ Seq sequence(const AttnParams& p, int b) {
  Seq s;
  s.first = min(max(p.q_start[b], 0), p.T);
  s.n = min(min(max(p.q_start[b + 1], s.first), p.T) - s.first, p.max_q);
  s.L = min(max(p.kv_len[b], 0), p.max_len);
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

// ---- many rows: a workgroup takes 256 rows of a key head (128 of wide heads) ----
//
// Waves of 32 rows share tiles of 64 keys, two buffers: the next tile is
// on its way while one is multiplied.

constexpr int kRowsKeys = 64;

template <int D, bool F8>
constexpr int rows_waves() {
  return D == 256 || (D == 64 && F8) ? 4 : 8;
}
template <int D, bool F8>
constexpr size_t rows_part() {  // bytes of a workgroup's results
  return (size_t)64 * rows_waves<D, F8>() * 4 * (D / 32 * 16 + 2);
}

template <int D, bool F8, int W>
__global__ __launch_bounds__(64 * W, W / 4) void attn_rows_kernel(AttnParams p) {
  typedef Cache<D, F8> L;
  constexpr int RT = 1;
  typedef Rows<D, F8, RT, 2> R;
  constexpr int BM = 32 * W, kStage = 2 * kRowsKeys * L::kRow;
  __shared__ __align__(1024) uint8_t lds[2 * kStage];
  __shared__ __align__(256) uint32_t ids[W][2][64];
  __shared__ uint32_t arrived;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), h = lane >> 5;

  int rest = (int)blockIdx.x;
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
  const int kal = klo & ~(kRowsKeys - 1);
  const int nk = khi > kal ? (khi - kal + kRowsKeys - 1) / kRowsKeys : 0;
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
  const uint32_t data = lds_offset(lds), id_lds = lds_offset(&ids[wave][0][0]);
  bool bad = false;
  const int last = khi - 1;
  if (j0 < j1) {
    issue_ids<64>(c, kal + 64 * j0, last, id_lds, lane);
    issue_ids<64>(c, kal + 64 * (j0 + 1), last, id_lds + 256, lane);
    wait_vmem<0>();
    bad = issue_tile<D, F8, 64, W>(c, kal + 64 * j0, last, ids[wave][0], data, wave, lane);
    issue_ids<64>(c, kal + 64 * (j0 + 2), last, id_lds, lane);
  }
  for (int j = j0; j < j1; ++j) {
    const int at = (j - j0) & 1, base = kal + 64 * j;
    wait_vmem<1>();  // this wave's share of tile j; the ids of j + 2 may be under way
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (j + 1 < j1) {
      bad |= issue_tile<D, F8, 64, W>(c, base + 64, last, ids[wave][at ^ 1], data + (uint32_t)(at ^ 1) * kStage, wave, lane);
      issue_ids<64>(c, base + 192, last, id_lds + (uint32_t)(at ^ 1) * 256, lane);
    }
    const uint8_t* const keys = lds + at * kStage;
    const uint32_t values = data + (uint32_t)at * kStage + kRowsKeys * L::kRow;
    w.template tile<W>(keys, values, base, base + 64 > see_min || base < lo_max, p.c, wave, lane);
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
    const uint32_t one = (uint32_t)rows_part<D, F8>();
    uint8_t* const base = p.part + (size_t)group * p.S * one;
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
    if (!arrive_last(p.cnt + (size_t)group * kOpsCounterStride, (uint32_t)p.S, &arrived)) return;
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
// of 32 keys a wave; the units of the whole call, one sequence after another, are
// dealt out in equal runs to a fixed number of workgroups, whatever the lengths
// are. A workgroup goes through its run head by head; its waves take the unit's
// keys by 32, each through two buffers of its own with no barrier, and meet at the
// head's end. A head that was cut between workgroups is joined by the last to
// arrive, from slots in the workspace, in the order of its keys.

constexpr int kFewRows = 32;

template <int D, bool F8>
constexpr int few_waves() {
  return D == 256 && !F8 ? 2 : 4;
}
template <int D>
constexpr size_t few_slot() {
  return (size_t)kFewRows * (D + 2) * 4;
}

// Units of a sequence for each key head, and the first key.
__device__ __forceinline__ int few_units(const AttnParams& p, const Seq& s, int unit, int* first) {
  if (s.n == 0 || s.n * p.G > p.few) return 0;
  const int lo = p.window > 0 ? max(0, s.L - s.n + 1 - p.window) & ~31 : 0;
  *first = lo;
  return s.L > lo ? (s.L - lo + unit - 1) / unit : 1;  // a row that sees no key is written too
}

template <int D, bool F8, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void attn_few_kernel(AttnParams p) {
  typedef Cache<D, F8> L;
  typedef Rows<D, F8, 1, 1> R;
  constexpr int kStage = 2 * 32 * L::kRow, kUnit = 32 * W, kLoads = 2 * 32 / L::kRows;
  constexpr int kRing = 2 * W * kStage, kMeet = W * D * 128;  // the waves' values at a head's end
  __shared__ __align__(1024) uint8_t lds[kRing > kMeet ? kRing : kMeet];
  __shared__ __align__(256) uint32_t ids[W][2][64];
  __shared__ float meet_m[W][64], meet_l[W][64];
  __shared__ uint32_t arrived;
  const int lane = (int)threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), h = lane >> 5, r = lane & 31;

  uint32_t total = 0;
  for (int at = 0; at < p.B; at += 64) {
    int units = 0, lo;
    if (at + lane < p.B) units = few_units(p, sequence(p, at + lane), kUnit, &lo);
    total += (uint32_t)uniform(__shfl(wave_scan(units, lane), 63));
  }
  total *= (uint32_t)p.Hkv;
  const uint32_t share = (total + gridDim.x - 1) / gridDim.x;
  uint32_t u = blockIdx.x * share;
  const uint32_t ue = min(total, u + share);
  uint32_t chunk_first = 0, chunk = 0;  // units before the 64 sequences that are looked at
  const uint32_t data = lds_offset(lds) + (uint32_t)wave * 2 * kStage, id_lds = lds_offset(&ids[wave][0][0]);
  const uint8_t* const my_lds = lds + wave * 2 * kStage;

  while (u < ue) {
    // The sequence, key head and unit of u.
    int b = -1;
    uint32_t start = 0, units = 0;
    for (;;) {
      int mine = 0, lo;
      if ((int)chunk + lane < p.B) mine = few_units(p, sequence(p, (int)chunk + lane), kUnit, &lo);
      const uint32_t end = chunk_first + (uint32_t)wave_scan(mine, lane) * (uint32_t)p.Hkv;
      const uint64_t past = __ballot(end > u);
      if (past != 0) {
        const int who = __builtin_ctzll(past);
        b = (int)chunk + who;
        units = (uint32_t)uniform(__shfl(mine, who));
        start = (uint32_t)uniform(__shfl((int)end, who)) - units * (uint32_t)p.Hkv;
        break;
      }
      chunk_first = (uint32_t)uniform(__shfl((int)end, 63));
      chunk += 64;
    }
    b = uniform(b);
    const int kvh = (int)((u - start) / units);
    start += (uint32_t)kvh * units;
    const int k0 = (int)(u - start), nu = (int)min(units - (uint32_t)k0, ue - u);
    const Seq seq = sequence(p, b);
    int kal;
    few_units(p, seq, kUnit, &kal);
    const int rows = seq.n * p.G, place = seq.L - seq.n + 1, khi = seq.L;
    const int lo_max = p.window > 0 ? seq.L - p.window : 0;

    R w;
    w.clear();
    const bool ok = r < rows;
    const int i = r / p.G, tok = seq.first + i, head = kvh * p.G + (r - i * p.G);
    w.hi[0] = ok ? place + i : 0;
    w.lo[0] = p.window > 0 ? place + i - p.window : 0;
    w.load_query(0, p.q + (size_t)tok * p.q_stride + (size_t)head * D * 2, ok, h);

    const Pages c = pages_of(p, b, kvh);
    const int first = kal + k0 * kUnit + 32 * wave, last = khi - 1;
    const int nt = khi > first ? min(nu, (khi - first + kUnit - 1) / kUnit) : 0;
    bool bad = false;
    if (nt > 0) {
      issue_ids<32>(c, first, last, id_lds, lane);
      issue_ids<32>(c, first + kUnit, last, id_lds + 256, lane);
      wait_vmem<0>();
      bad = issue_tile<D, F8, 32, 1>(c, first, last, ids[wave][0], data, 0, lane);
      issue_ids<32>(c, first + 2 * kUnit, last, id_lds, lane);
    }
    for (int j = 0; j < nt; ++j) {
      const int at = j & 1, base = first + j * kUnit;
      if (j + 1 < nt) {
        wait_vmem<kLoads + 1>();  // the ids of j + 1; after them came tile j and the ids of j + 2
        bad |= issue_tile<D, F8, 32, 1>(c, base + kUnit, last, ids[wave][at ^ 1], data + (uint32_t)(at ^ 1) * kStage, 0, lane);
        issue_ids<32>(c, base + 3 * kUnit, last, id_lds + (uint32_t)(at ^ 1) * 256, lane);
        wait_vmem<kLoads + 2>();  // tile j
      } else {
        wait_vmem<0>();
      }
      const uint8_t* const keys = my_lds + at * kStage;
      const uint32_t values = data + (uint32_t)at * kStage + 32 * L::kRow;
      w.template tile<1>(keys, values, base, base + 32 > place || base < lo_max, p.c, 0, lane);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before tile j + 2 lands there
    }
    w.lose();
    bad = __syncthreads_or(bad);  // and no wave reads its ring any more
    float l = xred_add<32>(w.l[0]);
    if (bad) l = __builtin_nanf("");
    meet_m[wave][lane] = w.m[0];
    meet_l[wave][lane] = l;
    f32x4* const meet = reinterpret_cast<f32x4*>(lds);  // [wave][32 values][quad of elements][lane]
#pragma unroll
    for (int d = 0; d < R::kDT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        meet[((wave * R::kDT + d) * 4 + e) * 64 + lane] =
            f32x4{w.o[0][d][4 * e], w.o[0][d][4 * e + 1], w.o[0][d][4 * e + 2], w.o[0][d][4 * e + 3]};
    __syncthreads();
    float m = meet_m[0][lane], by[W];
#pragma unroll
    for (int v = 1; v < W; ++v) m = fmaxf(m, meet_m[v][lane]);
    l = 0.0f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      by[v] = __builtin_amdgcn_exp2f(meet_m[v][lane] - m);
      l += by[v] * meet_l[v][lane];
    }
    // Wave v goes on with values 32 v .. and those 32 W further.
    const bool whole = (uint32_t)nu == units;
    constexpr size_t kSlot = few_slot<D>() / 4;
    const uint32_t wg0 = start / share, parts = (start + units - 1) / share - wg0 + 1;
    auto slot = [&](uint32_t k) {
      return reinterpret_cast<float*>(p.part) + (size_t)(2 * (wg0 + k) + (k == 0 ? 1 : 0)) * kSlot;
    };
    float* const to = slot(blockIdx.x - wg0);
    uint8_t* const row = p.o + (size_t)tok * p.o_stride + (size_t)head * D * 2;
    const int at = h * rows + r;  // in a slot: rows are packed
    for (int d = wave; d < R::kDT; d += W) {
      f32x16 o = {};
#pragma unroll
      for (int v = 0; v < W; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x4 q = meet[((v * R::kDT + d) * 4 + e) * 64 + lane];
#pragma unroll
          for (int f = 0; f < 4; ++f) o[4 * e + f] = fmaf(q[f], by[v], o[4 * e + f]);
        }
      if (!ok) continue;
      if (whole) {
        store_values(row, d, h, o, over_sum(p.v_scale, l));
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) coherent_store(to + (d * 16 + e) * 2 * rows + at, o[e]);
      }
    }
    bool write = whole;
    if (!whole) {
      if (ok && wave == 0) coherent_store(to + D * rows + at, h == 0 ? m : l);
      write = arrive_last(p.cnt + (size_t)wg0 * kOpsCounterStride, parts, &arrived);
      if (write && ok) {
        m = kFloor;
        for (uint32_t k = 0; k < parts; ++k) m = fmaxf(m, coherent_load(slot(k) + D * rows + r));
        l = 0.0f;
        for (uint32_t k = 0; k < parts; ++k)
          l += __builtin_amdgcn_exp2f(coherent_load(slot(k) + D * rows + r) - m) * coherent_load(slot(k) + D * rows + rows + r);
        for (int d = wave; d < R::kDT; d += W) {
          f32x16 o = {};
          for (uint32_t k = 0; k < parts; ++k) {
            const float* const from = slot(k);
            const float f = __builtin_amdgcn_exp2f(coherent_load(from + D * rows + r) - m);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(coherent_load(from + (d * 16 + e) * 2 * rows + at), f, o[e]);
          }
          store_values(row, d, h, o, over_sum(p.v_scale, l));
        }
      }
    }
    if (write && ok && p.lse != nullptr && h == 0 && wave == 0) p.lse[(size_t)tok * p.Hq + head] = lse_of(m, l);
    u += (uint32_t)nu;
    if (u < ue) __syncthreads();  // the meeting's LDS is the ring again
  }
}

// Tiles of the rows kernel at most: it has a workgroup for each, and those past
// what the lengths give end at once.
template <int D, bool F8>
int64_t tiles_bound(const AttnParams& p) {
  const int64_t BM = 32 * rows_waves<D, F8>();
  const int64_t by_rows = (int64_t)p.T * p.G / BM + p.B;
  const int64_t by_seq = (int64_t)p.B * (((int64_t)p.max_q * p.G + BM - 1) / BM);
  return by_rows < by_seq ? by_rows : by_seq;
}

// Workgroups that split the keys of each tile where the tiles alone leave CUs idle.
template <int D, bool F8>
int rows_splits(const AttnParams& p) {
  const int64_t groups = tiles_bound<D, F8>(p) * p.Hkv;
  if (groups <= 0 || groups > kOpsCounters) return 1;
  int64_t s = 2 * kChipCUs / groups;
  const int64_t tiles = (p.max_len + kRowsKeys - 1) / kRowsKeys;
  if (s > tiles / 4) s = tiles / 4;  // not below 256 keys each
  const int64_t room = (int64_t)(kOpsPartBytes / rows_part<D, F8>()) / groups;
  if (s > room) s = room;
  return s < 1 ? 1 : s > 64 ? 64 : (int)s;
}

// Workgroups of the few kernel: as many as the chip holds at once.
template <int D, bool F8>
constexpr int few_grid() {
  return D * (F8 ? 1 : 2) >= 256 ? kChipCUs : 2 * kChipCUs;
}

template <int D, bool F8>
hipError_t launch_format(AttnParams p, hipStream_t s) {
  static_assert((size_t)2 * few_grid<D, F8>() * few_slot<D>() <= kOpsPartBytes && few_grid<D, F8>() <= kOpsCounters, "slots fit");
  // A batch may hold sequences of both kinds; a single sequence goes by its bound.
  const bool many = (int64_t)p.max_q * p.G > kFewRows, few = !many || p.B > 1;
  p.few = few ? kFewRows : 0;
  if (many) {
    p.S = rows_splits<D, F8>(p);
    const int64_t grid = tiles_bound<D, F8>(p) * p.Hkv * p.S;
    const hipError_t e = launch(attn_rows_kernel<D, F8, rows_waves<D, F8>()>, dim3((unsigned)grid), dim3(64 * rows_waves<D, F8>()), 0, s, p);
    if (e != hipSuccess || !few) return e;
  }
  constexpr int W = few_waves<D, F8>(), kUnit = 32 * W;
  const int64_t units = (int64_t)p.B * p.Hkv * (p.max_len / kUnit + 1);
  const unsigned grid = (unsigned)(units < few_grid<D, F8>() ? units : few_grid<D, F8>());
  return launch(attn_few_kernel<D, F8, W>, dim3(grid), dim3(64 * W), 0, s, p);
}

}  // namespace

hipError_t launch_attention(const AttnParams& p, int D, bool codes, hipStream_t s) {
  switch (D) {
    case 64: return codes ? launch_format<64, true>(p, s) : launch_format<64, false>(p, s);
    case 128: return codes ? launch_format<128, true>(p, s) : launch_format<128, false>(p, s);
    default: return codes ? launch_format<256, true>(p, s) : launch_format<256, false>(p, s);
  }
}

}  // namespace skg
