// Log probabilities of given tokens with entropy and the best alternatives
// (skgemm_logprobs), and their gradient to the logits (skgemm_logprobs_grad).
//
// With m the largest logit x, c = scale / log 2 and d = (x - m) c:
//   s = sum 2^d, u = sum 2^d d,
//   lse = scale m + log s,  entropy = (log2 s - u / s) log 2,
//   logprob = scale (x[token] - m) - log s.
// Every term is built from d, so nothing cancels against m, and two parts of a row
// join by moving one to the other's reference:  with f = (m - m') c:  s' = s 2^f,
// u' = 2^f (u + f s). The pass over the data takes d as x c - ref in one fused
// operation a logit, with ref = m c rounded, and moves its sums from ref to m itself
// at the end. Where a product passes FP32's range (the type's lowest value as a
// mask, a large scale) a run's sums come out as 0 or not finite: it is then read
// again, with the difference before the scaling.
//
// Bound by memory for float logits (T=2048 V=131072: 163 us without alternatives,
// 6.6 TB/s) and by arithmetic for bf16: eight logits take about 80 vector slots,
// 32 of them the exponentials at a quarter rate, nearly the time of their read
// (T=4096 V=131072 with 8 alternatives 198 us, 5.4 TB/s, vector units nine tenths
// busy; 228 in the first twenty launches after a pause).
// The gradient reads and writes: T=4096 V=131072 bf16 400 us, 5.4 TB/s.

#include <algorithm>

#include "device/block.h"
#include "device/pack.h"
#include "ops_internal.h"
#include "skgemm.h"
#include "skgemm_internal.h"

namespace skg {

namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();
typedef unsigned long long u64;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// One row's 16-byte vectors: the row starts `head` elements into vector 0 and
// ends before element head + V. Only vector 0 and the last can be partial;
// those are read element by element, so nothing outside the row is read.
template <bool F32>
struct Row {
  static constexpr int kE = F32 ? 4 : 8;    // elements of a vector
  static constexpr int kSize = F32 ? 4 : 2;
  const uint8_t* base;  // vector 0, 16-byte aligned
  int head, V, nvec;

  __device__ __forceinline__ Row(const uint8_t* row, int v) {
    const int off = (int)((uintptr_t)row & 15u);
    base = row - off;
    head = off / kSize;
    V = v;
    nvec = (head + v + kE - 1) / kE;
  }
  __device__ __forceinline__ bool whole(int j) const { return j * kE >= head && (j + 1) * kE <= head + V; }
  // Index of element 0 of vector j (negative ahead of the row).
  __device__ __forceinline__ int index(int j) const { return j * kE - head; }
  __device__ __forceinline__ u32x4 load_whole(int j) const {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base) + j);
  }
  __device__ __forceinline__ static void unpack(u32x4 v, float* x) {
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(v[e]);
        x[2 * e + 1] = bf16_hi(v[e]);
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {  // element i of the row
    const uint8_t* p = base + (size_t)(head + i) * kSize;
    if constexpr (F32) return *reinterpret_cast<const float*>(p);
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  }
  // Vector j's elements; those outside the row are `fill`.
  __device__ __forceinline__ void load(int j, float* x, float fill) const {
    if (whole(j)) {
      unpack(load_whole(j), x);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int i = index(j) + e;
        x[e] = (i >= 0 && i < V) ? at(i) : fill;
      }
    }
  }
};

// ---- the sums ---------------------------------------------------------------

struct Sums {
  float m, s, u;  // reference (a logit), sum, weighted sum; m = -inf: no term yet
};

// Moves both parts to the larger reference and adds them. A part without a
// term has s = u = 0 and may have m = -inf.
__device__ __forceinline__ Sums join(Sums a, Sums b, float mul) {
  const float m = fmaxf(a.m, b.m);
  if (m == -kInf) return {m, a.s + b.s, a.u + b.u};  // + keeps a NaN
  const float da = (a.m - m) * mul, db = (b.m - m) * mul;
  const float ea = exp2_hw(da), eb = exp2_hw(db);
  // -inf times a zero sum would be NaN.
  return {m, a.s * ea + b.s * eb, ea * (a.u + fmaxf(da, -1e30f) * a.s) + eb * (b.u + fmaxf(db, -1e30f) * b.s)};
}

__device__ __forceinline__ float shfl_xor(float v, int off) { return __shfl_xor(v, off, 64); }

// The join of a workgroup's parts, in every thread. `part` is free again after
// the next barrier.
__device__ __forceinline__ void block_join(Sums& a, Sums* part, float mul) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) a = join(a, Sums{shfl_xor(a.m, off), shfl_xor(a.s, off), shfl_xor(a.u, off)}, mul);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  a = part[0];
  for (int i = 1; i < kThreads / 64; ++i) a = join(a, part[i], mul);
}

// ---- the best k ---------------------------------------------------------------
//
// Order: value first, then the lower index. A key holds both: the value's bits
// made monotonic (as unsigned) above the complement of the index, so keys are
// distinct and the larger key is the better element; 0 is no element.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 becomes 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ u64 make_key(float v, int i) { return ((u64)order_bits(v) << 32) | (uint32_t)~i; }
__device__ __forceinline__ int key_index(u64 k) { return (int)~(uint32_t)k; }

constexpr int kCand = 1024;  // candidates held in LDS

struct TopLds {
  u64 best[kThreads];
  int owners[kThreads];
  u64 cand[kCand + 8];
  u64 lowest;
  int n_own, n_cand, count;
};

// How a workgroup's vectors fall to 256 owners: owner o = (segment o / (256 / G),
// group o % (256 / G)) holds the vectors that the G = 1 << lg threads of the
// group take in `len` consecutive rounds of 256. G neighbouring vectors a round:
// with G = 8, whole 128-byte lines, so that reading an owner's vectors again
// moves no more than they hold.
struct Owners {
  int lg, len;
  __device__ __forceinline__ explicit Owners(int rounds) {
    lg = rounds >= 8 ? 3 : rounds >= 4 ? 2 : rounds >= 2 ? 1 : 0;
    len = (rounds + (1 << lg) - 1) >> lg;
  }
  __device__ __forceinline__ int items() const { return len << lg; }
  __device__ __forceinline__ int item(int o, int x) const {
    const int group = o & ((kThreads >> lg) - 1), seg = o >> (8 - lg);
    return (seg * len + (x >> lg)) * kThreads + (group << lg) + (x & ((1 << lg) - 1));
  }
};
static_assert(kThreads == 256, "owner numbers are 8 bits");

// Sorted best k of the keys that `src` holds, to out(rank, key), ranks 0 ..
// k-1 (fewer if fewer keys). l.best holds, for each owner of src's items, a
// bound below its best key of the same value, at most kE - 1 below it (the pass
// over the data notes the vector that holds the largest logit, not the
// element); 0: no key.
//
// If k of these bounds reach some b, then k keys reach it, so every key
// of the best k is at least b and lies with an owner whose bound + kE - 1 is.
// Only those owners' items are read again: about k of 256, a fraction k / 256
// of the data, whatever the values are, equal ones included. Should they hold
// more than kCand keys past b, the exact k-th key is searched bit by bit over
// the owners' items.
//
// The values are ordered, so no NaN is among them (fmaxf passes over one, a key
// orders it: reaches() and the keys would disagree, and the search would end
// with any number of candidates). The caller does not select from a run that
// holds one. The candidates are bounded by their buffer all the same, as the
// data are read twice and may change where a caller writes them meanwhile.
template <class Src, class Out>
__device__ __forceinline__ void block_top(const Src& src, const Owners& who, int k, TopLds& l, Out out) {
  const int tid = (int)threadIdx.x, lane = tid & 63;
  if (tid == 0) l.n_own = l.n_cand = 0;
  __syncthreads();
  // One wave finds b, four bounds a lane, one bit a step: first the value, then,
  // where many owners share it, the index. The common leading bits of all values
  // are skipped, and any b that k .. k + slack owners reach will do: half a dozen
  // steps as a rule. (All waves at it, exact: 53 steps; T=256 V=50001 34.8 instead
  // of 29.0 us.)
  if (tid < 64) {
    uint32_t v4[4], i4[4], most = 0, least = ~0u;
    int valid = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 b = l.best[lane + 64 * i];
      v4[i] = (uint32_t)(b >> 32);
      i4[i] = (uint32_t)b;
      most = max(most, v4[i]);
      least = min(least, v4[i] != 0 ? v4[i] : ~0u);
      valid += __popcll(__ballot(v4[i] != 0));
    }
    most = butterfly_umax(most);
    least = ~butterfly_umax(~least);
    uint32_t value = 0, index = 0;
    if (valid >= k) {
      const int slack = k / 2 + 8;
      most = (uint32_t)__builtin_amdgcn_readfirstlane((int)most);
      const uint32_t differ = most ^ (uint32_t)__builtin_amdgcn_readfirstlane((int)least);
      uint32_t bit = differ != 0 ? 0x80000000u >> __builtin_clz(differ) : 0u;
      value = bit != 0 ? most & ~(2u * bit - 1u) : most;
      int reach = valid;
      for (; bit != 0 && reach > k + slack; bit >>= 1) {
        const uint32_t c = value | bit;
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += __popcll(__ballot(v4[i] >= c));
        if (n >= k) {
          value = c;
          reach = n;
        }
      }
      if (reach > k + slack) {
        index = ~(uint32_t)(2 * SKGEMM_MAX_V - 1);  // an index is below SKGEMM_MAX_V + kE
        for (uint32_t low = SKGEMM_MAX_V; low != 0 && reach > k + slack; low >>= 1) {
          const uint32_t c = index | low;
          int n = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) n += __popcll(__ballot(v4[i] > value || (v4[i] == value && i4[i] >= c)));
          if (n >= k) {
            index = c;
            reach = n;
          }
        }
      }
    }
    if (lane == 0) l.lowest = ((u64)value << 32) | index;
  }
  __syncthreads();
  u64 lowest = l.lowest;
  const u64 bound = l.best[tid];
  if (bound != 0 && bound + (Src::kE - 1) >= lowest) l.owners[atomicAdd(&l.n_own, 1)] = tid;
  __syncthreads();
  // The owners' items over all threads, four loads of a thread in flight: a
  // wave's round takes 64 >> shift owners, 1 << shift items of each.
  const int n_own = l.n_own, per = who.items(), wave = tid >> 6;
  int shift = 0;
  while (shift < 6 && (1 << shift) < per) ++shift;
  const int width = 64 >> shift, groups = (n_own + width - 1) / width, chunks = (per + (1 << shift) - 1) >> shift;
  const int rounds = groups * chunks;
  auto each_key = [&](u64 at_least, auto f) {  // f of each key; those below at_least may be left out
    for (int r0 = wave; r0 < rounds; r0 += 4 * (kThreads / 64)) {
      int item[4];
      typename Src::Raw raw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + q * (kThreads / 64), group = r / chunks, chunk = r - group * chunks;
        const int own = group * width + (lane >> shift), j = (chunk << shift) + (lane & ((1 << shift) - 1));
        item[q] = (r < rounds && own < n_own && j < per) ? who.item(l.owners[own], j) : -1;
        raw[q] = src.load(item[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (!src.reaches(item[q], raw[q], (uint32_t)(at_least >> 32))) continue;
        u64 key[Src::kE];
        src.keys(item[q], raw[q], key);
#pragma unroll
        for (int e = 0; e < Src::kE; ++e) f(key[e]);
      }
    }
  };
  auto gather = [&]() {
    each_key(lowest, [&](u64 key) {
      if (key != 0 && key >= lowest) {
        const int at = atomicAdd(&l.n_cand, 1);
        if (at < kCand) l.cand[at] = key;
      }
    });
    __syncthreads();
  };
  gather();
  if (l.n_cand > kCand) {
    // The k-th largest key itself, one bit a step; then exactly k keys reach it.
    u64 kth = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const u64 c = kth | ((u64)1 << bit);
      if (tid == 0) l.count = 0;
      __syncthreads();
      int n = 0;
      each_key(c, [&](u64 key) { n += key >= c; });
      atomicAdd(&l.count, n);
      __syncthreads();
      if (l.count >= k) kth = c;
      __syncthreads();
    }
    lowest = kth;
    if (tid == 0) l.n_cand = 0;
    __syncthreads();
    gather();
  }
  const int n = min(l.n_cand, kCand);
  if (tid < 8) l.cand[n + tid] = 0;  // the ranks below are counted eight keys at a time
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const u64 key = l.cand[i];
    int rank = 0;
    for (int j = 0; j < n; j += 8) {
#pragma unroll
      for (int q = 0; q < 8; ++q) rank += l.cand[j + q] > key;
    }
    if (rank < k) out(rank, key);
  }
}

// A row's vectors first .. first + n as block_top's items.
template <bool F32>
struct RowItems {
  static constexpr int kE = Row<F32>::kE;
  const Row<F32>& row;
  int first, n;
  typedef u32x4 Raw;
  // Item `item` (none: negative, or past the run). A partial vector is read
  // element by element in keys().
  __device__ __forceinline__ Raw load(int item) const {
    if (item < 0 || item >= n || !row.whole(first + item)) return u32x4{0, 0, 0, 0};
    return row.load_whole(first + item);
  }
  // Whether a key of this item can have a value of at least `order`: for whole
  // vectors one comparison of the largest.
  __device__ __forceinline__ bool reaches(int item, Raw raw, uint32_t order) const {
    if (item < 0 || item >= n) return false;
    if (!row.whole(first + item)) return true;
    float x[kE], m;
    Row<F32>::unpack(raw, x);
    m = x[0];
#pragma unroll
    for (int e = 1; e < kE; ++e) m = fmaxf(m, x[e]);
    return order_bits(m) >= order;
  }
  __device__ __forceinline__ void keys(int item, Raw raw, u64* key) const {
#pragma unroll
    for (int e = 0; e < kE; ++e) key[e] = 0;
    if (item < 0 || item >= n) return;
    const int i0 = row.index(first + item);
    float x[kE];
    if (row.whole(first + item)) {
      Row<F32>::unpack(raw, x);
#pragma unroll
      for (int e = 0; e < kE; ++e) key[e] = make_key(x[e], i0 + e);
    } else {
      row.load(first + item, x, 0.0f);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (i0 + e >= 0 && i0 + e < row.V) key[e] = make_key(x[e], i0 + e);
    }
  }
};

// Keys in the workspace, kept by the workgroups of a row, as block_top's items.
struct KeyItems {
  static constexpr int kE = 1;
  typedef u64 Raw;
  u64* keys_;
  int n;
  __device__ __forceinline__ Raw load(int item) const {
    if (item < 0 || item >= n) return 0;
    return __hip_atomic_load(keys_ + item, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ bool reaches(int, Raw raw, uint32_t order) const { return (uint32_t)(raw >> 32) >= order; }
  __device__ __forceinline__ void keys(int, Raw raw, u64* key) const { key[0] = raw; }
};

__device__ __forceinline__ void store_agent(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float load_agent(float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A row, or where there are few rows one of p.parts runs of its vectors: the
// workgroup that finishes a row's last run joins the sums and the best k that
// the others left in the workspace.
template <bool F32, bool TOP>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobParams p) {
  __shared__ TopLds top;
  __shared__ Sums part[kThreads / 64];
  __shared__ uint32_t arrived;
  const int tid = (int)threadIdx.x;
  const size_t t = blockIdx.x / (unsigned)p.parts;
  const int run = (int)(blockIdx.x - (unsigned)t * (unsigned)p.parts);
  const Row<F32> row(p.logits + t * p.stride, p.V);
  constexpr int kE = Row<F32>::kE;
  const float mul = p.scale * kLog2e;
  const int first = run * p.per, n = max(0, min(p.per, row.nvec - first));
  Sums a = {-kInf, 0.0f, 0.0f};
  const int rounds = (n + kThreads - 1) / kThreads;
  const Owners who(TOP ? rounds : 1);
  float seg_m = -kInf;  // TOP: this segment's largest logit, and the first vector that holds it
  int at = -1;
  // The sums are kept against ref = m mul, rounded (one fused operation a logit
  // instead of two: the kernel is bound by its arithmetic at 2 bytes a logit),
  // and moved to m itself at the end. A product past FP32's range (the type's
  // lowest value, say) is held inside it; such a run's sums come out as 0 or not
  // finite and are taken again below.
  auto in_range = [](float v) { return fminf(fmaxf(v, -3e38f), 3e38f); };
  float ref = -3e38f;
  auto add = [&](int j, const float* x) {
    float m = x[0];
#pragma unroll
    for (int e = 1; e < kE; ++e) m = fmaxf(m, x[e]);
    if constexpr (TOP) {
      at = m > seg_m ? j : at;
      seg_m = fmaxf(seg_m, m);
    }
    if (m > a.m) {
      const float r = in_range(m * mul), d = ref - r, f = exp2_hw(d);
      a.u = f * (a.u + fmaxf(d, -1e30f) * a.s);
      a.s *= f;
      a.m = m;
      ref = r;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float d = fmaf(x[e], mul, -ref), w = exp2_hw(d);
      a.s += w;
      a.u = fmaf(w, fmaxf(d, -1e30f), a.u);  // 0 * -1e30 where 0 * -inf would be NaN
    }
  };
  {
    // Thread tid takes vector first + 256 i + tid in round i: whole ones four
    // loads at a time, the row's partial ends by themselves where they are this
    // thread's, in their segment and in order.
    const int last = row.nvec - 1;
    const int w0 = row.whole(0) ? 0 : 1, w1 = min(first + n, row.whole(last) ? row.nvec : last);
    const bool tail = last > 0 && !row.whole(last) && last < first + n;
    int i = 0;
    for (int seg = 0; seg < (1 << who.lg); ++seg) {
      const int i1 = TOP ? min(rounds, (seg + 1) * who.len) : rounds;
      const int j1 = first + i1 * kThreads;  // past this segment
      int j = first + i * kThreads + tid;
      if (j == 0 && n > 0 && w0 == 1) {
        float x[kE];
        row.load(0, x, -kInf);
        at = 0;
        add(0, x);
        j += kThreads;
        ++i;
      }
      const int end = min(j1, w1);
      // A segment of nothing but -inf keeps its first vector.
      if (at < 0 && j < min(j1, first + n)) at = j;
      for (; j + 3 * kThreads < end; j += 4 * kThreads) {
        u32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = row.load_whole(j + q * kThreads);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[kE];
          Row<F32>::unpack(v[q], x);
          add(j + q * kThreads, x);
        }
      }
      for (; j < end; j += kThreads) {
        float x[kE];
        Row<F32>::unpack(row.load_whole(j), x);
        add(j, x);
      }
      if (tail && j == last && last < j1) {
        float x[kE];
        row.load(last, x, -kInf);
        add(last, x);
      }
      i = i1;
      if constexpr (TOP) {
        // The group's best: its largest logit, the lowest vector among equals.
        const uint32_t v = at >= 0 ? order_bits(seg_m) : 0u;
        uint32_t most = v;
        if (who.lg > 0) most = xred_umax<1>(most);
        if (who.lg > 1) most = xred_umax<2>(most);
        if (who.lg > 2) most = xred_umax<4>(most);
        uint32_t low = at >= 0 && v == most ? ~(uint32_t)(row.index(at) + kE - 1) : 0u;
        if (who.lg > 0) low = xred_umax<1>(low);
        if (who.lg > 1) low = xred_umax<2>(low);
        if (who.lg > 2) low = xred_umax<4>(low);
        const u64 bound = ((u64)most << 32) | low;
        if ((tid & ((1 << who.lg) - 1)) == 0) top.best[seg * (kThreads >> who.lg) + (tid >> who.lg)] = bound;
        seg_m = -kInf;
        at = -1;
      }
    }
  }
  if (a.s != 0.0f) {  // to the reference m: d = (x mul - ref) - (m mul - ref)
    const float c = fmaf(a.m, mul, -ref), f = exp2_hw(-c);
    a.u = f * (a.u - c * a.s);
    a.s *= f;
  }
  block_join(a, part, mul);
  if (fabsf(a.m) < kInf && !(a.s > 0.0f && a.s < kInf)) {
    // Logits near the type's ends (or a NaN among finite ones): differences
    // first, with the run's largest logit as the reference.
    const float m = a.m;
    a = Sums{m, 0.0f, 0.0f};
    for (int j = first + tid; j < first + n; j += kThreads) {
      float x[kE];
      row.load(j, x, -kInf);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float d = (x[e] - m) * mul, w = exp2_hw(d);
        a.s += w;
        a.u = fmaf(w, fmaxf(d, -1e30f), a.u);
      }
    }
    __syncthreads();
    block_join(a, part, mul);
  }
  const RowItems<F32> items{row, first, n};
  // The row's sums, then its keys, of all runs.
  uint8_t* const work = p.part + t * (size_t)p.parts * kLogprobPart;
  u64* const kept = reinterpret_cast<u64*>(work + 16 * (size_t)p.parts);
  if (p.parts > 1) {
    float* const sums = reinterpret_cast<float*>(work);
    if (tid == 0) {
      store_agent(sums + 4 * run, a.m);
      store_agent(sums + 4 * run + 1, a.s);
      store_agent(sums + 4 * run + 2, a.u);
    }
    if constexpr (TOP) {
      // A NaN sum makes the row's ids -1: nothing is selected from such a run.
      const bool sound = a.s == a.s;
      u64* const keys = kept + run * p.k;
      if (sound)
        block_top(items, who, p.k, top, [&](int rank, u64 key) {
          __hip_atomic_store(keys + rank, key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        });
      // A run of fewer than k elements leaves the rest empty.
      if (tid >= (sound ? top.n_cand : 0) && tid < p.k)
        __hip_atomic_store(keys + tid, (u64)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_vmem_all();
    __syncthreads();
    if (tid == 0) {
      uint32_t* const cnt = p.cnt + t * kOpsCounterStride;
      const uint32_t c = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (c + 1 == (uint32_t)p.parts) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      arrived = c;
    }
    __syncthreads();
    if (arrived + 1 != (uint32_t)p.parts) return;
    handoff_order();
    a = Sums{-kInf, 0.0f, 0.0f};
    if (tid < p.parts) {  // at most 32: one wave
      float* const f = sums + 4 * tid;
      a = Sums{load_agent(f), load_agent(f + 1), load_agent(f + 2)};
    }
    if (tid < 64) {
#pragma unroll
      for (int off = 32; off > 0; off >>= 1)
        a = join(a, Sums{shfl_xor(a.m, off), shfl_xor(a.s, off), shfl_xor(a.u, off)}, mul);
      if (tid == 0) part[0] = a;
    }
    __syncthreads();
    a = part[0];
  }

  // s is NaN exactly where the row holds a NaN or +inf.
  const bool bad = !(a.s == a.s), empty = a.s == 0.0f;
  const float log_s = __builtin_amdgcn_logf(a.s);  // log2
  if (tid == 0) {
    if (p.lse != nullptr) p.lse[t] = bad ? a.s : empty ? -kInf : fmaf(a.m, p.scale, log_s * kLn2);
    if (p.entropy != nullptr) p.entropy[t] = empty ? 0.0f : (log_s - a.u / a.s) * kLn2;
    if (p.logprob != nullptr) {
      const int64_t tok = p.tokens[t];
      float v;
      if (tok < 0) v = 0.0f;
      else if (tok >= p.V || bad) v = __builtin_nanf("");
      else if (empty) v = -kInf;
      else v = (row.at((int)tok) - a.m) * p.scale - log_s * kLn2;
      p.logprob[t] = v;
    }
  }
  if constexpr (!TOP) return;
  float* tv = p.top_logprob + t * (size_t)p.k;
  int64_t* ti = p.top_ids + t * (size_t)p.k;
  if (bad) {
    if (tid < p.k) {
      tv[tid] = a.s;
      ti[tid] = -1;
    }
    return;
  }
  auto out = [&](int rank, u64 key) {
    const float v = order_value((uint32_t)(key >> 32));
    tv[rank] = empty ? -kInf : (v - a.m) * p.scale - log_s * kLn2;
    ti[rank] = key_index(key);
  };
  if (p.parts == 1) {
    block_top(items, who, p.k, top, out);
  } else {
    const KeyItems items2{kept, p.parts * p.k};
    u64 best = 0;
#pragma unroll 4
    for (int i = tid; i < items2.n; i += kThreads) {
      const u64 key = items2.load(i);
      best = key > best ? key : best;
    }
    __syncthreads();  // the run's own bounds have been read
    top.best[tid] = best;
    Owners each(1);  // thread t's keys t, t + 256, ...
    each.len = (items2.n + kThreads - 1) / kThreads;
    block_top(items2, each, p.k, top, out);
  }
}

// ---- the gradient -------------------------------------------------------------
//
//   d_j = scale * (g ([j == token] - p_j) - gH p_j (log p_j + H))
//       = p_j * (c0 + c1 log2 p_j) + [j == token] scale g,
//   c0 = -scale (g + gH H),  c1 = -scale gH ln 2.
// One workgroup takes a run of a row's vectors; elementwise, so d_logits may be
// the logits.
template <bool F32>
__global__ __launch_bounds__(kThreads) void logprobs_grad_kernel(LogprobGradParams p) {
  const size_t t = blockIdx.x / p.parts;
  const Row<F32> row(p.logits + t * p.stride, p.V);
  const Row<F32> out(p.d_logits + t * p.d_stride, p.V);
  constexpr int kE = Row<F32>::kE;
  const int64_t tok = p.tokens != nullptr ? p.tokens[t] : -1;
  const float lse = p.lse[t];
  const bool empty = lse == -kInf;
  float g = (p.g_logprob != nullptr && tok >= 0) ? p.g_logprob[t] : 0.0f;
  if (p.g_logprob != nullptr && tok >= p.V) g = __builtin_nanf("");
  const float gh = p.g_entropy != nullptr ? p.g_entropy[t] : 0.0f;
  const float ent = p.g_entropy != nullptr ? p.entropy[t] : 0.0f;
  const float ref = empty ? 0.0f : lse;
  // The clamp below would swallow a NaN lse, so it goes into c0; an lse of +inf
  // (scale * max past FP32's range) says nothing about the probabilities either.
  const float c0 = lse < kInf ? -p.scale * (g + gh * ent) : __builtin_nanf(""), c1 = -p.scale * gh * kLn2;
  const float hit = empty ? 0.0f : p.scale * g;
  const bool same = row.head == out.head;
  uint8_t* const base = p.d_logits + t * p.d_stride - (size_t)out.head * Row<F32>::kSize;
  const int hit_at = tok >= 0 && tok < p.V ? (int)tok + row.head : -1;  // counted from vector 0
  for (int j = (int)(blockIdx.x % p.parts * kThreads + threadIdx.x); j < row.nvec; j += (int)(p.parts * kThreads)) {
    float x[kE];
    row.load(j, x, 0.0f);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      // Past -150 the exponential is 0; -inf would make 0 * inf of it, and so would
      // a bound whose product with c1 passes FP32's range.
      const float lp = fmaxf(fmaf(x[e], p.scale, -ref) * kLog2e, -1024.0f);
      x[e] = exp2_hw(lp) * fmaf(c1, lp, c0);
    }
    if ((unsigned)(hit_at - j * kE) < (unsigned)kE) {
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (j * kE + e == hit_at) x[e] += hit;
    }
    if (same && row.whole(j)) {
      u32x4 w;
      if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(x[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = bf16_pair_hw(x[2 * e], x[2 * e + 1]);
      }
      reinterpret_cast<u32x4*>(base)[j] = w;
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int i = row.index(j) + e;
        if (i < 0 || i >= p.V) continue;
        if constexpr (F32)
          reinterpret_cast<float*>(base)[out.head + i] = x[e];
        else
          reinterpret_cast<uint16_t*>(base)[out.head + i] = (uint16_t)bf16_rne(x[e]);
      }
    }
  }
}

}  // namespace

// A row is split while there are fewer workgroups than keep the card busy, down
// to one vector a thread; at most 32 runs (one wave joins them). About 1024
// workgroups: with 2048 / 1024 / 512 / 256, T=67 V=50001 float took 21.2 / 17.7 /
// 17.9 / 23.9 us, T=300 V=131072 bf16 44.1 / 37.8 / 42.4 / 42.5 us (8
// alternatives); with up to 64 / 32 / 16 runs, T=1 V=131072 bf16 13.7 / 13.9 /
// 14.6 us for 8 and 31.7 / 22.5 / 20.8 us for 64 alternatives.
int logprob_parts(int T, int V, bool f32, int* per) {
  const int steps = (V / (f32 ? 4 : 8) + 2 + kThreads - 1) / kThreads;  // vectors a thread, partial ends included
  const int want = std::max(1, std::min(32, 1024 / std::max(T, 1)));
  const int each = (steps + want - 1) / want;
  *per = each * kThreads;
  return (steps + each - 1) / each;
}

hipError_t launch_logprobs(const LogprobParams& p, bool f32, hipStream_t s) {
  const dim3 grid((unsigned)p.T * (unsigned)p.parts);
  if (f32)
    return launch(p.k > 0 ? logprobs_kernel<true, true> : logprobs_kernel<true, false>, grid, dim3(kThreads), 0, s, p);
  return launch(p.k > 0 ? logprobs_kernel<false, true> : logprobs_kernel<false, false>, grid, dim3(kThreads), 0, s, p);
}

hipError_t launch_logprobs_grad(LogprobGradParams p, bool f32, hipStream_t s) {
  // Up to 16384 workgroups, down to one vector a thread (T=64 V=32001 float with 4
  // workgroups a row took 8.3 us, T=1 V=131072 bf16 7.6).
  const unsigned steps = ((unsigned)p.V / (f32 ? 4 : 8) + 2 + kThreads - 1) / kThreads;
  p.parts = std::max(1u, std::min(steps, 16384u / (unsigned)p.T));
  const dim3 grid((unsigned)p.T * p.parts);
  return launch(f32 ? logprobs_grad_kernel<true> : logprobs_grad_kernel<false>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace skg
