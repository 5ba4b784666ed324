// Product of 8-bit integers with a scale for each token and each output
// channel (skgemm_i8):
//   C[t, n] = x_scale[t] * w_scale[n] * sum_k Xq[t, k] Wq[n, k].
//
// v_mfma_i32_16x16x64_i8 with A = weights (rows = output features) and
// B = activations (columns = tokens): lane l = 16 g + i holds the 16 bytes of
// row (column) i at K block g, and D's rows 4g..4g+3 of column i. Sums of
// 32-bit integers are exact and commute, so K is split over waves freely.

#include <algorithm>

#include "device/block.h"
#include "device/pack.h"
#include "ops_internal.h"
#include "skgemm_internal.h"
#include "skgemm.h"

namespace skg {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Outputs n .. n+3 of token t from their integer sums. The sum is rounded to
// FP32, both products are FP32, and bf16 rounds once more.
__device__ __forceinline__ void store_sums(const I8Params& p, int t, int n, i32x4 s, float xs, const float* ws) {
  uint8_t* const row = p.c + (size_t)t * p.c_stride;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = (float)s[e] * xs * ws[e];
  if (p.c_quads && n + 3 < p.N) {  // every row's n is aligned for one store
    if (p.out_f32)
      *reinterpret_cast<f32x4*>(row + (size_t)n * 4) = f32x4{v[0], v[1], v[2], v[3]};
    else
      *reinterpret_cast<u32x2*>(row + (size_t)n * 2) = u32x2{bf16_pair_hw(v[0], v[1]), bf16_pair_hw(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    if (p.out_f32)
      reinterpret_cast<float*>(row)[n + e] = v[e];
    else
      reinterpret_cast<uint16_t*>(row)[n + e] = (uint16_t)bf16_pair_hw(v[e], 0.0f);
  }
}

// Few tokens: the weights' stream is everything. A workgroup of eight waves takes
// 16 features x 16 tokens, operands straight from memory into registers; the
// waves take the row's 128-byte units in turn and their sums meet in LDS, so K is
// split without a second pass.
//
// Both operands come as line pairs (device/types.h): 8 rows x 128 bytes a load,
// whole lines; one DPP move a register makes the two 16-row operands. With at
// most 8 tokens (LOW) the second load of the activations' pair is left out. U
// units are in flight in each wave: a slot is consumed, then refilled. Bound by the
// weights: T=1 N=18432 K=7168 23.5 us (5.6 TB/s), T=8 N=K=16384 51 us (5.2);
// below about 30 MB by launch and latency (T=1 N=2048 K=7168 6.6 us).
constexpr int kRowWaves = 8;
template <bool LOW, int U>
__global__ __launch_bounds__(64 * kRowWaves) void i8_rows_kernel(I8Params p) {
  constexpr int kXL = LOW ? 1 : 2;  // loads of 16 tokens
  __shared__ i32x4 part[kRowWaves][64];
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int li = lane & 15, g = lane >> 4;
  const int ntiles = (p.N + 15) / 16;
  const int tt = (int)blockIdx.x / ntiles;
  const int n0 = ((int)blockIdx.x - tt * ntiles) * 16, t0 = tt * 16;
  const int rows = min(16, p.N - n0), tokens = min(16, p.T - t0);
  const rsrc_t w = make_rsrc(p.w + (size_t)n0 * p.w_stride, (uint32_t)((rows - 1) * p.w_stride + p.K));
  const rsrc_t x = make_rsrc(p.x + (size_t)t0 * p.x_stride, (uint32_t)((tokens - 1) * p.x_stride + p.K));
  const int in_line = 64 * (li >> 3) + 16 * g;  // this lane's bytes of a unit
  // Rows past the tile's end read zeros.
  uint32_t woff[2], xoff[kXL];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = 8 * q + (li & 7);
    woff[q] = r < rows ? (uint32_t)(r * p.w_stride + in_line) : kOOB;
  }
#pragma unroll
  for (int q = 0; q < kXL; ++q) {
    const int r = 8 * q + (li & 7);
    xoff[q] = r < tokens ? (uint32_t)(r * p.x_stride + in_line) : kOOB;
  }
  u32x4 wv[U][2], xv[U][kXL];
  auto fill = [&](int u, int k) {  // k past the row's end: zeros
    const uint32_t past = k + in_line < p.K ? 0u : kOOB;
#pragma unroll
    for (int q = 0; q < kXL; ++q)
      xv[u][q] = __builtin_amdgcn_raw_buffer_load_b128(x, xoff[q] | past, k, kPolicyDefault);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      wv[u][q] = __builtin_amdgcn_raw_buffer_load_b128(w, woff[q] | past, k, kPolicyStream);
  };
  i32x4 acc = {};
  constexpr int kStep = 128 * kRowWaves;
#pragma unroll
  for (int u = 0; u < U; ++u) fill(u, 128 * wave + u * kStep);
  auto use = [&](int u) {
    u32x4 x0, x1, w0, w1;
    line_pair_to_operands(xv[u][0], LOW ? u32x4{0, 0, 0, 0} : xv[u][kXL - 1], x0, x1);
    line_pair_to_operands(wv[u][0], wv[u][1], w0, w1);
    acc = mfma_i8(w0, x0, acc);
    acc = mfma_i8(w1, x1, acc);
  };
  int k = 128 * wave;
  for (; k + U * kStep < p.K; k += U * kStep) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      use(u);
      fill(u, k + (U + u) * kStep);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) use(u);
  part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int v = 1; v < kRowWaves; ++v) acc += part[v][lane];
  const int t = t0 + li, n = n0 + 4 * g;
  float ws[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) ws[e] = n + e < p.N ? p.w_scale[n + e] : 0.0f;
  if (t < p.T) store_sums(p, t, n, acc, p.x_scale[t], ws);
}

// A tile of BT tokens x BN features, K in steps of 128 bytes through LDS.
//
// Each step's 128-byte row pieces come straight from memory into LDS
// (buffer_load ... lds, 16 bytes a lane, 8 whole lines an instruction) into one
// of STG buffers, STG - 1 steps ahead. Row r's 16-byte chunk c lies at position
// c ^ (r & 7) of its line: an operand read takes one chunk of 16 rows, and
// without the exchange all 16 would meet in the same banks. The exchange is on
// the memory side (lane l of a load fetches chunk (l % 8) ^ (l / 8) of row
// l / 8), as the LDS side of such a load is linear.
//
// WT x WN waves share the tile; a wave holds (BT / WT) x (BN / WN) sums in
// registers. One barrier a step: past it, every wave's loads of this step have
// landed and every wave has read the previous step's buffer, which the next
// loads then fill.
//
// Bound by the weights' stream for few tokens (T=32 N=18432 K=7168: 29.4 us, 4.5
// TB/s) and above that by the loads into LDS, up to 70 GB/s a CU (T=509 N=4100
// K=7168: 31.5 us). Loads counted by hand: left
// to the compiler, T=4096 N=18432 K=7168 took 664 instead of 582 us (before the
// kernel below took such calls).
//
// S workgroups may split K of a tile: each stores its sums to the workspace and
// the last to arrive adds the others' (integers: the order does not matter).
// Only the tiles past the last full round of workgroups are split, so that the
// last round is as full as the others.
template <int BT, int BN>
struct Tile {
  int slot, S, rank, t0, n0, tokens, rows, s0, s1;  // slot: this tile's place in the workspace (S > 1)
  u32x4 w, x;   // buffer resources of the tile's rows
  // No other tile reads these weights: they are loaded non-temporally (K=N=16384,
  // T=32 54.3 -> 51.0 us, T=64 58.5 -> 55.3, T=128 70.9 -> 68.0).
  bool stream;

  __device__ __forceinline__ explicit Tile(const I8Params& p) {
    // Workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles whose
    // operands its L2 then holds, four token tiles for each feature tile.
    const int ttiles = (p.T + BT - 1) / BT, ntiles = (p.N + BN - 1) / BN;
    int b = (int)blockIdx.x, total = p.whole, tile = 0;
    S = 1;
    if (b >= p.whole) {  // the tiles past the last full round of workgroups are split
      b -= p.whole;
      S = p.S;
      total = (ttiles * ntiles - p.whole) * S;
      tile = p.whole;
    }
    const int xcd = b & 7, idx = (b >> 3) + xcd * (total >> 3) + min(xcd, total & 7);
    rank = idx % S;
    slot = idx / S;
    tile += slot;
    const int group = tile / (4 * ntiles), in_group = tile - group * 4 * ntiles;
    const int gt = min(4, ttiles - 4 * group);
    t0 = (4 * group + in_group % gt) * BT;
    n0 = in_group / gt * BN;
    tokens = min(BT, p.T - t0);
    rows = min(BN, p.N - n0);
    stream = ttiles == 1;
    w = make_rsrc_words(p.w + (size_t)n0 * p.w_stride, (uint32_t)((rows - 1) * p.w_stride + p.K));
    x = make_rsrc_words(p.x + (size_t)t0 * p.x_stride, (uint32_t)((tokens - 1) * p.x_stride + p.K));
    const long steps = (p.K + 127) / 128;
    s0 = (int)(steps * rank / S);
    s1 = (int)(steps * (rank + 1) / S);
  }
};

// A wave's share of the loads of a step: kXL and kWL instructions.
template <int BT, int BN, int kWaves>
struct Loader {
  static constexpr int kXL = BT / 8 / kWaves, kWL = BN / 8 / kWaves;
  static constexpr int kStage = (BT + BN) * 128;
  static_assert(kXL >= 1 && kWL >= 1 && kXL * kWaves * 8 == BT && kWL * kWaves * 8 == BN, "whole loads");
  uint32_t xoff[kXL], woff[kWL];
  int chunk, wave;

  __device__ __forceinline__ Loader(const I8Params& p, const Tile<BT, BN>& t, int lane, int wave_) : wave(wave_) {
    const int row8 = lane >> 3;
    chunk = 16 * ((lane & 7) ^ row8);
    // A row past the tile's end loads zeros (out of range).
#pragma unroll
    for (int q = 0; q < kXL; ++q) {
      const int r = 8 * (wave * kXL + q) + row8;
      xoff[q] = r < t.tokens ? (uint32_t)(r * p.x_stride + chunk) : kOOB;
    }
#pragma unroll
    for (int q = 0; q < kWL; ++q) {
      const int r = 8 * (wave * kWL + q) + row8;
      woff[q] = r < t.rows ? (uint32_t)(r * p.w_stride + chunk) : kOOB;
    }
  }
  __device__ __forceinline__ void issue(const Tile<BT, BN>& t, int K, int s, uint32_t at) const {
    const uint32_t past = 128 * s + chunk < K ? 0u : kOOB;  // K ends inside the last step
#pragma unroll
    for (int q = 0; q < kWL; ++q) {
      const uint32_t to = at + BT * 128 + (wave * kWL + q) * 1024;
      if (t.stream)
        ld16_to_lds<true>(t.w, woff[q] | past, 128 * s, to);
      else
        ld16_to_lds(t.w, woff[q] | past, 128 * s, to);
    }
#pragma unroll
    for (int q = 0; q < kXL; ++q) ld16_to_lds(t.x, xoff[q] | past, 128 * s, at + (wave * kXL + q) * 1024);
  }
};

// Joins the sums of the S workgroups of a tile (true in the one that holds them
// all afterwards). Sums are stored as they lie in the registers: 16 bytes a
// lane, 1 KB a store.
template <int kTile, int kSums>
__device__ __forceinline__ bool join_ranks(const I8Params& p, int tile, int S, int rank, i32x4* acc, int lane, int wave) {
  __shared__ uint32_t arrived;
  const rsrc_t part = make_rsrc(p.part + (size_t)tile * S * kTile, (uint32_t)S * kTile);
  const uint32_t at = (uint32_t)(wave * kSums * 1024 + lane * 16);
#pragma unroll
  for (int k = 0; k < kSums; ++k)
    st16_coherent_if(true, __builtin_bit_cast(u32x4, acc[k]), part, (uint32_t)rank * kTile + at + k * 1024u);
  wait_vmem_all();
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* const cnt = p.cnt + (size_t)tile * kOpsCounterStride;
    const uint32_t a = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // Everyone has arrived: the counter is ready for the next call.
    if (a + 1 == (uint32_t)S) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    arrived = a;
  }
  __syncthreads();
  if (arrived + 1 != (uint32_t)S) return false;
  handoff_order();
  for (int r = 0; r < S; ++r) {
    if (r == rank) continue;
#pragma unroll
    for (int k = 0; k < kSums; ++k)
      acc[k] += __builtin_bit_cast(i32x4, ld16_coherent_if(true, part, (uint32_t)r * kTile + at + k * 1024u));
  }
  return true;
}

// The outputs of a wave's kNT x kMT blocks of 16 features x 16 tokens, block
// (0, 0) at feature n0 and token t0. A token's blocks go out one after another,
// so that the 32-byte pieces of a line meet in the L2.
template <int kNT, int kMT>
__device__ __forceinline__ void store_blocks(const I8Params& p, int t0, int n0, const i32x4* acc, int lane) {
  const int i = lane & 15, g = lane >> 4;
  float ws[kNT][4];
#pragma unroll
  for (int k = 0; k < kNT; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = n0 + 16 * k + 4 * g + e;
      ws[k][e] = n < p.N ? p.w_scale[n] : 0.0f;
    }
#pragma unroll
  for (int j = 0; j < kMT; ++j) {
    const int t = t0 + 16 * j + i;
    if (t >= p.T) continue;
    const float xs = p.x_scale[t];
#pragma unroll
    for (int k = 0; k < kNT; ++k) store_sums(p, t, n0 + 16 * k + 4 * g, acc[k * kMT + j], xs, ws[k]);
  }
}

template <int BT, int BN, int WT, int WN, int STG>
__global__ __launch_bounds__(64 * WT * WN) void i8_tile_kernel(I8Params p) {
  constexpr int kMT = BT / WT / 16, kNT = BN / WN / 16;
  typedef Loader<BT, BN, WT * WN> L;
  __shared__ __align__(1024) uint8_t lds[STG * L::kStage];
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const Tile<BT, BN> t(p);
  const L load(p, t, lane, wave);
  const uint32_t base = lds_offset(lds);
  i32x4 acc[kNT * kMT] = {};
  const int wt = wave / WN, wn = wave % WN;
  const int pos0 = i * 128 + 16 * (g ^ (i & 7)), pos1 = i * 128 + 16 * ((4 + g) ^ (i & 7));
  const int xbase = wt * (BT / WT) * 128, wbase = BT * 128 + wn * (BN / WN) * 128;
#pragma unroll
  for (int s = 0; s < STG - 1; ++s)
    if (t.s0 + s < t.s1) load.issue(t, p.K, t.s0 + s, base + s * L::kStage);
  int buf = 0;
  for (int s = t.s0; s < t.s1; ++s) {
    // The loads of steps s + 1 .. s + STG - 2 may stay in flight.
    if (s + STG - 2 < t.s1)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STG - 2) * (L::kXL + L::kWL)) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + STG - 1 < t.s1) load.issue(t, p.K, s + STG - 1, base + (buf == 0 ? STG - 1 : buf - 1) * L::kStage);
    const uint8_t* const at = lds + buf * L::kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int pos = h ? pos1 : pos0;
      u32x4 a[kNT], b[kMT];
#pragma unroll
      for (int j = 0; j < kNT; ++j) a[j] = *reinterpret_cast<const u32x4*>(at + wbase + j * 2048 + pos);
#pragma unroll
      for (int j = 0; j < kMT; ++j) b[j] = *reinterpret_cast<const u32x4*>(at + xbase + j * 2048 + pos);
#pragma unroll
      for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int k = 0; k < kNT; ++k) acc[k * kMT + j] = mfma_i8(a[k], b[j], acc[k * kMT + j]);
    }
    buf = buf + 1 == STG ? 0 : buf + 1;
  }
  if (t.S > 1 && !join_ranks<BT * BN * 4, kNT * kMT>(p, t.slot, t.S, t.rank, acc, lane, wave)) return;
  store_blocks<kNT, kMT>(p, t.t0 + wt * (BT / WT), t.n0 + wn * (BN / WN), acc, lane);
}

// The same tile for calls of many products: 256 x 256, two waves a SIMD that
// take turns. A step is four phases, each closed by a barrier: operands of the
// first 64 bytes of K from LDS (R0), their products (M0), the other 64 bytes
// (R1, M1). Waves 4-7 (the second of each SIMD) run one phase behind waves 0-3,
// so that while one wave of a SIMD multiplies the other reads, and only four
// waves at a time share the LDS (all eight in step: 591 against 561 us at
// T=N=K=8192).
// T=4096 N=18432 K=7168: 508 us, 2.13 POP/s, at 2.25 GHz once the clock is steady
// (the first twenty launches after a pause take about 575). The matrix units are
// busy 45 % of the cycles: a phase has 512 cycles of products and takes about 1130.
// Neither their rate nor the memory bounds it, then, but the phases, and most of
// that is in barriers and products themselves: T=N=K=8192 took 560 us, without the
// loads 430, without loads and LDS reads 404. What the waves wait for there has not
// been shown. The 32 x 32 x 32 instruction took 617 against 534 us, four stages of
// 64 bytes 602 against 560.
// With A's step s in phases 4s .. 4s+3 and B's one later, the last reads of
// step s - 1 are B's R1 in phase 4s - 1: from phase 4s on its buffer may be
// filled for step s + 1 (A issues in its R0, B in its M1 before), and the loads
// have to have landed by the end of phase 4s + 3 (A waits in its M1, B in its
// R1): four phases, about a microsecond.
__global__ __launch_bounds__(512) void i8_big_kernel(I8Params p) {
  constexpr int kMT = 8, kNT = 4;
  typedef Loader<256, 256, 8> L;
  __shared__ __align__(1024) uint8_t lds[2 * L::kStage];
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const Tile<256, 256> t(p);
  const L load(p, t, lane, wave);
  const uint32_t base = lds_offset(lds);
  const bool second = wave >= 4;
  // Two token halves x four feature quarters.
  const int wt = wave & 1, wn = wave >> 1;
  const int pos0 = i * 128 + 16 * (g ^ (i & 7)), pos1 = i * 128 + 16 * ((4 + g) ^ (i & 7));
  const int xbase = wt * 128 * 128, wbase = 256 * 128 + wn * 64 * 128;
  i32x4 acc[kNT * kMT] = {};
  u32x4 a[kNT], b[kMT];
  auto read = [&](const uint8_t* at, int pos) {
#pragma unroll
    for (int j = 0; j < kNT; ++j) a[j] = *reinterpret_cast<const u32x4*>(at + wbase + j * 2048 + pos);
#pragma unroll
    for (int j = 0; j < kMT; ++j) b[j] = *reinterpret_cast<const u32x4*>(at + xbase + j * 2048 + pos);
  };
  auto multiply = [&]() {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < kMT; ++j)
#pragma unroll
      for (int k = 0; k < kNT; ++k) acc[k * kMT + j] = mfma_i8(a[k], b[j], acc[k * kMT + j]);
    __builtin_amdgcn_s_setprio(0);
  };
  auto close = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto close_loads = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  if (t.s0 < t.s1) load.issue(t, p.K, t.s0, base);
  close_loads();
  if (second) {
    if (t.s0 + 1 < t.s1) load.issue(t, p.K, t.s0 + 1, base + L::kStage);
    close();
  }
  for (int s = t.s0; s < t.s1; ++s) {
    const uint32_t buf = (uint32_t)(s - t.s0) & 1u;
    const uint8_t* const at = lds + buf * L::kStage;
    if (!second && s + 1 < t.s1) load.issue(t, p.K, s + 1, base + (buf ^ 1u) * L::kStage);
    read(at, pos0);
    close();
    multiply();
    close();
    read(at, pos1);
    if (second) close_loads(); else close();
    if (second && s + 2 < t.s1) load.issue(t, p.K, s + 2, base + buf * L::kStage);
    multiply();
    if (!second) close_loads(); else close();
  }
  if (!second) close();  // the waves behind have one phase to go
  if (t.S > 1 && !join_ranks<256 * 256 * 4, kNT * kMT>(p, t.slot, t.S, t.rank, acc, lane, wave)) return;
  store_blocks<kNT, kMT>(p, t.t0 + wt * 128, t.n0 + wn * 64, acc, lane);
}

}  // namespace

namespace {

// The tile shapes and a score of each by which a call's shape and split are
// ranked. It has the form of a cost (a workgroup pays kStart and `alone` a step
// while the CU has room for it (`fit` at once), or `crowded` a step for each
// workgroup of the CU where they queue; the weights pass at kWeights; K split S
// ways adds kJoinRank S and the sums' traffic), but its numbers are no times: they
// were fitted to 7035 timed calls (T = 9..4096, N = 549..18432, K = 1024..16384) and
// then moved until the choices came out best (T=32 N=18432 K=7168 scores 18.8 and
// takes 31 us). Over those 216 sizes the choice is 1.9 % slower on average than the
// fastest found for each, 29 % at most (T=384 N=4096 K=7168 33.0 against 25.6 us).
// Nothing was fitted past them: at K=7168 with float output N=32001 takes 42.7 us
// for 32 tokens (the best shape pinned 40.7) and 92 for 256 (best 92), N=131072
// 168 (best 162) and 277 (best 277).
// Why these five, each where it is chosen against the best of the others (us):
// 256 x 256 T=N=4096 K=7168 119 / 134; 128 x 128 two to a CU T=800 N=18432 K=7168 132
// / 155; 128 x 128 with four buffers T=1024 N=4096 K=4096 25.5 / 30.9; 64 x 64 T=256
// N=7168 K=2048 13.1 / 14.6; 32 x 64 T=32 N=18432 K=7168 30.8 / 33.3. A shape of 256 x
// 128 was chosen for short K only and no faster there (T=3872 N=9563 K=512 90 / 84),
// though it was the fastest at some sizes that were not given to it (T=1024 N=18432
// K=7168 154 / 161).
struct TileShape {
  unsigned bt, bn, fit;
  float alone, crowded;  // a step of 128 bytes of K
};
constexpr TileShape kShapes[] = {
    {256, 256, 1, 2.081f, 1.922f}, {128, 128, 2, 0.956f, 0.532f}, {128, 128, 1, 0.499f, 0.634f},
    {64, 64, 2, 0.324f, 0.204f},   {32, 64, 3, 0.226f, 0.179f},
};
constexpr float kStart = 0.41f, kJoinRank = 0.222f;
constexpr float kWeights = 10.69e6f, kSums = 4.56e6f;  // bytes
constexpr int kShapeCount = (int)(sizeof(kShapes) / sizeof(kShapes[0]));
template <int BT, int BN, int WT, int WN, int STG>
hipError_t launch_tile(const I8Params& p, int grid, hipStream_t s) {
  return launch(i8_tile_kernel<BT, BN, WT, WN, STG>, dim3((unsigned)grid), dim3(64 * WT * WN), 0, s, p);
}

hipError_t launch_shape(int shape, const I8Params& p, int grid, hipStream_t s) {
  switch (shape) {
    case 0: return launch(i8_big_kernel, dim3((unsigned)grid), dim3(512), 0, s, p);
    case 1: return launch_tile<128, 128, 4, 2, 2>(p, grid, s);
    case 2: return launch_tile<128, 128, 2, 4, 4>(p, grid, s);
    case 3: return launch_tile<64, 64, 2, 4, 4>(p, grid, s);
    default: return launch_tile<32, 64, 1, 4, 4>(p, grid, s);
  }
}

template <bool LOW, int U>
hipError_t launch_rows(const I8Params& p, hipStream_t s) {
  const int ntiles = (p.N + 15) / 16, ttiles = (p.T + 15) / 16;
  return launch(i8_rows_kernel<LOW, U>, dim3((unsigned)(ntiles * ttiles)), dim3(64 * kRowWaves), 0, s, p);
}

// Units in flight: one load round of a wave where K is short (the workgroups of
// a CU hide each other's latency), seven from K = 4096 on. Measured with U = 1 /
// U = 7: T=1 N=4096 K=1024 3.4 / 4.7 us, T=1 N=16384 K=1024 5.5 / 11.5 us; T=8
// N=4096 K=7168 8.9 / 7.9 us, T=8 N=K=16384 60.8 / 51.3 us.
hipError_t launch_rows_for(const I8Params& p, hipStream_t s) {
  if (p.K < 4096) return p.T <= 8 ? launch_rows<true, 1>(p, s) : launch_rows<false, 1>(p, s);
  return p.T <= 8 ? launch_rows<true, 7>(p, s) : launch_rows<false, 7>(p, s);
}

}  // namespace

I8Tactic pick_i8(int T, int N, int K) {
  I8Tactic best;
  const int pinned = knob(kKnobI8Shape, -1), split = knob(kKnobI8Split, 0);
  // Few tokens, or little work: straight into registers (shape -1). Measured
  // against the best tile (us): T=8 N=K=4096 6.5 / 7.3; T=16 N=2048 K=4096 6.7 / 7.0,
  // past the border N=4096 K=8192 11.7 / 9.7; T=32 N=1024 K=2048 4.2 / 6.0, N=2048
  // K=4096 6.9 / 7.3. The borders lie below where the two meet (T=32 N=K=2048 4.3 /
  // 6.1), and for 8 tokens a very wide N is slower so (N=131072 K=7168 163 / 141).
  const long work = (long)N * K;
  const bool rows = T <= 8 || (T <= 16 && work <= 8L << 20) || (T <= 32 && work <= 2L << 20);
  if (pinned >= kShapeCount || (pinned < 0 && rows)) return best;
  const unsigned steps = std::max(1u, ((unsigned)K + 127) / 128);
  float least = 0.0f;
  for (int i = 0; i < kShapeCount; ++i) {
    if (pinned >= 0 && i != pinned) continue;
    const TileShape& sh = kShapes[i];
    // At most 2^16 x 2^12 tiles; 32-bit divisions, as this is on every call's way.
    const unsigned tiles = (((unsigned)T + sh.bt - 1) / sh.bt) * (((unsigned)N + sh.bn - 1) / sh.bn);
    // Only the tiles past the last full round of workgroups are split.
    const unsigned round = 256u * sh.fit, split_rest = tiles % round;
    const size_t bytes = (size_t)(sh.bt * sh.bn) * 4;
    for (unsigned S = 1; S <= 8; ++S) {
      if (split > 0 && S != std::min((unsigned)split, steps)) continue;
      if (S > steps) break;
      const unsigned rest = S > 1 ? split_rest : tiles, whole = tiles - rest;
      if (S > 1 && (rest == 0 || rest * S * bytes > kOpsPartBytes || rest > (unsigned)kOpsCounters)) continue;
      const unsigned m = (rest * S + 255) / 256, each = (steps + S - 1) / S;
      float score = std::max((float)((m + sh.fit - 1) / sh.fit) * (kStart + (float)each * sh.alone),
                             (float)m * (kStart + (float)each * sh.crowded));
      score += (float)(whole / 256) * (kStart + (float)steps * sh.crowded);
      score = std::max(score, ((float)N + (float)T) * (float)K / kWeights);
      if (S > 1) score += kJoinRank * (float)S + 8.0f * (float)(S * rest) * (float)(sh.bt * sh.bn) / kSums;
      if (best.shape < 0 || score < least) {
        least = score;
        best.shape = i;
        best.S = (int)S;
        best.whole = (int)whole;
        best.tiles = (int)tiles;
      }
    }
  }
  return best;
}

hipError_t launch_i8(const I8Params& q, const I8Tactic& tac, hipStream_t s) {
  I8Params p = q;
  p.S = tac.S;
  p.whole = tac.whole;
  const int per = p.out_f32 ? 16 : 8;  // bytes of four outputs
  p.c_quads = p.c_stride % per == 0;
  if (tac.shape < 0) return launch_rows_for(p, s);
  return launch_shape(tac.shape, p, tac.whole + (tac.tiles - tac.whole) * tac.S, s);
}

}  // namespace skg
