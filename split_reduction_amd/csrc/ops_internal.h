// Internal interface between the C-ABI layer (ops_api.hip) and the kernels of
// the operators around the layers and the head.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace skg {

struct NormParams {
  const uint8_t* x;      // bf16 [T, H]
  const uint8_t* r;      // bf16 [T, H] or null
  const uint8_t* g;      // bf16 [H] or null
  uint8_t* r_out;        // bf16 [T, H] or null
  uint8_t* y;            // bf16 or 8-bit codes [T, H]
  float* y_scale;        // [T] (8-bit codes)
  size_t x_stride, r_stride, r_out_stride, y_stride;  // bytes
  int T, H;
  float eps;
};

struct I8Params {
  const uint8_t* w;      // int8 [N, K]
  const uint8_t* x;      // int8 [T, K]
  const float* w_scale;  // [N]
  const float* x_scale;  // [T]
  uint8_t* c;            // bf16 or float [T, N]
  size_t w_stride, x_stride, c_stride;  // bytes
  int T, N, K;
  int out_f32;
  int c_quads;    // four outputs of a row are aligned for one store
  int S, whole;   // workgroups that split K of each tile past the first `whole`
  uint8_t* part;  // their sums [tiles - whole, S, tile] (S > 1)
  uint32_t* cnt;  // one arrival counter a tile, kOpsCounterStride words apart
};

// The workspace: partial results, then arrival counters, a 128-byte line each.
constexpr size_t kOpsPartBytes = (size_t)64 << 20;
constexpr int kOpsCounterStride = 32;
constexpr int kOpsCounters = 8192;

// How a call is run: tile shape (-1: operands straight into registers), and K
// split S ways in the tiles past the first `whole`.
struct I8Tactic {
  int shape = -1, S = 1, whole = 0, tiles = 0;
};
I8Tactic pick_i8(int T, int N, int K);

struct LogprobParams {
  const uint8_t* logits;  // bf16 or float [T, V]
  const int64_t* tokens;  // [T], null where logprob is
  float *logprob, *entropy, *lse;  // [T], each may be null
  float* top_logprob;     // [T, k]
  int64_t* top_ids;       // [T, k]
  size_t stride;          // bytes between rows of logits
  int T, V, k;
  float scale;
  int parts, per;  // workgroups a row, vectors a workgroup
  uint8_t* part;   // their results [T, parts], kLogprobPart bytes each (parts > 1)
  uint32_t* cnt;   // one arrival counter a row
};
constexpr size_t kLogprobPart = 16 + 64 * 8;  // three sums, the best 64 keys
int logprob_parts(int T, int V, bool f32, int* per);

struct LogprobGradParams {
  const uint8_t* logits;
  const int64_t* tokens;  // null: no logprob term
  const float *lse, *entropy, *g_logprob, *g_entropy;
  uint8_t* d_logits;
  size_t stride, d_stride;
  int T, V;
  unsigned parts;  // workgroups a row
  float scale;
};

// A cache's scale as the division by it needs it: scale = 2^e b, 1 <= b < 2.
struct CodeScale {
  float up, b, inv, most;  // 2^-e, b, 1 / b, 448 b
};

struct RopeParams {
  const uint8_t *q, *k, *v;  // bf16 rows of heads; k, v null where Hkv is 0
  const uint8_t *gq, *gk;    // bf16 [D] or null: no norm
  const float* freq;         // [rot / 2]
  const int64_t* pos;        // [T]
  const int64_t* slots;      // [T], below 0: not stored
  uint8_t *q_out, *kc, *vc;
  size_t q_stride, k_stride, v_stride, q_out_stride;   // bytes between tokens
  size_t page_stride, slot_stride, head_stride;        // bytes, of both caches
  int64_t n_slots;
  int T, Hq, Hkv, D, rot, page_shift;
  float eps, amplitude, by_d;  // by_d: 1 / D
  CodeScale k_by, v_by;
  int tokens, per;  // tokens of a workgroup; heads of one (blockIdx.y takes the next)
};

struct AttnParams {
  const uint8_t* q;        // bf16 [T, Hq, D]
  const uint8_t *kc, *vc;  // bf16 or E4M3 pages
  const int32_t* table;    // [B, max_pages]
  const int32_t* kv_len;   // [B]
  const int32_t* q_start;  // [B + 1]
  uint8_t* o;              // bf16 [T, Hq, D]
  float* lse;              // [T, Hq] or null
  size_t q_stride, o_stride, table_stride;  // bytes
  uint32_t page_stride, slot_stride, head_stride;
  int T, B, max_q, Hq, Hkv, G, n_pages, page_shift, max_len, window;
  float c, v_scale;  // scale * k_scale / log 2
  int few;           // rows (new tokens x G) of a sequence that attn_few_kernel takes
  int S;             // attn_rows_kernel: workgroups that split a tile's keys
  uint8_t* part;     // their results
  uint32_t* cnt;     // arrival counters, kOpsCounterStride words apart
};

// Tiles of 128 rows of a key head in sequences of more than 32, at most.
int64_t attention_tiles(int T, int B, int max_q, int G);
// Of all key heads: a launch of a workgroup of 256 threads for each, and of 512 beside
// them, stays below the 2^32 threads that a grid may have. (Where keys are split there
// are less workgroups than counters times 64.)
constexpr int64_t kMostTiles = ((int64_t)1 << 24) - 512;

hipError_t launch_rope(const RopeParams& p, bool inter, bool codes, hipStream_t s);
hipError_t launch_attention(const AttnParams& p, int D, bool codes, hipStream_t s);
hipError_t launch_logprobs(const LogprobParams& p, bool f32, hipStream_t s);
hipError_t launch_logprobs_grad(LogprobGradParams p, bool f32, hipStream_t s);
hipError_t launch_i8(const I8Params& p, const I8Tactic& t, hipStream_t s);
hipError_t launch_rmsnorm(const NormParams& p, int out_format, hipStream_t s);

// hip_fail and the retained error live with the other entry points (api.hip).
int hip_fail(hipError_t e);
// Frees the workspaces of ops_api.hip; part of skgemm_release.
int release_ops_workspaces();

}  // namespace skg
