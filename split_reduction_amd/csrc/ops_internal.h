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

hipError_t launch_logprobs(const LogprobParams& p, bool f32, hipStream_t s);
hipError_t launch_logprobs_grad(LogprobGradParams p, bool f32, hipStream_t s);
hipError_t launch_i8(const I8Params& p, const I8Tactic& t, hipStream_t s);
hipError_t launch_rmsnorm(const NormParams& p, int out_format, hipStream_t s);

// hip_fail and the retained error live with the other entry points (api.hip).
int hip_fail(hipError_t e);
// Frees the workspaces of ops_api.hip; part of skgemm_release.
int release_ops_workspaces();

}  // namespace skg
