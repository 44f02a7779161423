// Operators over voxel tokens (internal): per-head norm with position rotation,
// windowed attention with sinks. Launchers and argument structs.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "tr_sparseconv.h"

namespace trsc {

// Error text of the C ABI (api.hip): records the message, returns the code.
int fail(int code, const char* fmt, ...);
int hip_fail(hipError_t e, const char* where);

constexpr int kMaxHeadDim = 128;

// ---------------------------------------------------------------------------
// Norm and rotation. One side (queries or keys) of a call; strides in elements.
// ---------------------------------------------------------------------------
struct NormSide {
  const void* x;
  int64_t xts, xhs;
  const void* dy;  // backward only
  int64_t dts, dhs;
  void* y;  // forward: rotated output; backward: dx
  int64_t yts, yhs;
  const float* gain;  // null: no gain
  int gain_rows;      // 1 (shared by the heads) or heads
  float* dgain;       // backward, [gain_rows, dim]
  int heads;
};
struct NormArgs {
  NormSide q, k;
  const int32_t* pos;  // [tokens, axes], row stride pos_ts
  int64_t pos_ts;
  const float* freqs;  // [dim / 2]
  int c1, c2, c3;      // pairs [0, c1) turn with axis 0, [c1, c2) axis 1, [c2, c3) axis 2, the rest not
  int interleaved;
  float eps;
  int64_t tokens;
  int dim, dtype;
  float* partials;  // backward: norm_rope_partials(...) floats
};
hipError_t launch_norm_rope(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_rope_backward(const NormArgs& a, hipStream_t st);
int64_t norm_rope_partials(int64_t tokens, int heads, int dim);

// ---------------------------------------------------------------------------
// Windowed attention.
// ---------------------------------------------------------------------------
struct HeadsRef {
  const void* p;
  int64_t ts, hs;  // token and head strides, elements
};
struct AttnArgs {
  HeadsRef q, k, v, o, dout;  // o: output of the forward, input of the backward
  void *dq, *dk, *dv;         // contiguous [tokens, heads, dim]
  float* lse;                 // [q_heads, tokens_q]
  float2* stat;               // backward workspace: (shifted base-2 lse, delta) of row r = token, head of the group of
                              // each kv head, [kv_heads, tokens_q * group]
  int32_t* score_exp;         // backward workspace, fp16: exponent of the largest score gradient of every 32 rows
  float* part;                // forward splits: partial outputs, then their statistics
  float* sink_part;           // backward workspace: the sinks' partial gradients
  float* dkv_part;            // backward workspace: dk, dv of the parts of the row walk
  const int32_t *cu_q, *cu_k, *k_len;
  int batch;
  int32_t nq, nk;  // tokens of q and of k, v
  int hq, hk, dim, dtype;
  int32_t left, right, sinks;  // left, right <= kFar
  float scale;
};
constexpr int32_t kFar = (1 << 30) - 2;  // an unlimited window side; tokens <= 2^30, so sums of the two fit
constexpr int kMaxSinks = 128;           // one key tile of the backward
struct AttnPlan {
  bool token_form;  // few rows a sequence: the four waves of a workgroup share 32 rows and split the keys
  int splits;       // parts of the key axis in different workgroups
  size_t part_floats;
};
AttnPlan plan_attention(const AttnArgs& a);
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t st);
// Workspace of the backward, in floats (or as many 32-bit integers): the rows' statistics and, of fp16, their score
// gradients' exponents, the sinks' partials, the parts'.
size_t attention_backward_stat_floats(const AttnArgs& a);
size_t attention_backward_exponents(const AttnArgs& a);
size_t attention_backward_sink_floats(const AttnArgs& a);
size_t attention_backward_part_floats(const AttnArgs& a);
hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t st);

}  // namespace trsc
