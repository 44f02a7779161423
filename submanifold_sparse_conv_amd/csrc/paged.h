// Operators over a paged key-value cache (internal): launchers and argument structs.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "tokens.h"
#include "tr_sparseconv.h"

namespace trsc {

constexpr int kMinPageLog2 = 3, kMaxPageLog2 = 16;  // a wave's copy of up to 8 rows to LDS lies in one page

// The pages of a call; strides in elements.
struct PoolRef {
  void *k, *v;
  int64_t kps, kss, khs, vps, vss, vhs;  // page, slot and head strides
  int32_t pages;
  int log2;                // of the page size
  const int32_t* table;    // [batch, table_pages], row stride table_ts
  int64_t table_ts;
  int32_t table_pages;
  const int32_t* len;      // [batch]
};

// A call's sequences: cu [batch + 1], or null: each has `each` tokens of q.
struct Packed {
  const int32_t* cu;
  int batch;
  int32_t each;
};

struct AppendArgs {
  NormSide q, k;  // x, and q's y
  HeadsRef v;
  const int32_t* pos;
  int64_t pos_ts;
  const float* freqs;
  int c1, c2, c3;
  int interleaved, norm;
  float eps;
  int64_t tokens;
  int dim, dtype;
  PoolRef pool;
  Packed seqs;
};
hipError_t launch_norm_rope_append(const AppendArgs& a, hipStream_t st);

struct PagedArgs {
  HeadsRef q, o;
  PoolRef pool;
  Packed seqs;
  const int32_t* prefix;  // pages of the keys before every sequence's own
  int32_t prefix_len;
  float* lse;   // [hq, nq] or null
  float* part;  // workspace
  int32_t nq;
  int hq, hk, dim, dtype;
  int32_t left, right, sinks;
  float scale;
};
// shorts: a workgroup an item of 32 rows; whole_tiles: of 128; tokens, tiles: the items' units dealt to the chip's waves
// or workgroups; mixed: the prefix's to workgroups, the others to waves.
enum class PagedForm { shorts, whole_tiles, tokens, tiles, mixed };
struct PagedPlan {
  PagedForm form;
  int grid;
  size_t part_floats;  // of the workspace
  bool fits;           // the work list's numbers
};
PagedPlan plan_paged_attention(const PagedArgs& a);
hipError_t launch_paged_attention(const PagedArgs& a, const PagedPlan& plan, hipStream_t st);

}  // namespace trsc
