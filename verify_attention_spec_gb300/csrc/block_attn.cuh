// Attention over block-scaled pages: what paged_attn.cu hands to block_attn.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn_plan.cuh"

namespace vas {
namespace battn {

using attn::Divisor;

constexpr int kMaxRows = 32;  // query rows of a unit

// A partial of a cut unit: CTA k's first (a unit that began before its share) is record 2 k, its
// last (a unit that goes on behind it) 2 k + 1.
struct Record {
  int32_t head;                // KV head, or -1: no partial
  int32_t r0, rows, row0;      // first row, rows, the sequence's first query token
  int32_t begins, goes_on;     // from the unit's first tile; not to its last
  int32_t empty;               // no tile falls into the share
  int32_t pad;
};

struct Args {
  const void* q;
  void* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* query_lens;
  const uint64_t* tree_mask;
  const float* k_scale;
  const float* v_scale;
  int32_t B, T, Hq, Hkv, G, P, num_pages, maxp;
  float scale_log2;  // softmax scale * log2(e)
  int32_t* err;
  // Filled by launch().
  int32_t log2P, max_rows;
  int32_t parts, part_rows;  // parts of a group of heads, and heads of a part
  Divisor by_G;
  Record* records;
  float* part_lse;
  float* part_o;
};

size_t workspace_bytes(int head_dim);
// Returns a status code; the workspace holds workspace_bytes(head_dim).
int launch(Args a, const void* k_pages, const void* v_pages, int head_dim, bool fp8, void* workspace,
           cudaStream_t stream);

}  // namespace battn
}  // namespace vas
