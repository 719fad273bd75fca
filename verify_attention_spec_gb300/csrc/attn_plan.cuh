// What the planner of paged attention leaves in the workspace, shared by the attention
// kernels of paged_attn.cu and the shared-prefix kernel of prefix_attn.cu.
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>

namespace vas {
namespace attn {

struct SeqPlan {
  int32_t qrow0;         // first row of q / out / lse
  int32_t nsplit;        // partials of a row; 0 = nothing to compute (invalid or no query);
                         // negative: behind a shared prefix, merged by merge_shared_kernel
                         // and not by the last split
  int32_t partial_base;  // first partial row (nsplit > 1)
  int32_t len;           // L
  int32_t qlen;          // ql
  int32_t flags;         // kSeqInvalid
  int32_t nrb;           // row blocks
  int32_t item0;         // first work item (split 0, row block 0)
};

struct Item {
  int32_t seq, page_begin, page_end, split_rb;  // split << kRbBits | row block (| kItemPrecise)
};

struct PlanHeader {
  int32_t n_items;
  int32_t work_counter;
  int32_t chunk_pages;
  int32_t n_partial_rows;
  // Shared-prefix calls: groups that are shared, and how their work is dealt out.
  int32_t n_groups;
  int32_t span, share;
};

// A group of sequences whose shared pages are computed once.  Its rows, of one KV head, are
// its members' rows one after the other: row r is query token qrow0 + r / G, query head
// head * G + r % G.
//
// The work of all groups is one line of `span` units: a group's KV heads one behind the other
// from `base` on, head_units() each; of a head its blocks of kPrefixRows rows, a block `tiles`
// tiles of kPrefixTile tokens.  A tile takes two units, or one in a last block of at most
// kPrefixRows / 2 rows.  CTA k takes the units k * share .. (k + 1) * share - 1, so a block is
// computed in pieces by the CTAs its units fall to, piece j by the (j + 1)th of them.  share,
// base and head_units() are even, so no tile is cut.
struct PrefixGroup {
  int32_t qrow0;       // first query token
  int32_t rows;        // G * query tokens
  int32_t leader;      // sequence whose table names the shared pages
  int32_t pages;       // shared pages
  int32_t parts;       // partials of a row: the most pieces a block is cut into
  int32_t seq0, seq1;  // members
  int32_t tiles;       // of a block
  int32_t full, tail;  // blocks of a head whose tiles take two units; 1: and one of one unit
  int32_t base;
  __device__ __forceinline__ uint32_t head_units() const {
    return ((uint32_t)(2 * full + tail) * (uint32_t)tiles + 1) & ~1u;
  }
};
constexpr int kPrefixRows = 256;  // rows of a block
constexpr int kPrefixTile = 128;  // tokens of a tile

__host__ __device__ __forceinline__ int64_t prefix_blocks(int64_t R) {
  return (R + kPrefixRows - 1) / kPrefixRows;
}

// Partial rows of a sequence: [split][KV head][G * ql], from partial_base on.
__device__ __forceinline__ size_t partial_index(const SeqPlan& sp, int Hkv, int G, int split,
                                                int head, int r) {
  return (size_t)sp.partial_base + ((size_t)split * Hkv + head) * ((size_t)G * sp.qlen) + r;
}

// Division of 0 <= n < 2^31 by a divisor known to the host (Granlund and Montgomery, "Division
// by invariant integers using multiplication", PLDI 1994): with 2^(l-1) < d <= 2^l and
// m = floor(2^(31 + l) / d) + 1, n / d = floor(n m / 2^(31 + l)).
struct Divisor {
  uint32_t d, m, shift;
  explicit Divisor(uint32_t divisor) : d(divisor), shift(31) {
    while ((1ull << (shift - 31)) < d) ++shift;
    m = (uint32_t)((1ull << shift) / d + 1);
  }
  Divisor() = default;
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> shift);
  }
};

struct PrefixArgs {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const SeqPlan* seqplan;
  const int32_t* row0;  // [B + 1] first query token of each sequence
  const PrefixGroup* groups;
  const PlanHeader* header;
  float* part_o;
  float* part_lse;
  int32_t Hq, Hkv, G, maxp, num_pages, P;
  Divisor by_G;
  float scale_log2;  // softmax scale * log2(e)
  int32_t* err;
};

// The shared prefixes of a planned call: partial rows of every member (prefix_attn.cu).
// mk, mv: bf16 pools, boxes of one 64-column half of one page of one KV head; code pools,
// boxes of one page of one KV head.  Returns a status code; kv_dtype VAS_BF16,
// VAS_FP8_E4M3 or VAS_INT8.
int launch_prefix(const CUtensorMap& mk, const CUtensorMap& mv, const PrefixArgs& args,
                  int head_dim, int kv_dtype, void* stream);

}  // namespace attn
}  // namespace vas
