// Attention over shared prefixes (sm_103a): every query row of a group of sequences against
// the pages that all of them share, read once for the group.
//
// The rows of a group see all of its shared positions, so there is no mask: for a row q and
// the positions x of one split,
//     m = max_x s_x,  l = sum_x e^(s_x - m),  O = sum_x e^(s_x - m) v_x / l,  lse = m + ln l,
// written as one of the row's partials; the members' own splits (paged_attn.cu) and these
// are merged by lse there.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/vas.h"
#include "attn_plan.cuh"
#include "device_util.cuh"
#include "vas_internal.h"

namespace vas {
namespace attn {
namespace {

// The sequence that owns query token t of a group: the last member whose first token is at
// or below t (members without tokens start where their successor does).
__device__ __forceinline__ int member_of(const PrefixArgs& a, const PrefixGroup& g, int32_t t) {
  int lo = g.seq0, hi = g.seq1 - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.row0[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int KV>
__device__ __forceinline__ float kv_value(const void* base, size_t i) {
  if constexpr (KV == VAS_BF16) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  } else if constexpr (KV == VAS_FP8_E4M3) {
    return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(base)[i]);
  } else {
    return static_cast<float>(static_cast<const int8_t*>(base)[i]);
  }
}

// A piece of a block: what one CTA computes of it at a time.
struct Piece {
  PrefixGroup g;
  int head, r0, rows;      // KV head, first row and rows of the block
  int page_begin, n_tiles, tokens;  // of the group's shared pages
  int part;                // the piece's partial ...
  int empty;               // ... and how many behind it stay empty (O 0, lse -inf)
};

// The pieces of a CTA's share, in order.  Every warp walks them by itself.
struct Pieces {
  int64_t x, end, share;
  int e;
  __device__ __forceinline__ Pieces(const PrefixArgs& a, int lane) {
    share = a.header->share;
    x = (int64_t)blockIdx.x * share;
    end = min(x + share, a.header->span);
    e = 0;
    // The last entry whose base is at or below x, 32 entries at a time.
    const int n = a.header->n_groups;
    for (int s = 0; s < n; s += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, s + lane < n && a.groups[s + lane].base <= x);
      if (m == 0) break;
      e = s + 31 - __clz(m);
      if (m != 0xffffffffu) break;
    }
  }
  // False at the end of the share.  A group's span may end in one unit of padding.
  __device__ __forceinline__ bool next(const PrefixArgs& a, Piece& p) {
    while (x < end) {
      p.g = a.groups[e];
      const int64_t len = (int64_t)p.g.tiles * p.g.weight;
      const int64_t local = x - p.g.base, block = local / len;
      if (block >= p.g.blocks) {
        ++e;
        x = p.g.base + ((len * p.g.blocks + 1) & ~1ll);
        continue;
      }
      const int64_t first = p.g.base + block * len, stop = min(end, first + len);
      const int per_head = p.g.blocks / a.Hkv;
      p.head = (int)(block / per_head);
      p.r0 = (int)(block % per_head) * kPrefixRows;
      p.rows = min(kPrefixRows, p.g.rows - p.r0);
      const int t0 = (int)((x - first) / p.g.weight), t1 = (int)((stop - first) / p.g.weight);
      p.page_begin = t0 * (kPrefixTile / a.P);
      p.n_tiles = t1 - t0;
      p.tokens = min(p.g.pages * a.P, t1 * kPrefixTile) - t0 * kPrefixTile;
      p.part = (int)(blockIdx.x - first / share);
      p.empty = stop == first + len ? p.g.parts - 1 - p.part : 0;
      x = stop;
      return true;
    }
    return false;
  }
};

// Partial row of row r of a group, for partial `part` of its shared pages.
__device__ __forceinline__ size_t part_row(const PrefixArgs& a, const Piece& p, int r, int part) {
  const int t = p.g.qrow0 + r / a.G;
  const SeqPlan sp = a.seqplan[member_of(a, p.g, t)];
  return partial_index(sp, a.Hkv, a.G, sp.nsplit - p.g.parts + part, p.head,
                       (t - sp.qrow0) * a.G + r % a.G);
}
// Partial rows from one partial of a row to the next.
__device__ __forceinline__ size_t part_step(const PrefixArgs& a, const Piece& p, int r) {
  const int t = p.g.qrow0 + r / a.G;
  return (size_t)a.Hkv * ((size_t)a.G * a.seqplan[member_of(a, p.g, t)].qlen);
}

// One warp per row, CUDA-core arithmetic.
template <int D, int KV>
__global__ void __launch_bounds__(256) prefix_simple_kernel(const PrefixArgs a) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float qs[8][D];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  if (a.header->n_groups == 0) return;
  Pieces it(a, lane);
  Piece x;
  while (it.next(a, x)) {
    const int32_t* bt = a.block_table + (size_t)x.g.leader * a.maxp + x.page_begin;
    for (int rr = warp; rr < x.rows; rr += 8) {
      const int r = x.r0 + rr;
      const int t = x.g.qrow0 + r / a.G;
      const int hh = x.head * a.G + r % a.G;
      const __nv_bfloat16* q =
          static_cast<const __nv_bfloat16*>(a.q) + ((size_t)t * a.Hq + hh) * D;
      __syncwarp();
      for (int e = 0; e < E; ++e) qs[warp][lane + 32 * e] = __bfloat162float(q[lane + 32 * e]);
      __syncwarp();
      float acc[E] = {}, m = -INFINITY, l = 0.f;
      bool bad = false;
      for (int y0 = 0; y0 < x.tokens; y0 += 32) {
        const int y = y0 + lane;
        int page = -1;
        float s = -INFINITY;
        if (y < x.tokens) {
          page = bt[y / a.P];
          if (page < 0 || page >= a.num_pages) {
            bad = true;
            page = -1;
          } else {
            const size_t at = (((size_t)page * a.P + y % a.P) * a.Hkv + x.head) * D;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(qs[warp][d], kv_value<KV>(a.k_pages, at + d), dot);
            if constexpr (KV != VAS_BF16)
              dot *= a.k_scale[((size_t)page * a.Hkv + x.head) * a.P + y % a.P];
            s = dot * a.scale_log2;
          }
        }
        float mx = s;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - mu);
        float p = exp2f(s - mu);
        float ps = p;
        for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l = l * f + ps;
        m = mn;
        if constexpr (KV != VAS_BF16) {
          if (page >= 0) p *= a.v_scale[((size_t)page * a.Hkv + x.head) * a.P + y % a.P];
        }
        for (int e = 0; e < E; ++e) acc[e] *= f;
        for (int j = 0; j < 32 && y0 + j < x.tokens; ++j) {
          const float pj = __shfl_sync(0xffffffffu, p, j);
          const int pg = __shfl_sync(0xffffffffu, page, j);
          if (pg < 0) continue;
          const size_t at = (((size_t)pg * a.P + (y0 + j) % a.P) * a.Hkv + x.head) * D;
          for (int e = 0; e < E; ++e)
            acc[e] = fmaf(pj, kv_value<KV>(a.v_pages, at + lane + 32 * e), acc[e]);
        }
      }
      bad = __any_sync(0xffffffffu, bad);
      const size_t row = part_row(a, x, r, x.part);
      for (int e = 0; e < E; ++e)
        a.part_o[row * D + lane + 32 * e] = bad ? NAN : (l > 0.f ? acc[e] / l : 0.f);
      if (lane == 0) {
        a.part_lse[row] = bad ? NAN : (m + log2f(l)) * 0.6931471805599453f;
        if (bad) atomicOr(a.err, VAS_DEV_BAD_PAGE);
      }
      for (int k = 1; k <= x.empty; ++k) {
        const size_t none = row + k * part_step(a, x, r);
        for (int e = 0; e < E; ++e) a.part_o[none * D + lane + 32 * e] = 0.f;
        if (lane == 0) a.part_lse[none] = -INFINITY;
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// bf16 pages: both products on tcgen05
// ------------------------------------------------------------------------------------
// A CTA takes its pieces one at a time and walks each in tiles of 128 tokens.  Two streams
// of S = Q K^T, softmax, O += P V run against each other, so that the tensor cores compute
// one stream's products while the other stream's threads are in their softmax:
//   more than 128 rows: stream s holds rows 128 s .. 128 s + 127, every tile feeds both;
//   otherwise both hold the same rows and take the tiles in turn, and their two results are
//   merged in shared memory at the end of the piece.
// A stream is 256 threads: thread r of each half owns row r, TMEM lane r, with 64 of the
// tile's 128 scores; the halves exchange their maxima through shared memory.  (With one
// thread a row, two warps a scheduler left the issue slots 72 % idle and the tensor cores
// at 40 %.)  The scores come to registers and go back as bf16 pairs over the first columns
// of S, which are the A operand of the second product from there, so P never passes through
// shared memory.  TMEM: S 2 x 128, O 2 x D columns.  Shared memory: the query tiles and a
// ring of K and V tiles, 128-byte swizzled as the TMA boxes land.  A producer warp streams
// the pages, an MMA warp issues.
constexpr int kTile = kPrefixTile;          // tokens of a tile, rows of a stream
constexpr int kStreamThreads = 256, kStreamWarps = kStreamThreads / 32;
constexpr int kProducerWarp = 2 * kStreamWarps, kMmaWarp = kProducerWarp + 1;
constexpr int kPrefixThreads = 640;  // two warps idle: registers move by groups of four warps
// Registers a thread: what the launch gives is split between the streams, whose scores live
// in registers, and the other four warps.
constexpr int kStreamRegs = 104, kOtherRegs = 64, kLaunchRegs = 96;
static_assert(2 * kStreamThreads * kStreamRegs + 128 * kOtherRegs <= kPrefixThreads * kLaunchRegs,
              "setmaxnreg draws on the registers of the launch");
constexpr float kRebase = 8.f;  // a row's reference maximum may trail by this (log2 units)

template <int D>
struct PSmem {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kTile * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // one operand of a tile, a query tile
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kRingOff = 2 * kTileBytes;
  // [stream][half][row]: maxima, at the end of a piece the sums
  static constexpr int kStatOff = kRingOff + kSlots * kTileBytes;
  static constexpr int kBarOff = kStatOff + 4 * kTile * 4;
  // full[kSlots], empty[kSlots], s_full[2], p_full[2], o_full[2], q_full[2], fin | TMEM base
  static constexpr int kBytes = kBarOff + (2 * kSlots + 9) * 8 + 16;
  static constexpr int kDynBytes = kBytes;
  static_assert(kDynBytes <= 227 * 1024, "shared memory of one CTA");
  static_assert(kTile * D * 4 <= 2 * kTileBytes, "stream 1's O fits over the query tiles");
};

// 64 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,"
      "%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,"
      "%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]),
        "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]),
        "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]),
        "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

// The warps beside the streams hand registers over (every warp of the group executes it).
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

template <int D, int P>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const PrefixArgs a) {
  using S = PSmem<D>;
  constexpr int kSlots = S::kSlots;
  constexpr int kPages = kTile / P;  // pages of a tile
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle counts from 1024 bytes
  uint8_t* ring = smem + S::kRingOff;
  float* stat = reinterpret_cast<float*>(smem + S::kStatOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarOff);
  uint64_t* empty = full + kSlots;
  uint64_t* s_full = empty + kSlots;  // S of the stream is in TMEM, its last O product done
  uint64_t* p_full = s_full + 2;      // P of the stream is in TMEM
  uint64_t* o_full = p_full + 2;      // the stream's O of the unit is complete
  uint64_t* q_full = o_full + 2;      // the stream's query tile is staged
  uint64_t* fin = q_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kStreamWarps);
      mbar_init(&o_full[s], 1);
      mbar_init(&q_full[s], kStreamWarps);
    }
    mbar_init(fin, 1);
    mbar_fence_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
  }
  pdl_wait_prior_grid();  // the plan of this call is complete and visible
  pdl_launch_dependents();
  // The whole CTA, before it holds anything.
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) atomicOr(a.err, VAS_DEV_TIMEOUT);
    return;
  }
  if (a.header->n_groups == 0 || (int64_t)blockIdx.x * a.header->share >= a.header->span) return;
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_s = tmem, tmem_o = tmem + 2 * kTile;
  bool ok = true;

  if (warp == kProducerWarp) {
    // ------------------------------ producer ------------------------------
    give_registers();
    // Lane e of a tile's boxes: page e % kPages, column half e / kPages.  The order of the
    // ring is the order the MMA warp asks in: K first, by one tile (both streams) or two.
    static_assert(kPages * S::kHalves <= 32, "one box a lane");
    const uint64_t pol_once = l2_policy_evict_first(), pol_again = l2_policy_evict_normal();
    uint32_t fill = 0;
    Pieces it(a, lane);
    Piece x;
    while (ok && it.next(a, x)) {
      const bool both = x.rows > kTile;
      const int32_t* bt = a.block_table + (size_t)x.g.leader * a.maxp + x.page_begin;
      const int n_pages = x.tokens / P;
      const uint64_t pol = x.g.rows > kPrefixRows ? pol_again : pol_once;
      const int e_page = lane % kPages, e_half = lane / kPages;
      auto load = [&](const CUtensorMap* map, int tile) {
        const int slot = fill % kSlots;
        ok = ok && mbar_wait(&empty[slot], ((fill / kSlots) & 1) ^ 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          return;
        }
        const int pg = tile * kPages + e_page;
        int32_t id = -1;
        if (e_half < S::kHalves && pg < n_pages) id = bt[pg];
        const bool mine = id >= 0 && id < a.num_pages;  // bad pages: the rows end as NaN
        const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], boxes * (P * 128));
        __syncwarp();
        if (mine)
          tma_load_4d(ring + slot * S::kTileBytes + e_half * S::kHalfBytes + e_page * (P * 128), map,
                      &full[slot], 0, id * P, e_half, x.head, pol);
        __syncwarp();
        ++fill;
      };
      const int lead = min(both ? 1 : 2, x.n_tiles);
      for (int t = 0; t < lead && ok; ++t) load(&tm_k, t);
      for (int j = 0; j < x.n_tiles && ok; ++j) {
        load(&tm_v, j);
        if (ok && j + lead < x.n_tiles) load(&tm_k, j + lead);
      }
    }
    // Every copy this warp issued has landed before the CTA can exit.
    for (uint32_t f = fill > kSlots ? fill - kSlots : 0; f < fill; ++f)
      mbar_wait(&full[f % kSlots], (f / kSlots) & 1);
  } else if (warp == kMmaWarp) {
    // ------------------------------ MMA warp ------------------------------
    give_registers();
    // Per stream: S of its next tile is issued right behind the O product of the last one
    // (which is the last reader of the P it overwrites; products run in issue order), so
    // s_full also says that O may be rescaled.
    constexpr uint32_t kIdS = umma_idesc_bf16(128, kTile, false, false);
    constexpr uint32_t kIdO = umma_idesc_bf16(128, D, false, true);
    constexpr uint32_t kHi = umma_desc_hi_sw128(1024);
    const uint32_t q_lo = umma_desc_lo(smem_u32(smem), 16);
    const uint32_t ring_k = umma_desc_lo(smem_u32(ring), 16);
    const uint32_t ring_v = umma_desc_lo(smem_u32(ring), S::kHalfBytes);
    uint32_t use = 0, n_p[2] = {0, 0}, n_q = 0;
    auto landed = [&](uint32_t f) {
      ok = ok && mbar_wait_fast(&full[f % kSlots], (f / kSlots) & 1);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto scores = [&](int st, uint32_t f) {  // S of stream st from the K tile of fill f
      if (lane == 0) {
        tc_fence_after();
        const uint32_t k_lo = ring_k + (((f % kSlots) * S::kTileBytes) >> 4);
        const uint32_t a_lo = q_lo + ((st * S::kTileBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t step = ((ks >> 2) * S::kHalfBytes + (ks & 3) * 32) >> 4;
          umma_bf16_lh(tmem_s + st * kTile, a_lo + step, k_lo + step, kHi, kIdS, ks > 0);
        }
        umma_commit(&s_full[st]);
      }
      __syncwarp();
    };
    auto outputs = [&](int st, uint32_t f, int tokens, bool first) {  // O += P V
      ok = ok && mbar_wait_fast(&p_full[st], n_p[st] & 1);
      ok = __all_sync(0xffffffffu, ok);
      ++n_p[st];
      landed(f);
      if (!ok) return;
      if (lane == 0) {
        tc_fence_after();
        const uint32_t v_lo = ring_v + (((f % kSlots) * S::kTileBytes) >> 4);
        const uint32_t p = tmem_s + st * kTile, o = tmem_o + st * D;
        if (tokens == kTile) {
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            umma_ts_lh(o, p + 8 * ks, v_lo + ((ks * 2048) >> 4), kHi, kIdO, !first || ks > 0);
        } else {  // the V rows of pages that were not loaded are not read
          for (int ks = 0; ks < tokens / 16; ++ks)
            umma_ts_lh(o, p + 8 * ks, v_lo + ((ks * 2048) >> 4), kHi, kIdO, !first || ks > 0);
        }
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (lane == 0) umma_commit(bar);
      __syncwarp();
    };
    Pieces it(a, lane);
    Piece x;
    for (; ok && it.next(a, x); ++n_q) {
      const int n = x.n_tiles, all = x.tokens;
      for (int st = 0; st < 2 && ok; ++st) {
        ok = mbar_wait(&q_full[st], n_q & 1);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (x.rows > kTile) {
        landed(use);
        if (!ok) break;
        scores(0, use);
        scores(1, use);
        commit(&empty[use % kSlots]);
        ++use;
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t fv = use++;
          const bool more = j + 1 < n;
          const uint32_t fk = more ? use++ : 0;
          const int tokens = min(kTile, all - j * kTile);
          for (int st = 0; st < 2 && ok; ++st) {
            outputs(st, fv, tokens, j == 0);
            if (!ok) break;
            if (st == 1) commit(&empty[fv % kSlots]);
            if (more) {
              landed(fk);
              if (!ok) break;
              scores(st, fk);
              if (st == 1) commit(&empty[fk % kSlots]);
            } else {
              commit(&o_full[st]);
            }
          }
        }
      } else {
        for (int t = 0; t < min(2, n) && ok; ++t) {
          landed(use);
          if (!ok) break;
          scores(t, use);
          commit(&empty[use % kSlots]);
          ++use;
        }
        for (int j = 0; j < n && ok; ++j) {
          const int st = j & 1;
          const uint32_t fv = use++;
          const bool more = j + 2 < n;
          const uint32_t fk = more ? use++ : 0;
          outputs(st, fv, min(kTile, all - j * kTile), j < 2);
          if (!ok) break;
          commit(&empty[fv % kSlots]);
          if (more) {
            landed(fk);
            if (!ok) break;
            scores(st, fk);
            commit(&empty[fk % kSlots]);
          } else {
            commit(&o_full[st]);
          }
        }
      }
    }
    // Tensor memory is freed only after every product this warp issued has completed.
    commit(fin);
    if (!mbar_wait(fin, 0)) ok = false;
  } else if (warp < 2 * kStreamWarps) {
    // ------------------------------ softmax streams ------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStreamRegs));
    const int st = warp / kStreamWarps, half = (warp >> 2) & 1;
    const int row = threadIdx.x & (kTile - 1), tid = threadIdx.x & (kStreamThreads - 1);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem_s + lanes + st * kTile, o_at = tmem_o + lanes + st * D + half * (D / 2);
    float* const my_stat = stat + (2 * st + half) * kTile + row;
    const float* const other_stat = stat + (2 * st + 1 - half) * kTile + row;
    const float c = a.scale_log2;
    uint32_t n_s = 0, n_o = 0;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (ok) ok = mbar_wait_fast(bar, phase & 1);
      ok = __all_sync(0xffffffffu, ok);
    };
    Pieces it(a, lane);
    Piece x;
    while (it.next(a, x)) {
      const bool both = x.rows > kTile;
      const int base = x.r0 + (both ? st * kTile : 0);  // the stream's first row
      const int rows = min(kTile, x.r0 + x.rows - base);
      {
        // The query tile, K-major 128-byte swizzled.  Rows past the last keep whatever was
        // there: they feed only their own scores, which nobody reads.
        const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(a.q);
        uint8_t* qt = smem + st * S::kTileBytes;
        for (int e = tid; e < rows * (D / 8); e += kStreamThreads) {
          const int r = e / (D / 8), gc = e % (D / 8);
          const int rr = base + r;
          const uint4 v = *reinterpret_cast<const uint4*>(
              qg + ((size_t)(x.g.qrow0 + rr / a.G) * a.Hq + (size_t)x.head * a.G + rr % a.G) * D + gc * 8);
          *reinterpret_cast<uint4*>(qt + (gc >> 3) * S::kHalfBytes + r * 128 +
                                    (((gc & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        tc_fence_before();  // this stream's reads of O are over
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[st]);
      }
      // Bad pages of the piece: this thread looks at every 256th.
      bool bad = false;
      {
        const int32_t* bt = a.block_table + (size_t)x.g.leader * a.maxp + x.page_begin;
        for (int pg = tid; pg < x.tokens / P; pg += kStreamThreads) {
          const int32_t id = bt[pg];
          bad |= id < 0 || id >= a.num_pages;
        }
      }
      const int n_mine = both ? x.n_tiles : (x.n_tiles - st + 1) / 2;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n_mine; ++i, ++n_s) {
        const int tile = both ? i : 2 * i + st;
        const int nv = min(kTile, x.tokens - tile * kTile) - 64 * half;  // valid of this half
        wait(&s_full[st], n_s);
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld64(s_at + 64 * half, sr);
        if (nv < 64) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= nv) sr[e] = __float_as_uint(-INFINITY);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 2)
          mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;  // c > 0
        // The row's maximum over both halves.  (The next write of this tile's slot comes
        // after the next s_full, so after every thread's read here.)
        *my_stat = top;
        named_bar_sync(1 + st, kStreamThreads);
        top = fmaxf(top, *other_stat);
        const bool rebase = top > m + kRebase;
        const float alpha = rebase ? exp2f(m - top) : 1.f;
        if (rebase) {
          l *= alpha;
          m = top;
        }
        if (__any_sync(0xffffffffu, rebase && i > 0)) {
#pragma unroll 1
          for (int cc = 0; cc < D / 2; cc += 32) {
            uint32_t ov[32];
            tmem_ld32(o_at + cc, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(o_at + cc, ov);
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = pair(c, c), mu2 = pair(-mu, -mu);
        uint64_t sum[2] = {0, 0};
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          float p0, p1;
          unpair(fma2(pair(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), c2, mu2), p0, p1);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(p0, p1));
          p[e >> 1] = pack_bf16x2(p0, p1);
        }
        {
          float lo, hi;
          unpair(add2(sum[0], sum[1]), lo, hi);
          l += lo + hi;
        }
        // P lies over S: the halves' barrier above followed every thread's read of S.
        tmem_st32(s_at + 32 * half, p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[st]);
      }
      if (n_mine > 0) {
        wait(&o_full[st], n_o);
        ++n_o;
      }
      tc_fence_after();
      bad = named_bar_or(1 + st, kStreamThreads, bad);
      *my_stat = l;
      named_bar_sync(1 + st, kStreamThreads);
      l += *other_stat;

      // Results: normalised partial rows; each half of a stream writes half of the columns.
      float* dump = reinterpret_cast<float*>(smem) + half * (D / 2) * kTile;  // [D][128 rows]
      bool merge = false;
      float f0 = 1.f, f1 = 0.f;
      if (!both) {
        named_bar_sync(3, 2 * kStreamThreads);  // neither stream reads its query tile again
        if (st == 1 && half == 0) stat[row] = m;  // stream 0 has exchanged its sums
        if (st == 1 && n_mine > 0) {
#pragma unroll 1
          for (int cc = 0; cc < D / 2; cc += 32) {
            uint32_t ov[32];
            tmem_ld32(o_at + cc, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) dump[(cc + e) * kTile + row] = __uint_as_float(ov[e]);
          }
        }
        named_bar_sync(3, 2 * kStreamThreads);
        if (st == 0 && x.n_tiles > 1) {
          merge = true;
          const float m1 = stat[row], l1 = stat[2 * kTile + row] + stat[3 * kTile + row];
          const float mm = fmaxf(m, m1), mu = mm == -INFINITY ? 0.f : mm;
          f0 = exp2f(m - mu);
          f1 = exp2f(m1 - mu);
          l = l * f0 + l1 * f1;
          m = mm;
        }
      }
      if (both || st == 0) {
        const int r = base + row;
        const bool mine = row < rows;
        const size_t at = mine ? part_row(a, x, r, x.part) : 0;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // l NaN: NaN
#pragma unroll 1
        for (int cc = 0; cc < D / 2; cc += 32) {
          uint32_t ov[32];
          tmem_ld32(o_at + cc, ov);
          if (!mine) continue;
          float4* po = reinterpret_cast<float4*>(a.part_o + at * D + half * (D / 2) + cc);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float o = __uint_as_float(ov[4 * e + k]);
              if (merge) o = o * f0 + dump[(cc + 4 * e + k) * kTile + row] * f1;
              v[k] = bad ? NAN : o * inv;
            }
            po[e] = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        if (mine && half == 0) a.part_lse[at] = bad ? NAN : (m + log2f(l)) * 0.6931471805599453f;
        if (mine && x.empty > 0) {
          const size_t step = part_step(a, x, r);
          for (int k = 1; k <= x.empty; ++k) {
            float4* po = reinterpret_cast<float4*>(a.part_o + (at + k * step) * D + half * (D / 2));
            for (int e = 0; e < D / 8; ++e) po[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (half == 0) a.part_lse[at + k * step] = -INFINITY;
          }
        }
      }
      if (bad && tid == 0 && st == 0) atomicOr(a.err, VAS_DEV_BAD_PAGE);
      if (!both) named_bar_sync(3, 2 * kStreamThreads);  // the dump is read: Q may be staged
    }
  } else {
    give_registers();
  }
  if (!ok && lane == 0) atomicOr(a.err, VAS_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int P>
int launch_tc(const CUtensorMap& mk, const CUtensorMap& mv, const PrefixArgs& a, void* stream) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VAS_E_CUDA;
  std::call_once(once[dev & 63], [&] {
    cudaFuncAttributes fa;
    attr_err[dev & 63] = cudaFuncGetAttributes(&fa, prefix_kernel<D, P>);
    // Fewer registers than the split counts on would leave setmaxnreg waiting.
    if (attr_err[dev & 63] == cudaSuccess && fa.numRegs < kLaunchRegs)
      attr_err[dev & 63] = cudaErrorInvalidConfiguration;
    if (attr_err[dev & 63] == cudaSuccess)
      attr_err[dev & 63] = cudaFuncSetAttribute(
          prefix_kernel<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, PSmem<D>::kDynBytes);
  });
  if (attr_err[dev & 63] != cudaSuccess) return VAS_E_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms());
  cfg.blockDim = dim3(kPrefixThreads);
  cfg.dynamicSmemBytes = PSmem<D>::kDynBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prefix_kernel<D, P>, mk, mv, a) != cudaSuccess) {
    cudaGetLastError();
    return VAS_E_CUDA;
  }
  return VAS_OK;
}

template <typename K>
int launch(K kernel, const PrefixArgs& a, int grid, int threads, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return VAS_E_CUDA;
  }
  return VAS_OK;
}

}  // namespace

int launch_prefix(const CUtensorMap& mk, const CUtensorMap& mv, const PrefixArgs& a,
                  int head_dim, int kv_dtype, void* stream) {
  if (kv_dtype == VAS_BF16) {
    if (head_dim == 128)
      return a.P == 16 ? launch_tc<128, 16>(mk, mv, a, stream) : launch_tc<128, 32>(mk, mv, a, stream);
    return a.P == 16 ? launch_tc<64, 16>(mk, mv, a, stream) : launch_tc<64, 32>(mk, mv, a, stream);
  }
  const int grid = num_sms();
  if (head_dim == 128) {
    if (kv_dtype == VAS_FP8_E4M3)
      return launch(prefix_simple_kernel<128, VAS_FP8_E4M3>, a, grid, 256, stream);
    return launch(prefix_simple_kernel<128, VAS_INT8>, a, grid, 256, stream);
  }
  if (kv_dtype == VAS_FP8_E4M3)
    return launch(prefix_simple_kernel<64, VAS_FP8_E4M3>, a, grid, 256, stream);
  return launch(prefix_simple_kernel<64, VAS_INT8>, a, grid, 256, stream);
}

}  // namespace attn
}  // namespace vas
