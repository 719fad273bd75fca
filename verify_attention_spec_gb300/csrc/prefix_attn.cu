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
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "../../include/vas.h"
#include "attn_plan.cuh"
#include "device_util.cuh"
#include "packed_math.cuh"
#include "vas_internal.h"

namespace vas {
namespace attn {
namespace {

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
  uint32_t x, end, share;
  int e;
  __device__ __forceinline__ Pieces(const PrefixArgs& a, int lane) {
    share = a.header->share;
    x = blockIdx.x * share;
    end = min(x + share, (uint32_t)a.header->span);
    e = 0;
    // The last entry whose base is at or below x, 32 entries at a time.
    const int n = a.header->n_groups;
    for (int s = 0; s < n; s += 32) {
      const uint32_t m =
          __ballot_sync(0xffffffffu, s + lane < n && (uint32_t)a.groups[s + lane].base <= x);
      if (m == 0) break;
      e = s + 31 - __clz(m);
      if (m != 0xffffffffu) break;
    }
  }
  // False at the end of the share.
  __device__ __forceinline__ bool next(const PrefixArgs& a, Piece& p) {
    while (x < end) {
      p.g = a.groups[e];
      const uint32_t base = p.g.base, units = p.g.head_units(), two = 2 * p.g.tiles;
      const uint32_t head = (x - base) / units;
      if (head >= (uint32_t)a.Hkv) {
        ++e;
        continue;  // x is the next group's base
      }
      const uint32_t in_head = x - base - head * units;
      const uint32_t block = min(in_head / two, (uint32_t)p.g.full);
      const int wide = block < (uint32_t)p.g.full;
      // (A block of single units may end in one of padding.)
      const uint32_t len = wide ? two : (two / 2 + 1) & ~1u, first = base + head * units + block * two;
      const uint32_t stop = min(end, first + len);
      p.head = (int)head;
      p.r0 = (int)block * kPrefixRows;
      p.rows = min(kPrefixRows, p.g.rows - p.r0);
      const int t0 = (int)(x - first) >> wide, t1 = min((int)(stop - first) >> wide, p.g.tiles);
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

// Partial row of row r of a group for the piece's partial, and how far the next partial of
// the row is.  The whole warp, rows ascending with the lane: the member that owns the first
// lane's token is searched 32 at a time (the last member whose first token is at or below
// it; members without tokens start where their successor does), the others walk on from it.
__device__ __forceinline__ size_t part_row(const PrefixArgs& a, const Piece& p, int r, int lane,
                                           size_t* step) {
  const int j = (int)a.by_G.div(r), t = p.g.qrow0 + j;
  const int t_first = __shfl_sync(0xffffffffu, t, 0);
  int lo = p.g.seq0, n = p.g.seq1 - p.g.seq0;
  while (n > 1) {
    const int each = (n + 31) >> 5;
    const uint32_t m =
        __ballot_sync(0xffffffffu, lane * each < n && a.row0[lo + lane * each] <= t_first);
    const int c = 31 - __clz(m);
    lo += c * each;
    n = min(each, n - c * each);
  }
  while (lo + 1 < p.g.seq1 && a.row0[lo + 1] <= t) ++lo;
  const SeqPlan sp = a.seqplan[lo];
  *step = (size_t)a.Hkv * ((size_t)a.G * sp.qlen);
  return partial_index(sp, a.Hkv, a.G, -sp.nsplit - p.g.parts + p.part, p.head,
                       (t - sp.qrow0) * a.G + (r - j * a.G));
}

// ------------------------------------------------------------------------------------
// The kernel: both products on tcgen05
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
// shared memory.  (The rounding of P to bf16 is as in paged_attn.cu: 2^-8 of a weight at most,
// as much as the output's own; shared parts have 256 tokens or more, over which it averages.)
// TMEM: S 2 x 128, O 2 x D columns.  Shared memory: the query tiles and a ring of K and V tiles,
// 128-byte swizzled as the TMA boxes land.  A producer warp streams the pages, an MMA warp
// issues.
//
// Measured, 128 windows of 5 tokens and 64 heads on a 16384-token prefix (344 GFLOP, 67 MB of K
// and V): 241 us, 1.43 PFLOP/s, the tensor pipe 64 % busy.  Bounded by the MMA warp: products
// one behind the other and the waits between them (a copy without softmax took as long).
//
// Quantised pages (KV: VAS_FP8_E4M3, VAS_INT8): the producer lands a tile's codes beside its
// 16-bit slot (with 128-wide heads in the upper half of it) and the scales of its tokens with
// the V codes; two converter warps expand the codes, exact in f16, into the slot.  Products
// are f16 (a row of Q scaled into range by a power of two where it must be, P relative to the
// V scales by the references); scores are multiplied by the K scale of their token, P by its V
// scale.  Bounded by the softmax, whose warps read each scale as a broadcast: the whole call takes 472 us on FP8 pages, 370 on bf16.
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

template <int D, int KV>
struct PSmem {
  static constexpr bool kQuant = KV != VAS_BF16;
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kTile * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // one operand of a tile, a query tile
  static constexpr int kSlots = kQuant ? (D == 128 ? 4 : 6) : (D == 128 ? 5 : 8);
  static constexpr int kRingOff = 2 * kTileBytes;
  // Codes [128 tokens][D]: a token's 128 codes lie where the second half of its row goes, so
  // a row is expanded in place; its 64 codes have a place of their own.
  static constexpr int kCodeOff = kRingOff + (D == 128 ? kHalfBytes : kSlots * kTileBytes);
  static constexpr int kCodeStep = D == 128 ? kTileBytes : kTile * 64;
  // [slot] K scales, V scales of the tile whose V the slot holds
  static constexpr int kScaleOff =
      kRingOff + kSlots * (kTileBytes + (kQuant && D == 64 ? kTile * 64 : 0));
  // [slot] v_exponent of each half of those V scales
  static constexpr int kExpOff = kScaleOff + (kQuant ? kSlots * 2 * kTile * 4 : 0);
  // [stream][row] what a row's scores are multiplied by
  static constexpr int kBackOff = kExpOff + (kQuant ? kSlots * 8 : 0);
  // [stream][half][row]: maxima, at the end of a piece the sums
  static constexpr int kStatOff = kBackOff + (kQuant ? 2 * kTile * 4 : 0);
  static constexpr int kBarOff = kStatOff + 4 * kTile * 4;
  // full[kSlots], empty[kSlots], ready[kSlots], s_full[2], p_full[2], o_full[2], q_full[2],
  // fin | TMEM base
  static constexpr int kDynBytes = kBarOff + (3 * kSlots + 9) * 8 + 16;
  static_assert(kDynBytes <= 227 * 1024, "shared memory of one CTA");
  static_assert(kTile * D * 4 <= 2 * kTileBytes, "stream 1's O fits over the query tiles");
};

// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 16 columns of this thread's lane, not waited for.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]),
        "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]),
        "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The warps beside the streams hand registers over (every warp of the group executes it).
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

template <int D, int P, int KV>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const PrefixArgs a) {
  using S = PSmem<D, KV>;
  constexpr bool kQuant = S::kQuant;
  constexpr int kSlots = S::kSlots;
  constexpr int kPages = kTile / P;  // pages of a tile
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle counts from 1024 bytes
  uint8_t* ring = smem + S::kRingOff;
  float* stat = reinterpret_cast<float*>(smem + S::kStatOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarOff);
  uint64_t* empty = full + kSlots;
  uint64_t* ready = empty + kSlots;   // quantised: the slot's codes are expanded
  uint64_t* s_full = ready + kSlots;  // S of the stream is in TMEM, its last O product done
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
      mbar_init(&ready[s], 2);
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
      constexpr int kBoxes = kQuant ? 1 : S::kHalves;  // of a page and operand
      auto load = [&](bool v, int tile) {
        const int slot = fill % kSlots;
        ok = ok && mbar_wait(&empty[slot], ((fill / kSlots) & 1) ^ 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          return;
        }
        const int pg = tile * kPages + e_page;
        int32_t id = -1;
        if (e_half < kBoxes && pg < n_pages) id = bt[pg];
        const bool mine = id >= 0 && id < a.num_pages;  // bad pages: the rows end as NaN
        const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0)
          mbar_arrive_expect_tx(&full[slot],
                                boxes * (kQuant ? P * D + (v ? 2 * P * 4 : 0) : P * 128));
        __syncwarp();
        if (mine) {
          if constexpr (kQuant) {
            tma_load_3d(smem + S::kCodeOff + slot * S::kCodeStep + e_page * (P * D),
                        v ? &tm_v : &tm_k, &full[slot], 0, id * P, x.head, pol);
            if (v) {  // the tile's scales, of K too: they live as long as its V
              float* sc = reinterpret_cast<float*>(smem + S::kScaleOff) + slot * 2 * kTile + e_page * P;
              const size_t at = ((size_t)id * a.Hkv + x.head) * P;
              bulk_load(sc, a.k_scale + at, P * 4, &full[slot], pol);
              bulk_load(sc + kTile, a.v_scale + at, P * 4, &full[slot], pol);
            }
          } else {
            tma_load_4d(ring + slot * S::kTileBytes + e_half * S::kHalfBytes + e_page * (P * 128),
                        v ? &tm_v : &tm_k, &full[slot], 0, id * P, e_half, x.head, pol);
          }
        }
        __syncwarp();
        ++fill;
      };
      const int lead = min(both ? 1 : 2, x.n_tiles);
      for (int t = 0; t < lead && ok; ++t) load(false, t);
      for (int j = 0; j < x.n_tiles && ok; ++j) {
        load(true, j);
        if (ok && j + lead < x.n_tiles) load(false, j + lead);
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
    constexpr uint32_t kIdS = umma_idesc_bf16(128, kTile, false, false, kQuant);
    constexpr uint32_t kIdO = umma_idesc_bf16(128, D, false, true, kQuant);
    uint64_t* const landed_bar = kQuant ? ready : full;
    constexpr uint32_t kHi = umma_desc_hi_sw128(1024);
    const uint32_t q_lo = umma_desc_lo(smem_u32(smem), 16);
    const uint32_t ring_k = umma_desc_lo(smem_u32(ring), 16);
    const uint32_t ring_v = umma_desc_lo(smem_u32(ring), S::kHalfBytes);
    uint32_t use = 0, n_p[2] = {0, 0}, n_q = 0;
    auto landed = [&](uint32_t f) {
      ok = ok && mbar_wait_fast(&landed_bar[f % kSlots], (f / kSlots) & 1);
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
      landed(f);
      const uint32_t v_lo = ring_v + (((f % kSlots) * S::kTileBytes) >> 4);
      const uint32_t p = tmem_s + st * kTile, o = tmem_o + st * D;
      ok = ok && mbar_wait_fast(&p_full[st], n_p[st] & 1);
      ok = __all_sync(0xffffffffu, ok);
      ++n_p[st];
      if (!ok) return;
      if (lane == 0) {
        tc_fence_after();
        if (tokens == kTile) {
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            umma_ts_lh(o, p + 8 * ks + (ks >= 4 ? 32 : 0), v_lo + ((ks * 2048) >> 4), kHi, kIdO, !first || ks > 0);
        } else {  // the V rows of pages that were not loaded are not read
          for (int ks = 0; ks < tokens / 16; ++ks)
            umma_ts_lh(o, p + 8 * ks + (ks >= 4 ? 32 : 0), v_lo + ((ks * 2048) >> 4), kHi, kIdO, !first || ks > 0);
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
    // What scores are multiplied by: the softmax scale in log2 units, or (quantised) what was
    // taken out of Q, the scale being in the K scales.
    float c = a.scale_log2;
    uint32_t n_s = 0, n_o = 0;
    uint32_t used = 0;  // fills of the ring before the piece in hand (quantised)
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
        // The query tile, K-major 128-byte swizzled, zeros behind the last row.
        const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(a.q);
        uint8_t* qt = smem + st * S::kTileBytes;
        constexpr int kEach = kTile * (D / 8) / kStreamThreads;
        uint4 v[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int e = tid + k * kStreamThreads, r = e / (D / 8), gc = e % (D / 8);
          const int rr = base + r;
          v[k] = make_uint4(0, 0, 0, 0);
          if (r < rows)
            v[k] = *reinterpret_cast<const uint4*>(
                qg + ((size_t)x.g.qrow0 * a.Hq + (size_t)x.head * a.G + rr +
                      (size_t)a.by_G.div(rr) * (a.Hq - a.G)) * D + gc * 8);
        }
        if constexpr (kQuant) {
          // A row goes to f16 times 2^-e, the power of two that brings its largest |q| under
          // 2^15 (1 for any ordinary Q); its scores are scaled back through c.  By rows,
          // because the rows of a tile are those of several sequences.  D / 8 lanes hold one.
          float* const back = reinterpret_cast<float*>(smem + S::kBackOff) + st * kTile;
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            const int e = tid + k * kStreamThreads;
            float most = absmax_bf16x8(v[k]);
#pragma unroll
            for (int o = D / 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            float mul = 1.f, up = 1.f;
            if (most > 32768.f && most <= 3.0e38f) {
              int x2;
              frexpf(most, &x2);  // most < 2^x2
              mul = ldexpf(1.f, 15 - x2);
              up = ldexpf(1.f, x2 - 15);
            }
            v[k] = bf16x8_to_f16x8(v[k], mul);
            if (e % (D / 8) == 0) back[e / (D / 8)] = up;  // this piece's; the last one's are read
          }
          named_bar_sync(1 + st, kStreamThreads);
          c = back[row];
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int e = tid + k * kStreamThreads, r = e / (D / 8), gc = e % (D / 8);
          *reinterpret_cast<uint4*>(qt + (gc >> 3) * S::kHalfBytes + r * 128 +
                                    (((gc & 7) ^ (r & 7)) << 4)) = v[k];
        }
        fence_proxy_async_smem();
        tc_fence_before();  // this stream's reads of O are over
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[st]);
      }
      const int n_mine = both ? x.n_tiles : (x.n_tiles - st + 1) / 2;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n_mine; ++i, ++n_s) {
        const int tile = both ? i : 2 * i + st;
        const int nv = min(kTile, x.tokens - tile * kTile) - 64 * half;  // valid of this half
        wait(&s_full[st], n_s);
        tc_fence_after();
        // Quantised: scales of this thread's 64 tokens.  They came with the tile's V, fill f of
        // the ring, whose slot is not filled again before this tile's P is used.  (Not before S:
        // its K tile lies at most three fills before f, so the slot's last phase is over.)
        const float* ksc = nullptr;
        float ve = 0.f;  // a reference moves by the exponent of the V scales, as in paged_attn.cu
        if constexpr (kQuant) {
          const int lead = min(both ? 1 : 2, x.n_tiles);
          const uint32_t f = used + lead + tile + min(tile, x.n_tiles - lead);
          wait(&ready[f % kSlots], f / kSlots);
          ksc = reinterpret_cast<const float*>(smem + S::kScaleOff) + (f % kSlots) * 2 * kTile + 64 * half;
          const float2 e = *reinterpret_cast<const float2*>(smem + S::kExpOff + (f % kSlots) * 8);
          ve = fmaxf(e.x, e.y);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t sc[32];
          tmem_ld32(s_at + 64 * half + 32 * h, sc);
          if constexpr (kQuant) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(ksc + 32 * h + e);
              float y[4];
              unpair(mul2(pair(__uint_as_float(sc[e]), __uint_as_float(sc[e + 1])), k.x), y[0], y[1]);
              unpair(mul2(pair(__uint_as_float(sc[e + 2]), __uint_as_float(sc[e + 3])), k.y), y[2], y[3]);
#pragma unroll
              for (int d = 0; d < 4; ++d) sc[e + d] = __float_as_uint(y[d]);
            }
            // Back for the second reading: with the K scales loaded once more there, the copies
            // of a broadcast cost shared memory more than this (document on FP8 pages, 520 us
            // against 492).
            tmem_st32(s_at + 64 * half + 32 * h, sc);
          }
          if (nv < 64) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * h + e >= nv) sc[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(sc[e]), __uint_as_float(sc[e + 1]));
        }
        if constexpr (kQuant) tmem_wait_st();
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;  // c > 0
        // The row's maximum over both halves.  (The next write of this tile's slot comes
        // after the next s_full, so after every thread's read here.)
        *my_stat = top;
        named_bar_sync(1 + st, kStreamThreads);
        top = fmaxf(top, *other_stat);
        if constexpr (kQuant) top += ve;
        const bool rebase = top > m + kRebase;
        if (__any_sync(0xffffffffu, rebase)) {
          const float alpha = rebase ? exp2f(m - top) : 1.f;
          if (rebase) {
            l *= alpha;
            m = top;
          }
          if (i > 0) {
#pragma unroll 1
            for (int cc = 0; cc < D / 2; cc += 32) {
              uint32_t ov[32];
              tmem_ld32(o_at + cc, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st32(o_at + cc, ov);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = pair(c, c), mu2 = pair(-mu, -mu);
        uint64_t sum[2] = {0, 0};
        // P lies over the first half of this thread's own scores.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[16], sc[32];
          tmem_ld32(s_at + 64 * half + 32 * h, sc);  // again: held, they would leave no registers
          if (nv < 64) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * h + e >= nv) sc[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            ulonglong2 vs;
            if constexpr (kQuant) vs = *reinterpret_cast<const ulonglong2*>(ksc + kTile + 32 * h + e);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              const int f = e + 2 * d;
              float p0, p1;
              unpair(fma2(pair(__uint_as_float(sc[f]), __uint_as_float(sc[f + 1])), c2, mu2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              const uint64_t pp = pair(p0, p1);
              sum[d] = add2(sum[d], pp);
              if constexpr (kQuant) {
                float w0, w1;
                unpair(mul2(pp, d ? vs.y : vs.x), w0, w1);
                p[f >> 1] = pack_f16x2(w0, w1);
              } else {
                p[f >> 1] = pack_bf16x2(p0, p1);
              }
            }
          }
          tmem_st16(s_at + 64 * half + 16 * h, p);
        }
        {
          float lo, hi;
          unpair(add2(sum[0], sum[1]), lo, hi);
          l += lo + hi;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[st]);
      }
      used += 2 * x.n_tiles;
      // While the last products run: bad pages of the piece (this thread looks at every
      // 256th), where the row goes.
      bool bad = false;
      {
        const int32_t* bt = a.block_table + (size_t)x.g.leader * a.maxp + x.page_begin;
        for (int pg = tid; pg < x.tokens / P; pg += kStreamThreads) {
          const int32_t id = bt[pg];
          bad |= id < 0 || id >= a.num_pages;
        }
      }
      // Where this thread's row goes.
      size_t step;
      const size_t at = part_row(a, x, base + min(row, rows - 1), lane, &step);
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
        const bool mine = row < rows;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // l NaN: NaN
        // A thread holds a row, but memory wants rows written by warps: kWide columns of the
        // warp's 32 rows at a time go through shared memory, a line a row.  (A row a thread, 16
        // bytes at a time, took 3.6 us of a piece.)  The lines are the stream's query tile, or
        // in a merge the part of the dump that this warp alone reads.
        constexpr int kWide = D / 4, kPer = kWide / 4;  // columns, 16-byte chunks of a line
        constexpr int kAtOnce = 32 / kPer;              // lines of a store
        auto swizzle = [](int r) { return kWide == 32 ? r & 7 : (r >> 1) & 3; };
#pragma unroll 1
        for (int cc = 0; cc < D / 2; cc += kWide) {
          uint32_t ov[kWide];
          if constexpr (kWide == 32) tmem_ld32(o_at + cc, ov);
          else tmem_ld16(o_at + cc, ov);
          float4* lines;
          int step16;  // 16-byte chunks from line to line
          if (merge) {
#pragma unroll
            for (int e = 0; e < kWide; ++e)
              ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f0 + dump[(cc + e) * kTile + row] * f1);
            // Columns cc .. of rows 32 w ..: kWide lines of 128 bytes, two to a line if narrow.
            lines = reinterpret_cast<float4*>(dump + cc * kTile + (row & ~31));
            step16 = kTile / 4;
            __syncwarp();
          } else {
            lines = reinterpret_cast<float4*>(smem + st * S::kTileBytes) +
                    (warp % kStreamWarps) * (32 * kPer);
            step16 = 8;
          }
          auto line = [&](int r) {  // of row r of the warp's 32
            return kWide == 32 ? lines + r * step16 : lines + (r >> 1) * step16 + (r & 1) * kPer;
          };
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = bad ? NAN : __uint_as_float(ov[4 * e + k]) * inv;
            line(lane)[e ^ swizzle(lane)] = make_float4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
          const int r_last = rows - (row & ~31);  // of this warp's rows
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int r = k * kAtOnce + lane / kPer, e = lane % kPer;
            const size_t to = __shfl_sync(0xffffffffu, at, r);
            if (r < r_last)
              *reinterpret_cast<float4*>(a.part_o + to * D + half * (D / 2) + cc + 4 * e) =
                  line(r)[e ^ swizzle(r)];
          }
          __syncwarp();
        }
        if (mine && half == 0) a.part_lse[at] = bad ? NAN : (m + log2f(l)) * 0.6931471805599453f;
        if (mine && x.empty > 0) {
          for (int k = 1; k <= x.empty; ++k) {
            float4* po = reinterpret_cast<float4*>(a.part_o + (at + k * step) * D + half * (D / 2));
            for (int e = 0; e < D / 8; ++e) po[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (half == 0) a.part_lse[at + k * step] = -INFINITY;
          }
        }
      }
      if (bad && tid == 0 && st == 0) atomicOr(a.err, VAS_DEV_BAD_PAGE);
      // The dump, or the stream's lines, are read: the next query tile may be staged.
      if (both) named_bar_sync(1 + st, kStreamThreads);
      else named_bar_sync(3, 2 * kStreamThreads);
    }
  } else {
    // ------------------------------ converters ------------------------------
    // Two warps, each every other 16 bytes-by-row group of a tile.  A row's codes are read by
    // lanes of one warp before any of its f16 values is written.
    give_registers();
    if constexpr (kQuant) {
      constexpr int kChunks = D / 16;        // 16-code chunks of a row
      constexpr int kRows = 32 / kChunks;    // rows of a warp at a time: 4 or 8
      constexpr int kBatch = 4;
      // Of this lane: where its codes of a batch's first row lie, and its two 16-byte pieces
      // of f16, for rows 0..3 and 4..7 of a swizzle atom (with 8 rows at a time both are the
      // same).  Rows of a batch are immediates away.
      const int lr = lane / kChunks, lc = lane % kChunks;
      uint32_t at0[2], at1[2];
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int r = (lr + (kRows == 4 ? 4 * o : 0)) & 7;
        at0[o] = (2 * lc >> 3) * S::kHalfBytes + lr * 128 + (((2 * lc & 7) ^ r) << 4);
        at1[o] = (2 * lc >> 3) * S::kHalfBytes + lr * 128 + ((((2 * lc + 1) & 7) ^ r) << 4);
      }
      const int cw = warp - kMmaWarp - 1;
      uint32_t fill = 0;
      Pieces it(a, lane);
      Piece x;
      while (ok && it.next(a, x)) {
        for (int k = 0; k < 2 * x.n_tiles && ok; ++k, ++fill) {
          const int slot = fill % kSlots;
          ok = mbar_wait_fast(&full[slot], (fill / kSlots) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* codes = smem + S::kCodeOff + slot * S::kCodeStep + lr * D + lc * 16;
          uint8_t* out = ring + slot * S::kTileBytes;
#pragma unroll 1
          for (int r0 = cw * kRows * kBatch; r0 < kTile; r0 += 2 * kRows * kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              v[e] = *reinterpret_cast<const uint4*>(codes + (r0 + e * kRows) * D);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
              const int o = kRows == 4 ? e & 1 : 0;  // a batch begins at a multiple of 8 rows
              uint4 y0, y1;
              if constexpr (KV == VAS_FP8_E4M3) {
                e4m3x4_to_f16x4(v[e].x, y0.x, y0.y);
                e4m3x4_to_f16x4(v[e].y, y0.z, y0.w);
                e4m3x4_to_f16x4(v[e].z, y1.x, y1.y);
                e4m3x4_to_f16x4(v[e].w, y1.z, y1.w);
              } else {
                s8x4_to_f16x4(v[e].x, y0.x, y0.y);
                s8x4_to_f16x4(v[e].y, y0.z, y0.w);
                s8x4_to_f16x4(v[e].z, y1.x, y1.y);
                s8x4_to_f16x4(v[e].w, y1.z, y1.w);
              }
              uint8_t* row = out + (r0 + e * kRows) * 128;
              *reinterpret_cast<uint4*>(row + at0[o]) = y0;
              *reinterpret_cast<uint4*>(row + at1[o]) = y1;
            }
          }
          // The K scales of a tile (they came with its V) take the softmax scale along, in
          // log2 units.  Behind the last token, where anything may lie, the scales become 1 and
          // 0: scores of -inf then give weights of 0 by themselves.  (Checks at each weight
          // instead cost a tile 128 instructions a thread.)
          const int lead = min(x.rows > kTile ? 1 : 2, x.n_tiles);
          const bool is_v = k >= lead && (((k - lead) & 1) == 0 || k >= 2 * x.n_tiles - lead);
          if (is_v) {
            const int nv = x.tokens - ((k - lead + 1) >> 1) * kTile;
            float* sc = reinterpret_cast<float*>(smem + S::kScaleOff) + slot * 2 * kTile;
            float most = 0.f;
#pragma unroll
            for (int t = cw * 64 + lane; t < cw * 64 + 64; t += 32) {
              sc[t] = t < nv ? sc[t] * a.scale_log2 : 1.f;
              if (t < nv) most = fmaxf(most, fabsf(sc[kTile + t]));
              else sc[kTile + t] = 0.f;
            }
            most = v_exponent(most);
            if (lane == 0) reinterpret_cast<float*>(smem + S::kExpOff)[2 * slot + cw] = most;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ready[slot]);
        }
      }
    }
  }
  if (!ok && lane == 0) atomicOr(a.err, VAS_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int P, int KV>
int launch_kernel(const CUtensorMap& mk, const CUtensorMap& mv, const PrefixArgs& a, void* stream) {
  static std::once_flag once[64];
  static cudaError_t attr_err[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VAS_E_CUDA;
  std::call_once(once[dev & 63], [&] {
    cudaFuncAttributes fa;
    attr_err[dev & 63] = cudaFuncGetAttributes(&fa, prefix_kernel<D, P, KV>);
    // Fewer registers than the split counts on would leave setmaxnreg waiting.
    if (attr_err[dev & 63] == cudaSuccess && fa.numRegs < kLaunchRegs)
      attr_err[dev & 63] = cudaErrorInvalidConfiguration;
    if (attr_err[dev & 63] == cudaSuccess)
      attr_err[dev & 63] = cudaFuncSetAttribute(
          prefix_kernel<D, P, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, PSmem<D, KV>::kDynBytes);
  });
  if (attr_err[dev & 63] != cudaSuccess) return VAS_E_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms());
  cfg.blockDim = dim3(kPrefixThreads);
  cfg.dynamicSmemBytes = PSmem<D, KV>::kDynBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prefix_kernel<D, P, KV>, mk, mv, a) != cudaSuccess) {
    cudaGetLastError();
    return VAS_E_CUDA;
  }
  return VAS_OK;
}

}  // namespace

int launch_prefix(const CUtensorMap& mk, const CUtensorMap& mv, const PrefixArgs& a,
                  int head_dim, int kv_dtype, void* stream) {
  auto kind = [&](auto kv) {
    constexpr int KV = decltype(kv)::value;
    if (head_dim == 128)
      return a.P == 16 ? launch_kernel<128, 16, KV>(mk, mv, a, stream)
                       : launch_kernel<128, 32, KV>(mk, mv, a, stream);
    return a.P == 16 ? launch_kernel<64, 16, KV>(mk, mv, a, stream)
                     : launch_kernel<64, 32, KV>(mk, mv, a, stream);
  };
  switch (kv_dtype) {
    case VAS_BF16: return kind(std::integral_constant<int, VAS_BF16>{});
    case VAS_FP8_E4M3: return kind(std::integral_constant<int, VAS_FP8_E4M3>{});
    default: return kind(std::integral_constant<int, VAS_INT8>{});
  }
}

}  // namespace attn
}  // namespace vas
