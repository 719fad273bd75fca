// Writing and moving the paged KV cache (sm_103a): paged_kv_append, paged_kv_copy and
// paged_kv_keep_path.  All three move bytes once; what each kernel adds is said there.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/vas.h"
#include "device_util.cuh"
#include "packed_math.cuh"
#include "vas_internal.h"

namespace vas {
namespace cache {

// ------------------------------------------------------------------------------------
// Append: norms, rotation, store
// ------------------------------------------------------------------------------------
// A head row of D elements is held by D / 16 lanes, 16 elements each: two chunks of 8,
// `a` and `b`, chosen so that with the split-half rotation a's elements pair with b's and
// a rotation needs no exchange between lanes.  A warp works on 512 / D heads of one token
// at a time and keeps the token's cosines and sines and the weights in registers for all
// the heads it takes, so the table costs one read per warp and not one per head.
// Bytes bound it: T (2 Hq + 2 Hkv) D in and out and the pages' T 2 Hkv D; the arithmetic
// (a 16-term sum and 16 rotations a lane) hides behind the loads as long as tokens are many:
// 8192 tokens of 64/8 heads of 128 in bf16, 336 MB, 61 us, 5.5 TB/s; 768 on FP8 pages, 30 MB,
// 12.5 us, where the chain of one token's reads shows.
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendBlocks = 2;  // of an SM

struct AppendArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* q_weight;
  const void* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* query_lens;
  void* q_out;
  void* k_pages;
  void* v_pages;
  float* k_scale;
  float* v_scale;
  int64_t q_stride, k_stride, v_stride;
  int32_t B, T, Hq, Hkv, P, num_pages, maxp, rot, max_position;
  int32_t log2P;
  int32_t parts, iters;  // a token is `parts` tasks of `iters` groups of rows
  float eps;
  int32_t* err;
};

// Eight fp32 values as four pairs, the operands of the packed instructions.
struct F8 {
  uint64_t p[4];
};

__device__ __forceinline__ F8 load_f8(const float* p) {
  const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p);
  const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(p + 4);
  return {{u.x, u.y, w.x, w.y}};
}

// 16 (bf16) or 32 (fp32) raw bytes of each of a lane's two chunks: what waits in registers
// between the load and its use.
template <typename T>
struct Raw {
  uint4 a[sizeof(T) / 2], b[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int ca, int cb) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      a[i] = __ldcs(reinterpret_cast<const uint4*>(p + ca) + i);
      b[i] = __ldcs(reinterpret_cast<const uint4*>(p + cb) + i);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) a[i] = b[i] = make_uint4(0, 0, 0, 0);
  }
};
__device__ __forceinline__ F8 widen(const uint4 (&u)[1]) {
  return {{pair(bf16_lo_f32(u[0].x), bf16_hi_f32(u[0].x)), pair(bf16_lo_f32(u[0].y), bf16_hi_f32(u[0].y)),
           pair(bf16_lo_f32(u[0].z), bf16_hi_f32(u[0].z)), pair(bf16_lo_f32(u[0].w), bf16_hi_f32(u[0].w))}};
}
__device__ __forceinline__ F8 widen(const uint4 (&u)[2]) {
  auto f = [](uint32_t x, uint32_t y) { return pair(__uint_as_float(x), __uint_as_float(y)); };
  return {{f(u[0].x, u[0].y), f(u[0].z, u[0].w), f(u[1].x, u[1].y), f(u[1].z, u[1].w)}};
}
__device__ __forceinline__ F8 load_weights(const __nv_bfloat16* p) {
  const uint4 u[1] = {*reinterpret_cast<const uint4*>(p)};
  return widen(u);
}
__device__ __forceinline__ F8 load_weights(const float* p) { return load_f8(p); }

__device__ __forceinline__ uint32_t bf16_pair(uint64_t v) {
  float lo, hi;
  unpair(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& x) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16_pair(x.p[0]), bf16_pair(x.p[1]), bf16_pair(x.p[2]), bf16_pair(x.p[3]));
}
__device__ __forceinline__ void store8(float* p, const F8& x) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x.p[0], x.p[1]);
  *reinterpret_cast<ulonglong2*>(p + 4) = make_ulonglong2(x.p[2], x.p[3]);
}

// x / scale, rounded to nearest.  With the correctly rounded reciprocal r = 1 / scale, one
// correction of x r by its exact remainder gives the correctly rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34, 1990), three packed instructions for two elements; scales near the ends of the
// range, where r or the remainder could leave it, and the not finite ones divide.
__device__ __forceinline__ F8 quotients(const F8& x, float scale) {
  F8 y;
  if (scale > 0x1p-80f && scale < 0x1p80f) {
    const float r = __frcp_rn(scale);
    const uint64_t r2 = pair(r, r), ns2 = pair(-scale, -scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t q = mul2(x.p[i], r2);
      y.p[i] = fma2(fma2(q, ns2, x.p[i]), r2, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpair(x.p[i], lo, hi);
      y.p[i] = pair(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale));
    }
  }
  return y;
}

// 8 values as codes: E4M3 (round to nearest even, saturating; NaN stays NaN) or INT8.
template <int KV>
__device__ __forceinline__ uint2 codes8(const F8& x, float scale) {
  const F8 q = quotients(x, scale);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
    unpair(q.p[2 * h], y[0], y[1]);
    unpair(q.p[2 * h + 1], y[2], y[3]);
    if constexpr (KV == VAS_FP8_E4M3) {
      asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
          : "=r"(w[h])
          : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    } else {
      w[h] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // |y| <= 127 (1 + 2^-23), or NaN, which converts to 0 under a scale that is not
        // finite.
        const int c = max(-127, min(127, __float2int_rn(y[i])));
        w[h] |= (uint32_t)(c & 0xff) << (8 * i);
      }
    }
  }
  return make_uint2(w[0], w[1]);
}

// Where a token goes, or why it does not.
struct Place {
  int32_t page, slot, position;
  int32_t err;  // device error bits; the token is not stored and its q_out row is NaN
};

// The packing of a call, in shared memory: the first row of every `step`th sequence, and
// with step 1 (up to kAppendSeqs sequences) their lengths too.
constexpr int kAppendSeqs = 1024;
struct Packing {
  int32_t row0[kAppendSeqs + 1];  // clamped to INT_MAX; the last one is the total
  int32_t len[kAppendSeqs];
  int64_t wsum[kAppendWarps];
};

__device__ __forceinline__ bool lengths_ok(const AppendArgs& a, int32_t L, int32_t ql) {
  return ql >= 0 && ql <= a.T && L >= ql && (int64_t)L <= (int64_t)a.maxp * a.P;
}

__device__ __forceinline__ void scan_lengths(const AppendArgs& a, Packing& pk, int32_t step) {
  constexpr int kPer = kAppendSeqs / kAppendThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t mine[kPer], sum = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int c = tid * kPer + e;
    mine[e] = 0;
    if (step == 1) {
      if (c < a.B) {
        mine[e] = max(a.query_lens[c], 0);
        pk.len[c] = a.seq_lens[c];
      }
    } else {
      for (int64_t i = (int64_t)c * step; i < a.B && i < ((int64_t)c + 1) * step; ++i)
        mine[e] += max(a.query_lens[i], 0);
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int64_t n = mine[e];
    mine[e] = sum;
    sum += n;
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) pk.wsum[warp] = inc;
  __syncthreads();
  int64_t base = inc - sum;
#pragma unroll
  for (int w = 0; w < kAppendWarps; ++w)
    if (w < warp) base += pk.wsum[w];
  auto clamp = [](int64_t x) { return (int32_t)(x < INT_MAX ? x : INT_MAX); };
#pragma unroll
  for (int e = 0; e < kPer; ++e) pk.row0[tid * kPer + e] = clamp(base + mine[e]);
  if (tid == kAppendThreads - 1) pk.row0[kAppendSeqs] = clamp(base + sum);
  __syncthreads();
}

// The whole warp: the place of packed row t.  The last start at or below t is found in two
// rounds of 32 (sequences without tokens share their successor's start, so the last of
// equal starts is the one that has tokens).
__device__ __forceinline__ Place place_of(const AppendArgs& a, const Packing& pk, int32_t step,
                                          int32_t t, int lane) {
  Place p{0, 0, 0, 0};
  if (t >= pk.row0[kAppendSeqs]) {
    p.err = VAS_DEV_BAD_LENGTHS;  // a row that no sequence owns
    return p;
  }
  constexpr int kBlock = kAppendSeqs / 32;
  const int hi = __popc(__ballot_sync(0xffffffffu, pk.row0[lane * kBlock] <= t)) - 1;
  static_assert(kBlock == 32, "one start a lane in the second round");
  const int lo = __popc(__ballot_sync(0xffffffffu, pk.row0[hi * kBlock + lane] <= t)) - 1;
  const int c = hi * kBlock + lo;
  int64_t row = pk.row0[c];
  int32_t i = c, ql, L;
  if (step == 1) {
    // A negative length counts as none, so a sequence found here has its true one.
    ql = pk.row0[c + 1] - pk.row0[c];
    L = pk.len[c];
  } else {
    for (i = c * step; i < a.B; ++i) {
      ql = a.query_lens[i];
      const int64_t n = ql > 0 ? ql : 0;
      if (t < row + n) break;
      row += n;
    }
    if (i >= a.B) {
      p.err = VAS_DEV_BAD_LENGTHS;
      return p;
    }
    L = a.seq_lens[i];
  }
  if (!lengths_ok(a, L, ql) || row + ql > a.T) {
    p.err = VAS_DEV_BAD_LENGTHS;
    return p;
  }
  const int32_t pos = L - ql + (int32_t)(t - row);
  p.position = a.positions ? a.positions[t] : pos;
  if (a.rot && (p.position < 0 || p.position >= a.max_position)) p.err |= VAS_DEV_BAD_POSITION;
  p.page = a.block_table[(size_t)i * a.maxp + (pos >> a.log2P)];
  p.slot = pos & (a.P - 1);
  if (p.page < 0 || p.page >= a.num_pages) p.err |= VAS_DEV_BAD_PAGE;
  return p;
}

// KV: the pool's storage type; T: the activations' (float with VAS_F32, bf16 otherwise).
// ROWS: head rows a lane holds at a time, so a warp has a group of 512 / D * ROWS rows (q
// heads, then k, then v) in flight.  A task is `iters` consecutive groups of one token: one
// look-up of the token's place, one read of its table row.  A block scans the lengths once
// and its warps take tasks gridDim apart; as soon as a row has been taken from its
// registers the same row of the next group, or task, is fetched into them, so loads are
// always under way.  INTER: rotary pairs are neighbours.
template <typename T, int KV, int D, int ROWS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 16;     // lanes of a row
  constexpr int kSub = 32 / kLanes;  // rows of a warp at a time
  constexpr bool kQuant = KV == VAS_FP8_E4M3 || KV == VAS_INT8;
  __shared__ Packing pk;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = a.Hq + 2 * a.Hkv;
  const uint32_t n_tasks = (uint32_t)a.T * (uint32_t)a.parts;  // at most INT_MAX
  const uint32_t stride = gridDim.x * kAppendWarps;
  uint32_t task = blockIdx.x * kAppendWarps + warp;

  // This lane's chunks of a row.  Split halves: rotated pairs (8c + e, 8c + e + rot / 2)
  // first, then the rest of the head.  Neighbours: 16 consecutive elements.
  const int c = lane % kLanes, nrot = a.rot / 16;
  const bool turned = c < nrot;
  int ca, cb;
  if (INTER) {
    ca = 16 * c;
    cb = ca + 8;
  } else if (turned) {
    ca = 8 * c;
    cb = ca + a.rot / 2;
  } else {
    ca = a.rot + 8 * (c - nrot);
    cb = ca + (D - a.rot) / 2;
  }

  // A row's values are on their way while the place of its token is looked up (and, for
  // the first ones, while the block scans the lengths).
  Raw<T> x[ROWS];
  auto fetch = [&](Raw<T>& dst, int32_t t, int32_t r) {
    if (t < a.T && r < H) {
      const T* p;
      if (r < a.Hq) p = static_cast<const T*>(a.q) + t * a.q_stride + r * D;
      else if (r < a.Hq + a.Hkv) p = static_cast<const T*>(a.k) + t * a.k_stride + (r - a.Hq) * D;
      else p = static_cast<const T*>(a.v) + t * a.v_stride + (r - a.Hq - a.Hkv) * D;
      dst.load(p, ca, cb);
    } else {
      dst.zero();
    }
  };
  constexpr int kGroup = kSub * ROWS;
  int32_t t = (int32_t)(task / (uint32_t)a.parts);
  int32_t row0 = (int32_t)(task - (uint32_t)t * a.parts) * a.iters * kGroup + lane / kLanes;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) fetch(x[i], t, row0 + i * kSub);

  const int32_t step = (a.B + kAppendSeqs - 1) / kAppendSeqs;
  scan_lengths(a, pk, step);
  if (blockIdx.x == 0) {  // the call's lengths as a whole
    bool bad = threadIdx.x == 0 && pk.row0[kAppendSeqs] != a.T;
    for (int i = threadIdx.x; i < a.B; i += kAppendThreads)
      bad |= !lengths_ok(a, a.seq_lens[i], a.query_lens[i]);
    if (bad) atomicOr(a.err, VAS_DEV_BAD_LENGTHS);
  }
  F8 wa{}, wb{};  // the weights of this lane's chunks, and whose they are
  int kind = -1;  // 1: q, 0: k
  while (task < n_tasks) {
    const Place pl = place_of(a, pk, step, t, lane);
    if (pl.err && lane == 0) atomicOr(a.err, pl.err);

    // Cosines and sines of this lane's 8 pairs.
    const uint64_t one = pair(1.f, 1.f);
    F8 cs{{one, one, one, one}}, sn{{0, 0, 0, 0}};
    if (turned && !pl.err) {
      const float* row = a.cos_sin + (size_t)pl.position * a.rot + 8 * c;
      cs = load_f8(row);
      sn = load_f8(row + a.rot / 2);
    }

    task += stride;
    int32_t t_task = (int32_t)(task / (uint32_t)a.parts);
    const int32_t row_task =
        (int32_t)(task - (uint32_t)t_task * a.parts) * a.iters * kGroup + lane / kLanes;
    if (task >= n_tasks) t_task = a.T;
    for (int it = 0; it < a.iters; ++it) {
      const bool last = it + 1 == a.iters;
      const int32_t t_next = last ? t_task : t, row_next = last ? row_task : row0 + kGroup;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int r = row0 + i * kSub;
        // A warp's rows past H hold zeros and only take part in the shuffles.
        const bool is_v = r >= a.Hq + a.Hkv, is_q = r < a.Hq;
        F8 xa = widen(x[i].a), xb = widen(x[i].b);
        fetch(x[i], t_next, row_next + i * kSub);
        // Nothing for the whole warp (20 heads of 64, 10141 tokens: 21.3 -> 19.7 us).
        if (r - lane / kLanes >= H) continue;
        const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
        if (w != nullptr && kind != (int)is_q) {
          kind = is_q;
          wa = load_weights(w + ca);
          wb = load_weights(w + cb);
        }
        // Sum of squares over the row's lanes; every lane of the warp takes part.
        uint64_t s2 = mul2(xa.p[0], xa.p[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) s2 = fma2(xa.p[e], xa.p[e], s2);
#pragma unroll
        for (int e = 0; e < 4; ++e) s2 = fma2(xb.p[e], xb.p[e], s2);
        float ss, hi;
        unpair(s2, ss, hi);
        ss += hi;
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!is_v) {
          if (w != nullptr) {
            const float inv = rsqrtf(ss * (1.f / D) + a.eps);
            const uint64_t inv2 = pair(inv, inv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              xa.p[e] = mul2(mul2(xa.p[e], inv2), wa.p[e]);
              xb.p[e] = mul2(mul2(xb.p[e], inv2), wb.p[e]);
            }
          }
          if (turned) {
            if (INTER) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float c0, c1, s0, s1, u0, u1;
                unpair(cs.p[e], c0, c1);
                unpair(sn.p[e], s0, s1);
                // Pairs 2e and 2e + 1: chunk a holds pairs 0..3, chunk b 4..7.
                uint64_t& y0 = e < 2 ? xa.p[2 * (e & 1)] : xb.p[2 * (e & 1)];
                uint64_t& y1 = e < 2 ? xa.p[2 * (e & 1) + 1] : xb.p[2 * (e & 1) + 1];
                unpair(y0, u0, u1);
                y0 = pair(u0 * c0 - u1 * s0, u1 * c0 + u0 * s0);
                unpair(y1, u0, u1);
                y1 = pair(u0 * c1 - u1 * s1, u1 * c1 + u0 * s1);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint64_t u = xa.p[e], v = xb.p[e];
                xa.p[e] = sub2(mul2(u, cs.p[e]), mul2(v, sn.p[e]));
                xb.p[e] = fma2(v, cs.p[e], mul2(u, sn.p[e]));
              }
            }
          }
        }
        float scale = 1.f;
        if (kQuant && __any_sync(0xffffffffu, !is_q)) {
          // The largest magnitude of the row, by the order of the bits (NaN above infinity).
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y[4];
            unpair(xa.p[e], y[0], y[1]);
            unpair(xb.p[e], y[2], y[3]);
#pragma unroll
            for (int f = 0; f < 4; ++f) m = max(m, __float_as_uint(y[f]) & 0x7fffffffu);
          }
#pragma unroll
          for (int o = kLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          scale = __fdiv_rn(__uint_as_float(m), KV == VAS_FP8_E4M3 ? 448.f : 127.f);
          if (scale == 0.f) scale = 1.f;
        }
        if (r >= H) continue;
        if (is_q) {
          if (pl.err) {
#pragma unroll
            for (int e = 0; e < 4; ++e) xa.p[e] = xb.p[e] = pair(NAN, NAN);
          }
          T* p = static_cast<T*>(a.q_out) + ((size_t)t * a.Hq + r) * D;
          store8(p + ca, xa);
          store8(p + cb, xb);
          continue;
        }
        if (pl.err) continue;
        const int h = is_v ? r - a.Hq - a.Hkv : r - a.Hq;
        const size_t at = (((size_t)pl.page * a.P + pl.slot) * a.Hkv + h) * D;
        if constexpr (kQuant) {
          uint8_t* p = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + at;
          *reinterpret_cast<uint2*>(p + ca) = codes8<KV>(xa, scale);
          *reinterpret_cast<uint2*>(p + cb) = codes8<KV>(xb, scale);
          if (c == 0)
            (is_v ? a.v_scale : a.k_scale)[((size_t)pl.page * a.Hkv + h) * a.P + pl.slot] = scale;
        } else {
          T* p = static_cast<T*>(is_v ? a.v_pages : a.k_pages) + at;
          store8(p + ca, xa);
          store8(p + cb, xb);
        }
      }
      if (!last) row0 += kGroup;
    }
    t = t_task;
    row0 = row_task;
  }
}

// ------------------------------------------------------------------------------------
// Copies of pages
// ------------------------------------------------------------------------------------
// The pairs travel in the kernel's parameters, so the caller's lists are free when the
// call returns and no device copy of them is needed.  A page of one operand is contiguous;
// its first tokens are too.  A block moves segments of 16 KB, 4 x 16 bytes a thread in
// flight (bounded by HBM: every byte once in and once out; 2047 pages of 64 KB an operand,
// 537 MB in all, 80 us, 6.7 TB/s).
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopySeg = kCopyThreads * kCopyUnroll * 16;

template <int N>
struct CopyList {
  int32_t src[N], dst[N];
  uint8_t tokens[N];
};
constexpr int kCopySmall = 64, kCopyLarge = 2048;  // pairs of a launch

struct CopyArgs {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int32_t n, segs;      // pairs; segments of a page
  int32_t token_bytes;  // Hkv * D * element size
  int32_t P, Hkv, num_pages;
};

template <int N>
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const CopyArgs a, const __grid_constant__ CopyList<N> list) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int seg = blockIdx.x % a.segs, i = blockIdx.x / a.segs;
  const int layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int tokens = list.tokens[i];
  const size_t page_bytes = (size_t)a.token_bytes * a.P;
  const size_t from = (size_t)layer * a.num_pages + list.src[i];
  const size_t to = (size_t)layer * a.num_pages + list.dst[i];
  uint8_t* base = is_v ? a.v : a.k;
  const uint8_t* s = base + from * page_bytes;
  uint8_t* d = base + to * page_bytes;
  const int32_t bytes = a.token_bytes * tokens;
  const int32_t b0 = seg * kCopySeg + tid * 16;
  uint4 x[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int32_t b = b0 + u * kCopyThreads * 16;
    if (b < bytes) x[u] = __ldcs(reinterpret_cast<const uint4*>(s + b));
  }
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u) {
    const int32_t b = b0 + u * kCopyThreads * 16;
    if (b < bytes) __stcs(reinterpret_cast<uint4*>(d + b), x[u]);
  }
  if (a.ks != nullptr && seg == 0) {  // scales [Hkv][P]: the first tokens of each head
    float* sc = is_v ? a.vs : a.ks;
    const int n = a.Hkv * a.P;
    for (int e = tid; e < n; e += kCopyThreads)
      if (e % a.P < tokens) sc[to * n + e] = sc[from * n + e];
  }
}

// ------------------------------------------------------------------------------------
// Accepted draft paths
// ------------------------------------------------------------------------------------
// One block per (row of path, layer and operand); a thread owns 16-byte columns of the
// token row and takes the accepted nodes in order, kKeepUnroll at a time, all read before
// any is written.  That equals reading everything first: nodes ascend, so path[s] >= s + 1
// and a destination s + 1 is never the source of a later node (path[s'] >= s' + 1 > s + 1).
// Latency bounds it (a few tokens per sequence): one launch, and four dependent reads. (64
// windows of a layer 2.7 us.)
constexpr int kKeepThreads = 128;
constexpr int kKeepUnroll = 4;
constexpr int kKeepMaxNodes = 255;

struct KeepArgs {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* query_lens;
  const int32_t* seq_index;
  const int32_t* path;
  const int32_t* accepted_len;
  int32_t num_seqs, maxp, n, token_bytes, P, Hkv, num_pages;
  int32_t* err;
};

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepArgs a) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  // For node s: token index inside the pool (page * P + slot) of its source and target.
  __shared__ int64_t s_from[kKeepMaxNodes], s_to[kKeepMaxNodes];
  __shared__ int32_t s_err;
  const int tid = threadIdx.x, b = blockIdx.x;
  const int layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  if (tid == 0) s_err = 0;
  __syncthreads();
  const int32_t acc = a.accepted_len[b];
  if (acc <= 0) return;
  const int32_t i = a.seq_index ? a.seq_index[b] : b;
  int32_t err = 0;
  if (acc > a.n || i < 0 || i >= a.num_seqs) {
    err = VAS_DEV_BAD_TREE;
  } else {
    const int32_t L = a.seq_lens[i], ql = a.query_lens[i];
    if (ql < 1 || L < ql || (int64_t)L > (int64_t)a.maxp * a.P) {
      err = VAS_DEV_BAD_LENGTHS;
    } else {
      const int32_t* row = a.path + (size_t)b * a.n;
      const int32_t* bt = a.block_table + (size_t)i * a.maxp;
      for (int s = tid; s < acc; s += kKeepThreads) {
        const int32_t c = row[s], prev = s ? row[s - 1] : 0;
        // An ascending path has s + 1 <= c < ql, so that both positions lie inside the
        // sequence; one that fell before s may ascend here with c <= s.
        if (c <= prev || c <= s || c >= ql) {
          err |= VAS_DEV_BAD_TREE;
          continue;
        }
        const int32_t p0 = L - ql + c, p1 = L - ql + 1 + s;
        const int32_t g0 = bt[p0 / a.P], g1 = bt[p1 / a.P];
        if (g0 < 0 || g0 >= a.num_pages || g1 < 0 || g1 >= a.num_pages) {
          err |= VAS_DEV_BAD_PAGE;
          continue;
        }
        s_from[s] = (int64_t)g0 * a.P + p0 % a.P;
        s_to[s] = (int64_t)g1 * a.P + p1 % a.P;
      }
      if (a.seq_index)
        for (int r = tid; r < b; r += kKeepThreads)
          if (a.seq_index[r] == i) err |= VAS_DEV_BAD_TREE;
    }
  }
  if (err) atomicOr(&s_err, err);
  __syncthreads();
  if (s_err) {
    if (tid == 0 && blockIdx.y == 0) atomicOr(a.err, s_err);
    return;
  }
  const size_t pool = (size_t)layer * a.num_pages * a.P;  // tokens before this layer
  uint8_t* base = (is_v ? a.v : a.k) + pool * a.token_bytes;
  for (int32_t col = tid * 16; col < a.token_bytes; col += kKeepThreads * 16) {
    for (int s0 = 0; s0 < acc; s0 += kKeepUnroll) {
      uint4 x[kKeepUnroll];
#pragma unroll
      for (int u = 0; u < kKeepUnroll; ++u)
        if (s0 + u < acc)
          x[u] = *reinterpret_cast<const uint4*>(base + s_from[s0 + u] * a.token_bytes + col);
#pragma unroll
      for (int u = 0; u < kKeepUnroll; ++u)
        if (s0 + u < acc)
          *reinterpret_cast<uint4*>(base + s_to[s0 + u] * a.token_bytes + col) = x[u];
    }
  }
  if (a.ks != nullptr) {
    float* sc = (is_v ? a.vs : a.ks) + pool * a.Hkv;
    for (int h = tid; h < a.Hkv; h += kKeepThreads)
      for (int s = 0; s < acc; ++s) {
        const int64_t f = s_from[s], t = s_to[s];
        sc[((t / a.P) * a.Hkv + h) * a.P + t % a.P] = sc[((f / a.P) * a.Hkv + h) * a.P + f % a.P];
      }
  }
}

}  // namespace cache
}  // namespace vas

// ------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------
namespace {

using namespace vas::cache;

bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

bool is_quant(int32_t kv) { return kv == VAS_FP8_E4M3 || kv == VAS_INT8; }

int32_t element_size(int32_t kv) { return kv == VAS_F32 ? 4 : (kv == VAS_BF16 ? 2 : 1); }

// Launch as a programmatic dependent: the grid may be scheduled while the previous kernel
// of the stream ends, and waits for it before its first read.
template <typename... P, typename... A>
int launch(void (*kernel)(P...), dim3 grid, int threads, vas_stream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return VAS_E_CUDA;
  }
  return VAS_OK;
}

bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

template <typename T, int KV, int D, int ROWS, bool INTER>
int launch_append_rows(AppendArgs& a, vas_stream_t stream) {
  const int group = 32 / (D / 16) * ROWS;
  const int64_t warps = (int64_t)vas::num_sms() * kAppendBlocks * kAppendWarps;
  // Eight tasks a resident warp, where there are as many: the last round is then short
  // against the whole.  Fewer where the tokens do not give them; never less than a group.
  const int64_t groups = (a.Hq + 2 * a.Hkv + group - 1) / group;
  int64_t parts = (8 * warps + a.T - 1) / a.T;
  parts = parts < groups ? parts : groups;
  if (parts * a.T > INT_MAX / 2) parts = 1;  // 32-bit task numbers, with room for the stride
  a.iters = (int32_t)((groups + parts - 1) / parts);
  a.parts = (int32_t)((groups + a.iters - 1) / a.iters);
  const int64_t blocks = ((int64_t)a.T * a.parts + kAppendWarps - 1) / kAppendWarps;
  const int64_t most = warps / kAppendWarps;
  return launch(append_kernel<T, KV, D, ROWS, INTER>, dim3((unsigned)(blocks < most ? blocks : most)),
                kAppendThreads, stream, a);
}

// Rows of a lane at a time.  With one the most warps share a small step's rows; with four
// (fp32: two) a warp has the most bytes in flight and the fewest look-ups: a 768-token
// step over FP8 pages 12.4 us against 13.7 (one) and 13.0 (two), eight 1024-token chunks
// in bf16 60.9 against 62.7 and 65.1.
template <typename T, int KV, int D, bool INTER>
int launch_append_size(AppendArgs& a, vas_stream_t stream) {
  const int sub = 32 / (D / 16);
  const int64_t one = (int64_t)a.T * ((a.Hq + 2 * a.Hkv + sub - 1) / sub);
  const bool many = one > (int64_t)vas::num_sms() * 64;
  return many ? launch_append_rows<T, KV, D, sizeof(T) == 4 ? 2 : 4, INTER>(a, stream)
              : launch_append_rows<T, KV, D, 1, INTER>(a, stream);
}

template <typename T, int KV>
int launch_append(AppendArgs& a, int D, bool inter, vas_stream_t stream) {
  if (D == 128)
    return inter ? launch_append_size<T, KV, 128, true>(a, stream)
                 : launch_append_size<T, KV, 128, false>(a, stream);
  return inter ? launch_append_size<T, KV, 64, true>(a, stream)
               : launch_append_size<T, KV, 64, false>(a, stream);
}

// The checks that paged_kv_copy and paged_kv_keep_path share; *token_bytes of one operand.
int check_pool(const vas_pool_dims* d, const void* k, const void* v, const float* ks,
               const float* vs, int32_t* token_bytes) {
  if (!d) return VAS_E_INVALID_ARG;
  if (d->num_layers < 0 || d->num_pages < 0 || d->num_kv_heads <= 0) return VAS_E_INVALID_ARG;
  if ((d->head_dim != 64 && d->head_dim != 128) || (d->page_size != 16 && d->page_size != 32) ||
      d->kv_dtype < VAS_F32 || d->kv_dtype > VAS_INT8)
    return VAS_E_UNSUPPORTED;
  const int64_t tb = (int64_t)d->num_kv_heads * d->head_dim * element_size(d->kv_dtype);
  // Offsets inside a page are 32 bits, up to the end of its last segment.
  if (tb * d->page_size > INT32_MAX - kCopySeg || d->num_layers > 32767) return VAS_E_UNSUPPORTED;
  if (!k || !v || misaligned(k, 16) || misaligned(v, 16)) return VAS_E_INVALID_ARG;
  const bool quant = is_quant(d->kv_dtype);
  if (quant != (ks != nullptr) || quant != (vs != nullptr) || misaligned(ks, 16) ||
      misaligned(vs, 16))
    return VAS_E_INVALID_ARG;
  *token_bytes = (int32_t)tb;
  return VAS_OK;
}

// Whether the destinations are distinct and none is a source.  A few pairs are sorted, many
// are marked in a map of the pool (which is cleared for it: 0.1 ms for a million pages).
bool targets_apart(const int32_t* src, const int32_t* dst, int32_t n, int32_t num_pages) {
  if ((int64_t)n * 32 < num_pages) {
    std::vector<int32_t> d(dst, dst + n);
    std::sort(d.begin(), d.end());
    if (std::adjacent_find(d.begin(), d.end()) != d.end()) return false;
    for (int32_t i = 0; i < n; ++i)
      if (std::binary_search(d.begin(), d.end(), src[i])) return false;
    return true;
  }
  std::vector<uint8_t> seen(static_cast<size_t>(num_pages), 0);
  for (int32_t i = 0; i < n; ++i) seen[src[i]] = 1;
  for (int32_t i = 0; i < n; ++i) {
    if (seen[dst[i]]) return false;
    seen[dst[i]] = 1;
  }
  return true;
}

template <int N>
int launch_copy(CopyArgs a, const int32_t* src, const int32_t* dst, const int32_t* tokens,
                int32_t n, int32_t layers, vas_stream_t stream) {
  CopyList<N> list;
  memset(&list, 0, sizeof list);
  memcpy(list.src, src, sizeof(int32_t) * n);
  memcpy(list.dst, dst, sizeof(int32_t) * n);
  int32_t most = 0;
  for (int32_t i = 0; i < n; ++i) {
    list.tokens[i] = (uint8_t)(tokens ? tokens[i] : a.P);
    most = list.tokens[i] > most ? list.tokens[i] : most;
  }
  a.n = n;
  a.segs = (a.token_bytes * most + kCopySeg - 1) / kCopySeg;
  if ((int64_t)a.segs * n > INT32_MAX) return VAS_E_UNSUPPORTED;
  return launch(copy_kernel<N>, dim3((unsigned)(a.segs * n), (unsigned)(2 * layers)), kCopyThreads,
                stream, a, list);
}

}  // namespace

extern "C" {

int paged_kv_append(const void* q, const void* k, const void* v, const void* q_weight,
                    const void* k_weight, const float* cos_sin, const int32_t* positions,
                    const int32_t* block_table, const int32_t* seq_lens,
                    const int32_t* query_lens, void* q_out, void* k_pages, void* v_pages,
                    float* k_scale, float* v_scale, const vas_append_dims* dims,
                    vas_stream_t stream) {
  if (!dims) return VAS_E_INVALID_ARG;
  const vas_append_dims& d = *dims;
  if (d.num_seqs < 0 || d.total_tokens < 0 || d.num_q_heads < 0 || d.num_kv_heads <= 0 ||
      d.num_pages < 0 || d.max_pages_per_seq < 0 || d.rotary_dim < 0 || d.max_position < 0)
    return VAS_E_INVALID_ARG;
  if (!(d.eps >= 0.f) || std::isinf(d.eps)) return VAS_E_INVALID_ARG;
  if ((d.head_dim != 64 && d.head_dim != 128) || (d.page_size != 16 && d.page_size != 32) ||
      d.kv_dtype < VAS_F32 || d.kv_dtype > VAS_INT8 || d.rotary_dim % 16 ||
      d.rotary_dim > d.head_dim || (d.interleaved != 0 && d.interleaved != 1))
    return VAS_E_UNSUPPORTED;
  const int64_t heads = (int64_t)d.num_q_heads + 2 * (int64_t)d.num_kv_heads;
  if (heads * d.head_dim > INT32_MAX / 2) return VAS_E_INVALID_ARG;
  const bool quant = is_quant(d.kv_dtype);
  if (quant != (k_scale != nullptr) || quant != (v_scale != nullptr)) return VAS_E_INVALID_ARG;
  if (d.num_seqs == 0 || d.total_tokens == 0) return VAS_OK;
  if (!k || !v || !block_table || !seq_lens || !query_lens || !k_pages || !v_pages)
    return VAS_E_INVALID_ARG;
  if (d.num_q_heads > 0 && (!q || !q_out)) return VAS_E_INVALID_ARG;
  if (d.rotary_dim > 0 && !cos_sin) return VAS_E_INVALID_ARG;
  if (d.num_pages == 0 || d.max_pages_per_seq == 0) return VAS_E_INVALID_ARG;
  if ((int64_t)d.num_pages * d.page_size > INT32_MAX) return VAS_E_INVALID_ARG;
  const int es = d.kv_dtype == VAS_F32 ? 4 : 2;
  const int64_t qw = (int64_t)d.num_q_heads * d.head_dim, kw = (int64_t)d.num_kv_heads * d.head_dim;
  if (d.q_stride < qw || d.k_stride < kw || d.v_stride < kw) return VAS_E_INVALID_ARG;
  if ((d.num_q_heads > 0 && d.q_stride * es % 16) || d.k_stride * es % 16 || d.v_stride * es % 16)
    return VAS_E_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_weight, 16) ||
      misaligned(k_weight, 16) || misaligned(cos_sin, 16) || misaligned(positions, 4) ||
      misaligned(block_table, 4) || misaligned(seq_lens, 4) || misaligned(query_lens, 4) ||
      misaligned(q_out, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) ||
      misaligned(k_scale, 16) || misaligned(v_scale, 16))
    return VAS_E_INVALID_ARG;
  if (d.num_q_heads > 0) {
    // q_out is written while other rows are still to be read: either the same rows by the
    // same lanes, or apart.
    const int64_t T = d.total_tokens, out_bytes = T * qw * es;
    auto span = [&](int64_t stride, int64_t width) { return ((T - 1) * stride + width) * es; };
    const bool in_place = q_out == q && (d.q_stride == qw || T == 1);  // one row is contiguous
    if ((!in_place && overlap(q_out, out_bytes, q, span(d.q_stride, qw))) ||
        overlap(q_out, out_bytes, k, span(d.k_stride, kw)) ||
        overlap(q_out, out_bytes, v, span(d.v_stride, kw)))
      return VAS_E_INVALID_ARG;
  }
  AppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.query_lens = query_lens;
  a.q_out = q_out;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.q_stride = d.q_stride;
  a.k_stride = d.k_stride;
  a.v_stride = d.v_stride;
  a.B = d.num_seqs;
  a.T = d.total_tokens;
  a.Hq = d.num_q_heads;
  a.Hkv = d.num_kv_heads;
  a.P = d.page_size;
  a.num_pages = d.num_pages;
  a.maxp = d.max_pages_per_seq;
  a.rot = d.rotary_dim;
  a.max_position = d.max_position;
  a.log2P = d.page_size == 16 ? 4 : 5;
  a.parts = a.iters = 1;
  a.eps = d.eps;
  a.err = vas::device_error_word();
  if (!a.err || !vas::num_sms()) return VAS_E_CUDA;
  const bool inter = d.interleaved != 0;
  switch (d.kv_dtype) {
    case VAS_F32: return launch_append<float, VAS_F32>(a, d.head_dim, inter, stream);
    case VAS_BF16: return launch_append<__nv_bfloat16, VAS_BF16>(a, d.head_dim, inter, stream);
    case VAS_FP8_E4M3:
      return launch_append<__nv_bfloat16, VAS_FP8_E4M3>(a, d.head_dim, inter, stream);
    default: return launch_append<__nv_bfloat16, VAS_INT8>(a, d.head_dim, inter, stream);
  }
}

int paged_kv_copy(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                  const int32_t* src, const int32_t* dst, const int32_t* tokens, int32_t n,
                  const vas_pool_dims* dims, vas_stream_t stream) {
  CopyArgs a;
  const int st = check_pool(dims, k_pages, v_pages, k_scale, v_scale, &a.token_bytes);
  if (st != VAS_OK) return st;
  if (n < 0 || (n > 0 && (!src || !dst))) return VAS_E_INVALID_ARG;
  if (n == 0 || dims->num_layers == 0) return VAS_OK;
  for (int32_t i = 0; i < n; ++i) {
    if (src[i] < 0 || src[i] >= dims->num_pages || dst[i] < 0 || dst[i] >= dims->num_pages)
      return VAS_E_INVALID_ARG;
    if (tokens && (tokens[i] < 1 || tokens[i] > dims->page_size)) return VAS_E_INVALID_ARG;
  }
  try {
    if (!targets_apart(src, dst, n, dims->num_pages)) return VAS_E_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return VAS_E_NOMEM;
  }
  a.k = static_cast<uint8_t*>(k_pages);
  a.v = static_cast<uint8_t*>(v_pages);
  a.ks = k_scale;
  a.vs = v_scale;
  a.P = dims->page_size;
  a.Hkv = dims->num_kv_heads;
  a.num_pages = dims->num_pages;
  a.n = a.segs = 0;
  for (int32_t i = 0; i < n;) {
    const int32_t left = n - i;
    const int32_t m = left <= kCopySmall ? left : (left < kCopyLarge ? left : kCopyLarge);
    const int32_t* tk = tokens ? tokens + i : nullptr;
    const int r = m <= kCopySmall
                      ? launch_copy<kCopySmall>(a, src + i, dst + i, tk, m, dims->num_layers, stream)
                      : launch_copy<kCopyLarge>(a, src + i, dst + i, tk, m, dims->num_layers, stream);
    if (r != VAS_OK) return r;
    i += m;
  }
  return VAS_OK;
}

int paged_kv_keep_path(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                       const int32_t* block_table, const int32_t* seq_lens,
                       const int32_t* query_lens, int32_t num_seqs, int32_t max_pages_per_seq,
                       const int32_t* seq_index, const int32_t* path,
                       const int32_t* accepted_len, int32_t B, int32_t n,
                       const vas_pool_dims* dims, vas_stream_t stream) {
  KeepArgs a;
  const int st = check_pool(dims, k_pages, v_pages, k_scale, v_scale, &a.token_bytes);
  if (st != VAS_OK) return st;
  if (B < 0 || n < 1 || n > kKeepMaxNodes || num_seqs < 0 || max_pages_per_seq < 0)
    return VAS_E_INVALID_ARG;
  if (B == 0 || dims->num_layers == 0) return VAS_OK;
  if (!block_table || !seq_lens || !query_lens || !path || !accepted_len)
    return VAS_E_INVALID_ARG;
  if (!seq_index && B > num_seqs) return VAS_E_INVALID_ARG;
  if ((int64_t)dims->num_pages * dims->page_size > INT32_MAX) return VAS_E_INVALID_ARG;
  if (misaligned(block_table, 4) || misaligned(seq_lens, 4) || misaligned(query_lens, 4) ||
      misaligned(seq_index, 4) || misaligned(path, 4) || misaligned(accepted_len, 4))
    return VAS_E_INVALID_ARG;
  a.k = static_cast<uint8_t*>(k_pages);
  a.v = static_cast<uint8_t*>(v_pages);
  a.ks = k_scale;
  a.vs = v_scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.query_lens = query_lens;
  a.seq_index = seq_index;
  a.path = path;
  a.accepted_len = accepted_len;
  a.num_seqs = num_seqs;
  a.maxp = max_pages_per_seq;
  a.n = n;
  a.P = dims->page_size;
  a.Hkv = dims->num_kv_heads;
  a.num_pages = dims->num_pages;
  a.err = vas::device_error_word();
  if (!a.err) return VAS_E_CUDA;
  return launch(keep_kernel, dim3((unsigned)B, (unsigned)(2 * dims->num_layers)), kKeepThreads,
                stream, a);
}

}  // extern "C"
