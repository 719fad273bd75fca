// Writing and moving the paged KV cache (sm_103a): paged_kv_append, paged_kv_copy and
// paged_kv_keep_path.  All three move bytes once; what each kernel adds is said there.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/vas.h"
#include "device_util.cuh"
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
// (a 16-term sum and 16 rotations a lane) hides behind the loads.
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;

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
  int32_t groups;      // work items of one token (each kRows * heads_per_task heads)
  float eps;
  int32_t* err;
};

// 8 elements as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16_lo_f32(u.x);
  x[1] = bf16_hi_f32(u.x);
  x[2] = bf16_lo_f32(u.y);
  x[3] = bf16_hi_f32(u.y);
  x[4] = bf16_lo_f32(u.z);
  x[5] = bf16_hi_f32(u.z);
  x[6] = bf16_lo_f32(u.w);
  x[7] = bf16_hi_f32(u.w);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  const float4 w = *reinterpret_cast<const float4*>(p + 4);
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
  x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// 8 values as codes: E4M3 (round to nearest even, saturating; NaN stays NaN) or INT8.
template <int KV>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (KV == VAS_FP8_E4M3) {
      asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
          : "=r"(w[h])
          : "f"(y[4 * h]), "f"(y[4 * h + 1]), "f"(y[4 * h + 2]), "f"(y[4 * h + 3]));
    } else {
      w[h] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // |y| <= 127 (1 + 2^-23), or NaN, which converts to 0 under a scale that is not
        // finite.
        const int c = max(-127, min(127, __float2int_rn(y[4 * h + i])));
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

// Exclusive prefix sums of max(query_lens, 0) at kAppendThreads evenly spaced sequences,
// and whether all lengths are consistent.  sums[i] is the first packed row of sequence
// i * step; sums[kAppendThreads] the total.
__device__ __forceinline__ void scan_lengths(const AppendArgs& a, int64_t* sums, int32_t step) {
  __shared__ int64_t wsum[kAppendWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t mine = 0;
  for (int i = tid * step; i < min(a.B, (tid + 1) * step); ++i) {
    const int32_t ql = a.query_lens[i];
    mine += ql > 0 ? ql : 0;
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int64_t base = 0;
#pragma unroll
  for (int w = 0; w < kAppendWarps; ++w)
    if (w < warp) base += wsum[w];
  sums[tid] = base + inc - mine;
  if (tid == kAppendThreads - 1) sums[kAppendThreads] = base + inc;
  __syncthreads();
}

__device__ __forceinline__ bool lengths_ok(const AppendArgs& a, int32_t L, int32_t ql) {
  return ql >= 0 && ql <= a.T && L >= ql && (int64_t)L <= (int64_t)a.maxp * a.P;
}

__device__ __forceinline__ Place place_of(const AppendArgs& a, const int64_t* sums, int32_t step,
                                          int32_t t) {
  Place p{0, 0, 0, 0};
  if (t >= sums[kAppendThreads]) {
    p.err = VAS_DEV_BAD_LENGTHS;  // a row that no sequence owns
    return p;
  }
  int lo = 0, hi = kAppendThreads - 1;  // the last thread's start at or below t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  // Sequences without tokens share a start with their successor: the search above ends on
  // the last of equal starts, the walk below passes over the empty ones.
  int64_t row = sums[lo];
  int32_t i = lo * step, ql = 0;
  for (; i < a.B; ++i) {
    ql = a.query_lens[i];
    const int64_t n = ql > 0 ? ql : 0;
    if (t < row + n) break;
    row += n;
  }
  if (i >= a.B) {
    p.err = VAS_DEV_BAD_LENGTHS;
    return p;
  }
  const int32_t L = a.seq_lens[i];
  if (!lengths_ok(a, L, ql) || row + ql > a.T) {
    p.err = VAS_DEV_BAD_LENGTHS;
    return p;
  }
  const int32_t pos = L - ql + (int32_t)(t - row);
  p.position = a.positions ? a.positions[t] : pos;
  if (a.rot && (p.position < 0 || p.position >= a.max_position)) p.err |= VAS_DEV_BAD_POSITION;
  p.page = a.block_table[(size_t)i * a.maxp + pos / a.P];
  p.slot = pos % a.P;
  if (p.page < 0 || p.page >= a.num_pages) p.err |= VAS_DEV_BAD_PAGE;
  return p;
}

// KV: the pool's storage type; T: the activations' (float with VAS_F32, bf16 otherwise).
// ROWS: head rows a lane takes per task; a task is 512 / D * ROWS consecutive rows (q
// heads, then k, then v) of one token, one warp.  INTER: rotary pairs are neighbours.
template <typename T, int KV, int D, int ROWS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 16;     // lanes of a row
  constexpr int kSub = 32 / kLanes;  // rows of a warp at a time
  constexpr bool kQuant = KV == VAS_FP8_E4M3 || KV == VAS_INT8;
  __shared__ int64_t sums[kAppendThreads + 1];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t task = (int64_t)blockIdx.x * kAppendWarps + warp;
  const int32_t t = (int32_t)(task / a.groups);
  const int32_t row0 = (int32_t)(task % a.groups) * (kSub * ROWS) + lane / kLanes;
  const int H = a.Hq + 2 * a.Hkv;
  const bool live = t < a.T;

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

  // The rows' values first: the look-up of the token's place overlaps their latency.
  float xa[ROWS][8], xb[ROWS][8];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = row0 + i * kSub;
    if (live && r < H) {
      const T* p;
      if (r < a.Hq) p = static_cast<const T*>(a.q) + t * a.q_stride + r * D;
      else if (r < a.Hq + a.Hkv) p = static_cast<const T*>(a.k) + t * a.k_stride + (r - a.Hq) * D;
      else p = static_cast<const T*>(a.v) + t * a.v_stride + (r - a.Hq - a.Hkv) * D;
      load8(p + ca, xa[i]);
      load8(p + cb, xb[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) xa[i][e] = xb[i][e] = 0.f;
    }
  }

  const int32_t step = (a.B + kAppendThreads - 1) / kAppendThreads;
  scan_lengths(a, sums, step);
  if (blockIdx.x == 0) {  // the call's lengths as a whole
    bool bad = threadIdx.x == 0 && sums[kAppendThreads] != a.T;
    for (int i = threadIdx.x; i < a.B; i += kAppendThreads)
      bad |= !lengths_ok(a, a.seq_lens[i], a.query_lens[i]);
    if (bad) atomicOr(a.err, VAS_DEV_BAD_LENGTHS);
  }
  if (!live) return;
  Place pl{0, 0, 0, 0};
  if (lane == 0) {  // one lane looks the place up, the others take it from there
    pl = place_of(a, sums, step, t);
    if (pl.err) atomicOr(a.err, pl.err);
  }
  pl.page = __shfl_sync(0xffffffffu, pl.page, 0);
  pl.slot = __shfl_sync(0xffffffffu, pl.slot, 0);
  pl.position = __shfl_sync(0xffffffffu, pl.position, 0);
  pl.err = __shfl_sync(0xffffffffu, pl.err, 0);

  // Cosines and sines of this lane's 8 pairs.
  float cs[8], sn[8];
  if (turned && !pl.err) {
    const float* row = a.cos_sin + (size_t)pl.position * a.rot + 8 * c;
    load8(row, cs);
    load8(row + a.rot / 2, sn);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
  }

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = row0 + i * kSub;
    // Rows past H hold zeros and only take part in the shuffles.
    const bool is_v = r >= a.Hq + a.Hkv, is_q = r < a.Hq;
    const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
    // Sum of squares over the row's lanes; every lane of the warp takes part.
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(xa[i][e], xa[i][e], fmaf(xb[i][e], xb[i][e], ss));
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!is_v) {
      if (w != nullptr) {
        const float inv = __fdiv_rn(1.f, __fsqrt_rn(ss * (1.f / D) + a.eps));
        float wa[8], wb[8];
        load8(w + ca, wa);
        load8(w + cb, wb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xa[i][e] = xa[i][e] * inv * wa[e];
          xb[i][e] = xb[i][e] * inv * wb[e];
        }
      }
      if (turned) {
        if (INTER) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u0 = xa[i][2 * e], u1 = xa[i][2 * e + 1];
            xa[i][2 * e] = u0 * cs[e] - u1 * sn[e];
            xa[i][2 * e + 1] = u1 * cs[e] + u0 * sn[e];
            const float w0 = xb[i][2 * e], w1 = xb[i][2 * e + 1];
            xb[i][2 * e] = w0 * cs[4 + e] - w1 * sn[4 + e];
            xb[i][2 * e + 1] = w1 * cs[4 + e] + w0 * sn[4 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = xa[i][e], v = xb[i][e];
            xa[i][e] = u * cs[e] - v * sn[e];
            xb[i][e] = v * cs[e] + u * sn[e];
          }
        }
      }
    }
    float scale = 1.f;
    if constexpr (kQuant) {
      // The largest magnitude of the row, by the order of the bits (NaN above infinity).
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        m = max(m, max(__float_as_uint(xa[i][e]) & 0x7fffffffu, __float_as_uint(xb[i][e]) & 0x7fffffffu));
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      scale = __fdiv_rn(__uint_as_float(m), KV == VAS_FP8_E4M3 ? 448.f : 127.f);
      if (scale == 0.f) scale = 1.f;
    }
    if (r >= H) continue;
    if (is_q) {
      if (pl.err) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xa[i][e] = xb[i][e] = NAN;
      }
      T* p = static_cast<T*>(a.q_out) + ((size_t)t * a.Hq + r) * D;
      store8(p + ca, xa[i]);
      store8(p + cb, xb[i]);
      continue;
    }
    if (pl.err) continue;
    const int h = is_v ? r - a.Hq - a.Hkv : r - a.Hq;
    const size_t at = (((size_t)pl.page * a.P + pl.slot) * a.Hkv + h) * D;
    if constexpr (kQuant) {
      uint8_t* p = static_cast<uint8_t*>(is_v ? a.v_pages : a.k_pages) + at;
      *reinterpret_cast<uint2*>(p + ca) = codes8<KV>(xa[i], scale);
      *reinterpret_cast<uint2*>(p + cb) = codes8<KV>(xb[i], scale);
      if (c == 0)
        (is_v ? a.v_scale : a.k_scale)[((size_t)pl.page * a.Hkv + h) * a.P + pl.slot] = scale;
    } else {
      T* p = static_cast<T*>(is_v ? a.v_pages : a.k_pages) + at;
      store8(p + ca, xa[i]);
      store8(p + cb, xb[i]);
    }
  }
}

// ------------------------------------------------------------------------------------
// Copies of pages
// ------------------------------------------------------------------------------------
// The pairs travel in the kernel's parameters, so the caller's lists are free when the
// call returns and no device copy of them is needed.  A page of one operand is contiguous;
// its first tokens are too.  A block moves segments of 16 KB, 4 x 16 bytes a thread in
// flight (bounded by HBM: every byte once in and once out).
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
// Latency bounds it (a few tokens per sequence): one launch, and four dependent reads.
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
        if (c <= prev || c >= ql) {
          err |= VAS_DEV_BAD_TREE;
          continue;
        }
        // s + 1 <= c < ql: both positions lie inside the sequence.
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

// Rows of a lane per task.  With one row the most warps are in flight, which is what a
// small step needs; with four, one look-up of the token's place and one read of its
// table row serve four times the heads.
constexpr int kAppendRows = 4;

template <typename T, int KV, int D, bool INTER>
int launch_append_rows(AppendArgs& a, vas_stream_t stream) {
  const int sub = 32 / (D / 16);
  const int H = a.Hq + 2 * a.Hkv;
  const int sms = vas::num_sms();
  if (!sms) return VAS_E_CUDA;
  const int64_t one = (int64_t)a.T * ((H + sub - 1) / sub);
  const bool many = one > (int64_t)sms * 64;
  const int rows = many ? kAppendRows : 1;
  a.groups = (H + sub * rows - 1) / (sub * rows);
  const int64_t blocks = ((int64_t)a.T * a.groups + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT_MAX) return VAS_E_UNSUPPORTED;
  if (many)
    return launch(append_kernel<T, KV, D, kAppendRows, INTER>, dim3((unsigned)blocks),
                  kAppendThreads, stream, a);
  return launch(append_kernel<T, KV, D, 1, INTER>, dim3((unsigned)blocks), kAppendThreads, stream,
                a);
}

template <typename T, int KV>
int launch_append(AppendArgs& a, int D, bool inter, vas_stream_t stream) {
  if (D == 128)
    return inter ? launch_append_rows<T, KV, 128, true>(a, stream)
                 : launch_append_rows<T, KV, 128, false>(a, stream);
  return inter ? launch_append_rows<T, KV, 64, true>(a, stream)
               : launch_append_rows<T, KV, 64, false>(a, stream);
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
  if (tb * d->page_size > INT32_MAX || d->num_layers > 32767) return VAS_E_UNSUPPORTED;
  if (!k || !v || misaligned(k, 16) || misaligned(v, 16)) return VAS_E_INVALID_ARG;
  const bool quant = is_quant(d->kv_dtype);
  if (quant != (ks != nullptr) || quant != (vs != nullptr) || misaligned(ks, 16) ||
      misaligned(vs, 16))
    return VAS_E_INVALID_ARG;
  *token_bytes = (int32_t)tb;
  return VAS_OK;
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
    const bool in_place = q_out == q && d.q_stride == qw;
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
  a.groups = 0;
  a.eps = d.eps;
  a.err = vas::device_error_word();
  if (!a.err) return VAS_E_CUDA;
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
  // Every id in the pool, destinations distinct and apart from the sources.
  try {
    std::vector<uint8_t> seen(static_cast<size_t>(dims->num_pages), 0);  // 1 source, 2 target
    for (int32_t i = 0; i < n; ++i) {
      if (src[i] < 0 || src[i] >= dims->num_pages || dst[i] < 0 || dst[i] >= dims->num_pages)
        return VAS_E_INVALID_ARG;
      if (tokens && (tokens[i] < 1 || tokens[i] > dims->page_size)) return VAS_E_INVALID_ARG;
      seen[src[i]] |= 1;
    }
    for (int32_t i = 0; i < n; ++i) {
      if (seen[dst[i]]) return VAS_E_INVALID_ARG;
      seen[dst[i]] = 2;
    }
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
