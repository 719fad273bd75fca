// Logits of a verification window to the probabilities of the rejection rule (sm_103a):
// spec_logits.  Penalties for repeated tokens, a sparse bias, a grammar mask, temperature and
// softmax in one pass over the vocabulary.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/vas.h"
#include "device_util.cuh"
#include "vas_internal.h"

namespace vas {
namespace logits {

// Clusters of C CTAs stay on the GPU and take rows one after the other, a stretch of consecutive
// rows each; CTA r of a cluster holds slice r of the vocabulary, 8 NV logits a thread in registers
// as fp32 from the one read to the one write.  While a row is reduced and written, the next one's
// logits are on their way into shared memory by bulk copy.
// The logits of few tokens change by more than the mask and the temperature, so those are set
// apart: when a cluster comes to a sequence its token list is counted into a table in shared
// memory with a word for every token of the slice (each CTA reads 1 / C of the list and counts
// into the slices of all, through distributed shared memory), and a bit map says which words
// count.  A thread's dense logits leave those tokens out; the thread that owns their word of the
// map takes them, in both passes.  From row to row of a sequence only the drafts change.
// Exponentials are taken once, relative to the thread's own maximum, and scaled by one product
// when the row's maximum and sum are known.
// Bytes bound it: V (2 or 4 + 4) a row.  Vocabularies past the registers' reach (8 * 512 * 64 =
// 262144 logits) are taken in chunks, the table made anew and the logits read again for the
// second pass.
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxBias = 1024;
constexpr int kMaxTokens = 1 << 20;  // of a list: a count fits its field
constexpr int kMaxNodes = 255;
// A table word: count, prompt flag, bias entry + 1.
constexpr uint32_t kCountMask = (1u << 20) - 1, kPrompt = 1u << 20;
constexpr int kBiasShift = 21;

struct Args {
  const void* logits;
  const int32_t* tokens;
  const int32_t* token_lens;
  const int32_t* prompt_lens;
  const int32_t* drafts;
  const int32_t* parents;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_tokens;
  const float* bias;
  const uint32_t* mask;
  const float* temperature;
  float* out;
  int64_t row_stride;
  int32_t n, V, max_tokens, max_bias, mask_words;
  int32_t rows, clusters;          // rows of the call; clusters that share them
  int32_t cluster, slice, chunks;  // CTAs of a row; tokens of a CTA (a multiple of 32); chunks of it
  int32_t probs, counted;  // counted: penalties are in play
  int32_t out_vec;         // rows of out are 16-byte aligned
  int32_t staged;          // rows come by bulk copy; bytes of a slice's place
  int32_t words;           // of the table
  int32_t* err;
};

struct Shared {
  float bias[kMaxBias];
  int32_t bias_tok[kMaxBias];
  int32_t parent[kMaxNodes];
  uint8_t on_path[kMaxNodes + 1];
  float red_max[kWarps], red_sum[kWarps];
  int32_t red_at[kWarps];
  // Written by the cluster's CTAs, by the row's parity.
  float peer_max[2][kMaxCluster], peer_sum[2][kMaxCluster];
  int32_t peer_at[2][kMaxCluster];
  uint64_t landed;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_address(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_add(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_or(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// VEC: a thread's logits are runs of 8 neighbours, 16-byte aligned; else they are kThreads
// apart.
template <typename T, bool VEC, int NV>
struct Tile {
  static constexpr int kTokens = kThreads * 8 * NV;
  // Token (of the chunk) of this thread's value 8 v + e.
  static __device__ __forceinline__ int at(int v, int e) {
    return VEC ? (v * kThreads + (int)threadIdx.x) * 8 + e
               : (v * 8 + e) * kThreads + (int)threadIdx.x;
  }
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&y)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[2 * i] = bf16_lo_f32(w[i]), y[2 * i + 1] = bf16_hi_f32(w[i]);
}
__device__ __forceinline__ void load8(const float* p, float (&y)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w;
  y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
}
__device__ __forceinline__ float widen1(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen1(float x) { return x; }

template <typename T, bool VEC, int NV, bool MULTI>
__global__ void __launch_bounds__(kThreads, NV <= 4 && !MULTI ? 2 : 1) spec_logits_kernel(const Args a) {
  using L = Tile<T, VEC, NV>;
  constexpr int kKeep = 4;  // adjusted logits a thread keeps between the passes
  // The table's words, a bit for each, and the place of a row's slice.
  extern __shared__ __align__(16) uint32_t table[];
  uint32_t* const map = table + a.words;
  const T* const stage = reinterpret_cast<const T*>(map + a.words / 32);
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int C = a.cluster;
  const int cluster = (int)(blockIdx.x / (unsigned)C);
  const bool use_table = a.counted || a.max_bias > 0;
  const int nb = a.max_bias;
  auto clear_table = [&] {
    uint4* t4 = reinterpret_cast<uint4*>(table);
    for (int i = tid; i < a.words / 4 + a.words / 128; i += kThreads) t4[i] = make_uint4(0, 0, 0, 0);
  };
  if (tid == 0) {
    mbar_init(&s.landed, 1);
    mbar_fence_init();
  }
  if (use_table) clear_table();
  __syncthreads();
  // The cluster's CTAs are all there, and their tables clear, before the first word of a peer's
  // shared memory is touched: every arrival below has its wait.
  if (use_table || a.probs) cluster_arrive();
  bool arrived = use_table || a.probs;
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  const int first = rank * a.slice, last = min(a.V, first + a.slice);
  const int row0 = (int)((int64_t)a.rows * cluster / a.clusters);
  const int row1 = (int)((int64_t)a.rows * (cluster + 1) / a.clusters);
  auto row_in = [&](int row) { return static_cast<const T*>(a.logits) + (size_t)row * a.row_stride; };
  // One thread: row `row`'s slice to its place.  (Slices begin at multiples of 32 logits; the
  // rest of the last 16 bytes is read by the threads.)
  const uint32_t bulk = VEC && last > first ? (uint32_t)((last - first) * sizeof(T)) & ~15u : 0;
  auto fetch = [&](int row) {
    if (bulk) {
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&s.landed, bulk);
      bulk_load_plain(const_cast<T*>(stage), row_in(row) + first, bulk, &s.landed);
    }
  };
  if (a.staged && tid == 0 && row0 < row1) fetch(row0);

  int seq = -1;  // the sequence that the table counts
  uint32_t nth = 0;  // rows taken
  int32_t n_tok = 0, n_prompt = 0;
  float rep = 1.f, freq = 0.f, pres = 0.f, temp = 1.f;
  bool bad_seq = false;

  for (int row = row0; row < row1; ++row, ++nth) {
    const int b = row / (a.n + 1), j = row - b * (a.n + 1);
    const T* in = row_in(row);
    float* out = a.out + (size_t)row * a.V;
    const uint8_t* mask_bytes = reinterpret_cast<const uint8_t*>(a.mask + (size_t)row * a.mask_words);
    const bool other = b != seq;
    if (other) {
      rep = a.repetition ? a.repetition[b] : 1.f;
      freq = a.frequency ? a.frequency[b] : 0.f;
      pres = a.presence ? a.presence[b] : 0.f;
      temp = a.temperature ? a.temperature[b] : 1.f;
      bad_seq = false;
      n_tok = n_prompt = 0;
      if (a.counted && a.tokens) {
        n_tok = a.token_lens[b];
        n_prompt = a.prompt_lens ? a.prompt_lens[b] : 0;
        if (n_tok < 0 || n_tok > a.max_tokens || n_prompt < 0 || n_prompt > n_tok) {
          bad_seq = true;
          n_tok = n_prompt = 0;
          if (tid == 0 && rank == 0) atomicOr(a.err, VAS_DEV_BAD_LENGTHS);
        }
      }
    }
    bool bad = bad_seq;
    // The drafts on the way to row j: those before it, or its ancestors.  on_path: now and (bit 1)
    // at the row before of the same sequence.
    if (a.counted && a.n > 0) {
      __syncthreads();  // the row before is done with these
      for (int i = tid; i < a.n; i += kThreads) {
        if (other && a.parents) s.parent[i] = a.parents[(size_t)b * a.n + i];
        s.on_path[i] = (other ? 0 : (s.on_path[i] & 1) << 1) | (!a.parents && i < j);
      }
      __syncthreads();
      int e = 0;
      if (a.parents) {
        if (tid == 0)
          for (int u = j; u > 0;) {  // ascends: a parent precedes its child
            const int p = s.parent[u - 1];
            s.on_path[u - 1] |= 1;
            if (p < 0 || p >= u) {
              e = VAS_DEV_BAD_TREE;
              break;
            }
            u = p;
          }
        __syncthreads();
      }
      for (int i = tid; i < a.n; i += kThreads)
        if (s.on_path[i] & 1) {
          const int x = a.drafts[(size_t)b * a.n + i];
          if (x < 0 || x >= a.V) e |= VAS_DEV_BAD_TOKEN;
        }
      if (e && rank == 0) atomicOr(a.err, e);
      bad |= __syncthreads_or(e != 0) != 0;
    }

    // The table of chunk k: the cluster's counts of the sequence's list and its biases when the
    // table is another sequence's (or chunk's), and the row's drafts.
    auto make_table = [&](int k, bool anew) {
      const int base = first + k * L::kTokens;
      if (anew) {
        if (nb) {
          __syncthreads();
          for (int i = tid; i < nb; i += kThreads) {
            s.bias_tok[i] = a.bias_tokens[(size_t)b * nb + i];
            s.bias[i] = a.bias[(size_t)b * nb + i];
          }
        }
        if (!arrived) {
          __syncthreads();  // the table has been read
          clear_table();
          cluster_arrive();
        }
        __syncthreads();
        arrived = false;
        cluster_wait();  // all slices are clear
        if (a.counted) {
          for (int i = (int)rank * kThreads + tid; i < n_tok; i += C * kThreads) {
            const int32_t x = a.tokens[(size_t)b * a.max_tokens + i];
            if (x < 0 || x >= a.V) continue;  // no logit: a placeholder
            const uint32_t r = (uint32_t)x / (uint32_t)a.slice;
            const int at = x - (int)r * a.slice - k * L::kTokens;
            if (at < 0 || at >= L::kTokens) continue;
            const uint32_t word = peer_address(table + at, r);
            if (i < n_prompt) peer_or(word, kPrompt);
            else peer_add(word, 1);
            peer_or(peer_address(map + (at >> 5), r), 1u << (at & 31));
          }
        }
        // Biases of this slice: the first entry of a token stands for all of them.
        for (int i = tid; i < nb; i += kThreads) {
          const int x = s.bias_tok[i], at = x - base;
          if (x < first || x >= last || at < 0 || at >= L::kTokens) continue;
          bool head = true;
          for (int e = 0; e < i; ++e) head &= s.bias_tok[e] != x;
          if (head) {
            atomicOr(table + at, (uint32_t)(i + 1) << kBiasShift);
            atomicOr(map + (at >> 5), 1u << (at & 31));
          }
        }
      }
      if (a.counted)
        for (int i = tid; i < a.n; i += kThreads) {
          const int now = s.on_path[i] & 1, was = anew ? 0 : s.on_path[i] >> 1;
          if (now == was) continue;
          const int x = a.drafts[(size_t)b * a.n + i], at = x - base;
          if (x < first || x >= last || at < 0 || at >= L::kTokens) continue;
          atomicAdd(table + at, (uint32_t)(now - was));
          atomicOr(map + (at >> 5), 1u << (at & 31));
        }
      if (anew) {
        cluster_arrive();
        cluster_wait();
      } else {
        __syncthreads();
      }
    };
    auto adjusted = [&](float y, int x, int base) {
      const uint32_t w = table[x - base];
      if (w & (kCountMask | kPrompt)) y = y > 0.f ? y / rep : y * rep;
      if (w & kCountMask) y = y - freq * (float)(w & kCountMask) - pres;
      if (w >> kBiasShift) {
        const int head = (int)(w >> kBiasShift) - 1;
        float sum = s.bias[head];  // in list order
        for (int e = head + 1; e < nb; ++e)
          if (s.bias_tok[e] == x) sum += s.bias[e];
        y += sum;
      }
      if (a.mask && !((mask_bytes[x >> 3] >> (x & 7)) & 1)) y = -INFINITY;
      return y;
    };

    float z[NV][8], keep[kKeep];
    // Logits of chunk k: the dense ones in z, -inf where the mask or the table takes them away;
    // the table's, taken one by one by each(y, i), i counting this thread's.
    auto take_chunk = [&](int k, bool table_kept, auto&& each) {
      const int base = first + k * L::kTokens;
      uint32_t allowed[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int x0 = base + L::at(v, 0);
        allowed[v] = 0xff;
        if (VEC) {
          if (a.mask) allowed[v] = x0 < last ? mask_bytes[x0 >> 3] : 0;
        } else if (a.mask) {
          allowed[v] = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int x = base + L::at(v, e);
            if (x < last) allowed[v] |= (uint32_t)((mask_bytes[x >> 3] >> (x & 7)) & 1) << e;
          }
        }
      }
      if (use_table && !table_kept) make_table(k, other || MULTI);
      const bool staged = !MULTI && a.staged;
      if (staged && bulk && !mbar_wait(&s.landed, nth & 1) && lane == 0)
        atomicOr(a.err, VAS_DEV_TIMEOUT);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int x0 = base + L::at(v, 0);
        if (VEC && x0 + 8 <= last) {
          load8(staged ? stage + (x0 - first) : in + x0, z[v]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int x = base + L::at(v, e);
            z[v][e] = x < last ? widen1(in[x]) : -INFINITY;
          }
        }
      }
      if (use_table)
        for (int i = tid; i < a.words / 32; i += kThreads) {
          int nth_one = 0;
          for (uint32_t bits = map[i]; bits; bits &= bits - 1, ++nth_one) {
            const int x = base + 32 * i + __ffs(bits) - 1;
            each(adjusted(widen1(in[x]), x, base), i == tid ? nth_one : kKeep, x);
          }
        }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        uint32_t on = allowed[v];
        if (use_table) {
          // (The table ends with the slice, before the registers' last places may.)
          if (VEC) {
            const int at = L::at(v, 0);
            if (at < a.words) on &= ~(uint32_t)reinterpret_cast<const uint8_t*>(map)[at >> 3];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int at = L::at(v, e);
              if (at < a.words) on &= ~(((map[at >> 5] >> (at & 31)) & 1) << e);
            }
          }
        }
        if (on != 0xff) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!((on >> e) & 1)) z[v][e] = -INFINITY;
        }
      }
    };
    auto store_chunk = [&](int k) {
      const int base = first + k * L::kTokens;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int x0 = base + L::at(v, 0);
        if (VEC && a.out_vec && x0 + 8 <= last) {
          float4* p = reinterpret_cast<float4*>(out + x0);
          __stcs(p, make_float4(z[v][0], z[v][1], z[v][2], z[v][3]));
          __stcs(p + 1, make_float4(z[v][4], z[v][5], z[v][6], z[v][7]));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int x = base + L::at(v, e);
            if (x < last) __stcs(out + x, z[v][e]);
          }
        }
      }
    };
    // The table's tokens behind the dense ones, whose stores they replace.
    auto store_table = [&](int k, auto&& value) {
      if (!use_table) return;
      const int base = first + k * L::kTokens;
      __syncthreads();
      for (int i = tid; i < a.words / 32; i += kThreads) {
        int nth_one = 0;
        for (uint32_t bits = map[i]; bits; bits &= bits - 1, ++nth_one) {
          const int x = base + 32 * i + __ffs(bits) - 1;
          float y;
          if (!MULTI && i == tid && nth_one < kKeep)
            y = nth_one == 0 ? keep[0] : (nth_one == 1 ? keep[1] : (nth_one == 2 ? keep[2] : keep[3]));
          else y = adjusted(widen1(in[x]), x, base);
          out[x] = value(y, x);
        }
      }
    };
    auto held = [&](float y, int i) {
      if (i == 0) keep[0] = y;
      else if (i == 1) keep[1] = y;
      else if (i == 2) keep[2] = y;
      else if (i == 3) keep[3] = y;
    };
    // The next row into the place that all threads have read.
    auto fetch_next = [&] {
      if (MULTI || !a.staged) return;
      __syncthreads();
      if (tid == 0 && row + 1 < row1) fetch(row + 1);
    };

    const int chunks = MULTI ? a.chunks : 1;
    if (!a.probs) {
      for (int k = 0; k < chunks; ++k) {
        take_chunk(k, false, [&](float y, int i, int) { held(y, i); });
        fetch_next();
        if (bad) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[v][e] = NAN;
        }
        store_chunk(k);
        store_table(k, [&](float y, int) { return bad ? NAN : y; });
      }
      seq = b;
      continue;
    }

    // Softmax: m is the maximum of what a thread, a warp, a CTA, the cluster holds, sum its
    // exponentials relative to m (0, or NaN, without a finite value); with temperature 0 best is
    // the first token at the maximum, and sum only carries a NaN.
    const bool greedy = temp == 0.f;
    // (An infinite temperature keeps the sign of -inf.)
    const float c = temp > 0.f ? fmaxf(1.4426950408889634f / temp, 0x1p-149f) : NAN;
    float m = -INFINITY, sum = 0.f, ref = 0.f;  // ref: the thread's, 0 where that is not finite
    int best = 0x7fffffff;
    auto join = [&](float om, float os, int ob) {
      const float nm = fmaxf(m, om), r = nm == -INFINITY ? 0.f : nm;
      if (greedy) sum += os;
      else
        sum = (m == -INFINITY ? sum : sum * exp2f((m - r) * c)) +
              (om == -INFINITY ? os : os * exp2f((om - r) * c));
      best = om > m || (om == m && ob < best) ? ob : best;
      m = nm;
    };
    for (int k = 0; k < chunks; ++k) {
      take_chunk(k, false, [&](float y, int i, int x) {
        held(y, i);
        join(y, isnan(y) ? NAN : (greedy || y == -INFINITY ? 0.f : 1.f), x);
      });
      fetch_next();
      float cm = -INFINITY;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) cm = fmaxf(cm, z[v][e]);
      if (greedy) {
        int at = 0x7fffffff;
        float wild = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (isnan(z[v][e])) wild = NAN;
            if (z[v][e] == cm) at = min(at, first + k * L::kTokens + L::at(v, e));
          }
        join(cm, wild, at);
      } else {
        ref = cm == -INFINITY ? 0.f : cm;
        float cs = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = ex2_approx((z[v][e] - ref) * c);
            if (!MULTI) z[v][e] = y;
            cs += y;
          }
        join(cm, cs, 0);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
      join(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, sum, o),
           __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) {
      s.red_max[warp] = m;
      s.red_sum[warp] = sum;
      s.red_at[warp] = best;
    }
    __syncthreads();
    if (arrived) {  // no table: the cluster is there
      arrived = false;
      cluster_wait();
    }
    const int side = nth & 1;
    if (warp == 0) {
      m = lane < kWarps ? s.red_max[lane] : -INFINITY;
      sum = lane < kWarps ? s.red_sum[lane] : 0.f;
      best = lane < kWarps ? s.red_at[lane] : 0x7fffffff;
#pragma unroll
      for (int o = kWarps / 2; o; o >>= 1)
        join(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, sum, o),
             __shfl_xor_sync(0xffffffffu, best, o));
      if (lane < C) {
        peer_store(peer_address(&s.peer_max[side][rank], lane), __float_as_uint(m));
        peer_store(peer_address(&s.peer_sum[side][rank], lane), __float_as_uint(sum));
        peer_store(peer_address(&s.peer_at[side][rank], lane), (uint32_t)best);
      }
    }
    cluster_arrive();
    cluster_wait();
    m = s.peer_max[side][0], sum = s.peer_sum[side][0], best = s.peer_at[side][0];
    for (int r = 1; r < C; ++r) join(s.peer_max[side][r], s.peer_sum[side][r], s.peer_at[side][r]);
    const float row_ref = m == -INFINITY ? 0.f : m;
    const bool wild = bad || isnan(sum);
    // A row without a token is 0 throughout.
    const float inv = wild ? NAN : (m == -INFINITY ? 0.f : 1.f / sum);
    // What the held exponentials, relative to the thread's maximum, are short of the row's.
    const float f = exp2f((ref - row_ref) * c) * inv;
    auto hot = [&](int x) { return wild ? NAN : (x == best && m != -INFINITY ? 1.f : 0.f); };
    for (int k = 0; k < chunks; ++k) {
      if (MULTI) take_chunk(k, false, [](float, int, int) {});
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (greedy) z[v][e] = hot(first + k * L::kTokens + L::at(v, e));
          else if (MULTI) z[v][e] = ex2_approx((z[v][e] - row_ref) * c) * inv;
          else z[v][e] *= f;
        }
      store_chunk(k);
      store_table(k, [&](float y, int x) {
        return greedy ? hot(x) : ex2_approx((y - row_ref) * c) * inv;
      });
    }
    seq = b;
  }
  if (arrived) cluster_wait();
}

namespace {

bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

template <typename T, bool VEC, int NV, bool MULTI>
int launch(Args& a, cudaStream_t stream) {
  constexpr int kTokens = Tile<T, VEC, NV>::kTokens;
  constexpr int kMost = 200 * 1024;
  static std::once_flag once[kMaxCachedDevices];
  static cudaError_t attr_err[kMaxCachedDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxCachedDevices) return VAS_E_CUDA;
  std::call_once(once[dev], [&] {
    attr_err[dev] = cudaFuncSetAttribute(spec_logits_kernel<T, VEC, NV, MULTI>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  });
  if (attr_err[dev] != cudaSuccess) return VAS_E_CUDA;
  const bool table = a.counted || a.max_bias > 0;
  a.chunks = MULTI ? (a.slice + kTokens - 1) / kTokens : 1;
  // Whole 16-byte groups of map words.
  a.words = table ? ((MULTI ? kTokens : a.slice) + 127) / 128 * 128 : 0;
  const int fixed = a.words * 4 + a.words / 8;
  const int place = (int)((a.slice * sizeof(T) + 15) / 16 * 16);
  // Rows by bulk copy where two CTAs of an SM still have room for it.
  a.staged = VEC && !MULTI && fixed + place <= 100 * 1024;
  const int smem = fixed + (a.staged ? place : 0);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // As many clusters as are on the GPU at once; the answer for the last shape is kept.
  static std::atomic<uint64_t> known[kMaxCachedDevices];
  const uint64_t shape = ((uint64_t)smem << 8 | (uint64_t)a.cluster) << 20;
  uint64_t k = known[dev].load(std::memory_order_relaxed);
  if (k >> 20 != shape >> 20) {
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, spec_logits_kernel<T, VEC, NV, MULTI>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return VAS_E_CUDA;
    }
    k = shape | (uint64_t)std::max(1, std::min(n, 4096));
    known[dev].store(k, std::memory_order_relaxed);
  }
  const int most = (int)(k & 0xfffff);
  a.clusters = a.rows < most ? a.rows : most;
  cfg.gridDim = dim3((unsigned)(a.cluster * a.clusters));
  if (cudaLaunchKernelEx(&cfg, spec_logits_kernel<T, VEC, NV, MULTI>, a) != cudaSuccess) {
    cudaGetLastError();
    return VAS_E_CUDA;
  }
  return VAS_OK;
}

template <typename T, bool VEC>
int launch_size(Args& a, cudaStream_t stream) {
  // As many CTAs a row as have at least 8 logits a thread, at most a portable cluster.
  int cluster = (a.V + kThreads * 8 - 1) / (kThreads * 8);
  if (cluster > kMaxCluster) cluster = kMaxCluster;
  a.slice = ((a.V + cluster - 1) / cluster + 31) / 32 * 32;
  a.cluster = cluster;
  const int per = (a.slice + kThreads * 8 - 1) / (kThreads * 8);
  if (per <= 1) return launch<T, VEC, 1, false>(a, stream);
  if (per <= 4) return launch<T, VEC, 4, false>(a, stream);
  if (per <= 8) return launch<T, VEC, 8, false>(a, stream);
  return launch<T, VEC, 4, true>(a, stream);
}

}  // namespace
}  // namespace logits
}  // namespace vas

extern "C" int spec_logits(const void* logits, const int32_t* tokens, const int32_t* token_lens,
                           const int32_t* prompt_lens, const int32_t* draft_tokens,
                           const int32_t* parents, const float* repetition, const float* frequency,
                           const float* presence, const int32_t* bias_tokens, const float* bias,
                           const uint32_t* mask, const float* temperature, float* out,
                           const vas_logits_dims* dims, vas_stream_t stream) {
  using namespace vas::logits;
  if (!dims) return VAS_E_INVALID_ARG;
  const vas_logits_dims& d = *dims;
  if (d.num_seqs < 0 || d.num_drafts < 0 || d.num_drafts > kMaxNodes || d.vocab <= 0 ||
      d.max_tokens < 0 || d.max_bias < 0)
    return VAS_E_INVALID_ARG;
  if (d.out_kind != VAS_LOGITS && d.out_kind != VAS_PROBS) return VAS_E_INVALID_ARG;
  if ((d.dtype != VAS_F32 && d.dtype != VAS_BF16) || d.vocab > 1048576 ||
      d.max_tokens >= kMaxTokens - kMaxNodes || d.max_bias > kMaxBias)
    return VAS_E_UNSUPPORTED;
  if (d.row_stride < d.vocab) return VAS_E_INVALID_ARG;
  if (d.out_kind == VAS_LOGITS && temperature) return VAS_E_INVALID_ARG;
  if ((tokens != nullptr) != (token_lens != nullptr) || (prompt_lens && !tokens)) return VAS_E_INVALID_ARG;
  if ((bias_tokens != nullptr) != (bias != nullptr)) return VAS_E_INVALID_ARG;
  if (parents && !draft_tokens) return VAS_E_INVALID_ARG;
  if (d.num_seqs == 0) return VAS_OK;
  if (!logits || !out) return VAS_E_INVALID_ARG;
  const bool counted = repetition || frequency || presence;
  if (counted && d.num_drafts > 0 && !draft_tokens) return VAS_E_INVALID_ARG;
  const int es = d.dtype == VAS_F32 ? 4 : 2;
  if (misaligned(logits, es) || misaligned(tokens, 4) || misaligned(token_lens, 4) ||
      misaligned(prompt_lens, 4) || misaligned(draft_tokens, 4) || misaligned(parents, 4) ||
      misaligned(repetition, 4) || misaligned(frequency, 4) || misaligned(presence, 4) ||
      misaligned(bias_tokens, 4) || misaligned(bias, 4) || misaligned(mask, 4) ||
      misaligned(temperature, 4) || misaligned(out, 4))
    return VAS_E_INVALID_ARG;
  const int64_t rows = (int64_t)d.num_seqs * (d.num_drafts + 1);
  if (rows > INT32_MAX / kMaxCluster) return VAS_E_UNSUPPORTED;
  const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(out);
  const uintptr_t xn = (uintptr_t)(((rows - 1) * d.row_stride + d.vocab) * es);
  const uintptr_t yn = (uintptr_t)(rows * d.vocab * 4);
  if (x < y + yn && y < x + xn) return VAS_E_INVALID_ARG;  // read and written
  Args a;
  a.logits = logits;
  a.tokens = tokens;
  a.token_lens = token_lens;
  a.prompt_lens = prompt_lens;
  a.drafts = draft_tokens;
  a.parents = parents;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_tokens = bias_tokens;
  a.bias = bias;
  a.mask = mask;
  a.temperature = temperature;
  a.out = out;
  a.row_stride = d.row_stride;
  a.n = d.num_drafts;
  a.V = d.vocab;
  a.max_tokens = d.max_tokens;
  a.max_bias = bias_tokens ? d.max_bias : 0;
  a.mask_words = (d.vocab + 31) / 32;
  a.probs = d.out_kind == VAS_PROBS;
  a.counted = counted ? 1 : 0;
  a.out_vec = !misaligned(out, 16) && d.vocab % 4 == 0;
  a.err = vas::device_error_word();
  a.rows = (int)rows;
  if (!a.err || !vas::num_sms()) return VAS_E_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = !misaligned(logits, 16) && d.row_stride * es % 16 == 0;
  if (d.dtype == VAS_F32)
    return vec ? launch_size<float, true>(a, st) : launch_size<float, false>(a, st);
  return vec ? launch_size<__nv_bfloat16, true>(a, st)
             : launch_size<__nv_bfloat16, false>(a, st);
}
