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

// One warp per row, CUDA-core arithmetic.
template <int D, int KV>
__global__ void __launch_bounds__(256) prefix_simple_kernel(const PrefixArgs a) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float qs[8][D];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int32_t n_units = a.header->n_prefix_items * a.Hkv;
  for (int32_t u = blockIdx.x; u < n_units; u += gridDim.x) {
    const PrefixItem it = a.items[u / a.Hkv];
    const int head = u % a.Hkv;
    const PrefixGroup g = a.groups[it.group];
    const int split = it.split_rb >> kPrefixRbBits;
    const int r0 = (it.split_rb & ((1 << kPrefixRbBits) - 1)) * kPrefixRows;
    const int r1 = min(r0 + kPrefixRows, g.rows);
    const int32_t* bt = a.block_table + (size_t)g.leader * a.maxp;
    for (int r = r0 + warp; r < r1; r += 8) {
      const int t = g.qrow0 + r / a.G;
      const int hh = head * a.G + r % a.G;
      const __nv_bfloat16* q =
          static_cast<const __nv_bfloat16*>(a.q) + ((size_t)t * a.Hq + hh) * D;
      __syncwarp();
      for (int e = 0; e < E; ++e) qs[warp][lane + 32 * e] = __bfloat162float(q[lane + 32 * e]);
      __syncwarp();
      float acc[E] = {}, m = -INFINITY, l = 0.f;
      bool bad = false;
      for (int x0 = it.page_begin * a.P; x0 < it.page_end * a.P; x0 += 32) {
        const int x = x0 + lane;
        int page = -1;
        float s = -INFINITY;
        if (x < it.page_end * a.P) {
          page = bt[x / a.P];
          if (page < 0 || page >= a.num_pages) {
            bad = true;
            page = -1;
          } else {
            const size_t at = (((size_t)page * a.P + x % a.P) * a.Hkv + head) * D;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(qs[warp][d], kv_value<KV>(a.k_pages, at + d), dot);
            if constexpr (KV != VAS_BF16)
              dot *= a.k_scale[((size_t)page * a.Hkv + head) * a.P + x % a.P];
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
          if (page >= 0) p *= a.v_scale[((size_t)page * a.Hkv + head) * a.P + x % a.P];
        }
        for (int e = 0; e < E; ++e) acc[e] *= f;
        for (int j = 0; j < 32 && x0 + j < it.page_end * a.P; ++j) {
          const float pj = __shfl_sync(0xffffffffu, p, j);
          const int pg = __shfl_sync(0xffffffffu, page, j);
          if (pg < 0) continue;
          const size_t at = (((size_t)pg * a.P + (x0 + j) % a.P) * a.Hkv + head) * D;
          for (int e = 0; e < E; ++e)
            acc[e] = fmaf(pj, kv_value<KV>(a.v_pages, at + lane + 32 * e), acc[e]);
        }
      }
      bad = __any_sync(0xffffffffu, bad);
      const SeqPlan sp = a.seqplan[member_of(a, g, t)];
      const size_t row = partial_index(sp, a.Hkv, a.G, sp.nsplit - g.nsplit + split, head,
                                       (t - sp.qrow0) * a.G + r % a.G);
      for (int e = 0; e < E; ++e)
        a.part_o[row * D + lane + 32 * e] = bad ? NAN : (l > 0.f ? acc[e] / l : 0.f);
      if (lane == 0) {
        a.part_lse[row] = bad ? NAN : (m + log2f(l)) * 0.6931471805599453f;
        if (bad) atomicOr(a.err, VAS_DEV_BAD_PAGE);
      }
    }
  }
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

int launch_prefix(const CUtensorMap&, const CUtensorMap&, const PrefixArgs& a, int head_dim,
                  int kv_dtype, void* stream) {
  const int grid = 4 * num_sms();
  if (head_dim == 128) {
    if (kv_dtype == VAS_BF16) return launch(prefix_simple_kernel<128, VAS_BF16>, a, grid, 256, stream);
    if (kv_dtype == VAS_FP8_E4M3)
      return launch(prefix_simple_kernel<128, VAS_FP8_E4M3>, a, grid, 256, stream);
    return launch(prefix_simple_kernel<128, VAS_INT8>, a, grid, 256, stream);
  }
  if (kv_dtype == VAS_BF16) return launch(prefix_simple_kernel<64, VAS_BF16>, a, grid, 256, stream);
  if (kv_dtype == VAS_FP8_E4M3)
    return launch(prefix_simple_kernel<64, VAS_FP8_E4M3>, a, grid, 256, stream);
  return launch(prefix_simple_kernel<64, VAS_INT8>, a, grid, 256, stream);
}

}  // namespace attn
}  // namespace vas
