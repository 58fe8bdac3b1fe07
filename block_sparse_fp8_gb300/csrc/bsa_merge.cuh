// Join of attention results over disjoint sets of keys:
//   M = max_i LSE_i, w_i = exp(LSE_i - M), O = sum_i w_i O_i / sum_i w_i, LSE = M + ln sum_i w_i.
//
// The simplest form: one CTA per row, a thread per dimension.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>
#include <cstdint>

#include "bsa_common.cuh"

namespace bsa {
namespace merge {

constexpr int THREADS = 128;

struct Params {
  // no __restrict__: out may be one of outs, lse one of lses
  const __nv_bfloat16 *outs[BSA_MAX_MERGE];
  const float *lses[BSA_MAX_MERGE];
  __nv_bfloat16 *out;
  float *lse;
  int count, T, N1;
};

__global__ void __launch_bounds__(THREADS) merge_kernel(const Params p) {
  const int t = blockIdx.x / p.N1, h = blockIdx.x % p.N1, d = threadIdx.x;
  const size_t li = (size_t)h * p.T + t, oi = (size_t)blockIdx.x * HEAD_DIM + d;
  float m = -INFINITY;
  for (int i = 0; i < p.count; ++i)
    if (p.lses[i][li] != -FLT_MAX) m = fmaxf(m, p.lses[i][li]);
  float l = 0.f, o = 0.f;
  for (int i = 0; i < p.count; ++i) {
    const float x = p.lses[i][li];
    if (x == -FLT_MAX || x == -INFINITY) continue;
    const float w = expf(x - m);
    l += w;
    o += w * __bfloat162float(p.outs[i][oi]);
  }
  __syncthreads();  // every read of the row's LSE is done before it may be overwritten
  p.out[oi] = __float2bfloat16(l != 0.f ? o / l : 0.f);
  if (d == 0 && p.lse) p.lse[li] = l != 0.f ? m + logf(l) : -FLT_MAX;
}

}  // namespace merge
}  // namespace bsa
