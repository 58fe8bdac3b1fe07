// The paged e4m3 cache read back into contiguous rows: value = code * descale.
//
// The simplest form: one CTA per row, a thread per dimension.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "bsa_common.cuh"

namespace bsa {
namespace gather {

constexpr int THREADS = 128;

struct Params {
  const uint8_t *k_pages, *v_pages;
  const float *k_descale, *v_descale;
  const int *cu_seqlens, *cache_starts, *block_table;
  void *k_out, *v_out;
  int *dev_status;
  long long page_bytes, head_bytes, slot_bytes;
  int B, N2, ps, num_pages, L, total;
  int k_per_token, v_per_head;
};

template <typename Out>
__device__ __forceinline__ void put(void *out, size_t i, float v) {
  static_cast<Out *>(out)[i] = static_cast<Out>(v);
}

template <typename Out>
__global__ void __launch_bounds__(THREADS) gather_kernel(const Params p) {
  const int tok = blockIdx.x, d = threadIdx.x;
  if (tok >= p.cu_seqlens[p.B]) return;  // rows behind the last sequence stay as they are
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_seqlens[mid] <= tok) lo = mid; else hi = mid - 1;
  }
  const long long pos = (long long)(p.cache_starts ? p.cache_starts[lo] : 0) + tok -
                        p.cu_seqlens[lo];
  const long long lp = pos / p.ps;
  int pg = pos >= 0 && lp < p.L ? p.block_table[(size_t)lo * p.L + lp] : -1;
  if (pg < 0 || pg >= p.num_pages) {
    if (d == 0 && p.dev_status) atomicOr(p.dev_status, BSA_DEV_BAD_PAGE);
    pg = -1;
  }
  const int slot = (int)(pos % p.ps);
  for (int g = 0; g < p.N2; ++g) {
    float k = 0.f, v = 0.f;
    if (pg >= 0) {
      const size_t at = pg * p.page_bytes + g * p.head_bytes + slot * p.slot_bytes + d;
      __nv_fp8_e4m3 c;
      if (p.k_out) {
        c.__x = p.k_pages[at];
        k = static_cast<float>(c) * (p.k_per_token
                                         ? p.k_descale[((size_t)pg * p.N2 + g) * p.ps + slot]
                                         : p.k_descale[0]);
      }
      if (p.v_out) {
        c.__x = p.v_pages[at];
        v = static_cast<float>(c) * (p.v_per_head ? p.v_descale[g] : p.v_descale[0]);
      }
    }
    const size_t o = ((size_t)tok * p.N2 + g) * HEAD_DIM + d;
    if (p.k_out) put<Out>(p.k_out, o, k);
    if (p.v_out) put<Out>(p.v_out, o, v);
  }
}

}  // namespace gather
}  // namespace bsa
