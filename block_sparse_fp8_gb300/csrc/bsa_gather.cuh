// The paged e4m3 cache read back into contiguous rows: value = code * descale, one fp32 product,
// rounded once more for bf16.
//
// HBM-bound (a KV head's token: 256 bytes of codes and 4 of descale in, 512 or 1024 out).  A block
// takes a run of tokens.  Its first threads look the tokens up -- the sequence by binary search over
// cu_seqlens, then the block table -- and leave page and slot in shared memory, so that the
// dependent reads are paid once a token and not once a row.  Then a row of 128 values belongs to
// 16 lanes, each of which turns 8 codes into one 16-byte store (bf16: 8 neighbours) or two (fp32: 4
// neighbours of each half, so that either store covers 256 bytes in a row); a thread has the K and
// V codes of ROWS rows in flight.
//
// Measured (mean of back-to-back calls): 4 x 64K tokens x 8 heads to bf16 (1619 MB) 244 us, 6.63
// TB/s, 98% of the measured copy rate (two rows in flight: 247; one block a row, the first form: 1044);
// 22K tokens x 8 heads to fp32 (224 MB) 35 us, 94%.
//
// 4-bit pages (bsa_fp4.cuh) have a kernel of their own over the same blocks of tokens: there a thread
// has 16 codes of K or of V and their scale, and writes 32 bytes at once.  64K tokens x 8 heads to bf16
// (344 MB) 59 us, 87% (eight rows in flight a thread 89, two 63, blocks of 32 tokens 61).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_fp4.cuh"

namespace bsa {
namespace gather {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 32;  // tokens of a block
constexpr int ROWS = 4;         // rows in flight per thread

struct Params {
  const uint8_t *k_pages, *v_pages;
  const uint8_t *k_scales, *v_scales;  // 4-bit pages
  const float *k_descale, *v_descale;
  const int *cu_seqlens, *cache_starts, *block_table;
  void *k_out, *v_out;
  int *dev_status;
  long long page_bytes, head_bytes, slot_bytes;
  int B, N2, ps, num_pages, L, total;
  int k_per_token, k_per_head, v_per_head;
  int tokens;  // of a block, a power of two up to MAX_TOKENS
};

// Two e4m3 codes (the low 16 bits) as fp32.
__device__ __forceinline__ float2 values2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(codes));
  __half2 x;
  memcpy(&x, &h, 4);
  return __half22float2(x);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  uint32_t r;
  memcpy(&r, &x, 4);
  return r;
}

constexpr int LANES = 16;                // of a row
constexpr int STEP = THREADS / LANES;    // rows of a block's pass

// Lane li's 8 codes of the row at p.
template <bool F32>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int li) {
  if (!F32) return reinterpret_cast<const uint2 *>(p)[li];
  return make_uint2(reinterpret_cast<const uint32_t *>(p)[li],
                    reinterpret_cast<const uint32_t *>(p)[li + 16]);
}

// ... and their values, into the row at out.
template <bool F32>
__device__ __forceinline__ void store_values(void *out, size_t row, int li, uint2 c, float s) {
  const float2 a = values2(c.x), b = values2(c.x >> 16), d = values2(c.y), e = values2(c.y >> 16);
  if (F32) {
    float4 *o = static_cast<float4 *>(out) + row * (HEAD_DIM / 4) + li;
    __stcs(o, make_float4(a.x * s, a.y * s, b.x * s, b.y * s));
    __stcs(o + 16, make_float4(d.x * s, d.y * s, e.x * s, e.y * s));
  } else {
    __stcs(static_cast<uint4 *>(out) + row * (HEAD_DIM / 8) + li,
           make_uint4(bf16x2(a.x * s, a.y * s), bf16x2(b.x * s, b.y * s),
                      bf16x2(d.x * s, d.y * s), bf16x2(e.x * s, e.y * s)));
  }
}

// Page and slot of each of the block's tokens, in shared memory (a barrier after it).
__device__ __forceinline__ void look_up(const Params &p, int t0, int *s_page, int *s_slot) {
  const int tid = threadIdx.x;
  if (tid < p.tokens) {
    const int tok = t0 + tid;
    int page = -2, slot = 0;  // -2: a row behind the last sequence, left as it is
    if (tok < p.total && tok >= p.cu_seqlens[0] && tok < p.cu_seqlens[p.B]) {
      int lo = 0, hi = p.B - 1;  // the last b with cu_seqlens[b] <= tok
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[mid] <= tok) lo = mid; else hi = mid - 1;
      }
      const long long pos =
          (long long)(p.cache_starts ? p.cache_starts[lo] : 0) + (tok - p.cu_seqlens[lo]);
      const long long lp = pos / p.ps;
      page = pos >= 0 && lp < p.L ? p.block_table[(size_t)lo * p.L + lp] : -1;
      slot = (int)(pos & (p.ps - 1));
      if (page < 0 || page >= p.num_pages) {
        if (p.dev_status) atomicOr(p.dev_status, BSA_DEV_BAD_PAGE);
        page = -1;
      }
    }
    s_page[tid] = page;
    s_slot[tid] = slot;
  }
}

template <bool F32>
__global__ void __launch_bounds__(THREADS) gather_kernel(const Params p) {
  __shared__ int s_page[MAX_TOKENS], s_slot[MAX_TOKENS];
  const int tid = threadIdx.x, t0 = blockIdx.x * p.tokens;
  look_up(p, t0, s_page, s_slot);
  __syncthreads();
  // The block's rows (token, head), token-major: a thread's next row lies STEP rows on.
  const int li = tid % LANES, dt = STEP / p.N2, dg = STEP % p.N2;
  const float k_all = p.k_per_token || !p.k_out ? 0.f : p.k_descale[0];
  const float v_all = p.v_per_head || !p.v_out ? 0.f : p.v_descale[0];
  int t = tid / LANES / p.N2, g = tid / LANES - t * p.N2;
  while (t < p.tokens) {
    uint2 k[ROWS], v[ROWS];
    float ks[ROWS], vs[ROWS];
    int page[ROWS];
    size_t row[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      page[i] = t < p.tokens ? s_page[t] : -2;
      row[i] = (size_t)(t0 + t) * p.N2 + g;
      k[i] = v[i] = make_uint2(0, 0);
      ks[i] = k_all;
      vs[i] = v_all;
      if (page[i] >= 0) {
        const int slot = s_slot[t];
        const long long off = page[i] * p.page_bytes + g * p.head_bytes + slot * p.slot_bytes;
        if (p.k_out) {
          k[i] = load_codes<F32>(p.k_pages + off, li);
          if (p.k_per_token) ks[i] = p.k_descale[((size_t)page[i] * p.N2 + g) * p.ps + slot];
        }
        if (p.v_out) {
          v[i] = load_codes<F32>(p.v_pages + off, li);
          if (p.v_per_head) vs[i] = p.v_descale[g];
        }
      }
      t += dt;
      g += dg;
      if (g >= p.N2) {
        g -= p.N2;
        ++t;
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (page[i] == -2) continue;
      // a missing page's codes are zero: so are its values, whatever the descale
      const bool none = page[i] < 0;
      if (p.k_out) store_values<F32>(p.k_out, row[i], li, k[i], none ? 0.f : ks[i]);
      if (p.v_out) store_values<F32>(p.v_out, row[i], li, v[i], none ? 0.f : vs[i]);
    }
  }
}

// ------------------------------------------------------------------------------------------
// 4-bit pages: a thread has a block of 16 codes of K (lanes 0 to 7 of a row's 16) or of V.
// ------------------------------------------------------------------------------------------

// 16 codes times their scale, in fp16, exactly.
__device__ __forceinline__ void scaled16(uint2 c, uint32_t scale, uint32_t (&h)[8]) {
  uint32_t f;
  asm("{\n\t.reg .b16 s;\n\t"
      "cvt.u16.u32 s, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, s;\n\t}"
      : "=r"(f)
      : "r"(scale | scale << 8));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[4 * i]), "=r"(h[4 * i + 1]), "=r"(h[4 * i + 2]), "=r"(h[4 * i + 3])
        : "r"(i == 0 ? c.x : c.y));
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(f));
}

// 32 bytes at once; at least 16-byte aligned, 32 with `wide`.
__device__ __forceinline__ void store32(void *o, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4 *>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4 *>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <bool F32>
__global__ void __launch_bounds__(THREADS) gather_fp4_kernel(const Params p) {
  __shared__ int s_page[MAX_TOKENS], s_slot[MAX_TOKENS];
  const int tid = threadIdx.x, t0 = blockIdx.x * p.tokens;
  look_up(p, t0, s_page, s_slot);
  const int block = tid & (fp4::BLOCKS - 1);
  const bool is_v = tid & fp4::BLOCKS;
  void *const out = is_v ? p.v_out : p.k_out;
  const uint8_t *const pages = (is_v ? p.v_pages : p.k_pages) + block * (fp4::BLOCK / 2);
  const uint8_t *const scales = (is_v ? p.v_scales : p.k_scales) + block;
  const float *const descale = is_v ? p.v_descale : p.k_descale;
  const bool per_head = is_v ? p.v_per_head : p.k_per_head;
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  __syncthreads();
  if (!out) return;
  const int dt = STEP / p.N2, dg = STEP % p.N2;
  int t = tid / LANES / p.N2, g = tid / LANES - t * p.N2;
  while (t < p.tokens) {
    uint2 c[ROWS];
    uint32_t e[ROWS];
    float s[ROWS];
    int page[ROWS];
    size_t row[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      page[i] = t < p.tokens ? s_page[t] : -2;
      row[i] = (size_t)(t0 + t) * p.N2 + g;
      c[i] = make_uint2(0, 0);
      e[i] = 0u;
      s[i] = 0.f;
      if (page[i] >= 0) {
        const int slot = s_slot[t];
        const long long off = page[i] * p.page_bytes + g * p.head_bytes + slot * p.slot_bytes;
        c[i] = *reinterpret_cast<const uint2 *>(pages + off);
        e[i] = scales[(((size_t)page[i] * p.N2 + g) * p.ps + slot) * fp4::BLOCKS];
        s[i] = descale[per_head ? g : 0];
      }
      t += dt;
      g += dg;
      if (g >= p.N2) {
        g -= p.N2;
        ++t;
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (page[i] == -2) continue;
      uint32_t h[8], w[F32 ? 16 : 8];
      scaled16(c[i], e[i], h);
      const uint64_t ss = ptx::pk(s[i], s[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        __half2 x;
        memcpy(&x, &h[k], 4);
        const float2 y = __half22float2(x);
        float lo, hi;
        ptx::upk(ptx::mul2(ptx::pk(y.x, y.y), ss), lo, hi);
        if (F32) {
          w[2 * k] = __float_as_uint(lo);
          w[2 * k + 1] = __float_as_uint(hi);
        } else {
          w[k] = bf16x2(lo, hi);
        }
      }
      uint8_t *o = static_cast<uint8_t *>(out) + row[i] * HEAD_DIM * (F32 ? 4 : 2) +
                   block * fp4::BLOCK * (F32 ? 4 : 2);
      uint32_t part[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) part[k] = w[k];
      store32(o, part, wide);
      if (F32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) part[k] = w[F32 ? 8 + k : k];
        store32(o + 32, part, wide);
      }
    }
  }
}

}  // namespace gather
}  // namespace bsa
