// The 4-bit cache: a row of 128 values is 64 bytes of e2m1 codes (two to a byte, the first in the low
// half) and eight e4m3 scales, one for every 16 codes; value = code * scale * descale, with one fp32
// descale per tensor or KV head.  Here: new bf16 tokens quantised into it.
//
//   scale = the e4m3 number nearest to amax / (6 descale),  code = the e2m1 number nearest to
//   x / (scale * descale), ties to the even code, 448 and 6 the largest
//
// decided exactly, not on rounded quotients.  That matters more than it seems to: a descale is often some
// largest value over 6 * 448 = 2^7 * 21, so that quotients next to the borders at 7/4 and 7/2 are
// common (one value in six hundred), and fp32 puts them on the border.  A quotient estimated to
// 2^-21 is converted twice, nudged up and down by 2^-20; where the two codes differ the border between
// them, times scale and descale, is compared with the value itself by the sign of one fma, which rounds
// but never crosses zero.
//
// 256 bytes of a row read, 72 written.  A thread has one block of 16 values of K and the same of V,
// eight threads a row.  The integer pipe is what is busiest (71%; HBM 50%), much of it with this form's
// own work and not the operator's: two conversions of every value to find the rare ones next to a
// border, maxima of unpacked values.
//
// Measured: 64K tokens x 8 heads, NHD pages (344 MB) 74 us, 70% of the measured copy rate (with
// 64-bit divisions and the rare borders settled in four places 95).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_div.cuh"
#include "bsa_quant.cuh"
#include "ptx_sm103.cuh"

namespace bsa {
namespace fp4 {

constexpr int BLOCK = 16;                     // codes to a scale
constexpr int BLOCKS = HEAD_DIM / BLOCK;      // scales of a row
constexpr int ROW_BYTES = HEAD_DIM / 2;       // codes of a row
constexpr int THREADS = 256;

struct AppendParams {
  const __nv_bfloat16 *k_new, *v_new;
  long long k_stride, v_stride;  // elements from token to token
  const int *slot_map;
  const float *k_descale, *v_descale;
  uint8_t *k_pages, *v_pages, *k_scales, *v_scales;
  int *dev_status;
  uint32_t rows;  // tokens x KV heads, below 2^31
  Divisor heads;
  int N2, ps_shift, num_pages;
  int k_per_head, v_per_head, kv_nhd;
};

__device__ __forceinline__ uint32_t e4m3_of(float x) {  // of one non-negative value
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 c, %1, %1;\n\t"
      "cvt.u32.u16 %0, c;\n\t}"
      : "=r"(r)
      : "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float value_of_e4m3(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\t"
      "cvt.u16.u32 a, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(c & 0xffu));
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// e2m1 codes of eight values (as pairs), the first in the lowest half byte.
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t (&v)[4]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) ptx::upk(v[i], x[2 * i], x[2 * i + 1]);
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// The size of an e2m1 code (0 .. 7), doubled: 0 1 2 3 4 6 8 12.
__device__ __forceinline__ int twice_e2m1(uint32_t c) {
  const int e = c >> 1, m = c & 1;
  return e == 0 ? m : (2 + m) << (e - 1);
}

// 1 / x to 2^-22, 0 for an x of zero or next to it.
__device__ __forceinline__ float inverse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return x > 0x1p-120f ? r : 0.f;
}

constexpr float NUDGE_UP = 1.f + 0x1p-20f, NUDGE_DOWN = 1.f - 0x1p-20f;

// Which of two neighbouring codes (`down`, `down` + 1) is nearer: the sign of the value less the border
// between them, zero for a tie.
__device__ __forceinline__ uint32_t settle(uint32_t down, float above) {
  return above > 0.f || (above == 0.f && (down & 1u)) ? down + 1 : down;
}

// A power of two that brings a descale to where neither its reciprocal nor a product leaves fp32's
// normal numbers.  Values are multiplied by it too: exactly, but for those beyond fp32, which are
// beyond 448 * 6 descales, and those below 2^-149, which are below a code's first border.
__device__ __forceinline__ float lift_of(float descale) {
  return descale < 0x1p-60f ? 0x1p64f : descale > 0x1p60f ? 0x1p-64f : 1.f;
}

// The scale of a block whose largest magnitude is amax, as a code.
__device__ __forceinline__ uint32_t scale_of(float amax, float descale, float inv6) {
  const float t = amax * inv6;
  const uint32_t up = e4m3_of(t * NUDGE_UP), down = e4m3_of(t * NUDGE_DOWN);
  if (up == down) return up;
  const float border = 0.5f * (value_of_e4m3(down) + value_of_e4m3(up));
  return settle(down, fmaf(-6.f * border, descale, amax));
}

// Where the nudged codes of a block differ: the exact decision, a value at a time (read again from
// where it came: a register cannot be picked by number).
__device__ __forceinline__ void settle_codes(uint32_t (&up)[2], const uint32_t (&down)[2],
                                             const __nv_bfloat16 *x, float scale, float descale,
                                             float lift) {
  uint64_t w = (uint64_t)up[1] << 32 | up[0];
  const uint64_t other = (uint64_t)down[1] << 32 | down[0];
  uint64_t differ = (w ^ other) & 0x7777777777777777ull;
#pragma unroll 1
  while (differ) {
    const int i = (__ffsll((long long)differ) - 1) >> 2, at = 4 * i;
    const uint32_t u = (uint32_t)(w >> at) & 7u, d = (uint32_t)(other >> at) & 7u;
    // the border is (twice one + twice the other) / 4, exact with the scale
    const float border = 0.25f * (float)(twice_e2m1(u) + twice_e2m1(d)) * scale;
    const float size = fabsf(__bfloat162float(x[i])) * lift;
    w = (w & ~(7ull << at)) | (uint64_t)settle(d, fmaf(-border, descale, size)) << at;
    differ &= ~(0xfull << at);
  }
  up[0] = (uint32_t)w;
  up[1] = (uint32_t)(w >> 32);
}

// One block of 16 values, at x: their codes and scale.
__device__ __forceinline__ void store_block(const uint4 &a, const uint4 &b,
                                            const __nv_bfloat16 *from, float descale,
                                            uint8_t *codes, uint8_t *scale_at) {
  const float lift = lift_of(descale);
  descale *= lift;
  const uint32_t word[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float lo[8], hi[8], amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = __uint_as_float(word[i] << 16);
    hi[i] = __uint_as_float(word[i] & 0xffff0000u);
    amax = fmaxf(amax, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
  if (lift != 1.f) {
    amax *= lift;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] *= lift;
      hi[i] *= lift;
    }
  }
  const uint32_t s = scale_of(amax, descale, inverse(6.f * descale));
  const float scale = value_of_e4m3(s), d = scale * descale, r = inverse(d);
  const uint64_t up = ptx::pk(r * NUDGE_UP, r * NUDGE_UP),
                 down = ptx::pk(r * NUDGE_DOWN, r * NUDGE_DOWN);
  uint32_t w[2], other[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t u[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = ptx::pk(lo[4 * h + i], hi[4 * h + i]);
      u[i] = ptx::mul2(x, up);
      v[i] = ptx::mul2(x, down);
    }
    w[h] = e2m1x8(u);
    other[h] = e2m1x8(v);
  }
  if (w[0] != other[0] || w[1] != other[1]) settle_codes(w, other, from, scale, descale, lift);
  *reinterpret_cast<uint2 *>(codes) = make_uint2(w[0], w[1]);
  *scale_at = (uint8_t)s;
}

__global__ void __launch_bounds__(THREADS) append_kernel(const AppendParams p) {
  const int block = threadIdx.x & (BLOCKS - 1);
  const uint32_t row = blockIdx.x * (THREADS / BLOCKS) + threadIdx.x / BLOCKS;
  if (row >= p.rows) return;
  const uint32_t tok = p.heads.quotient(row);
  const int g = (int)(row - tok * p.N2);
  const int at = g * HEAD_DIM + block * BLOCK;
  const uint4 *k = reinterpret_cast<const uint4 *>(p.k_new + tok * p.k_stride + at);
  const uint4 *v = reinterpret_cast<const uint4 *>(p.v_new + tok * p.v_stride + at);
  const uint4 k0 = k[0], k1 = k[1], v0 = v[0], v1 = v[1];
  const int slot = p.slot_map[tok];
  const float kg = p.k_descale[p.k_per_head ? g : 0], vg = p.v_descale[p.v_per_head ? g : 0];
  if (slot < 0) return;  // a row without a place
  const int page = slot >> p.ps_shift, in = slot & ((1 << p.ps_shift) - 1);
  if (page >= p.num_pages) {
    if (p.dev_status) atomicOr(p.dev_status, BSA_DEV_BAD_PAGE);
    return;
  }
  const long long hnd = (((long long)page * p.N2 + g) << p.ps_shift) + in;
  const long long dst = p.kv_nhd ? (((long long)page << p.ps_shift) + in) * p.N2 + g : hnd;
  store_block(k0, k1, p.k_new + tok * p.k_stride + at, kg,
              p.k_pages + dst * ROW_BYTES + block * (BLOCK / 2), p.k_scales + hnd * BLOCKS + block);
  store_block(v0, v1, p.v_new + tok * p.v_stride + at, vg,
              p.v_pages + dst * ROW_BYTES + block * (BLOCK / 2), p.v_scales + hnd * BLOCKS + block);
}

}  // namespace fp4
}  // namespace bsa
