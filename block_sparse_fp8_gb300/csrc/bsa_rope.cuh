// Rotary positions: pairs of a head's first R values are turned by position x frequency,
//   (x, y) -> amplitude * (x cos a - y sin a, y cos a + x sin a),  a = 2 pi frac(position f_i),
// pair i being (i, i + R/2) or (2i, 2i + 1); the rest of the head is copied.  Either bf16 -> bf16 for Q
// and K at once, or bf16 -> e4m3 codes and a descale per row for Q (bsa_quant.cuh's rule on the
// turned values, which are not rounded to bf16 in between).
//
// A frequency is a 64-bit fixed-point fraction of a turn, and the product with the position is taken
// modulo a turn by the integers' own overflow: exact to 2^-33 turns for any 32-bit position, where an
// fp32 product at position 500,000 is off by up to 0.03 radians.
//
// HBM-bound (a row of 128 values: 256 bytes in, 256 or 132 out).  Eight threads have a row, two
// 16-byte vectors each, chosen so that a thread's vectors hold whole pairs and eight threads' loads
// lie side by side; eight frequencies serve a thread's sixteen values in either layout.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "bsa_common.cuh"
#include "bsa_quant.cuh"

namespace bsa {
namespace rope {

constexpr int THREADS = 256;
constexpr int LANES = 8;    // threads of a row
constexpr int VEC = 8;      // values of a 16-byte vector
constexpr int VECS = HEAD_DIM / VEC;

struct Params {
  const __nv_bfloat16 *q, *k;
  __nv_bfloat16 *q_out, *k_out;
  uint2 *codes;
  float *descale;
  const int *positions;
  const unsigned long long *freqs;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements from token to token
  long long units;  // tokens x groups of heads
  int N1, N2, R;
  int groups, heads;  // groups of `heads` heads that one thread serves
  int interleaved, ue8m0;
  float amplitude;
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  uint32_t r;
  memcpy(&r, &x, 4);
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                    bf16x2(v[6], v[7]));
}

constexpr int AHEAD = 4;  // heads in flight per thread

template <bool QUANT>
__global__ void __launch_bounds__(THREADS) rope_kernel(const Params p) {
  const int lane = threadIdx.x & (LANES - 1);
  // whole warps stay to the end: the rows' maxima go by shuffles
  const long long unit = (long long)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const bool live = unit < p.units;
  const int group = live ? (int)(unit % p.groups) : 0;
  const long long t = live ? unit / p.groups : 0;
  const int heads = p.N1 + p.N2, h0 = group * p.heads,
            h1 = live ? min(h0 + p.heads, heads) : h0;

  // the thread's vectors, and whether they are turned
  const int turned = p.R / VEC;  // vectors that hold pairs
  int v0 = lane, v1 = lane + LANES;
  bool turn0 = v0 < turned, turn1 = v1 < turned;
  if (!p.interleaved) {
    const int half = turned / 2, rest = lane - half;
    turn0 = turn1 = rest < 0;
    v0 = turn0 ? lane : turned + rest;
    v1 = turn0 ? lane + half : turned + rest + LANES - half;
  }

  const auto in = [&](int h) {
    return reinterpret_cast<const uint4 *>(
        h < p.N1 ? p.q + t * p.q_stride + (long long)h * HEAD_DIM
                 : p.k + t * p.k_stride + (long long)(h - p.N1) * HEAD_DIM);
  };
  uint4 a[AHEAD], b[AHEAD];
  const auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (h + i < h1) {
        const uint4 *x = in(h + i);
        a[i] = x[v0];
        b[i] = x[v1];
      }
    }
  };
  load(h0);

  // cosines and sines: in halves pair j of both vectors, interleaved four pairs of each vector
  float c[8], s[8];
  const unsigned long long pos = live ? (unsigned long long)(long long)p.positions[t] : 0ull;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = p.interleaved ? (j < 4 ? 4 * v0 + j : 4 * v1 + j - 4) : 8 * v0 + j;
    const bool on = j < 4 || !p.interleaved ? turn0 : turn1;
    const unsigned long long turns = on ? pos * p.freqs[i] : 0ull;
    // the nearer way round: [-1/2, 1/2) of a turn
    sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s[j], &c[j]);
    c[j] = on ? c[j] * p.amplitude : 1.f;
    s[j] = on ? s[j] * p.amplitude : 0.f;
  }

  // (with codes to make, whole warps walk the same heads: groups may be short, rows not)
  const int steps = (p.heads + AHEAD - 1) / AHEAD;
  for (int step = 0; step < steps; ++step) {
    const int h = h0 + step * AHEAD;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      float x[8], y[8];
      quant::unpack8(a[i], x);
      quant::unpack8(b[i], y);
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
          if (turn0) {
            x[2 * j] = x0 * c[j] - x1 * s[j];
            x[2 * j + 1] = x1 * c[j] + x0 * s[j];
          }
          if (turn1) {
            y[2 * j] = y0 * c[4 + j] - y1 * s[4 + j];
            y[2 * j + 1] = y1 * c[4 + j] + y0 * s[4 + j];
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = x[j], v = y[j];
          x[j] = u * c[j] - v * s[j];
          y[j] = v * c[j] + u * s[j];
        }
      }
      if constexpr (QUANT) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(x[j]), fabsf(y[j])));
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (h + i < h1) {
          const float d = quant::descale_of(m, p.ue8m0);
          const long long row = t * p.N1 + h + i;
          p.codes[row * VECS + v0] = quant::codes8(x, d);
          p.codes[row * VECS + v1] = quant::codes8(y, d);
          if (lane == 0) p.descale[row] = d;
        }
      } else if (h + i < h1) {
        uint4 *o = reinterpret_cast<uint4 *>(
            h + i < p.N1 ? p.q_out + t * p.q_out_stride + (long long)(h + i) * HEAD_DIM
                         : p.k_out + t * p.k_out_stride + (long long)(h + i - p.N1) * HEAD_DIM);
        o[v0] = turn0 ? pack8(x) : a[i];
        o[v1] = turn1 ? pack8(y) : b[i];
      }
    }
    if (step + 1 < steps) load(h + AHEAD);
  }
}

}  // namespace rope
}  // namespace bsa
