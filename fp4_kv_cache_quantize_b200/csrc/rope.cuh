// rope.cuh -- the rotation of a row's last channels by its position, shared by
// csa2_rope_rows and the cache extension so that both give the same bits.
//
// A pair (a, b) becomes (a c - b s, a s + b c) with (c, s) = table[pos][i].
// a and b are bf16 (8 significant bits), c and s fp32 (24): the products are
// exact in fp64 and their sum is off by at most 2^-53 of the larger one, so the
// one rounding that counts is the last, to fp32 and on to bf16.  In fp32 the
// two roundings of the products would decide now and then which FP4 code an
// entry gets, and differently for each order of the operations.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "fp4_codec.cuh"
#include "kernels.h"

namespace csa2 {

__device__ __forceinline__ float round_bf16(float v) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// The rotation of one pair, as fp32 (not yet rounded to bf16).
__device__ __forceinline__ float2 rotate_pair(float a, float b, float2 cs) {
  const double c = cs.x, s = cs.y;
  return make_float2((float)fma((double)a, c, -((double)b * s)),
                     (float)fma((double)a, s, (double)b * c));
}

// Row `pos` of the table, clamped into it (recorded in *status).
__device__ __forceinline__ const float2* rope_row(const RopeParams& r, int pos, uint32_t* status) {
  if (pos < 0 || pos >= r.n_pos) {
    set_status(status, ST_DEVICE_CHECK);
    pos = pos < 0 ? 0 : r.n_pos - 1;
  }
  return r.table + (int64_t)pos * (r.dims / 2);
}

// Channels [8 chunk, 8 chunk + 8) of the bf16 row `row` (ch channels) after
// rotation by the table row cs, rounded to bf16; r.table == NULL: unrotated.
__device__ __forceinline__ void rotated_chunk8(const RopeParams& r, const float2* cs,
                                               const uint16_t* row, int ch, int chunk,
                                               float (&f)[8]) {
  const uint4* rv = reinterpret_cast<const uint4*>(row);
  unpack_bf16x8(__ldg(rv + chunk), f);
  const int k = 8 * chunk - (ch - r.dims);
  if (r.table == nullptr || k < 0) return;
  if (r.style == CSA2_ROPE_PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 y = rotate_pair(f[2 * i], f[2 * i + 1], __ldg(cs + k / 2 + i));
      f[2 * i] = round_bf16(y.x);
      f[2 * i + 1] = round_bf16(y.y);
    }
  } else {
    const int half = r.dims / 2;
    const bool first = k < half;
    float g[8];
    unpack_bf16x8(__ldg(rv + chunk + (first ? half : -half) / 8), g);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float2 c = __ldg(cs + (first ? k : k - half) + i);
      const float2 y = first ? rotate_pair(f[i], g[i], c) : rotate_pair(g[i], f[i], c);
      f[i] = round_bf16(first ? y.x : y.y);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace csa2
