// rope.cu -- rotation of query and output rows by position (csa2_rope_rows).
#include "csa2_internal.cuh"
#include "rope.cuh"

namespace csa2 {

// One thread turns one unit of a (row, head): eight channels (four pairs), or
// in HALVES style the two 8-channel chunks whose channels pair up, so that a
// thread reads everything that it overwrites; the channels in front of the
// rotated ones are copied when y is another buffer.
__global__ void __launch_bounds__(256) rope_rows_kernel(const RopeRowsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int rot = p.rope.style == CSA2_ROPE_PAIRS ? p.rope.dims / 8 : p.rope.dims / 16;
  const int copy = p.in_place ? 0 : (p.ch - p.rope.dims) / 8;
  const int64_t units = p.rows * p.heads * (rot + copy);
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < units; u += stride) {
    const int64_t rh = u / (rot + copy);
    const int j = (int)(u - rh * (rot + copy));
    const uint4* x = reinterpret_cast<const uint4*>(p.x + rh * p.ch);
    uint4* y = reinterpret_cast<uint4*>(p.y + rh * p.ch);
    if (j < copy) {
      y[j] = x[j];
      continue;
    }
    const float2* cs = rope_row(p.rope, __ldg(p.pos + rh / p.heads), p.status);
    const int k = j - copy, at = (p.ch - p.rope.dims) / 8 + k;
    float f[8], g[8];
    unpack_bf16x8(x[at], f);
    if (p.rope.style == CSA2_ROPE_PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float2 c = __ldg(cs + 4 * k + i);
        if (p.inverse) c.y = -c.y;
        const float2 v = rotate_pair(f[2 * i], f[2 * i + 1], c);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    } else {
      const int other = at + p.rope.dims / 16;
      unpack_bf16x8(x[other], g);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float2 c = __ldg(cs + 8 * k + i);
        if (p.inverse) c.y = -c.y;
        const float2 v = rotate_pair(f[i], g[i], c);
        f[i] = v.x;
        g[i] = v.y;
      }
      y[other] = make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                            pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
    }
    y[at] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                       pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

cudaError_t launch_rope_rows(const RopeRowsParams& p, cudaStream_t st) {
  const int rot = p.rope.style == CSA2_ROPE_PAIRS ? p.rope.dims / 8 : p.rope.dims / 16;
  const int64_t units =
      p.rows * p.heads * (rot + (p.in_place ? 0 : (p.ch - p.rope.dims) / 8));
  if (units == 0) return cudaSuccess;
  const int64_t want = (units + 255) / 256, cap = (int64_t)num_sms() * 8;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < cap ? want : cap));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  trace_mark("rope_rows", st);
  return cudaLaunchKernelEx(&cfg, rope_rows_kernel, p);
}

}  // namespace csa2
