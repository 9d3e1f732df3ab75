// rope.cu -- rotation of query and output rows by position (csa2_rope_rows).
//
// Bytes bound it: each rotated channel is read and written once (in place; into
// another buffer each channel).  What comes next are the conversions to and from
// fp64, six per pair at a quarter of the ALU's rate, two of them for the table.
// All heads of a row turn by the same angles, so a thread takes the same channels of
// several heads: the position, the table's entries and their conversions once, and
// the heads' loads on their way together.  8,192 rows x 16 heads, 64 of 512 channels in
// place (33.5 MB): 14.4 us with the 5 of an empty launch (one head at a time 18.5);
// 8,000 x 16 heads into another buffer (262 MB) 55 us, 4.7 TB/s (one head: 103, two: 69).
// HALVES holds 16 channels a head and twice the angles: two heads, 14 to 16 us, which
// still spill 72 bytes of the 64 registers that four CTAs an SM leave (four heads spill
// 264 and take 18).
#include "csa2_internal.cuh"
#include "rope.cuh"

namespace csa2 {

constexpr int RR_NT = 256;

// Heads per thread, and CTAs per SM that have to fit.
__host__ __device__ constexpr int rr_heads(bool halves) { return halves ? 2 : 4; }
constexpr int RR_CTAS = 4;

// Units of a row and its heads: eight channels (four pairs), or in HALVES style the
// two 8-channel chunks whose channels pair up, so that a thread reads everything
// that it overwrites; and the chunks in front of the rotated channels, copied when
// y is another buffer.
__host__ __device__ inline int rope_rot(const RopeRowsParams& p) {
  return p.rope.style == CSA2_ROPE_PAIRS ? p.rope.dims / 8 : p.rope.dims / 16;
}
__host__ __device__ inline int rope_copy(const RopeRowsParams& p) {
  return p.in_place ? 0 : (p.ch - p.rope.dims) / 8;
}
__host__ __device__ inline int64_t rope_units(const RopeRowsParams& p) {
  const int n = rr_heads(p.rope.style != CSA2_ROPE_PAIRS);
  return p.rows * ((p.heads + n - 1) / n) * (rope_rot(p) + rope_copy(p));
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

template <bool HALVES>
__global__ void __launch_bounds__(RR_NT, RR_CTAS) rope_rows_kernel(const RopeRowsParams p) {
  constexpr int RR_HEADS = rr_heads(HALVES);
  pdl_launch_dependents();
  pdl_wait();
  const int copy = rope_copy(p), per = rope_rot(p) + copy;
  const int per_row = (p.heads + RR_HEADS - 1) / RR_HEADS * per;
  const int64_t units = rope_units(p);
  const int64_t stride = (int64_t)gridDim.x * RR_NT;
  for (int64_t u = (int64_t)blockIdx.x * RR_NT + threadIdx.x; u < units; u += stride) {
    const int64_t row = units >> 32 ? u / per_row : (int64_t)((uint32_t)u / (uint32_t)per_row);
    const int in_row = (int)(u - row * per_row), h0 = in_row / per * RR_HEADS, j = in_row % per;
    const int n = min(RR_HEADS, p.heads - h0), step = p.ch / 8;  // a head's 16-byte pieces
    const uint4* x = reinterpret_cast<const uint4*>(p.x + (row * p.heads + h0) * p.ch);
    uint4* y = reinterpret_cast<uint4*>(p.y + (row * p.heads + h0) * p.ch);
    const int k = j - copy, at = k < 0 ? j : (p.ch - p.rope.dims) / 8 + k;
    uint4 v[RR_HEADS];
#pragma unroll
    for (int h = 0; h < RR_HEADS; h++)
      if (h < n) v[h] = x[h * step + at];
    if (k < 0) {
#pragma unroll
      for (int h = 0; h < RR_HEADS; h++)
        if (h < n) y[h * step + at] = v[h];
      continue;
    }
    const float2* cs = rope_row(p.rope, __ldg(p.pos + row), p.status);
    const float sign = p.inverse ? -1.0f : 1.0f;
    if (!HALVES) {
      float2 c[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        c[i] = __ldg(cs + 4 * k + i);
        c[i].y *= sign;
      }
#pragma unroll
      for (int h = 0; h < RR_HEADS; h++) {
        float f[8];
        if (h >= n) break;
        unpack_bf16x8(v[h], f);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float2 r = rotate_pair(f[2 * i], f[2 * i + 1], c[i]);
          f[2 * i] = r.x;
          f[2 * i + 1] = r.y;
        }
        y[h * step + at] = pack_bf16x8(f);
      }
    } else {
      const int other = at + p.rope.dims / 16;
      float2 c[8];
      uint4 w[RR_HEADS];
#pragma unroll
      for (int h = 0; h < RR_HEADS; h++)
        if (h < n) w[h] = x[h * step + other];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        c[i] = __ldg(cs + 8 * k + i);
        c[i].y *= sign;
      }
#pragma unroll
      for (int h = 0; h < RR_HEADS; h++) {
        float f[8], g[8];
        if (h >= n) break;
        unpack_bf16x8(v[h], f);
        unpack_bf16x8(w[h], g);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float2 r = rotate_pair(f[i], g[i], c[i]);
          f[i] = r.x;
          g[i] = r.y;
        }
        y[h * step + at] = pack_bf16x8(f);
        y[h * step + other] = pack_bf16x8(g);
      }
    }
  }
}

cudaError_t launch_rope_rows(const RopeRowsParams& p, cudaStream_t st) {
  const int64_t units = rope_units(p);
  if (units == 0) return cudaSuccess;
  const int64_t want = (units + RR_NT - 1) / RR_NT, cap = (int64_t)num_sms() * 8;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < cap ? want : cap));
  cfg.blockDim = dim3(RR_NT);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  trace_mark("rope_rows", st);
  return p.rope.style == CSA2_ROPE_PAIRS ? cudaLaunchKernelEx(&cfg, rope_rows_kernel<false>, p)
                                         : cudaLaunchKernelEx(&cfg, rope_rows_kernel<true>, p);
}

}  // namespace csa2
