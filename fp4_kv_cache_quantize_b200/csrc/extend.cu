// extend.cu -- the ragged, rotated cache append (csa2_cache_extend).
//
// Token i of sequence b's run goes to position n_rows[b] + i: its entry is
// rotated by position and packed to FP4, its indexer key x W is summed in fp32,
// rotated and rounded once, and the last 128 tokens of the run go to every
// layer's E4M3 window ring.  A sequence whose run does not fit is left alone as
// a whole, so every CTA that writes for a sequence first checks the sequence's
// whole run; extend_commit_kernel makes the same check and advances counters.
#include "csa2_internal.cuh"
#include "rope.cuh"

namespace csa2 {

constexpr int EX_NT = 256;
constexpr int EX_LAYERS_PER_CTA = EX_NT / 64;

// Tokens [lo, hi) of sequence b; false if the offsets are out of order or do
// not start at 0.
__device__ __forceinline__ bool run_of(const ExtendParams& p, int b, int& lo, int& hi) {
  if (!p.cu) {
    lo = b;
    hi = b + 1;
    return true;
  }
  lo = __ldg(p.cu + b);
  hi = __ldg(p.cu + b + 1);
  return lo >= 0 && hi >= lo && hi <= p.total && (b > 0 || lo == 0);
}

// The sequence of token i (cu[b] <= i < cu[b + 1]), or -1.
__device__ __forceinline__ int seq_of(const ExtendParams& p, int i) {
  if (!p.cu) return i;
  int lo = 0, hi = p.batch;  // the last b with cu[b] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid) <= i) lo = mid; else hi = mid;
  }
  return i >= __ldg(p.cu + lo) && i < __ldg(p.cu + lo + 1) ? lo : -1;
}

// Pool row of position pos of sequence b, or -1.
__device__ __forceinline__ int64_t extend_row(const ExtendParams& p, int b, int64_t pos) {
  int64_t row;
  if (p.page_table) {
    const int64_t page = pos >> 6;
    if (page >= p.max_pages) return -1;
    const int64_t pid = __ldg(p.page_table + (int64_t)b * p.max_pages + page);
    if (pid < 0) return -1;
    row = pid * 64 + (pos & 63);
  } else {
    if (pos >= p.seq_stride) return -1;
    row = (int64_t)b * p.seq_stride + pos;
  }
  return row < p.pool_rows ? row : -1;
}

// Whether lane `first` of `step` finds the run of sequence b in order: `step`
// threads together look at every page that it touches, and at the counters.
__device__ __forceinline__ bool run_fits(const ExtendParams& p, int b, int count, int first,
                                         int step) {
  if (p.swa && (__ldg(p.swa_pos + b) < 0 || __ldg(p.swa_pos + b) > 0x7FFFFFFF - count)) return false;
  if (!p.x) return true;
  const int64_t n0 = p.n_rows[b], end = n0 + count;
  if (n0 < 0 || end > 0x7FFFFFFF) return false;
  if (count == 0) return true;
  if (!p.page_table) return extend_row(p, b, end - 1) >= 0;
  bool ok = end <= (int64_t)p.max_pages * 64;
  for (int64_t page = (n0 >> 6) + first; ok && page <= (end - 1) >> 6; page += step) {
    // the last row of the page that the run uses
    const int64_t last = min(page * 64 + 63, end - 1);
    ok = extend_row(p, b, last) >= 0;
  }
  return ok;
}

// One CTA per token: part 0 packs the entry and projects its key (256 threads:
// 8 outputs x 16 channels each, partial sums reduced in a fixed order); parts
// 1.. convert four layers' window entries each (64 threads per layer).
__global__ void __launch_bounds__(EX_NT) extend_token_kernel(const ExtendParams p) {
  __shared__ float xs[CSA2_D];
  __shared__ float part[32][CSA2_DI + 1];
  __shared__ float ks[CSA2_DI];
  const int t = threadIdx.x, tok = blockIdx.x;
  const bool main_part = p.x != nullptr && blockIdx.y == 0;
  pdl_launch_dependents();
  pdl_wait();

  const int b = seq_of(p, tok);
  if (b < 0) return;  // behind the last run (extend_commit_kernel records bad offsets)
  int lo, hi;
  const bool in_order = run_of(p, b, lo, hi);
  if (!__syncthreads_and(in_order && run_fits(p, b, hi - lo, t, EX_NT))) return;

  if (main_part) {
    const int64_t pos = (int64_t)p.n_rows[b] + (tok - lo);
    const int64_t row = extend_row(p, b, pos);
    const int rp = p.pos ? __ldg(p.pos + tok) : (int)pos;
    const uint16_t* x = p.x + (int64_t)tok * CSA2_D;
    if (t < CSA2_D / 8) {
      float f[8];
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(x) + t), f);
#pragma unroll
      for (int k = 0; k < 8; k++) xs[8 * t + k] = f[k];
      const float2* cs = p.rope.table ? rope_row(p.rope, rp, p.status) : nullptr;
      rotated_chunk8(p.rope, cs, x, CSA2_D, t, f);
      float amax = amax8(f);
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      uint8_t sb;
      const uint32_t packed = fp4_encode8(f, amax, &sb);
      reinterpret_cast<uint32_t*>(p.codes + row * (CSA2_D / 2))[t] = packed;
      if ((t & 1) == 0) p.scales[row * (CSA2_D / 16) + (t >> 1)] = sb;
    }
    __syncthreads();
    const int jg = t & 7, c16 = t >> 3;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint4* wp = reinterpret_cast<const uint4*>(p.w_idx) + (int64_t)(16 * c16) * 8 + jg;
    uint4 wv[16];
#pragma unroll
    for (int c = 0; c < 16; c++) wv[c] = __ldg(wp + c * 8);
#pragma unroll
    for (int c = 0; c < 16; c++) {
      float wf[8];
      unpack_bf16x8(wv[c], wf);
      const float xc = xs[16 * c16 + c];
#pragma unroll
      for (int k = 0; k < 8; k++) acc[k] = fmaf(xc, wf[k], acc[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; k++) part[c16][8 * jg + k] = acc[k];
    __syncthreads();
    if (t < CSA2_DI) {
      float sum = 0.f;
#pragma unroll 8
      for (int i = 0; i < 32; i++) sum += part[i][t];
      ks[t] = sum;
    }
    __syncthreads();
    if (t < CSA2_DI / 2) {  // pair t of the key: its two channels, rotated or not
      const int n = p.rope_idx.table ? p.rope_idx.dims / 2 : 0, plain = CSA2_DI - 2 * n;
      int i = 2 * t, j = 2 * t + 1;
      if (2 * t >= plain && p.rope_idx.style == CSA2_ROPE_HALVES) {
        i = plain + (t - plain / 2);
        j = i + n;
      }
      float2 v = make_float2(ks[i], ks[j]);
      if (2 * t >= plain)
        v = rotate_pair(v.x, v.y, __ldg(rope_row(p.rope_idx, rp, p.status) + (t - plain / 2)));
      p.idx_k[row * CSA2_DI + i] = __bfloat16_as_ushort(__float2bfloat16_rn(v.x));
      p.idx_k[row * CSA2_DI + j] = __bfloat16_as_ushort(__float2bfloat16_rn(v.y));
    }
    return;
  }

  const int l = (blockIdx.y - (p.x ? 1 : 0)) * EX_LAYERS_PER_CTA + (t >> 6);
  if (l >= p.n_layers || tok < hi - CSA2_W) return;
  const int spos = __ldg(p.swa_pos + b) + (tok - lo), ch = t & 63;
  const float2* cs = p.rope_swa.table
                         ? rope_row(p.rope_swa, p.pos ? __ldg(p.pos + tok) : spos, p.status)
                         : nullptr;
  float f[8];
  rotated_chunk8(p.rope_swa, cs, p.x_swa + ((int64_t)l * p.total + tok) * CSA2_D, CSA2_D, ch, f);
  uint32_t w2[4];
#pragma unroll
  for (int k = 0; k < 4; k++)
    w2[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * k], f[2 * k + 1]), __NV_SATFINITE,
                                               __NV_E4M3);
  uint8_t* dst = p.swa + (((int64_t)l * p.batch + b) * CSA2_W + spos % CSA2_W) * CSA2_D + 8 * ch;
  *reinterpret_cast<uint2*>(dst) = make_uint2((w2[0] & 0xFFFFu) | (w2[1] << 16),
                                              (w2[2] & 0xFFFFu) | (w2[3] << 16));
}

// Advances the counters once every write of the step has landed: one warp per
// sequence.
__global__ void __launch_bounds__(EX_NT) extend_commit_kernel(const ExtendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = (blockIdx.x * EX_NT + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (b >= p.batch) return;
  int lo, hi;
  bool ok = run_of(p, b, lo, hi);
  ok = __all_sync(0xffffffffu, ok && run_fits(p, b, hi - lo, lane, 32));
  if (lane != 0) return;
  if (!ok) {
    set_status(p.status, ST_DEVICE_CHECK);
    return;
  }
  if (p.x) p.n_rows[b] += hi - lo;
  if (p.swa) {
    const int spos = p.swa_pos[b] + (hi - lo);
    p.swa_pos[b] = spos;
    p.swa_len[b] = spos < CSA2_W ? spos : CSA2_W;
  }
}

cudaError_t launch_extend(const ExtendParams& p, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(EX_NT);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (p.total > 0) {
    cfg.gridDim = dim3(p.total, (p.x ? 1 : 0) +
                                    (p.n_layers + EX_LAYERS_PER_CTA - 1) / EX_LAYERS_PER_CTA);
    trace_mark("extend", st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, extend_token_kernel, p);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3((p.batch * 32 + EX_NT - 1) / EX_NT);
  trace_mark("extend_commit", st);
  return cudaLaunchKernelEx(&cfg, extend_commit_kernel, p);
}

}  // namespace csa2
