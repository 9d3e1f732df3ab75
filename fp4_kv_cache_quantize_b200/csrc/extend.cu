// extend.cu -- the ragged, rotated cache append (csa2_cache_extend).
//
// Token i of sequence b's run goes to position n_rows[b] + i: its entry is
// rotated by position and packed to FP4, its indexer key x W is summed in fp32,
// rotated and rounded once, and the last 128 tokens of the run go to every
// layer's E4M3 window ring.  A sequence whose run does not fit is left alone as
// a whole, so every CTA that writes for a sequence first checks the sequence's
// whole run; what advances the counters makes the same check.
#include "csa2_internal.cuh"
#include "extend_runs.cuh"
#include "umma_m64.cuh"
#include "rope.cuh"

namespace csa2 {

constexpr int EX_NT = 256;
constexpr int EX_LAYERS_PER_CTA = EX_NT / 64;
constexpr int EX_COMMIT_BATCH = 512;  // sequences whose counters the last CTA advances
// Tokens up to which each has CTAs of its own.  Both ways in a graph, one run without
// window layers: 256 tokens 6.8 us (tiles: 10.5), 512 11.3 (10.5), 1,024 15.7 (10.4);
// with 20 layers 512 15.8 (15.9), 1,024 23 (16).  Runs of one or two tokens never fill a
// tile's places and windows: 1,024 sequences x 20 layers 37 us (tiles: 100).
constexpr int EX_FEW = 512;
// CTAs per SM up to which a token's layers are spread (512 sequences x 20 layers 32 us,
// 1,024 37; four layers to a CTA always: 46, 57; batches of 64 and fewer alike).
constexpr int EX_ROOM = 4;

__device__ __forceinline__ int seq_of(const ExtendParams& p, int i, int& lo, int& hi) {
  return seq_of(p.cu, p.batch, p.total, i, lo, hi);
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
  if (p.swa && (p.swa_pos[b] < 0 || p.swa_pos[b] > 0x7FFFFFFF - count)) return false;
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

// Advances the counters of all sequences, once every write of the step has
// landed: a thread per sequence whose run is short, a warp per one whose run is
// not (`threads` threads, whole warps).  sorted: no offset descends.
__device__ __forceinline__ void extend_commit(const ExtendParams& p, int t, int threads,
                                              bool sorted) {
  constexpr int SHORT = 128;  // at most three pages
  auto advance = [&](int b, int count, bool ok) {
    if (!ok) {
      set_status(p.status, ST_DEVICE_CHECK);
      return;
    }
    if (p.x) p.n_rows[b] += count;
    if (p.swa) {
      const int spos = p.swa_pos[b] + count;
      p.swa_pos[b] = spos;
      p.swa_len[b] = spos < CSA2_W ? spos : CSA2_W;
    }
  };
  auto run_of = [&](int b, int& lo, int& hi) {
    return run_pair(p.cu, p.total, b, lo, hi) &&
           (sorted || run_clear(p.cu, p.batch, b, lo, hi));
  };
  for (int b = t; b < p.batch; b += threads) {
    int lo, hi;
    const bool order = run_of(b, lo, hi);
    if (!order) {
      advance(b, 0, false);
    } else if (hi - lo <= SHORT) {
      advance(b, hi - lo, run_fits(p, b, hi - lo, 0, 1));
    }
  }
  if (p.total <= SHORT) return;
  for (int b = t >> 5; b < p.batch; b += threads >> 5) {
    int lo, hi;
    if (!run_of(b, lo, hi) || hi - lo <= SHORT) continue;
    const bool ok = __all_sync(0xffffffffu, run_fits(p, b, hi - lo, t & 31, 32));
    if ((t & 31) == 0) advance(b, hi - lo, ok);
  }
}

// The last CTA of a launch to get here advances the counters: a launch less than
// with a commit kernel.  Every CTA arrives after its last read of them; the
// arrival counter (workspace header) is left at zero.
__device__ __forceinline__ void extend_arrive(const ExtendParams& p) {
  __shared__ int last;
  if (!p.commit) return;
  __syncthreads();
  bool rise = true;  // the other warps look at the offsets while the first one counts
  if (threadIdx.x >= 32) {
    for (int b = threadIdx.x - 32; b < p.batch; b += blockDim.x - 32) {
      int lo, hi;
      run_pair(p.cu, p.total, b, lo, hi);
      rise = rise && lo <= hi;
    }
  } else if (threadIdx.x == 0) {
    __threadfence();
    const uint32_t n = gridDim.x * gridDim.y * gridDim.z;
    last = atomicAdd(p.status + CSA2_WS_ARRIVE_WORD, 1u) == n - 1;
    if (last) p.status[CSA2_WS_ARRIVE_WORD] = 0u;
  }
  const bool sorted = __syncthreads_and(rise);
  if (!last) return;
  extend_commit(p, threadIdx.x, blockDim.x, sorted);
}

// Eight channels of one window entry: rotated, E4M3, into its ring slot.
__device__ __forceinline__ void window_row(const ExtendParams& p, int b, int l, int tok, int spos,
                                           int ch) {
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

// CTAs for one token (few tokens): part 0 packs the entry and projects its key (256 threads:
// 8 outputs x 16 channels each, partial sums reduced in a fixed order); parts
// 1.. convert the window entries, four layers at a time (64 threads per layer).
__device__ __forceinline__ void extend_token(const ExtendParams& p) {
  __shared__ float xs[CSA2_D];
  __shared__ float part[32][CSA2_DI + 1];
  __shared__ float ks[CSA2_DI];
  const int t = threadIdx.x, tok = blockIdx.x;
  const bool main_part = p.x != nullptr && blockIdx.y == 0;

  int lo, hi;
  const int b = seq_of(p, tok, lo, hi);
  if (b < 0) return;  // no run's token (extend_commit records bad offsets)
  if (!__syncthreads_and(run_fits(p, b, hi - lo, t, EX_NT))) return;

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

  const int z0 = p.x ? 1 : 0, step = (gridDim.y - z0) * EX_LAYERS_PER_CTA;
  if (tok < hi - CSA2_W) return;
  const int spos = p.swa_pos[b] + (tok - lo);
#pragma unroll 4
  for (int l = (blockIdx.y - z0) * EX_LAYERS_PER_CTA + (t >> 6); l < p.n_layers; l += step)
    window_row(p, b, l, tok, spos, t & 63);
}

__global__ void __launch_bounds__(EX_NT) extend_token_kernel(const ExtendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  extend_token(p);
  extend_arrive(p);
}

// ------------------------------------------------- many tokens: tiles of 32
// One CTA per SM, four groups of eight warps that each walk tiles of 32 tokens.
// cp.async brings a tile's raw rows into the swizzled layout that the MMA reads:
// the key x W of the tokens is one tcgen05 product, M = 64, N = 64, K = 512, with
// one W in shared memory for all groups.  (Rows 32.. of the product are whatever
// lies behind a chunk, the next chunk or W; their sums are not read.)  Under it the
// rows are packed from the same tile, first the pieces (8 channels) in front of the
// rotated ones, then the rotated ones, all lanes busy whatever their share of a row,
// in loops short enough to stay in the instruction cache.
//
// What bounds it: memory allows 1,440 bytes a token at its rate, 32K tokens in
// 7.2 us; they take 27 in a graph (31 cold).  20,000 of the 57,000 cycles are issue
// slots (some 20 instructions a value: packing, fp64 rotation), 10,000 the first tiles'
// way from memory, and the rest the dependent phases of a tile (rows, packing, turning,
// keys).  Two groups of 64 tokens took 2 us more, tiles of 16 tokens 11, shares of the
// packing handed out to warps one by one 4.  With few tokens the tiles are shorter (16),
// so that every SM has some.  A paged run costs more the longer it is, since et_check
// looks at all of its pages for every tile: 32K tokens 40 us, 128K 233 (contiguous: 83).
constexpr int ET_GROUPS = 4;
constexpr int ET_GT = 256;                              // threads of a group
constexpr int ET_NT = ET_GROUPS * ET_GT;
constexpr int ET_TOK = 32;                              // most tokens of a tile
constexpr int ET_M = 64;                                // rows of the product
constexpr int ET_KB = ET_TOK * 128;                     // one 64-channel chunk of the tile

struct EtGroup {
  int64_t row[2][ET_TOK];                    // by tile parity: pool row, -1: not written
  int pos[2][ET_TOK];                        // rotation position
  int seq_lo, seq_hi;                        // lowest and highest sequence of the tile
  uint64_t mbar;
};
struct EtSmem {
  alignas(1024) uint8_t a[ET_GROUPS][8 * ET_KB];  // raw bf16 rows: chunk kb, 32 rows of 128 B, swizzled
  alignas(1024) uint8_t w[CSA2_D * 128];          // W: 512 rows (K) of 64 outputs, swizzled
  EtGroup g[ET_GROUPS];
  uint32_t tmem_base;
};
constexpr size_t ET_SMEM = sizeof(EtSmem);

__device__ __forceinline__ uint32_t et_at(int row, int piece) {
  return (uint32_t)((piece >> 3) * ET_KB + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

// Packs the eight channels of a piece; lanes 2 j and 2 j + 1 hold one scale
// group.  row < 0: nothing is written.
__device__ __forceinline__ void et_pack(const ExtendParams& p, const float (&f)[8], int64_t row,
                                        int piece) {
  float amax = amax8(f);
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  uint8_t sb;
  const uint32_t packed = fp4_encode8(f, amax, &sb);
  if (row < 0) return;
  reinterpret_cast<uint32_t*>(p.codes + row * (CSA2_D / 2))[piece] = packed;
  if ((piece & 1) == 0) p.scales[row * (CSA2_D / 16) + (piece >> 1)] = sb;
}

__device__ __forceinline__ void prefetch_l2(const void* a) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}
// The table row of a position that a later step reads (clamped alike).
__device__ __forceinline__ void prefetch_rope(const RopeParams& r, int pos) {
  if (r.table == nullptr) return;
  pos = min(max(pos, 0), r.n_pos - 1);
  const char* a = reinterpret_cast<const char*>(r.table + (int64_t)pos * (r.dims / 2));
  for (int i = 0; i < r.dims * 4; i += 128) prefetch_l2(a + i);
}

// The rows and positions of a tile's tokens (the group's first warp).
__device__ __forceinline__ void et_places(const ExtendParams& p, EtGroup& g, int tile, int buf,
                                          int t) {
  const int tok = tile * p.tile + t;
  int seq = -1, pos = 0;
  int64_t row = -1;
  if (t < p.tile && tok < p.total) {
    const char* x = reinterpret_cast<const char*>(p.x + (int64_t)tok * CSA2_D);
    for (int i = 0; i < CSA2_D * 2; i += 128) prefetch_l2(x + i);
    int lo, hi;
    seq = seq_of(p, tok, lo, hi);
    if (seq >= 0) {
      const int64_t at = (int64_t)p.n_rows[seq] + (tok - lo);
      if (at >= 0) row = extend_row(p, seq, at);
      pos = p.pos ? __ldg(p.pos + tok) : (int)at;
      prefetch_rope(p.rope, pos);
      prefetch_rope(p.rope_idx, pos);
    }
  }
  g.row[buf][t] = row;
  g.pos[buf][t] = pos;
  const int a = __reduce_min_sync(0xffffffffu, seq < 0 ? p.batch : seq);
  const int z = __reduce_max_sync(0xffffffffu, seq);
  if (t == 0) {
    g.seq_lo = a;
    g.seq_hi = z;
  }
}

// A run that does not fit is not written at all: a warp per sequence of the tile
// checks all of its pages (none where every token lies behind the last run: then
// the range is [batch, -1]).
__device__ __forceinline__ void et_check(const ExtendParams& p, EtGroup& g, int tile, int buf,
                                         int warp, int lane) {
  const int tok0 = tile * p.tile, seq_hi = g.seq_hi;
  for (int b = g.seq_lo + warp; b <= seq_hi; b += ET_GT / 32) {
    int lo, hi;
    if (!run_pair(p.cu, p.total, b, lo, hi) || lo == hi) continue;
    if (!__all_sync(0xffffffffu, run_clear_lane(p.cu, p.batch, b, lane, lo, hi)))
      continue;  // (no token has its row)
    if (!__all_sync(0xffffffffu, run_fits(p, b, hi - lo, lane, 32)))
      for (int k = max(lo - tok0, 0) + lane; k < min(hi - tok0, p.tile); k += 32)
        g.row[buf][k] = -1;
  }
}

// The scale groups in front of the rotated channels, packed: 256 / tile threads
// per row, one 16-channel group each in turn (a quarter-warp's 16-byte reads meet
// different banks, a row's codes are written 32 bytes at a time or more).
__device__ __forceinline__ void et_plain(const ExtendParams& p, const uint8_t* a, const EtGroup& g,
                                         int buf, int plain, int t) {
  const int per_row = ET_GT / p.tile, r = (t >> 2) & (p.tile - 1);
  const int64_t row = g.row[buf][r];
  if (row < 0) return;
#pragma unroll 2
  for (int q = (t & 3) + t / (4 * p.tile) * 4; q < plain / 2; q += per_row) {
    uint8_t sb;
    const uint2 codes = fp4_encode16(*reinterpret_cast<const uint4*>(a + et_at(r, 2 * q)),
                                     *reinterpret_cast<const uint4*>(a + et_at(r, 2 * q + 1)), &sb);
    reinterpret_cast<uint2*>(p.codes + row * (CSA2_D / 2))[q] = codes;
    p.scales[row * (CSA2_D / 16) + q] = sb;
  }
}

// The rotated pieces of a tile, turned from the raw rows and packed.
__device__ __forceinline__ void et_turn(const ExtendParams& p, const uint8_t* a, const EtGroup& g,
                                        int buf, int plain, int t) {
  const int per = 64 - plain;
  for (int i = t; i < p.tile * per; i += ET_GT) {  // (whole warps: a multiple of 16 * 4)
    const int r = i / per, piece = plain + i - r * per, k = 8 * (piece - plain);
    float f[8];
    unpack_bf16x8(*reinterpret_cast<const uint4*>(a + et_at(r, piece)), f);
    const float2* cs = rope_row(p.rope, g.pos[buf][r], p.status);
    if (p.rope.style == CSA2_ROPE_PAIRS) {
      const float4* c4 = reinterpret_cast<const float4*>(cs + k / 2);
      const float4 c[2] = {__ldg(c4), __ldg(c4 + 1)};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float2 y = rotate_pair(f[2 * j], f[2 * j + 1],
                                     (j & 1) ? make_float2(c[j >> 1].z, c[j >> 1].w)
                                             : make_float2(c[j >> 1].x, c[j >> 1].y));
        f[2 * j] = round_bf16(y.x);
        f[2 * j + 1] = round_bf16(y.y);
      }
    } else {
      const int half = p.rope.dims / 2;
      const bool first = k < half;
      float h[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(a + et_at(r, piece + (first ? half : -half) / 8)), h);
      const float4* c4 = reinterpret_cast<const float4*>(cs + (first ? k : k - half));
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float4 c = __ldg(c4 + j);
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float2 cc = e ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
          float& fj = f[2 * j + e];
          const float2 y = first ? rotate_pair(fj, h[2 * j + e], cc) : rotate_pair(h[2 * j + e], fj, cc);
          fj = round_bf16(first ? y.x : y.y);
        }
      }
    }
    et_pack(p, f, g.row[buf][r], piece);
  }
}

// The keys of a tile: the sums rotated in fp64, rounded once.  Warp (quad, part):
// tokens 16 quad + lane / 4 and + 8, column blocks of 8 that hold whole pairs.
__device__ __forceinline__ void et_keys(const ExtendParams& p, const EtGroup& g, int buf,
                                        uint32_t tmem, int warp, int lane) {
  const int quad = warp & 3, part = warp >> 2;
  if (16 * quad >= p.tile) return;
  const int rk = p.rope_idx.table ? p.rope_idx.dims : 0;  // 0, 32 or 64
  const bool halves = rk && p.rope_idx.style == CSA2_ROPE_HALVES;
  // blocks 2 part, 2 part + 1, + 4, + 5: with HALVES of 64 block n pairs with n +
  // 4; of 32, blocks 4, 5 pair with 6, 7: part 0 takes 0..3 then, part 1 the rest
  const int b0 = halves && rk == 32 ? 4 * part : 2 * part, up = halves && rk == 32 ? 2 : 4;
  uint32_t acc[4][4];
#pragma unroll
  for (int n = 0; n < 4; n++)
    tmem_ld_16x256b_x1(tmem + ((uint32_t)(32 * quad) << 16) + 8 * (b0 + (n & 1) + (n >> 1) * up), acc[n]);
  tmem_ld_wait();
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int r = 16 * quad + (lane >> 2) + 8 * h;
    const int64_t row = g.row[buf][r];
    if (row < 0) continue;
    float2 y[4];  // block n: columns 8 block + 2 (lane % 4) + {0, 1}
#pragma unroll
    for (int n = 0; n < 4; n++)
      y[n] = make_float2(__uint_as_float(acc[n][2 * h]), __uint_as_float(acc[n][2 * h + 1]));
    if (rk) {
      const float2* cs = rope_row(p.rope_idx, g.pos[buf][r], p.status);
      if (!halves) {
#pragma unroll
        for (int n = 0; n < 4; n++) {
          const int c = 8 * (b0 + (n & 1) + (n >> 1) * up) - (CSA2_DI - rk);
          if (c >= 0) y[n] = rotate_pair(y[n].x, y[n].y, __ldg(cs + c / 2 + (lane & 3)));
        }
      } else {
#pragma unroll
        for (int n = 0; n < 2; n++) {
          const int c = 8 * (b0 + n) - (CSA2_DI - rk);
          if (c < 0) continue;  // (dims 32, part 0: nothing is rotated)
          const float4 a = __ldg(reinterpret_cast<const float4*>(cs + c) + (lane & 3));
          const float2 u = rotate_pair(y[n].x, y[n + 2].x, make_float2(a.x, a.y));
          const float2 w = rotate_pair(y[n].y, y[n + 2].y, make_float2(a.z, a.w));
          y[n] = make_float2(u.x, w.x);
          y[n + 2] = make_float2(u.y, w.y);
        }
      }
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.idx_k + row * CSA2_DI) + (lane & 3);
#pragma unroll
    for (int n = 0; n < 4; n++)
      dst[4 * (b0 + (n & 1) + (n >> 1) * up)] = pack_bf16x2(y[n].x, y[n].y);
  }
}

__global__ void __launch_bounds__(ET_NT, 1) extend_tile_kernel(const ExtendParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // (not rounded up: a generic pointer then)
  EtSmem& s = *reinterpret_cast<EtSmem*>(smem_raw);
  const int grp = __shfl_sync(0xffffffffu, threadIdx.x / ET_GT, 0);
  const int t = threadIdx.x % ET_GT, lane = t & 31, warp = __shfl_sync(0xffffffffu, t >> 5, 0);
  const int n_tiles = (p.total + p.tile - 1) / p.tile, step = gridDim.x * ET_GROUPS;
  EtGroup& g = s.g[grp];
  uint8_t* const a = s.a[grp];
  if (t == 0) {
    mbar_init(&g.mbar, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    tmem_alloc(&s.tmem_base, 64 * ET_GROUPS);
    tmem_relinquish();
  }
  pdl_wait();
  for (int i = threadIdx.x; i < CSA2_D * 8; i += ET_NT)
    cp_async16(s.w + (i >> 3) * 128 + (((i & 7) ^ ((i >> 3) & 7)) << 4),
               reinterpret_cast<const uint8_t*>(p.w_idx) + 16 * i);
  cp_async_commit();

  auto fetch = [&](int tile) {  // the tile's rows (those behind the last token: any)
    const int n = min(p.tile, p.total - tile * p.tile) * 64;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x + (int64_t)tile * p.tile * CSA2_D);
    for (int i = t; i < n; i += ET_GT) cp_async16(a + et_at(i >> 6, i & 63), x + 16 * i);
    cp_async_commit();
  };
  // neighbouring tiles go to different CTAs: few tiles spread over all SMs
  int tile = blockIdx.x + grp * gridDim.x;
  fetch(tile);
  if (warp == 0) et_places(p, g, tile, 0, t);
  cp_async_wait_all();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();  // W, the tensor memory's base, the first places
  tc_fence_after();
  pdl_launch_dependents();  // (with the tensor memory in hand: a kernel that waits for this one may want some)
  const uint32_t tmem = s.tmem_base + 64 * grp;
  et_check(p, g, tile, 0, warp, lane);
  const int turned = p.rope.table ? p.rope.dims : 0;  // rotated channels, at the end of a row
  const int plain = (CSA2_D - turned) / 8;            // pieces in front of them (even)
  bool alive = true;
  bar_sync<ET_GT>(1 + grp);
  for (uint32_t n = 0; tile < n_tiles && alive; tile += step, n++) {
    const int buf = n & 1;
    if (warp == 0) {
      tc_fence_after();
      if (elect_one()) {
        const uint64_t da = sdesc_k128(smem_u32(a)), db = sdesc_mn128(smem_u32(s.w), 65536, 1024);
        constexpr uint32_t id = idesc_bf16_f32(ET_M, CSA2_DI) | (1u << 16);  // W is read MN-major
#pragma unroll
        for (uint32_t k = 0; k < 32; k++)
          umma_bf16(tmem, da + (((k >> 2) * ET_KB + 32 * (k & 3)) >> 4), db + ((k * 2048) >> 4), id,
                    k != 0);
        umma_commit(&g.mbar);
      }
      __syncwarp();
    }
    const bool more = tile + step < n_tiles;
    if (more && warp == 0) et_places(p, g, tile + step, buf ^ 1, t);
    et_plain(p, a, g, buf, plain, t);
    et_turn(p, a, g, buf, plain, t);
    const bool ok = mbar_wait(&g.mbar, n & 1, nullptr);
    __syncwarp();
    tc_fence_after();
    if (ok) et_keys(p, g, buf, tmem, warp, lane);
    tc_fence_before();
    alive = bar_and<ET_GT>(1 + grp, ok);  // the rows are done with
    if (more) fetch(tile + step);
    if (more) et_check(p, g, tile + step, buf ^ 1, warp, lane);
    cp_async_wait_all();
    fence_proxy_async_smem();
    bar_sync<ET_GT>(1 + grp);
  }
  if (!alive && t == 0) set_status(p.status, ST_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc(s.tmem_base, 64 * ET_GROUPS);
  }
  extend_arrive(p);
}

// The window entries of many tokens: gridDim.z CTAs share the last 128 tokens of a
// sequence's run and layer, 16 at a time, 64 threads per row.
constexpr int EW_TOK = 16;
__device__ __forceinline__ void extend_window(const ExtendParams& p) {
  const int t = threadIdx.x, b = blockIdx.x, l = blockIdx.y, ch = t & 63;
  int lo, hi;
  if (!run_pair(p.cu, p.total, b, lo, hi) || hi - (int)blockIdx.z * EW_TOK <= lo) return;
  if (!__syncthreads_and(run_clear_lane(p.cu, p.batch, b, t, lo, hi) &&
                         run_fits(p, b, hi - lo, t, EX_NT)))
    return;
  const int spos0 = p.swa_pos[b];
  const int end = max(lo, hi - CSA2_W);
  for (int last = hi - blockIdx.z * EW_TOK; last > end; last -= gridDim.z * EW_TOK)
    for (int tok = max(end, last - EW_TOK) + (t >> 6); tok < last; tok += EX_NT / 64)
      window_row(p, b, l, tok, spos0 + (tok - lo), ch);
}

__global__ void __launch_bounds__(EX_NT, 4) extend_window_kernel(const ExtendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  extend_window(p);
  extend_arrive(p);
}

// The same for large batches.
__global__ void __launch_bounds__(EX_NT) extend_commit_kernel(const ExtendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  extend_commit(p, blockIdx.x * EX_NT + threadIdx.x, gridDim.x * EX_NT, false);
}

cudaError_t launch_extend(const ExtendParams& params, cudaStream_t st) {
  ExtendParams p = params;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(EX_NT);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e;
  // the last launch that writes also advances the counters, unless one CTA would
  // be long at it
  const bool in_last = p.batch <= EX_COMMIT_BATCH;
  const int sms = num_sms();
  if (p.total <= EX_FEW || p.total / 2 <= p.batch) {
    p.commit = in_last;
    // a token's layers are spread over CTAs as long as those find room
    const int quads = (p.n_layers + EX_LAYERS_PER_CTA - 1) / EX_LAYERS_PER_CTA;
    const int room = EX_ROOM * sms / p.total, most = room > 1 ? room : 1;
    cfg.gridDim = dim3(p.total, (p.x ? 1 : 0) + (quads < most ? quads : most));
    trace_mark("extend", st);
    if ((e = cudaLaunchKernelEx(&cfg, extend_token_kernel, p)) != cudaSuccess) return e;
  } else {
    if (p.n_layers > 0) {
      p.commit = in_last && !p.x;
      // as many as a run of twice the average length keeps busy
      const int mean = (p.total - 1) / p.batch + 1, most = mean < CSA2_W / 2 ? 2 * mean : CSA2_W;
      cfg.gridDim = dim3(p.batch, p.n_layers, (most + EW_TOK - 1) / EW_TOK);
      trace_mark("extend_window", st);
      if ((e = cudaLaunchKernelEx(&cfg, extend_window_kernel, p)) != cudaSuccess) return e;
    }
    if (p.x) {
      static PerDeviceOnce attr;
      e = attr.run([](int&) {
        return cudaFuncSetAttribute(extend_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)ET_SMEM);
      });
      if (e != cudaSuccess) return e;
      p.commit = in_last;
      p.tile = 16;
      while (p.tile < ET_TOK && (p.total + p.tile - 1) / p.tile > sms * ET_GROUPS) p.tile *= 2;
      const int tiles = (p.total + p.tile - 1) / p.tile;
      cfg.gridDim = dim3(tiles < sms ? tiles : sms);
      cfg.blockDim = dim3(ET_NT);
      cfg.dynamicSmemBytes = ET_SMEM;
      trace_mark("extend", st);
      if ((e = cudaLaunchKernelEx(&cfg, extend_tile_kernel, p)) != cudaSuccess) return e;
      cfg.blockDim = dim3(EX_NT);
      cfg.dynamicSmemBytes = 0;
    }
  }
  if (in_last) return cudaSuccess;
  cfg.gridDim = dim3((p.batch * 32 + EX_NT - 1) / EX_NT);
  trace_mark("extend_commit", st);
  return cudaLaunchKernelEx(&cfg, extend_commit_kernel, p);
}

}  // namespace csa2
