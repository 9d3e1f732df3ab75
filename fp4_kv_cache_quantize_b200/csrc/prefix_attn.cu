// prefix_attn.cu -- dense attention of a batch that shares a prefix
// (csa2_prefix_attn).
//
// Every query head of the batch meets the shared rows, so a key tile is read
// and dequantised once for 64 query rows: S^T = K Q'^T (keys on the MMA's M
// axis) and O^T = V^T P^T (channels on it), fp16 operands, fp32 accumulators
// in tensor memory.  E2M1 x E4M3 products and E4M3 window values are exact in
// fp16; a query head is scaled by a power of two into fp16's range.
//
// Softmax in one pass: with a reference m per row, p_j = 2^(s_j - m + 7),
// O += p_j v_j, l += p_j.  m only has to be near the maximum: it is raised (and
// O, l scaled) when some s_j exceeds it by 8, so p <= 2^15 fits fp16, and the
// +7 keeps p to 2^-31 of the row's largest before it is lost: a million keys
// lose at most 2^-12 of the sum together.  l sums the rounded p, so the weights
// that multiply V are exactly normalised.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "csa2_internal.cuh"
#include "kernels.h"
#include "prefix_plan.cuh"

namespace csa2 {

constexpr int PA_NT = 512;
constexpr int PA_KB = PA_KEYS * 128;   // one 64-channel block of the key tile
constexpr int PA_QKB = PA_ROWS * 128;  // one 64-channel block of the queries
constexpr uint32_t PA_S_COL = 256;     // TMEM: O^T in columns [0, 256), S^T behind
constexpr uint32_t PA_TMEM_COLS = 512;
constexpr float PA_SHIFT = 7.0f, PA_SLACK = 8.0f;
constexpr float PA_NONE = -1e30f;  // reference of a row that has met no key

struct PaSmem {
  // K = V in fp16: channel block kb at kb * PA_KB, 128 rows (keys) of 128 B,
  // 16-byte chunks swizzled by row % 8
  alignas(1024) uint8_t tile[8 * PA_KB];
  alignas(1024) uint8_t q[8 * PA_QKB];       // Q': block kb, 64 rows of 128 B
  alignas(1024) uint8_t p[PA_KEYS * 128];    // P: [key][64 query rows] fp16
  alignas(16) float scl1[PA_ROWS], scl2[PA_ROWS];  // logit = acc * scl1 * scl2 (log2 units)
  alignas(16) float m[PA_ROWS];
  alignas(16) int lo[PA_ROWS], hi[PA_ROWS];  // keys [lo, hi) are visible to the row
  uint32_t bad[PA_KEYS];  // byte qq: quarter qq of the key row holds a NaN
  float red[4][PA_ROWS];
  int cum[CSA2_PREFIX_MAX_BATCH + 1];        // own key tiles of sequences < b
  int wsum[PA_NT / 32];
  uint64_t mbar;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t PA_SMEM = sizeof(PaSmem) + 1024;
static_assert(PA_SMEM <= 232448, "shared memory of one CTA");

__device__ __forceinline__ uint32_t pa_h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t pa_sw(int r, int cc) {
  return (uint32_t)(r * 128 + ((cc ^ (r & 7)) << 4));
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One contiguous run of key tiles of one segment.
struct PaRun {
  int row0, n_rows;  // first query row of the batch, rows (a multiple of 16)
  int seq;           // sequence whose row map is used
  int kt, kt_end;    // key tiles
  int own_tiles;     // tiles at or past this are window tiles (own segments)
  int first_pos;     // position of key 0 of tile 0
  int win_lo;        // first window row of tile own_tiles
  bool own;
  int64_t slot;
};

// This thread's quarter of one key row: raw bytes of key r, channels
// [128 qq, 128 qq + 128).
struct PaRaw {
  uint4 v[8];
  uint2 s;
  bool ok;      // the key exists
  bool window;  // E4M3 bytes, otherwise FP4 codes
};

__device__ __forceinline__ void pa_load(const PrefixParams& p, const PaRun& run, int kt, int r,
                                        int qq, int n_own, int n_win, PaRaw& raw) {
  raw.ok = false;
  raw.window = run.own && kt >= run.own_tiles;
  if (!raw.window) {
    const int pos = run.first_pos + kt * PA_KEYS + r;
    if (pos >= n_own) return;
    int64_t row;
    if (p.page_table) {
      const int page = pos >> 6;
      const int64_t pid =
          page < p.max_pages ? (int64_t)__ldg(p.page_table + (int64_t)run.seq * p.max_pages + page)
                             : -1;
      row = pid < 0 ? -1 : pid * 64 + (pos & 63);
    } else {
      row = (int64_t)run.seq * p.seq_stride + pos;
    }
    if (row < 0 || row >= p.pool_rows) {
      set_status(p.status, ST_DEVICE_CHECK);
      return;
    }
    raw.ok = true;
    const uint4* c = reinterpret_cast<const uint4*>(p.codes + row * (CSA2_D / 2) + 64 * qq);
#pragma unroll
    for (int i = 0; i < 4; i++) raw.v[i] = __ldg(c + i);
    raw.s = __ldg(reinterpret_cast<const uint2*>(p.scales + row * (CSA2_D / 16) + 8 * qq));
  } else {
    const int j = run.win_lo + (kt - run.own_tiles) * PA_KEYS + r;
    if (j >= n_win) return;
    raw.ok = true;
    const uint4* w = reinterpret_cast<const uint4*>(
        p.swa + ((int64_t)run.seq * p.swa_rows + j) * CSA2_D + 128 * qq);
#pragma unroll
    for (int i = 0; i < 8; i++) raw.v[i] = __ldg(w + i);
  }
}

// Whether a byte of w is an E4M3 NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
}

// A key that is not there, or whose values hold a NaN, becomes zeros: P = 0 of a
// row that must not see it would otherwise turn NaN in the product.  Returns
// whether it was a NaN: the rows that see the key then get NaN weights.
__device__ __forceinline__ bool pa_dequant(const PaRaw& raw, uint8_t* tile, int r, int qq) {
  uint8_t* trow = tile + r * 128;
  const int sw = r & 7;
  bool nan = false;
  if (raw.ok && !raw.window) nan = has_nan(raw.s.x) || has_nan(raw.s.y);
  if (raw.ok && raw.window) {
#pragma unroll
    for (int j = 0; j < 8; j++)
      nan |= has_nan(raw.v[j].x) || has_nan(raw.v[j].y) || has_nan(raw.v[j].z) ||
             has_nan(raw.v[j].w);
  }
  if (!raw.ok || nan) {
#pragma unroll
    for (int j = 0; j < 16; j++)
      *reinterpret_cast<uint4*>(trow + (2 * qq + (j >> 3)) * PA_KB + (((j & 7) ^ sw) << 4)) =
          make_uint4(0, 0, 0, 0);
  } else if (!raw.window) {
#pragma unroll
    for (int i = 0; i < 4; i++) {  // 16 code bytes: channels 128 qq + 32 i + [0, 32)
      const uint32_t words[4] = {raw.v[i].x, raw.v[i].y, raw.v[i].z, raw.v[i].w};
      const uint32_t sb = ((i < 2 ? raw.s.x : raw.s.y) >> (16 * (i & 1))) & 0xFFFFu;
      const __half2 sc = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)sb, __NV_E4M3));
      uint8_t* dst = trow + (2 * qq + (i >> 1)) * PA_KB;
#pragma unroll
      for (int c = 0; c < 4; c++) {  // 8 channels per 16-byte store
        const __half2 s2 = c < 2 ? __low2half2(sc) : __high2half2(sc);
        uint32_t hv[4];
#pragma unroll
        for (int k = 0; k < 4; k++)
          hv[k] = pa_h2u(__hmul2(__half2(__nv_cvt_fp4x2_to_halfraw2(
                                     (__nv_fp4x2_storage_t)((words[c] >> (8 * k)) & 0xFF),
                                     __NV_E2M1)),
                                 s2));
        *reinterpret_cast<uint4*>(dst + (((4 * (i & 1) + c) ^ sw) << 4)) =
            make_uint4(hv[0], hv[1], hv[2], hv[3]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {  // 16 E4M3 bytes: channels 128 qq + 16 j + [0, 16)
      const uint32_t wv[4] = {raw.v[j].x, raw.v[j].y, raw.v[j].z, raw.v[j].w};
      uint32_t hv[8];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        hv[2 * k] = pa_h2u(__half2(
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(wv[k] & 0xFFFF), __NV_E4M3)));
        hv[2 * k + 1] = pa_h2u(
            __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(wv[k] >> 16), __NV_E4M3)));
      }
      uint8_t* dst = trow + (2 * qq + (j >> 2)) * PA_KB;
      const int cc = 2 * (j & 3);
      *reinterpret_cast<uint4*>(dst + ((cc ^ sw) << 4)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
      *reinterpret_cast<uint4*>(dst + (((cc + 1) ^ sw) << 4)) = make_uint4(hv[4], hv[5], hv[6], hv[7]);
    }
  }
  return nan;
}

// S^T and O^T products; n: query rows of the tile.  P is read MN-major (its
// rows are keys, the K axis of the second product).
__device__ __forceinline__ uint32_t pa_idesc(int n, bool pv) {
  return (1u << 4) | (pv ? (1u << 15) | (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

__global__ void __launch_bounds__(PA_NT, 1) prefix_attn_kernel(const PrefixParams p) {
  extern __shared__ uint8_t smem_raw[];
  PaSmem& s = *reinterpret_cast<PaSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~uintptr_t(1023));
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  pdl_launch_dependents();
  if (t == 0) {
    mbar_init(&s.mbar, 1);
    fence_mbar_init();
    s.abort = 0;
  }
  if (warp == 0) {
    tmem_alloc(&s.tmem_base, PA_TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();

  // ---- the plan: prefix sums of the sequences' own key tiles
  PaPlan pl = pa_plan(p);
  {
    int v[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int b = 2 * t + k;
      if (b < p.batch) {
        const int n = p.n_rows[b];
        if ((n < 0 || n > p.max_rows) && blockIdx.x == 0) set_status(p.status, ST_DEVICE_CHECK);
        v[k] = pa_own_tiles(p, n) + pl.win_tiles;
      }
    }
    int incl = v[0] + v[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s.wsum[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int before = 0;
    for (int w = 0; w < warp; w++) before += s.wsum[w];
    if (2 * t < p.batch) s.cum[2 * t + 1] = before + incl - v[1];
    if (2 * t + 1 < p.batch) s.cum[2 * t + 2] = before + incl;
    if (t == 0) s.cum[0] = 0;
    __syncthreads();
  }
  pl.finish(s.cum[p.batch]);
  const uint32_t tmem = s.tmem_base;
  const int r = t & (PA_KEYS - 1), qq = t >> 7;  // key row, quarter; also TMEM lane, column group
  const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;

  int64_t tile = pl.total > 0 ? pl.tile_at(blockIdx.x) : 0;
  const int64_t tile_end = pl.total > 0 ? pl.tile_at(blockIdx.x + 1) : 0;
  bool alive = true;
  while (tile < tile_end && alive) {
    // ---- the segment of this tile and the run of it that is ours
    PaRun run;
    int n_own, n_win = 0;  // keys of the row map, rows of the window
    int64_t seg_end;
    if (tile < pl.shared) {
      const int seg = (int)(tile / pl.prefix_tiles);
      run.own = false;
      run.seq = 0;
      run.row0 = seg * PA_ROWS;
      run.n_rows = min(PA_ROWS, p.batch * p.nq * CSA2_H - run.row0);
      run.kt = (int)(tile - (int64_t)seg * pl.prefix_tiles);
      run.own_tiles = pl.prefix_tiles;
      run.first_pos = 0;
      run.win_lo = 0;
      run.slot = pl.shared_slot(seg, blockIdx.x);
      seg_end = (int64_t)(seg + 1) * pl.prefix_tiles;
      n_own = p.prefix;
    } else {
      const int64_t u = tile - pl.shared;
      int lo = 0, hi = p.batch;  // the last b with q_blocks * cum[b] <= u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)s.cum[mid] * pl.q_blocks <= u) lo = mid; else hi = mid;
      }
      const int b = lo, kts = s.cum[b + 1] - s.cum[b];
      const int64_t rem = u - (int64_t)s.cum[b] * pl.q_blocks;
      const int qb = (int)(rem / kts);
      run.own = true;
      run.seq = b;
      run.row0 = (b * p.nq + qb * PA_QB) * CSA2_H;
      run.n_rows = min(PA_QB, p.nq - qb * PA_QB) * CSA2_H;
      run.kt = (int)(rem - (int64_t)qb * kts);
      run.own_tiles = kts - pl.win_tiles;
      run.first_pos = p.prefix;
      run.slot = pl.own_slot(b * pl.q_blocks + qb, blockIdx.x);
      seg_end = tile - run.kt + kts;
      const int n = p.n_rows[b];
      n_own = n < 0 ? 0 : min(n, p.max_rows);
      run.win_lo = 0;
      if (p.swa) {
        n_win = p.swa_len[b];
        if (n_win < 0 || n_win > p.swa_rows) {
          if (t == 0) set_status(p.status, ST_DEVICE_CHECK);
          n_win = n_win < 0 ? 0 : p.swa_rows;
        }
        run.win_lo = max(0, n_win - (p.nq - 1 - qb * PA_QB) - CSA2_W);
      }
    }
    run.kt_end = run.kt + (int)(min(seg_end, tile_end) - tile);
    tile += run.kt_end - run.kt;

    PaRaw raw;
    pa_load(p, run, run.kt, r, qq, n_own, n_win, raw);

    // ---- Q' = Q * 2^e in fp16, max |Q'| of a row in [2^14, 2^15): one warp per
    // row, 16 channels per lane
    for (int h = warp; h < run.n_rows; h += PA_NT / 32) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(run.row0 + h) * CSA2_D) +
                         2 * lane;
      uint4 v[2];
      uint32_t mx = 0u;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        v[k] = __ldg(src + k);
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; j++) mx = max(mx, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      const int e = q_pow2_exponent(mx);
      const int e1 = e / 2, e2 = e - e1;
      const float f = pow2i(e1), f2 = pow2i(e2);
      if (lane == 0) {
        s.scl1[h] = pow2i(-e1);
        s.scl2[h] = p.scale_log2 * pow2i(-e2);
      }
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o4[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
          o4[j] = pa_h2u(__floats2half2_rn(__uint_as_float(w[j] << 16) * f * f2,
                                           __uint_as_float(w[j] & 0xFFFF0000u) * f * f2));
        *reinterpret_cast<uint4*>(s.q + (lane >> 2) * PA_QKB + pa_sw(h, 2 * (lane & 3) + k)) =
            make_uint4(o4[0], o4[1], o4[2], o4[3]);
      }
    }
    float l[16];
#pragma unroll
    for (int j = 0; j < 16; j++) l[j] = 0.0f;
    if (t < PA_ROWS) s.m[t] = PA_NONE;
    bool window_limits = false;
    const int kt0 = run.kt;
#pragma unroll 1
    for (int kt = kt0; kt < run.kt_end && alive; kt++) {
      // ---- visible keys of every row: positions, or window rows
      const bool win = run.own && kt >= run.own_tiles;
      if ((kt == kt0 || win != window_limits) && t < run.n_rows) {
        const int qi = (run.row0 + t) / CSA2_H, b = qi / p.nq, later = p.nq - 1 - (qi - b * p.nq);
        if (win) {
          s.hi[t] = max(0, n_win - later);
          s.lo[t] = max(0, n_win - later - CSA2_W);
        } else {
          const int n = p.n_rows[b];
          s.hi[t] = min((n < 0 ? 0 : min(n, p.max_rows)) - later, n_own);
          s.lo[t] = 0;
        }
      }
      window_limits = win;
      // ---- the fp16 tile
      reinterpret_cast<uint8_t*>(&s.bad[r])[qq] = pa_dequant(raw, s.tile, r, qq);
      const bool key_ok = raw.ok;
      const int key = win ? run.win_lo + (kt - run.own_tiles) * PA_KEYS + r
                          : run.first_pos + kt * PA_KEYS + r;
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      // ---- S^T = K Q'^T: K = 512 in 32 steps
      if (t == 0) {
        tc_fence_after();
        const uint64_t da = sdesc_k128(smem_u32(s.tile)), db = sdesc_k128(smem_u32(s.q));
        const uint32_t id = pa_idesc(run.n_rows, false);
#pragma unroll 1
        for (uint32_t i = 0; i < 32; i++)
          umma_bf16(tmem + PA_S_COL, da + (((i >> 2) * PA_KB + 32 * (i & 3)) >> 4),
                    db + (((i >> 2) * PA_QKB + 32 * (i & 3)) >> 4), id, i != 0);
        umma_commit(&s.mbar);
      }
      if (kt + 1 < run.kt_end) pa_load(p, run, kt + 1, r, qq, n_own, n_win, raw);
      if (!mbar_wait(&s.mbar, 0, nullptr)) s.abort = 1;
      __syncwarp();
      tc_fence_after();
      // ---- softmax: one key and 16 query rows per thread
      const bool active = 16 * qq < run.n_rows;  // per warp
      float x[16];
      float over = -INFINITY;
      if (active) {
        uint32_t acc[16];
        tmem_ld_x16(tmem + lane_base + PA_S_COL + 16 * qq, acc);
        tmem_ld_wait();
        const bool bad = s.bad[r] != 0;
#pragma unroll
        for (int j = 0; j < 16; j++) {
          const int c = 16 * qq + j;
          const bool see = key_ok && key >= s.lo[c] && key < s.hi[c];
          const float v = __uint_as_float(acc[j]) * s.scl1[c] * s.scl2[c];
          x[j] = see ? (bad ? __int_as_float(0x7FC00000) : v) : -INFINITY;
          over = fmaxf(over, x[j] - s.m[c]);
        }
      }
      if (__syncthreads_or(over > PA_SLACK)) {
        // some logit is far above its reference: raise the references to the
        // rows' maxima and scale what was summed
        if (active) {
#pragma unroll
          for (int j = 0; j < 16; j++) {
            const float mx = warp_max_f32(x[j]);
            if (lane == 0) s.red[warp & 3][16 * qq + j] = mx;
          }
        }
        __syncthreads();
        if (active) {
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; j++) {
            const int c = 16 * qq + j;
            const float old = s.m[c];
            const float mx = fmaxf(fmaxf(s.red[0][c], s.red[1][c]), fmaxf(s.red[2][c], s.red[3][c]));
            f[j] = exp2f(old - fmaxf(old, mx));
            l[j] *= f[j];
          }
          if (kt != kt0) {
#pragma unroll 1
            for (int cb = 0; cb < 4; cb++) {
              uint32_t o[16];
              tmem_ld_x16(tmem + lane_base + 64 * cb + 16 * qq, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * f[j]);
              tmem_st_x16(tmem + lane_base + 64 * cb + 16 * qq, o);
            }
            tmem_st_wait();
          }
        }
        __syncthreads();
        if (t < run.n_rows)
          s.m[t] = fmaxf(s.m[t], fmaxf(fmaxf(s.red[0][t], s.red[1][t]),
                                       fmaxf(s.red[2][t], s.red[3][t])));
        __syncthreads();
      }
      if (active) {
        uint32_t hv[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const int c = 16 * qq + 2 * j;
          const __half2 h = __floats2half2_rn(exp2f(x[2 * j] - s.m[c] + PA_SHIFT),
                                              exp2f(x[2 * j + 1] - s.m[c + 1] + PA_SHIFT));
          const float2 g = __half22float2(h);
          l[2 * j] += g.x;
          l[2 * j + 1] += g.y;
          hv[j] = pa_h2u(h);
        }
        *reinterpret_cast<uint4*>(s.p + pa_sw(r, 2 * qq)) = make_uint4(hv[0], hv[1], hv[2], hv[3]);
        *reinterpret_cast<uint4*>(s.p + pa_sw(r, 2 * qq + 1)) =
            make_uint4(hv[4], hv[5], hv[6], hv[7]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      // ---- O^T += V^T P^T: four channel blocks of 128, K = 128 keys in 8 steps
      if (t == 0) {
        tc_fence_after();
        const uint64_t da = sdesc_mn128(smem_u32(s.tile), PA_KB, 1024),
                       db = sdesc_mn128(smem_u32(s.p), PA_KEYS * 128, 1024);
        const uint32_t id = pa_idesc(run.n_rows, true);
#pragma unroll 1
        for (uint32_t i = 0; i < 32; i++) {
          const uint32_t cb = i & 3, ks = i >> 2;
          umma_bf16(tmem + 64 * cb, da + ((cb * 2 * PA_KB + ks * 2048) >> 4),
                    db + ((ks * 2048) >> 4), id, kt != kt0 || ks != 0);
        }
        umma_commit(&s.mbar);
      }
      if (!mbar_wait(&s.mbar, 1, nullptr)) s.abort = 1;
      __syncwarp();
      tc_fence_after();
      __syncthreads();
      alive = s.abort == 0;
    }
    if (!alive) {
      if (t == 0) set_status(p.status, ST_TIMEOUT);
      break;
    }

    // ---- the run's partial: O [row][channel], (max, sum) per row
    if (16 * qq < run.n_rows) {
#pragma unroll
      for (int j = 0; j < 16; j++) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], o);
        if (lane == 0) s.red[warp & 3][16 * qq + j] = l[j];
      }
#pragma unroll 1
      for (int cb = 0; cb < 4; cb++) {
        uint32_t o[16];
        tmem_ld_x16(tmem + lane_base + 64 * cb + 16 * qq, o);
        tmem_ld_wait();
        float* dst = p.part_o + (run.slot + 16 * qq) * CSA2_D + 128 * cb + r;
#pragma unroll
        for (int j = 0; j < 16; j++) dst[j * CSA2_D] = __uint_as_float(o[j]);
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (t < run.n_rows) {
      p.part_ml[2 * (run.slot + t)] = s.m[t];
      p.part_ml[2 * (run.slot + t) + 1] =
          (s.red[0][t] + s.red[1][t]) + (s.red[2][t] + s.red[3][t]);
    }
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, PA_TMEM_COLS);
  }
}

// One CTA per query row: out = sum_i w_i O_i / sum_i w_i l_i over the row's
// partials, w_i = 2^(m_i - max m).  Four groups of 128 threads (four channels
// each) take every fourth partial; their sums join in a fixed order.
constexpr int PM_NT = 512;
__global__ void __launch_bounds__(PM_NT) prefix_merge_kernel(const PrefixParams p) {
  __shared__ int64_t slot[2 * PA_MAX_GRID];
  __shared__ float w[2 * PA_MAX_GRID];
  __shared__ int sums[2];
  __shared__ float red[PM_NT / 32];
  __shared__ float total_l;
  __shared__ float4 acc_s[3][128];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, row = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  if (t < 2) sums[t] = 0;
  __syncthreads();
  const int qi = row / CSA2_H, b = qi / p.nq, tq = qi - b * p.nq;
  PaPlan pl = pa_plan(p);
  int before = 0, all = 0;
  for (int i = t; i < p.batch; i += PM_NT) {
    const int k = pa_own_tiles(p, p.n_rows[i]) + pl.win_tiles;
    all += k;
    if (i < b) before += k;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    atomicAdd(&sums[0], all);  // whole numbers: any order gives the same sum
    atomicAdd(&sums[1], before);
  }
  __syncthreads();
  pl.finish(sums[0]);
  const int kts = pa_own_tiles(p, p.n_rows[b]) + pl.win_tiles;

  // ---- the row's partials: shared segment, then own segment
  const int qb = tq / PA_QB, seg = row / PA_ROWS, oseg = b * pl.q_blocks + qb;
  const int64_t ts[2] = {(int64_t)seg * pl.prefix_tiles,
                         pl.shared + (int64_t)sums[1] * pl.q_blocks + (int64_t)qb * kts};
  const int64_t te[2] = {ts[0] + pl.prefix_tiles, ts[1] + kts};
  int first[2] = {0, 0}, count[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; k++) {
    if (te[k] > ts[k]) {
      first[k] = pl.cta_of(ts[k]);
      count[k] = pl.cta_of(te[k] - 1) - first[k] + 1;
    }
  }
  const int n = count[0] + count[1];
  float m = -INFINITY, l = 0.0f;
  int64_t at = 0;
  if (t < n) {  // n <= 2 * PA_MAX_GRID <= PM_NT
    const int k = t < count[0] ? 0 : 1, c = first[k] + (k ? t - count[0] : t);
    const int64_t a = max(pl.tile_at(c), ts[k]), z = min(pl.tile_at(c + 1), te[k]);
    if (a < z) {
      at = k ? pl.own_slot(oseg, c) + (tq - qb * PA_QB) * CSA2_H + row % CSA2_H
             : pl.shared_slot(seg, c) + row % PA_ROWS;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
      if (ml.y > 0.0f || ml.y != ml.y) {  // a NaN sum stays one
        m = ml.x;
        l = ml.y;
      }
    }
  }
  {
    const float v = warp_max_f32(m);
    if (lane == 0) red[warp] = v;
  }
  __syncthreads();
  float M = red[0];
#pragma unroll
  for (int i = 1; i < PM_NT / 32; i++) M = fmaxf(M, red[i]);
  const float wt = m == -INFINITY ? 0.0f : exp2f(m - M);
  if (t < n) {
    slot[t] = at;
    w[t] = wt;
  }
  float sl = wt * l;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sl += __shfl_xor_sync(0xffffffffu, sl, o);
  __syncthreads();
  if (lane == 0) red[warp] = sl;
  __syncthreads();
  if (t == 0) {
    float v = 0.0f;
    for (int i = 0; i < PM_NT / 32; i++) v += red[i];
    total_l = v;
  }
  // ---- the weighted sum
  const int g = t >> 7, ch = 4 * (t & 127);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = g; i < n; i += 4) {
    if (w[i] == 0.0f) continue;
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot[i] * CSA2_D + ch);
    acc.x = fmaf(w[i], v.x, acc.x);
    acc.y = fmaf(w[i], v.y, acc.y);
    acc.z = fmaf(w[i], v.z, acc.z);
    acc.w = fmaf(w[i], v.w, acc.w);
  }
  if (g > 0) acc_s[g - 1][t & 127] = acc;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int k = 0; k < 3; k++) {
      const float4 v = acc_s[k][t];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float tl = total_l;
    const float inv = tl == 0.0f ? 0.0f : 1.0f / tl;
    const __nv_bfloat162 o0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 o1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + (int64_t)row * CSA2_D + ch) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&o0), *reinterpret_cast<const uint32_t*>(&o1));
  }
}

int prefix_grid(const PrefixParams& p, int num_sms) {
  const PaPlan pl = pa_plan(p);
  const int64_t own = (int64_t)p.batch * pl.q_blocks *
                      ((p.max_rows - p.prefix + PA_KEYS - 1) / PA_KEYS + pl.win_tiles);
  const int64_t most = num_sms < PA_MAX_GRID ? num_sms : PA_MAX_GRID;
  const int64_t tiles = pl.shared + own;
  return (int)(tiles < 1 ? 1 : (tiles < most ? tiles : most));
}

size_t prefix_partial_rows(const PrefixParams& p) {
  const PaPlan pl = pa_plan(p);
  return (size_t)(pl.row_blocks + pl.grid) * PA_ROWS +
         ((size_t)p.batch * pl.q_blocks + pl.grid) * pl.own_rows;
}

cudaError_t launch_prefix_attn(const PrefixParams& p, cudaStream_t st) {
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([](int&) {
    return cudaFuncSetAttribute(prefix_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)PA_SMEM);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(PA_NT);
  cfg.dynamicSmemBytes = PA_SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  trace_mark("prefix_attn", st);
  if ((e = cudaLaunchKernelEx(&cfg, prefix_attn_kernel, p)) != cudaSuccess) return e;
  cfg.gridDim = dim3(p.batch * p.nq * CSA2_H);
  cfg.blockDim = dim3(PM_NT);
  cfg.dynamicSmemBytes = 0;
  trace_mark("prefix_merge", st);
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel, p);
}

}  // namespace csa2
