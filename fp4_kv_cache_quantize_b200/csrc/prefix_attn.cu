// prefix_attn.cu -- dense attention of a batch that shares a prefix
// (csa2_prefix_attn).
//
// Every query head of the batch meets the shared rows, so a key tile is read
// and dequantised once for 64 query rows, or, where there are many blocks of those,
// once for all of them by a kernel in front: S^T = K Q'^T (keys on the MMA's M
// axis) and O^T = V^T P^T (channels on it), fp16 operands, fp32 accumulators
// in tensor memory.  E2M1 x E4M3 products and E4M3 window values are exact in
// fp16; a query head is scaled by a power of two into fp16's range.
//
// Softmax in one pass: with a reference m per row, p_j = 2^(c (a_j - m) + 7),
// O += p_j v_j, l += p_j, where a_j are the products' accumulators and c >= 0 the
// row's scale (a negative sm_scale turns the queries' signs instead).  m only has to
// be near the maximum: it is raised (and O, l scaled) when some c a_j exceeds c m by
// 8, so p <= 2^15 fits fp16, and the +7 keeps p to 2^-31 of the row's largest before
// it is lost: a million keys lose at most 2^-12 of the sum together.  (fp16 rounds
// each p by 2^-11 of itself where bf16 would by 2^-8; l sums them unrounded, in
// fp32.)  m is one of the a_j, not a logit: c m rounded to fp32 would be off by more
// than the 8 from 2^28 on, and no logit has to fit fp32 this way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa2_internal.cuh"
#include "kernels.h"
#include "prefix_plan.cuh"
#include "umma_m64.cuh"

namespace csa2 {

// What bounds it.  At 64 query rows a 64-key tile costs 1,792 cycles of tensor core
// (32 S^T steps of 32 cycles, 16 O^T steps of 48).  Where row blocks turn their own
// tiles to fp16 it takes 3,300: shared memory's path is busy for 2,840 of them (the
// products read K, V, Q' and P, the warps write K and P), each scheduler issues for
// 2,200.  With the images there it takes 2,600: the chain of a tile buffer, which is
// its copy (1,500 from request to first byte, 2,600 to last), S^T, softmax (1,300 with
// its waits) and O^T, one after another but for the parts; there are two buffers.
// The L2 is not what they wait for: over a 16K-row prefix and 64 sequences it gives 23%
// of its rate (its busiest slice 26%), 83% of it hits.
//   128K-row prefix, 64 sequences (1,024 rows): 381 us, 0.73 PFLOP/s; 390 to 400 call
//   after call, when the power limit takes the clock below 1.85 GHz
//   16K-row prefix, 2 x 256 queries (8,192 rows): 372 us, 0.77 PFLOP/s, 1.9 GHz
//   1M-row prefix, 4 sequences (64 rows, no images): 229 us, 1.26 TB/s of cache rows
//   2K-row prefix, 4 sequences: 17 us, the latencies of one tile a CTA (lengths,
//   plan, page, rows, products, softmax, partial) and of the merge
//
// Roles of a CTA: eight warps turn key tiles into fp16 (or one of them copies images:
// all eight took 402 us instead of 389, in power), sixteen run the softmax, one thread
// issues the S^T products and one the O^T products, one warp works out which tiles
// come next.  Key tiles are 64 keys so that two fit next to the queries: while one is
// multiplied, the next is written.  S^T then is an M = 64 product at half the tensor
// core's rate, but one that shared memory could not
// feed faster anyway (4 KB of operands in 32 cycles); a single 128-key tile,
// filled, multiplied and filled again, took twice as long.
constexpr int PA_DQ_WARPS = 8, PA_SM_WARPS = 16;
constexpr int PA_PART = 4 * PA_ROWS / PA_SM_WARPS;  // query rows of a softmax warp
constexpr int PA_COLS = PA_PART / 4;                // and of a thread
constexpr int PA_MMA_WARP = PA_DQ_WARPS + PA_SM_WARPS;
constexpr int PA_NT = 32 * (PA_MMA_WARP + 3);
// A tile is written, multiplied and freed in parts of 128 channels: S^T begins with
// the first part, and the first part is filled again while the others are still in
// the O^T products (2 x 256 queries 374 us with two parts, 356 with four).  Warps that
// turn codes into fp16 finish two parts at once: each costs them a fence and waits
// (a million rows: one part 247 us, two 238, four of their own 293).
constexpr int PA_PARTS = 4;
constexpr int PA_KB = PA_KEYS * 128;   // one 64-channel chunk of a key tile
constexpr int PA_COPY = 8 * PA_KB / PA_PARTS;  // a part of an image
constexpr int PA_QKB = PA_ROWS * 128;  // one 64-channel chunk of the queries
constexpr uint32_t PA_S_COL = 256;     // TMEM: O^T in columns [0, 256), two S^T behind
constexpr uint32_t PA_TMEM_COLS = 512;
constexpr float PA_SHIFT = 7.0f, PA_SLACK = 8.0f;
// Reference of a row that has met no key.  The first one raises it, except where c is
// so small (2^-125) that all its p are 2^7 to the last bit.
constexpr float PA_NONE = -3.402823466e38f;
constexpr float PA_MOST = 3.402823466e38f;
// The scale of 1 / 256 that keeps sm_scale log2(e) finite until a row's is made of it.
constexpr float PA_PRE_SCALE = 256.0f;

// mbar_wait that sleeps until the phase completes, in naps of up to 20 us: the
// waits' polling otherwise takes issue slots from the warps that work.
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  auto nap = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
  };
  if (nap()) return true;
  const long long t0 = clock64();
  while (!nap()) {
    if (*abort || clock64() - t0 > kWaitCycles) return false;
  }
  return true;
}

// One contiguous run of key tiles of one segment.
struct PaRun {
  int row0, n_rows;  // first query row of the batch, rows (a multiple of 16)
  int seq;           // sequence whose row map is used
  int kt, kt_end;    // key tiles (none if kt_end <= kt)
  int line;          // how far the run goes on the line
  int own_tiles;     // tiles at or past this are window tiles (own segments)
  int kt_cache;      // cache tiles of the run end here
  int first_pos;     // position of key 0 of tile 0
  int n_keys;        // positions of the row map end here
  int win_lo, n_win; // first window row of tile own_tiles, rows of the window
  bool own, image;   // image: the run's tiles are there in fp16
  bool valid;        // false: no run is left
  int64_t slot;
};

struct PaSmem {
  // K = V in fp16, two tiles: channel chunk kb at kb * PA_KB, 64 rows (keys) of
  // 128 B, 16-byte pieces swizzled by row % 8
  alignas(1024) uint8_t tile[2][8 * PA_KB];
  alignas(1024) uint8_t q[8 * PA_QKB];        // Q': chunk kb, 64 rows of 128 B
  alignas(1024) uint8_t p[2][PA_KEYS * 128];  // P: [key][64 query rows] fp16
  alignas(16) float scl[PA_ROWS];             // logit = acc * scl (log2 units), >= 0
  alignas(16) float fac[PA_ROWS];             // what a raised reference scales O by
  alignas(16) int lo[2][PA_ROWS], hi[2][PA_ROWS];  // cache, window: visible keys [lo, hi)
  int lo_max[2], hi_min[2];                   // keys [lo_max, hi_min) are visible to all rows
  // per tile: whether a key is missing (1) or holds a NaN (2), by reading thread
  alignas(16) uint8_t key[2][PA_KEYS][4];
  float red[4][PA_ROWS];
  int cum[CSA2_PREFIX_MAX_BATCH + 1];         // own tiles on the line of sequences < b
  int wsum[32];
  uint64_t full[2][PA_PARTS], empty[2][PA_PARTS];  // part of a tile: written, multiplied
  uint64_t s_full[2], p_full[2];
  uint64_t run_full[2], run_empty[2];  // run planned, done with by every role
  uint32_t tmem_base;
  int abort;
  PaRun run[2];
};
constexpr size_t PA_SMEM = sizeof(PaSmem);
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
// Barrier of 128 threads that also tells whether any of them said so.
__device__ __forceinline__ bool bar_or_128(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// Loads that stay where they are written: a plain read-only load may be moved
// down to its use, one tile later, which put a whole memory latency in front of
// every block.
__device__ __forceinline__ uint4 ld_now_v4(const void* a) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a));
  return v;
}
__device__ __forceinline__ float4 ld_now_f4(const float* a) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_now_u16(const void* a) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(a));
  return v;
}

__device__ __forceinline__ uint32_t ld_now_u8(const void* a) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}
__device__ __forceinline__ int ld_now_s32(const void* a) {
  int v;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(a));
  return v;
}

// The row map in two steps, so that the page id's latency has a tile's time:
// the page id of a position (not waited for), then its pool row.  -1: none (a
// mapping outside the pool is recorded).  A thread holds its key's part of the run:
// position pos + 64 kt of sequence seq, if below n_keys and kt below kt_cache.
struct PaMap {
  int pos, n_keys, kt_cache, seq;
};
__device__ __forceinline__ int pa_page(const PrefixParams& p, const PaMap& m, int kt) {
  const int pos = m.pos + kt * PA_KEYS;
  if (kt >= m.kt_cache || pos >= m.n_keys) return -1;
  if (!p.page_table) return 0;
  const int page = pos >> 6;
  if (page >= p.max_pages) return -2;
  return ld_now_s32(p.page_table + (int64_t)m.seq * p.max_pages + page);
}
__device__ __forceinline__ int64_t pa_row(const PrefixParams& p, const PaMap& m, int kt, int pid) {
  const int pos = m.pos + kt * PA_KEYS;
  if (kt >= m.kt_cache || pos >= m.n_keys) return -1;
  const int64_t row = p.page_table ? (int64_t)pid * 64 + (pos & 63)
                                   : (int64_t)m.seq * p.seq_stride + pos;
  if (pid < 0 || row >= p.pool_rows) {
    set_status(p.status, ST_DEVICE_CHECK);
    return -1;
  }
  return row;
}

// Whether a byte of w is an E4M3 NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
}
// Two E4M3 bytes at bits 0 and 16 of w as fp16 times 2^-8: the four exponent
// and three mantissa bits keep their places below the fp16 exponent's top bit,
// which is right for E4M3's subnormals too.
__device__ __forceinline__ __half2 e4m3x2_as_f16(uint32_t w) {
  const uint32_t h = ((w & 0x007F007Fu) << 7) | ((w & 0x00800080u) << 8);
  return *reinterpret_cast<const __half2*>(&h);
}
// Tile values are 2^-7 of the key's, so that the factor fits fp16 (below); the
// logits' and the outputs' scales give it back.
constexpr float PA_TILE_SCALE = 128.0f;
// Eight FP4 codes (one word) times the scale f as fp16.  A code's bits s, eem go
// to the fp16 sign and to bits 9..11, which reads as 2^-14 of the E2M1 value
// (subnormal 0.5 included): by shifts and masks into the upper byte of the fp16,
// four codes at once, then bytes to halves (the conversion instruction has a small
// share of the ALU's rate: with it the kernel spent 86% of its time in that unit).
// f = scale * 2^7 <= 57,344 makes the product value * scale * 2^-7: five significant
// bits above 2^-18, exact.  Codes come out in the order 0 2 4 6 1 3 5 7; Q' has the
// same and the outputs are stored through pa_channel.
__device__ __forceinline__ uint4 pa_fp4x8(uint32_t w, __half2 f) {
  const uint32_t even = ((w << 4) & 0x80808080u) | ((w << 1) & 0x0E0E0E0Eu);
  const uint32_t odd = (w & 0x80808080u) | ((w >> 3) & 0x0E0E0E0Eu);
  uint32_t h[4] = {__byte_perm(even, 0, 0x1404), __byte_perm(even, 0, 0x3424),
                   __byte_perm(odd, 0, 0x1404), __byte_perm(odd, 0, 0x3424)};
#pragma unroll
  for (int k = 0; k < 4; k++) h[k] = pa_h2u(__hmul2(*reinterpret_cast<__half2*>(&h[k]), f));
  return make_uint4(h[0], h[1], h[2], h[3]);
}
// Channel at place c of a tile row (within its group of eight).
__device__ __forceinline__ int pa_channel(int c) {
  return (c & ~7) | ((c & 3) << 1) | ((c >> 2) & 1);
}
// Two E4M3 scales (bits 0 and 16) as pa_fp4x8's factors.
__device__ __forceinline__ __half2 pa_scale(uint32_t sc) {
  return __hmul2(e4m3x2_as_f16(sc),
                 __half2(__ushort_as_half(0x7800), __ushort_as_half(0x7800)));  // 2^15
}
// 32 FP4 codes (16 bytes) with their two E4M3 scales (low half of sc) into four
// 16-byte pieces cc .. cc + 3 of a swizzled row.
__device__ __forceinline__ void pa_put_fp4(uint8_t* row, int sw, int cc, uint4 v, uint32_t sc) {
  const __half2 s2 = pa_scale((sc & 0xFFu) | ((sc & 0xFF00u) << 8));
  const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int c = 0; c < 4; c++)
    *reinterpret_cast<uint4*>(row + (((cc + c) ^ sw) << 4)) =
        pa_fp4x8(words[c], c < 2 ? __low2half2(s2) : __high2half2(s2));
}
// Eight E4M3 values (two words) as tile values.
__device__ __forceinline__ uint4 pa_e4m3x8(uint32_t a, uint32_t b) {
  const __half2 two = __half2(__ushort_as_half(0x4000), __ushort_as_half(0x4000));
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; k++)
    h[k] = pa_h2u(__hmul2(e4m3x2_as_f16((k & 1 ? b : a) >> (k & 2 ? 8 : 0)), two));
  return make_uint4(h[0], h[1], h[2], h[3]);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The same into the L2, one tile ahead (128K-row prefix x 64 sequences 394 -> 385 us).
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// umma_bf16 with the descriptors as two words: only the low one (the start
// address) changes from product to product, so a step costs one 32-bit addition
// per operand.
struct PaDesc {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit PaDesc(uint64_t d) : lo((uint32_t)d), hi((uint32_t)(d >> 32)) {}
};
__device__ __forceinline__ void pa_umma(uint32_t d_tmem, PaDesc a, uint32_t a_off, PaDesc b,
                                        uint32_t b_off, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a.lo + a_off), "r"(a.hi), "r"(b.lo + b_off), "r"(b.hi), "r"(idesc),
      "r"((uint32_t)accumulate)
      : "memory");
}

// S^T (M = 64 keys) and O^T (M = 128 channels) products; n: query rows of the
// tile.  P is read MN-major (its rows are keys, the K axis of the second
// product).
__device__ __forceinline__ uint32_t pa_idesc(int n, bool pv) {
  return (1u << 4) | (pv ? (1u << 15) | (1u << 16) : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)((pv ? 128 : PA_KEYS) >> 4) << 24);
}

// (a - m) scl + PA_SHIFT of two rows, as packed pairs: as many instructions as one
// product and sum each (unpacked, 64 x 1 queries over 128K rows 399 us instead of 393).
__device__ __forceinline__ float2 pa_exponents(float2 a, float m0, float m1, float s0, float s1) {
  float2 y;
  asm("{\n\t.reg .b64 a, m, s, h;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 m, {%4, %5};\n\tmov.b64 s, {%6, %7};\n\t"
      "mov.b64 h, {%8, %8};\n\t"
      "add.rn.f32x2 a, a, m;\n\tfma.rn.f32x2 a, a, s, h;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(-m0), "f"(-m1), "f"(s0), "f"(s1), "f"(PA_SHIFT));
  return y;
}

// The run that begins at `tile`: the segment of that tile as far as this CTA's
// share [.., tile_end) goes.
__device__ __forceinline__ PaRun pa_next_run(const PrefixParams& p, const PaPlan& pl,
                                             const int* cum, int64_t tile, int64_t tile_end,
                                             bool stop) {
  PaRun run;
  run.valid = tile < tile_end && !stop;
  run.image = pl.images && tile < pl.shared;
  if (!run.valid) return run;
  int64_t seg_end;
  run.n_win = run.win_lo = 0;
  if (tile < pl.shared) {
    const int64_t in_band = (int64_t)pl.band * pl.row_blocks;
    const int band = (int)pa_div(tile, in_band), len = pl.band_tiles(band);
    const int at = (int)(tile - band * in_band), block = at / len;
    run.own = false;
    run.seq = 0;
    run.row0 = block * PA_ROWS;
    run.n_rows = min(PA_ROWS, p.batch * p.nq * CSA2_H - run.row0);
    run.kt = band * pl.band + at - block * len;
    run.own_tiles = pl.prefix_tiles;
    run.first_pos = 0;
    run.slot = pl.shared_slot(band * pl.row_blocks + block, blockIdx.x);
    seg_end = tile + (block + 1) * len - at;
    run.n_keys = p.prefix;
  } else {
    const int64_t u = tile - pl.shared;
    int lo = 0, hi = p.batch;  // the last b with q_blocks * cum[b] <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)cum[mid] * pl.q_blocks <= u) lo = mid; else hi = mid;
    }
    const int b = lo, kts = cum[b + 1] - cum[b];
    const int64_t rem = u - (int64_t)cum[b] * pl.q_blocks;
    const int qb = (int)pa_div(rem, kts);
    run.own = true;
    run.seq = b;
    run.row0 = (b * p.nq + qb * PA_QB) * CSA2_H;
    run.n_rows = min(PA_QB, p.nq - qb * PA_QB) * CSA2_H;
    run.kt = (int)(rem - (int64_t)qb * kts) - PA_SEG;  // < 0: an empty tile
    run.own_tiles = kts - PA_SEG - pl.win_tiles;
    run.first_pos = p.prefix;
    run.slot = pl.own_slot(b * pl.q_blocks + qb, blockIdx.x);
    seg_end = tile - run.kt + kts - PA_SEG;
    const int n = p.n_rows[b];
    run.n_keys = n < 0 ? 0 : min(n, p.max_rows);
    if (p.swa) {
      run.n_win = p.swa_len[b];
      if (run.n_win < 0 || run.n_win > p.swa_rows) {
        if ((threadIdx.x & 31) == 0) set_status(p.status, ST_DEVICE_CHECK);
        run.n_win = run.n_win < 0 ? 0 : p.swa_rows;
      }
      run.win_lo = max(0, run.n_win - (p.nq - 1 - qb * PA_QB) - CSA2_W);
    }
  }
  run.kt_end = run.kt + (int)(min(seg_end, tile_end) - tile);
  run.line = run.kt_end - run.kt;
  run.kt = max(run.kt, 0);
  run.kt_cache = min(run.kt_end, run.own_tiles);
  return run;
}

// The softmax warps bring a run's queries and limits into shared memory.
__device__ __forceinline__ void pa_queries(const PrefixParams& p, const PaRun& run, PaSmem& s,
                                           int warp, int lane) {
  // Q' = Q * 2^e in fp16, max |Q'| of a row in [2^14, 2^15): one warp per row,
  // 16 channels per lane, four rows' loads in flight
#pragma unroll 1
  for (int h0 = warp; h0 < run.n_rows; h0 += 4 * PA_SM_WARPS) {
    uint4 v[4][2];
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int h = min(h0 + u * PA_SM_WARPS, run.n_rows - 1);
      const uint4* src =
          reinterpret_cast<const uint4*>(p.q + (int64_t)(run.row0 + h) * CSA2_D) + 2 * lane;
      v[u][0] = __ldg(src);
      v[u][1] = __ldg(src + 1);
    }
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const int h = h0 + u * PA_SM_WARPS;
      if (h >= run.n_rows) break;
      uint32_t mx = 0u;
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const uint32_t w[4] = {v[u][k].x, v[u][k].y, v[u][k].z, v[u][k].w};
#pragma unroll
        for (int j = 0; j < 4; j++) mx = max(mx, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      const int e = q_pow2_exponent(mx);
      const int e1 = e / 2, e2 = e - e1;
      const float f = p.scale_log2 < 0.0f ? -pow2i(e1) : pow2i(e1), f2 = pow2i(e2);
      // Below fp32's range the logits are below 2^-80 anyway.  Above it only the largest
      // counts, with PA_MOST too: two sums that differ do so by 2^-41 or more (Q' has
      // 2^-24, tiles 2^-17 for their last place).  A head that is not finite gives NaN.
      if (lane == 0)
        s.scl[h] = mx >= 0x7F80u
                       ? __int_as_float(0x7FC00000)
                       : fminf(fabsf(p.scale_log2) * pow2i(-e1) * pow2i(-e2) *
                                   (PA_PRE_SCALE * PA_TILE_SCALE), PA_MOST);
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const uint32_t w[4] = {v[u][k].x, v[u][k].y, v[u][k].z, v[u][k].w};
        float g[8];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          g[2 * j] = __uint_as_float(w[j] << 16) * f * f2;
          g[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * f * f2;
        }
        uint32_t o4[4];  // the tile's order of channels
#pragma unroll
        for (int j = 0; j < 4; j++)
          o4[j] = pa_h2u(__floats2half2_rn(g[pa_channel(2 * j)], g[pa_channel(2 * j + 1)]));
        *reinterpret_cast<uint4*>(s.q + (lane >> 2) * PA_QKB + pa_sw(h, 2 * (lane & 3) + k)) =
            make_uint4(o4[0], o4[1], o4[2], o4[3]);
      }
    }
  }
  // visible keys of every row: cache positions, and window rows
  const int t = 32 * warp + lane;
  if (warp < 2) {
    int lo[2] = {0, 0}, hi[2] = {0x7FFFFFFF, 0x7FFFFFFF};
    if (t < run.n_rows) {
      const int qi = (run.row0 + t) / CSA2_H, b = qi / p.nq, later = p.nq - 1 - (qi - b * p.nq);
      const int n = p.n_rows[b];
      hi[0] = min((n < 0 ? 0 : min(n, p.max_rows)) - later, run.n_keys);
      hi[1] = max(0, run.n_win - later);
      lo[1] = max(0, run.n_win - later - CSA2_W);
    }
#pragma unroll
    for (int w = 0; w < 2; w++) {
      s.lo[w][t] = lo[w];
      s.hi[w][t] = hi[w];
    }
  }
  fence_proxy_async_smem();
  bar_sync<32 * PA_SM_WARPS>(5);
  if (warp == 0) {  // over all 64 rows
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const int a = __reduce_max_sync(0xffffffffu, max(s.lo[w][lane], s.lo[w][lane + 32]));
      const int z = __reduce_min_sync(0xffffffffu, min(s.hi[w][lane], s.hi[w][lane + 32]));
      if (lane == 0) {
        s.lo_max[w] = a;
        s.hi_min[w] = z;
      }
    }
  }
}

__global__ void __launch_bounds__(PA_NT, 1) prefix_attn_kernel(const PrefixParams p) {
  // declared with its alignment rather than rounded up to it: a rounded pointer is
  // a generic one, whose 64-bit addresses cost the inner loops a third of their time
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  PaSmem& s = *reinterpret_cast<PaSmem*>(smem_raw);
  const int t = threadIdx.x, lane = t & 31, warp = __shfl_sync(0xffffffffu, t >> 5, 0);
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
      for (int c = 0; c < PA_PARTS; c++) {
        mbar_init(&s.full[i][c], PA_DQ_WARPS);
        mbar_init(&s.empty[i][c], 1);
      }
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], PA_SM_WARPS);
      mbar_init(&s.run_full[i], 1);
      mbar_init(&s.run_empty[i], PA_MMA_WARP + 2);
    }
    fence_mbar_init();
    s.abort = 0;
  }
  if (warp == PA_MMA_WARP) {
    tmem_alloc(&s.tmem_base, PA_TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();

  // ---- the plan: prefix sums of the sequences' own key tiles
  PaPlan pl = pa_plan(p);
  {
    constexpr int PER = (CSA2_PREFIX_MAX_BATCH + PA_NT - 1) / PA_NT;
    int v[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; k++) {
      const int b = PER * t + k;
      v[k] = 0;
      if (b < p.batch) {
        const int n = p.n_rows[b];
        if ((n < 0 || n > p.max_rows) && blockIdx.x == 0) set_status(p.status, ST_DEVICE_CHECK);
        v[k] = pa_own_line(p, pl, n);
      }
      sum += v[k];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s.wsum[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    static_assert(PA_NT <= 32 * 32, "a lane per warp");
    int before = incl - sum + (int)__reduce_add_sync(0xffffffffu, lane < warp ? s.wsum[lane] : 0);
#pragma unroll
    for (int k = 0; k < PER; k++) {
      const int b = PER * t + k;
      if (b < p.batch) s.cum[b] = before;
      before += v[k];
      if (b == p.batch - 1) s.cum[p.batch] = before;
    }
    __syncthreads();
  }
  pl.finish(s.cum[p.batch]);
  const uint32_t tmem = s.tmem_base;

  // The runs of tiles, planned one ahead; a role goes on to the next run when its
  // part of this one is done (the tiles' barriers keep it from running away).
  // Tile i of the CTA uses buffers i & 1; their barriers' phase is (i >> 1) & 1.
  // Named barriers 1 to 4: the softmax warps of 16 rows, 5: all softmax warps,
  // BAR_Q: a run's queries are in shared memory (softmax and MMA warps), 7: an image
  // run is on its way (the warps that fill tiles).
  constexpr int BAR_Q = 6, Q_THREADS = 32 * (PA_SM_WARPS + 2);
  uint32_t n_run = 0;
  // Waits for the next run's plan.  The planner always gives one (after an expired
  // wait anywhere: that there is none), and every role goes by its `valid` alone, so
  // all reach the same barriers.
  auto next_run = [&]() -> const PaRun& {
    const uint32_t k = n_run++;
    mbar_wait(&s.run_full[k & 1], (k >> 1) & 1, nullptr, 2 * kWaitCycles);
    return s.run[k & 1];
  };
  auto done_run = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.run_empty[(n_run - 1) & 1]);
  };
  uint32_t i = 0;
  if (warp < PA_DQ_WARPS) {
    // ------------------------------------------------ key tiles to fp16
    // Lane (seg, r8) of a warp has key r8 of the warp's eight and 32 channels (16
    // code bytes) of each 128-channel block: a load of the warp touches 8 rows by
    // 64 consecutive bytes, and a quarter-warp's 16-byte stores go to 8 rows, whose
    // swizzle gives them different banks.  The next tile's codes are on their way
    // while this one's wait for a free buffer and are turned.
    const int seg = lane >> 3, r = 8 * warp + (lane & 7), sw = lane & 7, cc = 4 * (seg & 1);
    // before and after the tile's 128-channel block b is written
    auto begin_part = [&](int b) {
      if (b % 2 == 0 && i >= 2) {
        pa_wait(&s.empty[i & 1][b], ((i >> 1) - 1) & 1, &s.abort);
        pa_wait(&s.empty[i & 1][b + 1], ((i >> 1) - 1) & 1, &s.abort);
      }
    };
    auto end_part = [&](int b) {
      if (b % 2 != 1) return;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.full[i & 1][b - 1]);
        mbar_arrive(&s.full[i & 1][b]);
      }
    };
    for (;;) {
      const PaRun& run = next_run();
      if (!run.valid) break;
      const int kt_end = run.kt_end;
      if (run.image) {
        // the tiles are there: one warp copies them for all eight
        if (warp == 0) {
          const uint8_t* src = p.image + (int64_t)run.kt * PREFIX_IMAGE;
          const uint8_t* key = p.image_key + (int64_t)run.kt * PA_KEYS + lane;
          uint32_t flag0 = ld_now_u8(key), flag1 = ld_now_u8(key + 32);
#pragma unroll 1
          for (int kt = run.kt; kt < kt_end; kt++, i++, src += PREFIX_IMAGE) {
            const uint32_t now0 = flag0, now1 = flag1;
            if (kt + 1 < kt_end) {
              key += PA_KEYS;
              flag0 = ld_now_u8(key);
              flag1 = ld_now_u8(key + 32);
              if (lane < PA_PARTS) bulk_prefetch(src + PREFIX_IMAGE + lane * PA_COPY, PA_COPY);
            }
#pragma unroll
            for (int c = 0; c < PA_PARTS; c++) {
              const bool ok = i < 2 || pa_wait(&s.empty[i & 1][c], ((i >> 1) - 1) & 1, &s.abort);
              if (c == 0) {
                *reinterpret_cast<uint32_t*>(s.key[i & 1][lane]) = now0;
                *reinterpret_cast<uint32_t*>(s.key[i & 1][lane + 32]) = now1;
              }
              __syncwarp();
              if (lane == 0) {
                if (ok) {
                  mbar_arrive_expect_tx(&s.full[i & 1][c], PA_COPY);
                  bulk_load(s.tile[i & 1] + c * PA_COPY, src + c * PA_COPY, PA_COPY,
                            &s.full[i & 1][c]);
                } else {
                  mbar_arrive(&s.full[i & 1][c]);
                }
                mbar_arrive_n(&s.full[i & 1][c], PA_DQ_WARPS - 1);
              }
            }
          }
          // after an expired wait nobody else may look for the last copies
          if (s.abort)
            for (uint32_t k = i - min(i, 2u); k < i; k++)
              for (int c = 0; c < PA_PARTS; c++) mbar_wait(&s.full[k & 1][c], (k >> 1) & 1, nullptr);
        } else {
          i += (uint32_t)(kt_end - run.kt);
        }
        // the others' next waits are for phases that come after this run's
        bar_sync<32 * PA_DQ_WARPS>(7);
        done_run();
        continue;
      }
      const PaMap map = {run.first_pos + r, run.n_keys, run.kt_cache, run.seq};
      uint4 v[4], nv[4];       // by block: this tile's codes, the next one's
      uint32_t sc[4], nsc[4];  // the two scales of the same 32 channels
      auto load = [&](int64_t row) {
        if (row < 0) return;
        const uint8_t* c = p.codes + row * (CSA2_D / 2) + 16 * seg;
        const uint8_t* f = p.scales + row * (CSA2_D / 16) + 2 * seg;
#pragma unroll
        for (int b = 0; b < 4; b++) {
          nv[b] = ld_now_v4(c + 64 * b);
          nsc[b] = ld_now_u16(f + 8 * b);
        }
      };
#pragma unroll
      for (int b = 0; b < 4; b++) {
        nv[b] = make_uint4(0u, 0u, 0u, 0u);
        nsc[b] = 0u;
      }
      int pid = pa_page(p, map, run.kt), pid1 = pa_page(p, map, run.kt + 1);
      int64_t row, next = pa_row(p, map, run.kt, pid);
      load(next);
      int kt = run.kt;
#pragma unroll 1
      for (; kt < map.kt_cache; kt++, i++) {
        pid = pid1;
        pid1 = pa_page(p, map, kt + 2);
        row = next;
#pragma unroll
        for (int b = 0; b < 4; b++) {
          v[b] = nv[b];
          sc[b] = nsc[b];
        }
        next = pa_row(p, map, kt + 1, pid);
        load(next);
        // A key that is not there, or whose values hold a NaN, becomes zeros: the
        // P = 0 of a row that must not see it would turn NaN in the product
        const bool nan = has_nan(sc[0] | (sc[1] << 16)) || has_nan(sc[2] | (sc[3] << 16));
        const bool zero = row < 0 || nan;
        uint8_t* dst = s.tile[i & 1] + (seg >> 1) * PA_KB + r * 128;
#pragma unroll
        for (int b = 0; b < 4; b++) {
          begin_part(b);
          if (b == 0) s.key[i & 1][r][seg] = (uint8_t)(row < 0 ? 1 : (nan ? 2 : 0));
          if (!zero) {
            pa_put_fp4(dst + 2 * b * PA_KB, sw, cc, v[b], sc[b]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; c++)
              *reinterpret_cast<uint4*>(dst + 2 * b * PA_KB + (((cc + c) ^ sw) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
          end_part(b);
        }
      }
#pragma unroll 1
      for (; kt < kt_end; kt++, i++) {  // window tiles
        const int w = run.win_lo + (kt - run.own_tiles) * PA_KEYS + r;
        uint4 a[8];
        bool nan = false;
#pragma unroll
        for (int b = 0; b < 8; b++) a[b] = make_uint4(0u, 0u, 0u, 0u);
        if (w < run.n_win) {
          const uint4* src = reinterpret_cast<const uint4*>(
              p.swa + ((int64_t)run.seq * p.swa_rows + w) * CSA2_D + 32 * seg);
#pragma unroll
          for (int b = 0; b < 8; b++) a[b] = __ldg(src + 8 * (b >> 1) + (b & 1));
#pragma unroll
          for (int b = 0; b < 8; b++)
            nan |= has_nan(a[b].x) || has_nan(a[b].y) || has_nan(a[b].z) || has_nan(a[b].w);
        }
        uint8_t* dst = s.tile[i & 1] + (seg >> 1) * PA_KB + r * 128;
#pragma unroll
        for (int b = 0; b < 8; b++) {
          if (b % 2 == 0) begin_part(b / 2);
          if (b == 0) s.key[i & 1][r][seg] = (uint8_t)(w >= run.n_win ? 1 : (nan ? 2 : 0));
          if (nan) a[b] = make_uint4(0u, 0u, 0u, 0u);
          uint8_t* d = dst + 2 * (b >> 1) * PA_KB;
          const int c = cc + 2 * (b & 1);
          *reinterpret_cast<uint4*>(d + ((c ^ sw) << 4)) = pa_e4m3x8(a[b].x, a[b].y);
          *reinterpret_cast<uint4*>(d + (((c + 1) ^ sw) << 4)) = pa_e4m3x8(a[b].z, a[b].w);
          if (b % 2 == 1) end_part(b / 2);
        }
      }
      done_run();
    }
  } else if (warp < PA_MMA_WARP) {
    // --------------------------------------------------------- softmax
    // Warp (quad, part): keys 16 quad + [0, 16), query rows PA_PART part + [0, PA_PART).  An
    // M = 64 accumulator has its rows in lanes 0..15 of each TMEM quarter; read as
    // 16 x 256 bits, a thread holds keys lane / 4 and lane / 4 + 8 by columns
    // 8 n + 2 (lane % 4) + {0, 1}, n < PA_PART / 8.
    const int w = warp - PA_DQ_WARPS, quad = w & 3, part = w >> 2;
    const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
    const int c0 = PA_PART * part + 2 * (lane & 3), k0 = 16 * quad + (lane >> 2);
    for (;;) {
      const PaRun& run = next_run();
      if (!run.valid) break;
      bar_sync<32 * PA_SM_WARPS>(5);  // all have left the last run
      pa_queries(p, run, s, w, lane);
      bar_sync<Q_THREADS>(BAR_Q);
      const bool active = PA_PART * part < run.n_rows;  // per warp
      float scl[PA_COLS], m[PA_COLS], l[PA_COLS];
#pragma unroll
      for (int j = 0; j < PA_COLS; j++) {
        const int c = c0 + 8 * (j >> 1) + (j & 1);
        scl[j] = c < run.n_rows ? s.scl[c] : 0.0f;
        m[j] = PA_NONE;
        l[j] = 0.0f;
      }
#pragma unroll 1
      for (int kt = run.kt; kt < run.kt_end; kt++, i++) {
        const bool win = run.own && kt >= run.own_tiles;
        const int first = win ? run.win_lo + (kt - run.own_tiles) * PA_KEYS
                              : run.first_pos + kt * PA_KEYS;
        // the keys' flags are there before S^T is
        if (!pa_wait(&s.full[i & 1][0], (i >> 1) & 1, &s.abort)) s.abort = 1;
        const uint32_t f0 = *reinterpret_cast<const uint32_t*>(s.key[i & 1][k0]);
        const uint32_t f1 = *reinterpret_cast<const uint32_t*>(s.key[i & 1][k0 + 8]);
        const bool plain = first >= s.lo_max[win] && first + PA_KEYS <= s.hi_min[win] &&
                           __all_sync(0xffffffffu, (f0 | f1) == 0);
        if (!pa_wait(&s.s_full[i & 1], (i >> 1) & 1, &s.abort)) s.abort = 1;
        __syncwarp();
        tc_fence_after();
        if (active) {
          // x[4 n + 2 k + e]: key k0 + 8 k, row c0 + 8 n + e: the exponent of its p, or
          // its accumulator
          auto logits = [&](bool sums, float(&x)[2 * PA_COLS]) {
            uint32_t acc[2 * PA_COLS];
            tmem_ld_16x256b(tmem + lane_base + PA_S_COL + PA_ROWS * (i & 1) + PA_PART * part, acc);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 2 * PA_COLS; j += 2) {
              const int c = 2 * (j >> 2);
              const float2 a = make_float2(__uint_as_float(acc[j]), __uint_as_float(acc[j + 1]));
              const float2 y = sums ? a : pa_exponents(a, m[c], m[c + 1], scl[c], scl[c + 1]);
              x[j] = y.x;
              x[j + 1] = y.y;
            }
            if (!plain) {
#pragma unroll
              for (int j = 0; j < 2 * PA_COLS; j++) {
                const int c = c0 + 8 * (j >> 2) + (j & 1), key = first + k0 + 8 * ((j >> 1) & 1);
                const uint32_t bad = (j >> 1) & 1 ? f1 : f0;
                const bool see = !(bad & 1u) && key >= s.lo[win][c] && key < s.hi[win][c];
                x[j] = see ? (bad ? __int_as_float(0x7FC00000) : x[j]) : -INFINITY;
              }
            }
          };
          float x[2 * PA_COLS];
          logits(false, x);
          float over = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2 * PA_COLS; j += 2) over = fmaxf(over, fmaxf(x[j], x[j + 1]));
          if (bar_or_128(1 + part, over > PA_SHIFT + PA_SLACK)) {
            // some logit is far above its reference: raise the references to the
            // rows' maxima and scale what was summed
            logits(true, x);
#pragma unroll
            for (int j = 0; j < PA_COLS; j++) {
              float mx = fmaxf(x[4 * (j >> 1) + (j & 1)], x[4 * (j >> 1) + 2 + (j & 1)]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              if (lane < 4) s.red[quad][c0 + 8 * (j >> 1) + (j & 1)] = mx;
            }
            bar_or_128(1 + part, false);
#pragma unroll
            for (int j = 0; j < PA_COLS; j++) {
              const int c = c0 + 8 * (j >> 1) + (j & 1);
              const float mx = fmaxf(fmaxf(s.red[0][c], s.red[1][c]), fmaxf(s.red[2][c], s.red[3][c]));
              const float top = fmaxf(m[j], mx), f = ex2((m[j] - top) * scl[j]);
              m[j] = top;
              l[j] *= f;
              if (quad == 0 && lane < 4) s.fac[c] = f;
            }
            bar_or_128(1 + part, false);
            if (kt != run.kt) {
              // the products up to the last tile's are in O
              if (!pa_wait(&s.empty[(i - 1) & 1][PA_PARTS - 1], ((i - 1) >> 1) & 1, &s.abort)) s.abort = 1;
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int g = 0; g < 4 * PA_PART / 16; g++) {  // channel block, 16 rows
                const int c = PA_PART * part + 16 * (g >> 2);
                const uint32_t at = tmem + lane_base + 64 * (g & 3) + c;
                uint32_t o[16];
                tmem_ld_x16(at, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; j++)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * s.fac[c + j]);
                tmem_st_x16(at, o);
              }
              tmem_st_wait();
            }
            logits(false, x);
          }
          uint8_t* dst = s.p[i & 1] + k0 * 128 + 4 * (lane & 3);
#pragma unroll
          for (int n = 0; n < PA_COLS / 2; n++) {
            const float p0 = ex2(x[4 * n]), p1 = ex2(x[4 * n + 1]);
            const float p2 = ex2(x[4 * n + 2]), p3 = ex2(x[4 * n + 3]);
            l[2 * n] += p0 + p2;
            l[2 * n + 1] += p1 + p3;
            const uint32_t at = (uint32_t)((PA_PART / 8 * part + n) ^ (k0 & 7)) << 4;  // (k0 + 8 alike)
            *reinterpret_cast<uint32_t*>(dst + at) = pa_h2u(__floats2half2_rn(p0, p1));
            *reinterpret_cast<uint32_t*>(dst + 1024 + at) = pa_h2u(__floats2half2_rn(p2, p3));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[i & 1]);
      }
      // ---- the run's partial: O [row][channel], (max, sum) per row.  The last
      // tile's commit covers every product.
      if (!pa_wait(&s.empty[(i - 1) & 1][PA_PARTS - 1], ((i - 1) >> 1) & 1, &s.abort)) s.abort = 1;
      __syncwarp();
      tc_fence_after();
      if (active) {
#pragma unroll
        for (int j = 0; j < PA_COLS; j++) {
          float v = l[j];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane < 4) {
            const int c = c0 + 8 * (j >> 1) + (j & 1);
            s.red[quad][c] = v;
            if (quad == 0) s.fac[c] = m[j];
          }
        }
        bar_or_128(1 + part, false);
        const int c = PA_PART * part + lane;
        if (quad == 0 && lane < PA_PART && c < run.n_rows) {
          p.part_scl[run.slot + c] = s.scl[c];
          p.part_ml[2 * (run.slot + c)] = s.fac[c];
          p.part_ml[2 * (run.slot + c) + 1] =
              (s.red[0][c] + s.red[1][c]) + (s.red[2][c] + s.red[3][c]);
        }
#pragma unroll
        for (int g = 0; g < 4 * PA_PART / 16; g++) {  // channel block, 16 rows
          const int r0 = PA_PART * part + 16 * (g >> 2);
          if (r0 >= run.n_rows) continue;
          uint32_t o[16];
          tmem_ld_x16(tmem + lane_base + 64 * (g & 3) + r0, o);
          tmem_ld_wait();
          float* dst = p.part_o + (run.slot + r0) * CSA2_D + 128 * (g & 3) +
                       pa_channel(32 * quad + lane);
#pragma unroll
          for (int j = 0; j < 16; j++) dst[j * CSA2_D] = __uint_as_float(o[j]) * PA_TILE_SCALE;
        }
        tc_fence_before();
      }
      done_run();
    }
  } else if (warp == PA_MMA_WARP + 2) {
    // ------------------------------------------------------- the planner
    const int64_t share = pl.total > 0 ? pl.tile_at(blockIdx.x + (lane & 1)) : 0;
    int64_t tile = __shfl_sync(0xffffffffu, share, 0);
    const int64_t tile_end = __shfl_sync(0xffffffffu, share, 1);
    for (bool valid = true; valid; n_run++) {
      PaRun r;
      do {  // skips what holds empty tiles only
        r = pa_next_run(p, pl, s.cum, tile, tile_end, s.abort != 0);
        if (r.valid) tile += r.line;
      } while (r.valid && r.kt_end <= r.kt);
      valid = r.valid;
      const uint32_t k = n_run;
      if (k >= 2 && !pa_wait(&s.run_empty[k & 1], ((k >> 1) - 1) & 1, &s.abort)) s.abort = 1;
      valid = __all_sync(0xffffffffu, valid && !s.abort);
      if (lane == 0) {
        if (valid) s.run[k & 1] = r;
        s.run[k & 1].valid = valid;  // (alone: a role may still be at the run before last)
        mbar_arrive(&s.run_full[k & 1]);
      }
    }
  } else {
    // ------------------------------------------------------ the products
    // S^T from one warp, O^T from another: each waits for its own input only (one
    // thread that took them in turn would hold up the other's), and the loops stay
    // small.  A tile's buffers are free again once its O^T step is done, which
    // follows its S^T and its softmax.
    for (;;) {
      const PaRun& run = next_run();
      if (!run.valid) break;
      const uint32_t begin = i, end = i + (uint32_t)(run.kt_end - run.kt);
      const uint32_t id = pa_idesc(run.n_rows, warp != PA_MMA_WARP);
      bar_sync<Q_THREADS>(BAR_Q);
      tc_fence_after();
      const bool leader = elect_one();
      if (warp == PA_MMA_WARP) {
        const PaDesc qd(sdesc_k128(smem_u32(s.q))), kd(sdesc_k128(smem_u32(s.tile[0])));
#pragma unroll 1
        for (; i < end; i++) {
          const uint32_t a = (i & 1) * ((8 * PA_KB) >> 4);
          const uint32_t d = tmem + PA_S_COL + PA_ROWS * (i & 1);
#pragma unroll
          for (uint32_t c = 0; c < PA_PARTS; c++) {  // S^T = K Q'^T: K = 512
            if (!pa_wait(&s.full[i & 1][c], (i >> 1) & 1, &s.abort)) s.abort = 1;
            __syncwarp();
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (uint32_t j = 0; j < 32 / PA_PARTS; j++) {
                const uint32_t k = c * (32 / PA_PARTS) + j;
                pa_umma(d, kd, a + (((k >> 2) * PA_KB) >> 4) + 2 * (k & 3), qd,
                        (((k >> 2) * PA_QKB) >> 4) + 2 * (k & 3), id, k != 0);
              }
              if (c == PA_PARTS - 1) umma_commit(&s.s_full[i & 1]);
            }
            __syncwarp();
          }
        }
      } else {
        const PaDesc pd(sdesc_mn128(smem_u32(s.p[0]), PA_KEYS * 128, 1024));
        const PaDesc vd(sdesc_mn128(smem_u32(s.tile[0]), PA_KB, 1024));
#pragma unroll 1
        for (; i < end; i++) {
          if (!pa_wait(&s.p_full[i & 1], (i >> 1) & 1, &s.abort)) s.abort = 1;
          __syncwarp();
          tc_fence_after();
          if (leader) {  // O^T += V^T P^T: K = 64 keys in four steps, four channel blocks
            const uint32_t a = (i & 1) * ((8 * PA_KB) >> 4), b = (i & 1) * ((PA_KEYS * 128) >> 4);
#pragma unroll
            for (uint32_t k = 0; k < 16; k++) {
              const uint32_t c = k >> 2, j = k & 3;  // channel block, 16 keys
              pa_umma(tmem + 64 * c, vd, a + ((c * 2 * PA_KB + j * 2048) >> 4), pd,
                      b + ((j * 2048) >> 4), id, i != begin || j != 0);
              if (k % (16 / PA_PARTS) == 16 / PA_PARTS - 1)
                umma_commit(&s.empty[i & 1][c * PA_PARTS / 4]);
            }
          }
          __syncwarp();
        }
      }
      done_run();
    }
  }
  // The merge's blocks start where this block's end; started earlier they only took
  // registers and issue slots (512 queries: 487 us instead of 461)
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (s.abort && t == 0) set_status(p.status, ST_TIMEOUT);
  if (warp == PA_MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, PA_TMEM_COLS);
  }
}

// The images of the prefix's tiles: a CTA per tile, a warp per eight keys, lane (key of
// four, piece) with eight channels of each 64-channel chunk, so that a warp writes
// whole 128-byte lines.
constexpr int PI_NT = 256;
__global__ void __launch_bounds__(PI_NT) prefix_image_kernel(const PrefixParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, piece = lane & 7, kt = blockIdx.x;
  pdl_wait();
  uint8_t* image = p.image + (int64_t)kt * PREFIX_IMAGE;
  uint32_t w[2][8], sc[2][8];
  int64_t row[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int r = 8 * warp + 4 * h + (lane >> 3);
    const PaMap map = {r, p.prefix, (int)gridDim.x, 0};
    row[h] = pa_row(p, map, kt, pa_page(p, map, kt));
#pragma unroll
    for (int kb = 0; kb < 8; kb++) {
      w[h][kb] = sc[h][kb] = 0u;
      if (row[h] < 0) continue;
      w[h][kb] = __ldg(reinterpret_cast<const uint32_t*>(p.codes + row[h] * (CSA2_D / 2)) + 8 * kb + piece);
      sc[h][kb] = __ldg(reinterpret_cast<const uint32_t*>(p.scales + row[h] * (CSA2_D / 16)) + kb);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int r = 8 * warp + 4 * h + (lane >> 3);
    bool nan = false;  // of the whole key: every lane has all of its scales
#pragma unroll
    for (int kb = 0; kb < 8; kb++) nan |= has_nan(sc[h][kb]);
    if (piece == 0) p.image_key[kt * PA_KEYS + r] = (uint8_t)(row[h] < 0 ? 1 : (nan ? 2 : 0));
#pragma unroll
    for (int kb = 0; kb < 8; kb++) {
      const uint32_t b = nan ? 0u : (sc[h][kb] >> (8 * (piece >> 1))) & 0xFFu;
      *reinterpret_cast<uint4*>(image + kb * PA_KB + pa_sw(r, piece)) =
          pa_fp4x8(nan ? 0u : w[h][kb], pa_scale(b | (b << 16)));
    }
  }
  pdl_launch_dependents();
}

// out = sum_i w_i O_i / sum_i w_i l_i over a row's partials, w_i = 2^(c (m_i - max m)),
// c the row's scale.
// All heads of a query share the list of partials.  A CTA takes HEADS heads of one
// query: all 16 where the queries alone fill the GPU (a CTA's look at the plan
// costs more than a row's sum), else one, its partials dealt to four groups of 128
// threads (four channels each) whose sums join in a fixed order and whose first
// partials are loaded while the weights are found (2K-row prefix: 22 -> 18 us with
// the plan moved before the wait and its divisions to 32 bits; more registers for
// more of them cost blocks per SM: 7 x 3 queries 32 us with 3, 36 with 6).
constexpr int PM_NT = 512, PM_AHEAD = 3;
constexpr int PM_PARTS = PA_MAX_GRID + PA_MAX_BANDS + 1;  // partials of a row
static_assert(PM_PARTS <= PM_NT, "a thread finds each");
template <int HEADS>
__global__ void __launch_bounds__(PM_NT) prefix_merge_kernel(const PrefixParams p) {
  __shared__ int64_t slot[PM_PARTS];
  __shared__ float w[PM_PARTS][HEADS];
  __shared__ int seg_first[PA_MAX_BANDS + 1], seg_end[PA_MAX_BANDS + 1];
  __shared__ int sums[2];
  __shared__ float inv[HEADS];
  __shared__ float4 acc_s[3][128];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int qi = blockIdx.x / (CSA2_H / HEADS), h0 = blockIdx.x % (CSA2_H / HEADS) * HEADS;
  pdl_launch_dependents();
  if (t < 2) sums[t] = 0;
  __syncthreads();
  const int b = qi / p.nq, tq = qi - b * p.nq;
  PaPlan pl = pa_plan(p);
  int before = 0, all = 0;
  for (int i = t; i < p.batch; i += PM_NT) {
    const int k = pa_own_line(p, pl, p.n_rows[i]);
    all += k;
    if (i < b) before += k;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0 && (all | before) != 0) {
    atomicAdd(&sums[0], all);  // whole numbers: any order gives the same sum
    atomicAdd(&sums[1], before);
  }
  __syncthreads();
  pl.finish(sums[0]);
  const int kts = pa_own_line(p, pl, p.n_rows[b]);

  // ---- the query's partials (row of head 0): its shared segments', then its own's;
  // at most one for each CTA and one more for each segment
  const int qb = tq / PA_QB, row0 = qi * CSA2_H, block = row0 / PA_ROWS, oseg = b * pl.q_blocks + qb;
  auto tiles_of = [&](int k, int64_t& ts, int64_t& te) {  // of band k, or k = bands: own
    ts = k < pl.bands ? pl.shared_tile(k, block)
                      : pl.shared + (int64_t)sums[1] * pl.q_blocks + (int64_t)qb * kts;
    te = ts + (k < pl.bands ? (pl.prefix_tiles > 0 ? pl.band_tiles(k) : 0) : kts);
  };
  if (t <= pl.bands) {
    int64_t ts, te;
    tiles_of(t, ts, te);
    seg_first[t] = te > ts ? pl.cta_of(ts) : 0;
    seg_end[t] = te > ts ? pl.cta_of(te - 1) - seg_first[t] + 1 : 0;  // (its count)
  }
  __syncthreads();
  if (t == 0)
    for (int k = 1; k <= pl.bands; k++) seg_end[k] += seg_end[k - 1];
  __syncthreads();
  const int n = seg_end[pl.bands];
  if (t < n) {
    int k = 0;
    while (t >= seg_end[k]) k++;
    const int c = seg_first[k] + t - (k > 0 ? seg_end[k - 1] : 0);
    const bool own = k == pl.bands;
    int64_t ts, te;
    tiles_of(k, ts, te);
    const int64_t from = max(pl.tile_at(c), ts + (own ? PA_SEG : 0)), to = min(pl.tile_at(c + 1), te);
    slot[t] = from >= to ? -1
              : own      ? pl.own_slot(oseg, c) + (tq - qb * PA_QB) * CSA2_H
                         : pl.shared_slot(k * pl.row_blocks + block, c) + row0 % PA_ROWS;
  }
  __syncthreads();
  pdl_wait();  // for the partials; the lengths prefix_attn_kernel itself has waited for
  // The first partials of a lone head, on their way while the weights are found
  const int g = t >> 7, ch = 4 * (t & 127);
  float4 ahead[PM_AHEAD];
#pragma unroll
  for (int k = 0; k < PM_AHEAD; k++) {
    const int i = g + 4 * k;
    ahead[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (HEADS == 1 && i < n && slot[i] >= 0)
      ahead[k] = ld_now_f4(p.part_o + (slot[i] + h0) * CSA2_D + ch);
  }
  // ---- weights: a warp per head (a NaN sum stays one)
  if (warp < HEADS) {
    float M = -INFINITY, scl = 0.0f;
    for (int i = lane; i < n; i += 32) {
      float m = -INFINITY;
      if (slot[i] >= 0) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (slot[i] + h0 + warp));
        if (ml.y > 0.0f || ml.y != ml.y) m = ml.x;
        scl = p.part_scl[slot[i] + h0 + warp];  // (alike in all of them)
      }
      w[i][warp] = m;
      M = fmaxf(M, m);
    }
    M = warp_max_f32(M);
    float sum = 0.0f;
    for (int i = lane; i < n; i += 32) {
      const float wt = w[i][warp] == -INFINITY ? 0.0f : exp2f((w[i][warp] - M) * scl);
      w[i][warp] = wt;
      if (slot[i] >= 0 && M != -INFINITY) {
        const float l = p.part_ml[2 * (slot[i] + h0 + warp) + 1];
        if (wt != 0.0f || l != l) sum += wt * l;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) inv[warp] = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  __syncthreads();
  // ---- the weighted sums
  auto store = [&](int h, float4 acc) {
    const float f = inv[h];
    const __nv_bfloat162 o0 = __floats2bfloat162_rn(acc.x * f, acc.y * f);
    const __nv_bfloat162 o1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
    *reinterpret_cast<uint2*>(p.out + (int64_t)(row0 + h0 + h) * CSA2_D + ch) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&o0), *reinterpret_cast<const uint32_t*>(&o1));
  };
  auto add_v = [&](float wt, float4 v, float4& acc) {
    acc.x = fmaf(wt, v.x, acc.x);
    acc.y = fmaf(wt, v.y, acc.y);
    acc.z = fmaf(wt, v.z, acc.z);
    acc.w = fmaf(wt, v.w, acc.w);
  };
  // (a partial of weight zero is loaded and not added: no branch holds up the next
  // ones' loads)
  auto add = [&](int h, int i, float4& acc) {
    const int64_t at = max(slot[i], (int64_t)0) + h0 + h;
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * CSA2_D + ch);
    if (w[i][h] != 0.0f) add_v(w[i][h], v, acc);
  };
  if (HEADS > 1) {
#pragma unroll 1
    for (int h = g; h < HEADS; h += 4) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < n; i++) add(h, i, acc);
      store(h, acc);
    }
  } else {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < PM_AHEAD; k++) {
      const int i = g + 4 * k;
      if (i < n && w[i][0] != 0.0f) add_v(w[i][0], ahead[k], acc);
    }
#pragma unroll 4
    for (int i = g + 4 * PM_AHEAD; i < n; i += 4) add(0, i, acc);
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
      store(0, acc);
    }
  }
}

int prefix_grid(const PrefixParams& p, int num_sms) {
  const PaPlan pl = pa_plan(p);
  const int64_t own = (int64_t)p.batch * pl.q_blocks *
                      ((p.max_rows - p.prefix + PA_KEYS - 1) / PA_KEYS + pl.win_tiles + PA_SEG);
  const int64_t most = num_sms < PA_MAX_GRID ? num_sms : PA_MAX_GRID;
  const int64_t tiles = pl.shared + own;
  return (int)(tiles < 1 ? 1 : (tiles < most ? tiles : most));
}

size_t prefix_partial_rows(const PrefixParams& p) {
  const PaPlan pl = pa_plan(p);
  return (size_t)(pl.row_blocks * pl.bands + pl.grid) * PA_ROWS +
         ((size_t)p.batch * pl.q_blocks + pl.grid) * pl.own_rows;
}

size_t prefix_image_tiles(const PrefixParams& p) {
  const PaPlan pl = pa_plan(p);
  return pl.images ? pl.prefix_tiles : 0;
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
  const size_t images = prefix_image_tiles(p);
  if (images > 0) {
    cfg.gridDim = dim3((unsigned)images);
    cfg.blockDim = dim3(PI_NT);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    trace_mark("prefix_image", st);
    if ((e = cudaLaunchKernelEx(&cfg, prefix_image_kernel, p)) != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(PA_NT);
  cfg.dynamicSmemBytes = PA_SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  trace_mark("prefix_attn", st);
  if ((e = cudaLaunchKernelEx(&cfg, prefix_attn_kernel, p)) != cudaSuccess) return e;
  const int queries = p.batch * p.nq;
  const bool whole = queries >= num_sms();
  cfg.gridDim = dim3(whole ? queries : queries * CSA2_H);
  cfg.blockDim = dim3(PM_NT);
  cfg.dynamicSmemBytes = 0;
  trace_mark("prefix_merge", st);
  return whole ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<CSA2_H>, p)
               : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<1>, p);
}

}  // namespace csa2
