// prefix_plan.cuh -- how csa2_prefix_attn cuts its work, the same arithmetic
// for the kernel that computes the partials and the one that merges them.
//
// A tile is 64 keys against up to 64 query rows (a row is one head of one
// query).  A segment is the key tiles of one row block: first the blocks of 64
// rows of the whole batch against the shared prefix, band by band of it, then, per
// sequence, its blocks of up to four queries against its own rows and its window.  The tiles
// lie on one line in segment order, each as long as it costs, and CTA i of G
// takes the tiles that start in [i C / G, (i + 1) C / G): every CTA gets an
// equal share whatever the lengths, and one partial per segment that it touches.
// (segment + CTA) rises along the line, so it numbers the partials.  An own
// segment begins with PA_SEG empty tiles: what starting and ending it costs.
#pragma once

#include <stdint.h>

#include "kernels.h"

namespace csa2 {

constexpr int PA_KEYS = 64;      // keys per tile: the MMA's M
constexpr int PA_ROWS = 64;      // query rows per tile: the MMA's N
constexpr int PA_QB = PA_ROWS / CSA2_H;  // queries per row block
constexpr int PA_MAX_GRID = 192;
constexpr int PA_SEG = 6;  // (2 x 256 queries: 544 us with 4, 498 with 6; 64 x 1 477 and 479)

// Whether the prefix is turned into fp16 tiles once, by a kernel of its own, instead of
// by every row block again.  A tile of 64 rows costs 2.6 ns (of all SMs' time) less
// with its image there, an image 13 ns and the kernel 4.5 us: 16 row blocks of 2,048
// tiles 395 us (without: 449), 2 of 2,048 102 (80), 8 of 128 47 (46), 6 of 79 35 (32).
__host__ __device__ inline bool pa_images(int row_blocks, int prefix_tiles) {
  return (int64_t)(row_blocks - 5) * prefix_tiles >= 2048;
}

// Bands of the prefix: one, but with images several, so that CTAs which run at the
// same time read the same ones while they are in the L2: about as long as a CTA's
// share, and at most 512 tiles (32 MB), as far as PA_MAX_BANDS go.  In one band the
// row blocks meet an image a whole prefix apart, and 134 MB of them (128K rows) came
// from memory four times: 64 sequences took as long while the GPU was cool, but 440
// us instead of 403 call after call, at its power limit.
constexpr int PA_MAX_BANDS = 16;
__host__ __device__ inline int pa_bands(bool images, int row_blocks, int prefix_tiles, int grid) {
  if (!images) return 1;
  const int a = grid / row_blocks, b = (prefix_tiles + 511) / 512, n = a > b ? a : b;
  return n < 1 ? 1 : n < PA_MAX_BANDS ? n : PA_MAX_BANDS;
}

// What a tile of n rows costs, relative to others; with its image there already (64 x
// 1 and 2 x 256 queries: 428 and 372 us with 8, 396 and 358 with 11, 390 and 393 with 13).
constexpr int PA_IMAGE_COST = 11;
__host__ __device__ inline int pa_cost(int n_rows) { return 14 + n_rows / 32; }

// a / b for a >= 0, b > 0: a 64-bit division takes several times a 32-bit one's
// instructions, and a call's first tiles wait for a handful of them.
__host__ __device__ inline int64_t pa_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

struct PaPlan {
  int row_blocks;   // blocks of 64 rows over the whole batch
  int prefix_tiles; // key tiles of the shared prefix
  bool images;      // their fp16 images are made first
  int band, bands;  // tiles of a band (the last may have fewer), bands
  int q_blocks;     // row blocks per sequence for its own rows
  int own_rows;     // rows of a partial of an own segment
  int win_tiles;    // window tiles per own segment
  int shared;       // tiles of the shared segments
  int cost_p, cost_o;
  int64_t base, total;  // costs of the shared tiles, and of all
  int grid;

  // own: key tiles of all sequences' own rows and windows, per row block
  __host__ __device__ void finish(int64_t own) {
    base = (int64_t)shared * cost_p;
    total = base + own * q_blocks * cost_o;
  }
  __host__ __device__ int64_t tile_at(int i) const {  // first tile of CTA i
    const int64_t x = pa_div(total * i, grid);
    if (x <= base) return pa_div(x + cost_p - 1, cost_p);
    return shared + pa_div(x - base + cost_o - 1, cost_o);
  }
  __host__ __device__ int64_t cost_before(int64_t tile) const {
    return tile < shared ? tile * cost_p : base + (tile - shared) * cost_o;
  }
  __host__ __device__ int cta_of(int64_t tile) const {
    return (int)pa_div((cost_before(tile) + 1) * grid - 1, total);
  }
  // segment k row_blocks + b is row block b's of band k
  __host__ __device__ int band_tiles(int k) const {
    return prefix_tiles - k * band < band ? prefix_tiles - k * band : band;
  }
  __host__ __device__ int64_t shared_tile(int k, int b) const {  // its first on the line
    return (int64_t)k * band * row_blocks + (int64_t)b * band_tiles(k);
  }
  // first row of the partial of CTA c for a shared / an own segment
  __host__ __device__ int64_t shared_slot(int seg, int c) const {
    return (int64_t)(seg + c) * PA_ROWS;
  }
  __host__ __device__ int64_t own_slot(int seg, int c) const {
    return (int64_t)(row_blocks * bands + grid) * PA_ROWS + (int64_t)(seg + c) * own_rows;
  }
};

__host__ __device__ inline PaPlan pa_plan(const PrefixParams& p) {
  PaPlan pl;
  const int rows = p.batch * p.nq * CSA2_H;
  pl.row_blocks = (rows + PA_ROWS - 1) / PA_ROWS;
  pl.prefix_tiles = (p.prefix + PA_KEYS - 1) / PA_KEYS;
  pl.q_blocks = (p.nq + PA_QB - 1) / PA_QB;
  pl.own_rows = CSA2_H * (p.nq < PA_QB ? p.nq : PA_QB);
  // the windows of a block of k queries span 128 + k - 1 rows
  pl.win_tiles =
      p.swa == nullptr ? 0 : (CSA2_W + (p.nq < PA_QB ? p.nq : PA_QB) - 1 + PA_KEYS - 1) / PA_KEYS;
  pl.shared = pl.row_blocks * pl.prefix_tiles;
  pl.images = pa_images(pl.row_blocks, pl.prefix_tiles);
  pl.bands = pa_bands(pl.images, pl.row_blocks, pl.prefix_tiles, p.grid);
  pl.band = (pl.prefix_tiles + pl.bands - 1) / pl.bands;
  if (pl.band > 0) pl.bands = (pl.prefix_tiles + pl.band - 1) / pl.band;
  pl.cost_p = pl.images ? PA_IMAGE_COST : pa_cost(rows < PA_ROWS ? rows : PA_ROWS);
  pl.cost_o = pa_cost(pl.own_rows);
  pl.base = pl.total = 0;
  pl.grid = p.grid;
  return pl;
}

// Key tiles of sequence b's own rows (beyond the prefix), without its window.
__host__ __device__ inline int pa_own_tiles(const PrefixParams& p, int n_rows) {
  const int n = n_rows < 0 ? 0 : (n_rows > p.max_rows ? p.max_rows : n_rows);
  return n > p.prefix ? (n - p.prefix + PA_KEYS - 1) / PA_KEYS : 0;
}

// Tiles of an own segment of sequence b on the line, the empty ones included.
__host__ __device__ inline int pa_own_line(const PrefixParams& p, const PaPlan& pl, int n_rows) {
  const int n = pa_own_tiles(p, n_rows) + pl.win_tiles;
  return n > 0 ? n + PA_SEG : 0;
}

}  // namespace csa2
