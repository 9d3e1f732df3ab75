// The work plan of csa2_prefix_attn, walked on the CPU: every key tile of every
// segment belongs to exactly one CTA, a CTA's tiles are one range, the partials
// that the merge looks for are the ones that are written, no two share rows, and
// all lie inside the workspace.  Built and called by test_prefix_plan.py.
#include <algorithm>
#include <cstdint>
#include <set>
#include <utility>
#include <vector>

#define __forceinline__ inline
#include "prefix_plan.cuh"

using namespace csa2;

extern "C" int plan_check(int batch, int nq, int prefix, int max_rows, const int32_t* n_rows,
                          int window, int grid, int64_t* most_cost, int64_t* mean_cost) {
  PrefixParams p{};
  p.batch = batch;
  p.nq = nq;
  p.prefix = prefix;
  p.max_rows = max_rows;
  p.swa = window ? reinterpret_cast<const uint8_t*>(16) : nullptr;
  p.grid = grid;
  PaPlan pl = pa_plan(p);
  std::vector<int> cum(batch + 1, 0);
  for (int b = 0; b < batch; b++) cum[b + 1] = cum[b] + pa_own_line(p, pl, n_rows[b]);
  pl.finish(cum[batch]);
  const int64_t tiles = pl.shared + (int64_t)cum[batch] * pl.q_blocks;
  if (tiles == 0) return pl.total == 0 ? 0 : 1;
  if (pl.tile_at(0) != 0 || pl.tile_at(grid) != tiles) return 2;
  std::vector<int64_t> at(grid + 1);
  for (int c = 0; c <= grid; c++) at[c] = pl.tile_at(c);
  *most_cost = 0;
  for (int c = 0; c < grid; c++) {
    if (at[c] > at[c + 1]) return 3;
    const int64_t cost = pl.cost_before(at[c + 1]) - pl.cost_before(at[c]);
    if (cost > *most_cost) *most_cost = cost;
    for (int64_t t = at[c]; t < at[c + 1]; t++)
      if (pl.cta_of(t) != c) return 4;
  }
  *mean_cost = pl.total / grid;
  // slots: workspace rows as prefix_partial_rows counts them
  const int64_t rows = (int64_t)(pl.row_blocks * pl.bands + grid) * PA_ROWS +
                       ((int64_t)batch * pl.q_blocks + grid) * pl.own_rows;
  std::set<std::pair<int64_t, int64_t>> taken;
  auto segment = [&](int64_t ts, int64_t te, int seg, bool own) {
    if (te <= ts) return 0;
    const int64_t real = own ? ts + PA_SEG : ts;
    if (real >= te) return 8;
    for (int c = pl.cta_of(ts); c <= pl.cta_of(te - 1); c++) {
      if (!(std::max(at[c], real) < std::min(at[c + 1], te))) continue;
      const int64_t s = own ? pl.own_slot(seg, c) : pl.shared_slot(seg, c);
      const int64_t n = own ? pl.own_rows : PA_ROWS;
      if (s < 0 || s + n > rows) return 5;
      auto it = taken.lower_bound({s, 0});
      if (it != taken.end() && it->first < s + n) return 6;
      if (it != taken.begin() && (--it)->second > s) return 7;
      taken.insert({s, s + n});
    }
    return 0;
  };
  int64_t next = 0;
  if (pl.bands < 1 || pl.bands > PA_MAX_BANDS) return 9;
  if (pl.prefix_tiles > 0)
    for (int k = 0; k < pl.bands; k++)
      for (int i = 0; i < pl.row_blocks; i++) {
        const int64_t ts = pl.shared_tile(k, i), te = ts + pl.band_tiles(k);
        if (ts != next || te <= ts) return 10;
        next = te;
        if (int e = segment(ts, te, k * pl.row_blocks + i, false)) return e;
      }
  if (next != pl.shared) return 11;
  for (int b = 0; b < batch; b++) {
    const int kts = cum[b + 1] - cum[b];
    for (int qb = 0; qb < pl.q_blocks; qb++) {
      const int64_t ts = pl.shared + (int64_t)cum[b] * pl.q_blocks + (int64_t)qb * kts;
      if (int e = segment(ts, ts + kts, b * pl.q_blocks + qb, true)) return e;
    }
  }
  return 0;
}
