// Which tokens the cache extension takes for which sequence (csrc/extend_runs.cuh),
// on the CPU.  Built and called by test_extend_runs.py.
#include <cstdint>

#include <cuda_runtime.h>
#undef __forceinline__
#define __forceinline__ inline
#include "extend_runs.cuh"

extern "C" int run_of(const int32_t* cu, int batch, int total, int b, int32_t* lo, int32_t* hi) {
  if (!csa2::run_pair(cu, total, b, *lo, *hi)) return 0;
  const bool ok = csa2::run_clear(cu, batch, b, *lo, *hi);
  bool lanes = true;
  for (int lane = 0; lane < 32; lane++)
    lanes &= csa2::run_clear_lane(cu, batch, b, lane, *lo, *hi);
  return lanes == ok ? ok : 2;
}
extern "C" int seq_of(const int32_t* cu, int batch, int total, int i) {
  int lo, hi;
  const int b = csa2::seq_of(cu, batch, total, i, lo, hi);
  return b >= 0 && (lo != cu[b] || hi != cu[b + 1]) ? -2 : b;
}
