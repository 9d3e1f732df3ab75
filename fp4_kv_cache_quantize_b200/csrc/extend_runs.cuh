// extend_runs.cuh -- which tokens of a ragged batch belong to which sequence, the
// same arithmetic for every kernel of the cache extension.
//
// A token's sequence is where a binary search in the offsets ends.  Offsets that
// descend would let that search and a look at one pair of offsets disagree, and a
// counter advance over rows that nobody wrote.  So a run counts as in order only if
// each offset that the search meets on its way to this sequence lies on the right
// side of the whole run: then the search takes that way for the run's first token
// and for its last, hence for every token between them, and no token belongs to two
// sequences.
#pragma once

#include <stdint.h>

namespace csa2 {

__host__ __device__ __forceinline__ int run_offset(const int32_t* cu, int b) {
#ifdef __CUDA_ARCH__
  return __ldg(cu + b);
#else
  return cu[b];
#endif
}

__host__ __device__ __forceinline__ bool run_inside(int total, int b, int lo, int hi) {
  return lo >= 0 && hi >= lo && hi <= total && (b > 0 || lo == 0);
}

// Tokens [lo, hi) of sequence b < batch; false if its own two offsets are out of order,
// do not start at 0 or end behind the tokens.  cu NULL: one token each.
__host__ __device__ __forceinline__ bool run_pair(const int32_t* cu, int total, int b, int& lo,
                                                  int& hi) {
  lo = cu ? run_offset(cu, b) : b;
  hi = cu ? run_offset(cu, b + 1) : b + 1;
  return !cu || run_inside(total, b, lo, hi);
}

// Whether the offsets on the search's way to b leave the run [lo, hi) to it.  (Where no
// offset of the batch descends they always do.)
__host__ __device__ __forceinline__ bool run_clear(const int32_t* cu, int batch, int b, int lo,
                                                   int hi) {
  constexpr int STEPS = 5;  // the way depends on b alone: so many loads together
  bool ok = true;
#pragma unroll 1
  for (int l = 0, z = cu ? batch : 1; z - l > 1;) {
    int c[STEPS];
    bool right[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; k++) {
      const int mid = (l + z) >> 1;  // (at the way's end: b itself)
      c[k] = run_offset(cu, mid);
      right[k] = mid <= b;
      if (right[k]) l = mid; else z = mid;
    }
#pragma unroll
    for (int k = 0; k < STEPS; k++) ok = ok && (right[k] ? c[k] <= lo : c[k] >= hi);
  }
  return ok;
}

// The same by 16 lanes or more, each with one offset of the way, which depends on b
// alone (a batch has fewer than 2^16 sequences): true if all of them say so.
__host__ __device__ __forceinline__ bool run_clear_lane(const int32_t* cu, int batch, int b,
                                                        int lane, int lo, int hi) {
  if (!cu) return true;
  int l = 0, z = batch, mid = z >> 1;
  for (int k = 0; k < lane && z - l > 1; k++) {
    if (mid <= b) l = mid; else z = mid;
    mid = (l + z) >> 1;
  }
  const int c = run_offset(cu, mid);
  return mid <= b ? c <= lo : c >= hi;
}

// The sequence of token i and its tokens [lo, hi); -1 if there is none (behind the
// last run, or in front of the first) or its run is not in order.
__host__ __device__ __forceinline__ int seq_of(const int32_t* cu, int batch, int total, int i,
                                               int& lo, int& hi) {
  if (!cu) {
    lo = i;
    hi = i + 1;
    return i;
  }
  int b = 0, z = batch, below = 0, above = 0x7FFFFFFF;  // the offsets on the way
  while (z - b > 1) {
    const int mid = (b + z) >> 1, c = run_offset(cu, mid);
    if (c <= i) {
      b = mid;
      below = c > below ? c : below;
    } else {
      z = mid;
      above = c < above ? c : above;
    }
  }
  lo = run_offset(cu, b);
  hi = run_offset(cu, b + 1);
  return run_inside(total, b, lo, hi) && lo <= i && i < hi && below <= lo && hi <= above ? b : -1;
}

}  // namespace csa2
