// paged_masks.cuh — which keys a row sees (internal to libfpd).
#pragma once

#include "paged_sched.cuh"

namespace fpd {

__device__ __forceinline__ bool row_sees(const PagedShape& s, int row, int pos) {
  return (!s.window || pos < s.sinks || row - pos < s.window) && (!s.causal || pos <= row);
}

// Keys [lo, hi) of a tile that a window hides from every row of the unit.
__device__ __forceinline__ void hidden_from_all(const PagedShape& s, const PagedUnit& u, const PagedTile& t, int& lo, int& hi) {
  lo = hi = 0;
  if (!s.window) return;
  lo = max(0, s.sinks - t.pos);
  hi = max(lo, min(t.valid, u.p0 - s.window + 1 - t.pos));
}

}  // namespace fpd
