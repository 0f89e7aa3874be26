// Modified scores (pkv_score_mod): what a row sees and what its scores become.
#pragma once

#include <cuda_runtime.h>

#include "pkv_internal.h"

namespace pkv {
namespace {

// Keys [lo, hi) that packed row `row` at position p of a slot of L keys sees; lo = hi = 0 for none.
__device__ __forceinline__ void row_sees(const StepArgs &a, int64_t row, int p, int L, int &lo, int &hi) {
  lo = a.key_begin ? max(0, __ldg(a.key_begin + row)) : 0;
  if (a.window > 0) lo = max(lo, p - a.window + 1);
  hi = a.key_end ? min(L, __ldg(a.key_end + row)) : p + 1;
  if (lo >= hi) lo = hi = 0;
}

}  // namespace
}  // namespace pkv
