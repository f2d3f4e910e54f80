// Second step of a sum over rows: the partial rows part[p][n] fp32, p < parts, that a first kernel's blocks wrote, added
// up in a fixed order (unlike atomics, the same call gives the same bits).  Columns below `split` go to out,
// the others to out2 at n - split (dropped where out2 is null).
#pragma once

#include "common.h"

namespace sfp8 {

void launch_col_reduce(const float* part, int parts, int64_t n, float* out, int64_t split, float* out2, hipStream_t st);

}  // namespace sfp8
