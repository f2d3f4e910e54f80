// Second step of a sum over rows: a first kernel's blocks wrote partial rows, part[p][seg][pitch] fp32 for p < parts;
// added up in a fixed order (unlike atomics, the same call gives the same bits), the first n columns of segment 0
// go to out and those of segment 1 to out2.  Without out2, `segs` tells whether the rows have a second segment.
#pragma once

#include "common.h"

namespace sfp8 {

void launch_col_reduce(const float* part, int parts, int segs, int64_t pitch, int64_t n, float* out, float* out2,
                       hipStream_t st);

}  // namespace sfp8
