// norm_range.h - rows whose squares 32 bits do not hold: the factor their
// elements are multiplied by, and the block's choice to look at them again.
// Host and device.
#pragma once

#include "plan.h"

namespace vdn {

// Any row of up to 2^20 finite elements, not all zero, is brought into range: a sum that overflows has an element of 2^54
// or more, and 2^20 elements below 2^128 come to 2^116 after 2^-80; a sum below 2^-80 has elements below 2^-40 (2^112
// after 2^96), the smallest of which, 2^-149, has a square of 2^-106.
constexpr float kBigDown = 0x1p-80f, kSmallUp = 0x1p96f;

// Factor that brings a row's elements back where 32 bits hold their squares: 1
// unless the sum of squares has overflowed, or vanishes and eps does not cover it.
VDN_HD float norm_rescue(float sum, float eps) {
  if (!(sum <= 3.40282347e38f)) return kBigDown;
  return sum < 0x1p-80f && eps < 0x1p-80f ? kSmallUp : 1.f;
}

// Whether a block of kRows rows, kWarps warps to each, goes through its registers once more, from the warps' sums of
// squares.  The second look has barriers, so the answer may not depend on which thread asks: it is made of what all of
// them see, the sums of the rows that exist (the first `real` ones) and the call's eps.
template <int kRows, int kWarps>
VDN_HD bool norm_look_again(const float* sums, int real, float eps) {
  bool again = false;
#ifdef __CUDA_ARCH__
#pragma unroll
#endif
  for (int r = 0; r < kRows; ++r) {
    float s = sums[r * kWarps];
    for (int i = 1; i < kWarps; ++i) s += sums[r * kWarps + i];
    again = again || (r < real && norm_rescue(s, eps) != 1.f);
  }
  return again;
}

}  // namespace vdn
