// What the two kernels of linear_fp8_block share.
#pragma once

#include <type_traits>

#include "block.h"
#include "kernels.h"
#include "tcgen05.cuh"

namespace gbf {

// The activations are fast_act's (common.cuh), as in the static Linears: the error of
// the hardware's tanh, |a| 2^-11.9, or of an erf of 1.5e-7, and not a rounding of the
// result itself where a GELU's result is small beside a.  Forms that are right to a
// few 2^-23 of the result (a logistic function; the gated activation's erfc) take 455
// us for 418 with the tanh GELU, 502-508 for 478-494 with the erf's (8192 x 16384 x
// 4096), and 16.2 for 15.4 on 32 rows.
//
// Calls f with the activation as a constant: chosen once a tile, not at each
// value, where the branches kept the values' chains apart (8192 x 16384 x 4096
// with the tanh GELU: 451 -> 422 us).
template <typename F>
GBF_DEVICE void with_act(int act, F f) {
  switch (act) {
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    case kActGeluErf: f(std::integral_constant<int, kActGeluErf>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    default: f(std::integral_constant<int, kActNone>()); break;
  }
}

}  // namespace gbf
