// What the two kernels of linear_fp8_block share.
#pragma once

#include <type_traits>

#include "block.h"
#include "kernels.h"
#include "tcgen05.cuh"

namespace gbf {

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
