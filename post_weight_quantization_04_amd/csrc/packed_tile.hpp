// Products with packed few-bit weights, many tokens: declared here, compiled once
// for each input type.
#pragma once

#include "packed_common.hpp"

namespace gptq {

// fine: groups that are no multiple of 128
template <typename T, int kBits>
hipError_t launch_packed_tile(const PmArgs& a, bool fine, hipStream_t s);

}  // namespace gptq
