// Launchers of the products with packed few-bit weights, compiled once for each
// input type.
#pragma once

#include "packed_common.hpp"

namespace gptq {

// tokens x weight rows of a workgroup
enum PmKernel { kPmFew, kPm32x64, kPm64x128, kPm128x384 };

// fine: groups that are no multiple of 128
template <typename T, int kBits>
hipError_t launch_packed_few(const PmArgs& a, bool fine, hipStream_t s);
template <typename T, int kBits>
hipError_t launch_packed_tile(const PmArgs& a, int kernel, bool fine, hipStream_t s);

}  // namespace gptq
