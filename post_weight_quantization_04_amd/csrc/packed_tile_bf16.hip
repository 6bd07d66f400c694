// Products with packed few-bit weights for many tokens, bfloat16 activations.
#include "packed_tile_kernel.hpp"

namespace gptq {

template hipError_t launch_packed_tile<bf16_t, 2>(const PmArgs&, int, bool, hipStream_t);
template hipError_t launch_packed_tile<bf16_t, 3>(const PmArgs&, int, bool, hipStream_t);
template hipError_t launch_packed_tile<bf16_t, 4>(const PmArgs&, int, bool, hipStream_t);
template hipError_t launch_packed_tile<bf16_t, 5>(const PmArgs&, int, bool, hipStream_t);
template hipError_t launch_packed_tile<bf16_t, 6>(const PmArgs&, int, bool, hipStream_t);
template hipError_t launch_packed_tile<bf16_t, 7>(const PmArgs&, int, bool, hipStream_t);
template hipError_t launch_packed_tile<bf16_t, 8>(const PmArgs&, int, bool, hipStream_t);

}  // namespace gptq
