// Products with packed few-bit weights for few tokens, float16 activations.
#include "packed_few_kernel.hpp"

namespace gptq {

template hipError_t launch_packed_few<half_t, 2>(const PmArgs&, bool, hipStream_t);
template hipError_t launch_packed_few<half_t, 3>(const PmArgs&, bool, hipStream_t);
template hipError_t launch_packed_few<half_t, 4>(const PmArgs&, bool, hipStream_t);
template hipError_t launch_packed_few<half_t, 5>(const PmArgs&, bool, hipStream_t);
template hipError_t launch_packed_few<half_t, 6>(const PmArgs&, bool, hipStream_t);
template hipError_t launch_packed_few<half_t, 7>(const PmArgs&, bool, hipStream_t);
template hipError_t launch_packed_few<half_t, 8>(const PmArgs&, bool, hipStream_t);

}  // namespace gptq
