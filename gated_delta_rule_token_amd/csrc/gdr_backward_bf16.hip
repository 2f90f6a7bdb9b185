// gdr_backward_bf16.hip -- the backward pass's kernels for bf16 activations.
#include "gdr_backward.hpp"

namespace gdr {

hipError_t launch_back_bf16(const BackParams &a, bool retrieves, hipStream_t s) { return launch_back_act<bf16_t>(a, retrieves, s); }

}  // namespace gdr
