// gdr_backward_f16.hip -- the backward pass's kernels for f16 activations.
#include "gdr_backward.hpp"

namespace gdr {

hipError_t launch_back_f16(const BackParams &a, bool retrieves, hipStream_t s) { return launch_back_act<half_t>(a, retrieves, s); }

}  // namespace gdr
