// gdr_backward_f32.hip -- the backward pass's kernels for f32 activations.
#include "gdr_backward.hpp"

namespace gdr {

hipError_t launch_back_f32(const BackParams &a, bool retrieves, hipStream_t s) { return launch_back_act<float>(a, retrieves, s); }

}  // namespace gdr
