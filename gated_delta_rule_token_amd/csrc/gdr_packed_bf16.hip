// gdr_packed_bf16.hip -- the step on a state cache in bf16 (gdr_packed.hpp).
#include "gdr_packed.hpp"

namespace gdr {

hipError_t launch_packed_step_bf16(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s)
{
    return packed_step_typed<CACHE_BF16>(a, rule, per_key, act, s);
}

}  // namespace gdr
