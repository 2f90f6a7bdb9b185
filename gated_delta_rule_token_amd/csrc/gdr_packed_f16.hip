// gdr_packed_f16.hip -- the step on a state cache in f16 (gdr_packed.hpp).
#include "gdr_packed.hpp"

namespace gdr {

hipError_t launch_packed_step_f16(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s)
{
    return packed_step_typed<CACHE_F16>(a, rule, per_key, act, s);
}

}  // namespace gdr
