// gdr_packed_e4m3.hip -- the step on a state cache in e4m3 (gdr_packed.hpp).
#include "gdr_packed.hpp"

namespace gdr {

hipError_t launch_packed_step_e4m3(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s)
{
    return packed_step_typed<CACHE_E4M3>(a, rule, per_key, act, s);
}

}  // namespace gdr
