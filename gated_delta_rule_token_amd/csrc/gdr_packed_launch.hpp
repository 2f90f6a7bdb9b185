// gdr_packed_launch.hpp -- argument blocks and launchers of the state cache in
// 16 or 8 bits (internal to libgdr).
#pragma once

#include "gdr_launch.hpp"

namespace gdr {

// Types of the cache's values, as in gdr_dtype.
enum : int { CACHE_F16 = 1, CACHE_BF16 = 2, CACHE_E4M3 = 3 };

// A cache of p.num_slots x p.HV states of p.dv rows of p.dk values at `data`;
// e4m3 values are in units of 2^(scale - 127), one byte a row.
struct PackedParams {
    Params p;            // slot_ids, sizes, requests and, for a step, its tensors; p.init and p.state are not used
    void *data;
    uint8_t *scale;
    int32_t type;
    float *states;       // (B, HV, dv, dk): packed from, unpacked to
    int32_t *ids;        // unpack: b, or -1 where a slot id is out of range (or nullptr)
    int32_t skip_empty;  // pack: requests without tokens keep their slots
};

// Workgroups of pack and unpack at most; a step takes no more.  A launch has fewer than
// 2^32 threads, 256 a workgroup.
int64_t pack_blocks(int batch, int heads, int dv);
constexpr int64_t PACK_BLOCKS_MAX = (int64_t{1} << 24) - 1;

hipError_t launch_pack(const PackedParams &a, hipStream_t s);
hipError_t launch_unpack(const PackedParams &a, hipStream_t s);
// rule: as gdr_update_rule; act: 0 fp32, 1 fp16, 2 bf16
hipError_t launch_packed_step(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s);
hipError_t launch_packed_step_f16(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s);
hipError_t launch_packed_step_bf16(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s);
hipError_t launch_packed_step_e4m3(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s);

}  // namespace gdr
