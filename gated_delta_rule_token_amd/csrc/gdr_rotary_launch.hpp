// gdr_rotary_launch.hpp -- argument blocks and launchers of the norm and
// rotation of queries and keys (internal to libgdr).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gdr_device.hpp"

namespace gdr {

constexpr int ROTARY_MAX_DIM = 256;
constexpr int ROTARY_MAX_AXES = 4;

// One of q and k: `heads` heads a token, `stride` elements from token to
// token of x, `out_stride` of y (forward: the result; backward: the gradient
// of x); d_y, backward, has no gaps.
struct RotaryPart {
    const void *x, *weight, *d_y;
    void *y;
    float *d_weight, *partial;  // backward: rotary_back_blocks x dim floats, or nullptr
    int64_t stride, out_stride;
    int32_t heads;
    int32_t block, blocks;          // backward: tokens a workgroup takes at a time, workgroups
};

// dt, weight_dt: 0 fp32, 1 fp16, 2 bf16; weight_dt is dt or 0.
struct RotaryParams {
    RotaryPart part[2];
    int64_t tokens;
    int32_t dim, half, axes;        // half: pairs that are turned
    int32_t neighbours, norm, dt, weight_dt;
    int32_t block;                  // forward: tokens a workgroup takes
    int64_t first;                  // forward: token of the launch's first workgroup
    float eps;
    const int32_t *positions, *axis_of;
    const float *freq;
};

int rotary_back_blocks(int64_t tokens, int64_t heads, int64_t all_heads, int64_t dim);
hipError_t launch_rotary(const RotaryParams &p, hipStream_t s);
hipError_t launch_rotary_backward(const RotaryParams &p, hipStream_t s);

}  // namespace gdr
