// gdr_norm_launch.hpp -- argument blocks and launchers of the root-mean-square
// norm (internal to libgdr).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "gdr_device.hpp"

namespace gdr {

constexpr int64_t NORM_MAX_WIDTH = 32768;  // columns a row's threads hold in registers

// dt, weight_dt: 0 fp32, 1 fp16, 2 bf16; weight_dt is dt or 0.
struct NormParams {
    int64_t rows;
    int32_t width, dt, weight_dt;
    int32_t eight;              // 1: y is e4m3 with scales
    int32_t group, groups;      // columns of a scale (0: the row), scales of a row
    float eps;
    const void *x, *residual, *weight;
    void *y, *residual_out;
    float *scale, *inv_rms;
};

struct NormBackParams {
    int64_t rows;
    int32_t width, dt, weight_dt;
    const void *d_y, *x, *weight, *d_residual;
    const float *inv_rms;
    void *d_x;
    float *d_weight;            // or nullptr (then partial too)
    float *partial;             // norm_back_blocks x width floats
};

int norm_back_blocks(int64_t rows, int64_t width);
hipError_t launch_norm(const NormParams &p, hipStream_t s);
hipError_t launch_norm_backward(const NormBackParams &p, hipStream_t s);

}  // namespace gdr
