// gdr_norm.hip -- root-mean-square norm of rows, with the residual's addition
// and an output in 8 bits with scales, and its backward pass.
//
//   r = x + residual (rounded to the activations' type, the value that is
//       kept and that the backward pass sees; r = x without a residual)
//   y = r inv w,   inv = 1 / sqrt(mean r^2 + eps)
//   8 bits: scale = max |y| / 448 over the row or each group of columns (1
//       where the maximum is 0), y8 = e4m3(y / scale)
// and backwards, with h = r inv and t = w dy,
//   dx = inv (t - h mean(t h)) + d_residual,   dw = sum over rows of dy h
//
// Bound by memory: one pass over the data.  A row lies in the registers of
// TPR threads, NV vectors of 8 elements each, between its load and its store;
// the sums and the maxima go over lanes (and, past one wave, over LDS).
// Vectors are loaded whatever the row's alignment (16-bit rows of odd width
// start at any even byte); only the vector that holds the row's end is loaded
// by element.
#include "gdr_norm_launch.hpp"

namespace gdr {
namespace {

constexpr float E4M3_MAX = 448.f;

template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) Vec8 { T x[8]; };

template <typename T>
__device__ __forceinline__ void load8(const T *row, int col, int width, float (&out)[8])
{
    if (col + 8 <= width) {
        const Vec8<T> v = *reinterpret_cast<const Vec8<T> *>(row + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = to_f32(v.x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = col + i < width ? to_f32(row[col + i]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *row, int col, int width, const float (&v)[8])
{
    if (col + 8 <= width) {
        Vec8<T> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.x[i] = from_f32<T>(v[i]);
        *reinterpret_cast<Vec8<T> *>(row + col) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < width) row[col + i] = from_f32<T>(v[i]);
    }
}

// Eight values as e4m3, rounded to nearest even; |v| <= 448 but for NaN,
// which stays NaN.
struct __attribute__((packed, aligned(1))) Bytes8 { uint32_t x[2]; };

__device__ __forceinline__ Bytes8 to_e4m3(const float (&v)[8])
{
    Bytes8 b;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * n], v[4 * n + 1], 0, false);
        b.x[n] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * n + 2], v[4 * n + 3], w, true);
    }
    return b;
}

struct Add { __device__ __forceinline__ float operator()(float a, float b) const { return a + b; } };
// the larger; NaN if either is
struct Max { __device__ __forceinline__ float operator()(float a, float b) const { return a > b || a != a ? a : b; } };

// Over the TPR threads of a row; every one of them gets the result.
template <int TPR, typename Op>
__device__ __forceinline__ float row_reduce(float x, Op op, float *s)
{
    constexpr int LANES = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) x = op(x, __shfl_xor(x, o));
    if constexpr (TPR > 64) {
        __syncthreads();  // the last use of s
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        x = s[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) x = op(x, s[w]);
    }
    return x;
}

constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }

template <typename T, typename TW, int TPR, int NV>
__global__ __launch_bounds__(threads_of(TPR)) void k_norm(const NormParams p)
{
    __shared__ float s_red[16];
    constexpr int ROWS = threads_of(TPR) / TPR;
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (ROWS > 1 && row >= p.rows) return;  // whole groups of TPR lanes; no barrier below when ROWS > 1
    const size_t base = (size_t)row * p.width;
    const T *x = static_cast<const T *>(p.x) + base;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + base : nullptr;
    float r[NV][8], w[NV][8], sum = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = (lane + TPR * n) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[n][i] = 0.f;
        if (col < p.width) {
            load8(x, col, p.width, r[n]);
            if (res) {
                float y[8];
                load8(res, col, p.width, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) r[n][i] = to_f32(from_f32<T>(r[n][i] + y[i]));
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = (lane + TPR * n) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[n][i] = 1.f;
        if (col < p.width) {
            if (p.weight) load8(static_cast<const TW *>(p.weight), col, p.width, w[n]);
            if (p.residual_out) store8(static_cast<T *>(p.residual_out) + base, col, p.width, r[n]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += r[n][i] * r[n][i];
    }
    sum = row_reduce<TPR>(sum, Add(), s_red);
    const float inv = 1.f / sqrtf(sum / (float)p.width + p.eps);
    if (p.inv_rms && lane == 0) p.inv_rms[row] = inv;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) r[n][i] = r[n][i] * inv * w[n][i];

    if (!p.eight) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (lane + TPR * n) * 8;
            if (col < p.width) store8(static_cast<T *>(p.y) + base, col, p.width, r[n]);
        }
        return;
    }
    float top[NV], all = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        top[n] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((lane + TPR * n) * 8 + i < p.width) top[n] = Max()(fabsf(r[n][i]), top[n]);
        all = Max()(top[n], all);
    }
    const int lanes = p.group / 8;  // lanes of a group, a power of two
    const bool whole = p.group == 0 || p.group >= p.width;
    if (whole) all = row_reduce<TPR>(all, Max(), s_red);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float m = all;
        if (!whole) {
            m = top[n];
            for (int o = 1; o < lanes; o <<= 1) m = Max()(m, __shfl_xor(m, o));
        }
        float scale = m / E4M3_MAX;
        if (scale == 0.f) scale = 1.f;
        const int v = lane + TPR * n, col = v * 8;
        if (col >= p.width) continue;
        if (whole ? v == 0 : v % lanes == 0) p.scale[(size_t)row * p.groups + (whole ? 0 : v / lanes)] = scale;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = r[n][i] / scale;
            // a rounding of the quotient may pass the largest value by an ulp
            q[i] = t > E4M3_MAX ? E4M3_MAX : t < -E4M3_MAX ? -E4M3_MAX : t;
        }
        const Bytes8 b = to_e4m3(q);
        uint8_t *out = static_cast<uint8_t *>(p.y) + base;
        if (col + 8 <= p.width) *reinterpret_cast<Bytes8 *>(out + col) = b;
        else
            for (int i = 0; i < 8; ++i)
                if (col + i < p.width) out[col + i] = (uint8_t)(b.x[i / 4] >> (8 * (i % 4)));
    }
}

// ---------------------------------------------------------------- backward
// A workgroup takes rows blockIdx.x * ROWS + group, + gridDim.x * ROWS, ...;
// a thread's columns are the same for all of them, so that the weight's
// gradient stays in its registers until the end.  Its sums over the
// workgroup's row groups and then (second kernel) over the workgroups have a
// fixed order.
template <typename T, typename TW, int TPR, int NV>
__global__ __launch_bounds__(threads_of(TPR)) void k_norm_back(const NormBackParams p)
{
    __shared__ float s_red[16];
    __shared__ float s_dw[TPR < 256 ? 256 * 8 : 1];
    constexpr int ROWS = threads_of(TPR) / TPR;
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
    float w[NV][8], dw[NV][8];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = (lane + TPR * n) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[n][i] = 1.f;
            dw[n][i] = 0.f;
        }
        if (p.weight && col < p.width) load8(static_cast<const TW *>(p.weight), col, p.width, w[n]);
    }
    for (int64_t row = (int64_t)blockIdx.x * ROWS + group; row < p.rows; row += (int64_t)gridDim.x * ROWS) {
        const size_t base = (size_t)row * p.width;
        const float inv = p.inv_rms[row];
        float h[NV][8], t[NV][8], sum = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (lane + TPR * n) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[n][i] = t[n][i] = 0.f;
            if (col < p.width) {
                load8(static_cast<const T *>(p.x) + base, col, p.width, h[n]);
                load8(static_cast<const T *>(p.d_y) + base, col, p.width, t[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[n][i] *= inv;
                dw[n][i] += t[n][i] * h[n][i];
                t[n][i] *= w[n][i];
                sum += t[n][i] * h[n][i];
            }
        sum = row_reduce<TPR>(sum, Add(), s_red) / (float)p.width;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (lane + TPR * n) * 8;
            if (col >= p.width) continue;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = 0.f;
            if (p.d_residual) load8(static_cast<const T *>(p.d_residual) + base, col, p.width, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] += inv * (t[n][i] - h[n][i] * sum);
            store8(static_cast<T *>(p.d_x) + base, col, p.width, d);
        }
    }
    if (!p.partial) return;
    float *out = p.partial + (size_t)blockIdx.x * p.width;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int col = (lane + TPR * n) * 8;
        if constexpr (ROWS > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) s_dw[threadIdx.x * 8 + i] = dw[n][i];
            __syncthreads();
            if (group == 0)
                for (int g = 1; g < ROWS; ++g)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dw[n][i] += s_dw[(g * TPR + lane) * 8 + i];
        }
        if (group == 0 && col < p.width) store8(out, col, p.width, dw[n]);
    }
}

// Workgroup: 64 columns, four threads a column, each every fourth partial row.
__global__ __launch_bounds__(256) void k_norm_back_sums(const NormBackParams p, int blocks)
{
    __shared__ float s[256];
    const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    float sum = 0.f;
    if (col < p.width)
        for (int b = threadIdx.x >> 6; b < blocks; b += 4) sum += p.partial[(size_t)b * p.width + col];
    s[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < 64 && col < p.width)
        p.d_weight[col] = (s[threadIdx.x] + s[threadIdx.x + 64]) + (s[threadIdx.x + 128] + s[threadIdx.x + 192]);
}

// Threads and vectors of a row.  Up to 64 vectors of 8 a row takes the power
// of two of lanes that covers it; up to 4,096 columns one wave; past that a
// workgroup.
template <typename F>
hipError_t by_width(int64_t width, F &&f)
{
    const int64_t v = (width + 7) / 8;
    if (v <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (v <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
    if (v <= 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (v <= 128) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    if (v <= 256) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
    if (v <= 512) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
    if (v <= 1024) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
    return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
}

template <typename T, typename TW>
hipError_t norm_typed(const NormParams &p, hipStream_t s)
{
    return by_width(p.width, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, ROWS = threads_of(TPR) / TPR;
        hipLaunchKernelGGL((k_norm<T, TW, TPR, NV>), dim3((unsigned)((p.rows + ROWS - 1) / ROWS)), dim3(threads_of(TPR)), 0, s, p);
        return hipGetLastError();
    });
}

template <typename T, typename TW>
hipError_t norm_back_typed(const NormBackParams &p, hipStream_t s)
{
    return by_width(p.width, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const int blocks = norm_back_blocks(p.rows, p.width);
        hipLaunchKernelGGL((k_norm_back<T, TW, TPR, NV>), dim3((unsigned)blocks), dim3(threads_of(TPR)), 0, s, p);
        if (p.partial)
            hipLaunchKernelGGL(k_norm_back_sums, dim3((unsigned)((p.width + 63) / 64)), dim3(256), 0, s, p, blocks);
        return hipGetLastError();
    });
}

template <typename P, typename F>
hipError_t by_types(const P &p, F &&f)
{
    if (p.dt == 1) return p.weight_dt == 1 ? f(half_t(), half_t()) : f(half_t(), float());
    if (p.dt == 2) return p.weight_dt == 2 ? f(bf16_t(), bf16_t()) : f(bf16_t(), float());
    return f(float(), float());
}

}  // namespace

int norm_back_blocks(int64_t rows, int64_t width)
{
    const int64_t n = rows * width / 16384;  // elements a workgroup, up to four workgroups per CU
    return n < 1 ? 1 : n > 1024 ? 1024 : (int)n;
}

hipError_t launch_norm(const NormParams &p, hipStream_t s)
{
    if (p.rows == 0) return hipSuccess;
    return by_types(p, [&](auto t, auto w) { return norm_typed<decltype(t), decltype(w)>(p, s); });
}

hipError_t launch_norm_backward(const NormBackParams &p, hipStream_t s)
{
    return by_types(p, [&](auto t, auto w) { return norm_back_typed<decltype(t), decltype(w)>(p, s); });
}

}  // namespace gdr
