// gdr_norm.hip -- root-mean-square norm of rows, with the residual's addition
// and an output in 8 bits with scales, and its backward pass.
//
//   r = x + residual (rounded to the activations' type, the value that is
//       kept and that the backward pass sees; r = x without a residual)
//   y = r inv w,   inv = 1 / sqrt(mean r^2 + eps)
//   8 bits: scale = max |y| / 448 over the row or each group of columns (1
//       where that is 0), y8 = e4m3(y / scale), the fp32 quotient
// and backwards, with h = r inv and t = w dy,
//   dx = inv (t - h mean(t h)) + d_residual,   dw = sum over rows of dy h
//
// Bound by memory: one pass over the data.  A row lies in the registers of
// TPR threads, NV vectors of 8 elements each, between its load and its store;
// the sums and the maxima go over lanes (and, past one wave, over LDS).  The
// next row is on its way, as it lies in memory, while one is worked on.
// Vectors are loaded whatever the row's alignment (16-bit rows of odd width
// start at any even byte), the last one of a row from 8 elements before its
// end, so that no load stands under a condition.
#include "gdr_norm_launch.hpp"

namespace gdr {
namespace {

constexpr float E4M3_MAX = 448.f;
constexpr int64_t NORM_BLOCKS = 256 * 8;  // workgroups of the forward pass: eight a CU

// 16 bytes from any even address.
typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements as they lie in memory: whole registers (as elements, 16-bit
// ones would take a register each).
template <typename T> struct Raw8 {
    static constexpr int WORDS = 2 * sizeof(T);
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *src)
    {
#pragma unroll
        for (int n = 0; n < WORDS / 4; ++n) {
            const v4 x = reinterpret_cast<const v4 *>(src)[n];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * n + i] = x[i];
        }
    }
    // What was widened before is forgotten: else it would be kept in fp32.
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[i]);
        else return to_f32(__builtin_bit_cast(T, (uint16_t)(w[i / 2] >> (16 * (i % 2)))));
    }
    __device__ __forceinline__ void set(int i, T x)
    {
        if constexpr (sizeof(T) == 4) w[i] = __builtin_bit_cast(uint32_t, x);
        else if (i % 2 == 0) w[i / 2] = __builtin_bit_cast(uint16_t, x);
        else w[i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, x) << 16;
    }
};

// A thread's vector of a row: columns col .. col + 7, of which [lo, hi) are
// its own, loaded from column `base` on.  EXACT: the width is a multiple of 8.
template <bool EXACT> struct Place {
    int col, base, lo, hi;
    __device__ __forceinline__ Place(int vector, int width)
    {
        col = vector * 8;
        base = col + 8 <= width ? col : width < 8 ? 0 : width - 8;
        lo = col < width ? col - base : 8;
        hi = width < 8 ? width : 8;
    }
    __device__ __forceinline__ bool on() const { return lo < 8; }
    __device__ __forceinline__ bool own(int i) const { return EXACT ? on() : i >= lo && i < hi; }
    __device__ __forceinline__ bool full() const { return EXACT ? on() : lo == 0 && hi == 8; }
    template <typename T> __device__ __forceinline__ void load(Raw8<T> &r, const T *row) const
    {
        if (EXACT || hi == 8) {
            r.load(row + base);
        } else {  // a row narrower than a vector
#pragma unroll
            for (int i = 0; i < 8; ++i) r.set(i, row[i < hi ? i : 0]);
        }
    }
    template <typename T> __device__ __forceinline__ void widen(const Raw8<T> &r, float (&out)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = own(i) ? r.get(i) : 0.f;
    }
    template <typename T> __device__ __forceinline__ void store(T *row, const float (&v)[8]) const
    {
        if (full()) {
            Raw8<T> o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o.set(i, from_f32<T>(v[i]));
    #pragma unroll
            for (int n = 0; n < Raw8<T>::WORDS / 4; ++n)
                reinterpret_cast<v4 *>(row + base)[n] = v4{o.w[4 * n], o.w[4 * n + 1], o.w[4 * n + 2], o.w[4 * n + 3]};
        } else if (!EXACT && on()) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (own(i)) row[base + i] = from_f32<T>(v[i]);
        }
    }
};

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

// A workgroup takes rows blockIdx.x * ROWS + group, + gridDim.x * ROWS, ...
template <typename T, typename TW, int TPR, int NV, bool EXACT>
__global__ __launch_bounds__(threads_of(TPR)) void k_norm(const NormParams p)
{
    __shared__ float s_red[16];
    constexpr int ROWS = threads_of(TPR) / TPR;
    constexpr bool AHEAD = TPR < 1024;  // the widest rows leave no registers for the next one
    const int lane = threadIdx.x % TPR, width = p.width;
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    if (ROWS > 1 && row >= p.rows) return;  // whole groups of TPR lanes; no barrier below when ROWS > 1
    Raw8<TW> w[NV];
    Raw8<T> x[NV], a[NV];
    auto fetch = [&](int64_t row) {
        const size_t at = (size_t)row * width;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const Place<EXACT> v(lane + TPR * n, width);
            v.load(x[n], static_cast<const T *>(p.x) + at);
            if (p.residual) v.load(a[n], static_cast<const T *>(p.residual) + at);
        }
    };
    if (AHEAD) fetch(row);
    if (p.weight)
#pragma unroll
        for (int n = 0; n < NV; ++n) Place<EXACT>(lane + TPR * n, width).load(w[n], static_cast<const TW *>(p.weight));
    for (; row < p.rows; row += stride) {
        if (!AHEAD) fetch(row);
        const size_t at = (size_t)row * width;
        float r[NV][8], sum = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const Place<EXACT> v(lane + TPR * n, width);
            v.widen(x[n], r[n]);
            if (p.residual) {
                float y[8];
                v.widen(a[n], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) r[n][i] = to_f32(from_f32<T>(r[n][i] + y[i]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += r[n][i] * r[n][i];
        }
        if (AHEAD) fetch(row + stride < p.rows ? row + stride : row);
        sum = row_reduce<TPR>(sum, Add(), s_red);
        // every load of the row has come back: residual_out may be the residual itself
        if (p.residual_out)
#pragma unroll
            for (int n = 0; n < NV; ++n) Place<EXACT>(lane + TPR * n, width).store(static_cast<T *>(p.residual_out) + at, r[n]);
        const float inv = 1.f / sqrtf(sum / (float)width + p.eps);
        if (p.inv_rms && lane == 0) p.inv_rms[row] = inv;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) r[n][i] = p.weight ? r[n][i] * inv * w[n].get(i) : r[n][i] * inv;

        if (!p.eight) {
#pragma unroll
            for (int n = 0; n < NV; ++n) Place<EXACT>(lane + TPR * n, width).store(static_cast<T *>(p.y) + at, r[n]);
            continue;
        }
        float top[NV], all = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const Place<EXACT> v(lane + TPR * n, width);
            top[n] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (v.own(i)) top[n] = Max()(fabsf(r[n][i]), top[n]);
            all = Max()(top[n], all);
        }
        const int lanes = p.group / 8;  // lanes of a group, a power of two
        const bool whole = p.group == 0 || p.group >= width;
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
            const int vec = lane + TPR * n;
            const Place<EXACT> v(vec, width);
            if (v.on() && (whole ? vec == 0 : vec % lanes == 0))
                p.scale[(size_t)row * p.groups + (whole ? 0 : vec / lanes)] = scale;
            // The code of the quotient that a division gives, by the reciprocal and
            // one step on the remainder: the two differ at no border of two codes for
            // any of the scale's 2^23 mantissas (each tried, with the nine floats
            // round the border; the reciprocal alone errs at 6 % of these).  The
            // reciprocal alone, this and a division: rows of 4,096 in groups of 128,
            // 174, 174 and 171 us (29,273 of them); of 2,050 in groups of 64, 259, 266
            // and 299 (60,000); of 128, 95, 101 and 115 (936,736).
            const float up = scale < 0x1p-60f ? 0x1p64f : 1.f;  // else remainders, or the reciprocal, would be denormal
            const float sc = scale * up, inv_scale = 1.f / sc, minus = sc < __builtin_huge_valf() ? -sc : 0.f;
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = r[n][i] * up, t0 = y * inv_scale, t = fmaf(fmaf(t0, minus, y), inv_scale, t0);
                // the scale's rounding may take the largest value past the type's
                q[i] = t > E4M3_MAX ? E4M3_MAX : t < -E4M3_MAX ? -E4M3_MAX : t;
            }
            const Bytes8 b = to_e4m3(q);
            uint8_t *out = static_cast<uint8_t *>(p.y) + at + v.base;
            if (v.full()) *reinterpret_cast<Bytes8 *>(out) = b;
            else if (!EXACT)
                for (int i = 0; i < 8; ++i)
                    if (v.own(i)) out[i] = (uint8_t)(b.x[i / 4] >> (8 * (i % 4)));
        }
    }
}

// ---------------------------------------------------------------- backward
// A workgroup takes rows blockIdx.x * ROWS + group, + gridDim.x * ROWS, ...;
// a thread's columns are the same for all of them, so that the weight's
// gradient stays in its registers until the end.  Its sums over the
// workgroup's row groups and then (second kernel) over the workgroups have a
// fixed order.
template <typename T, typename TW, int TPR, int NV, bool EXACT>
__global__ __launch_bounds__(threads_of(TPR)) void k_norm_back(const NormBackParams p)
{
    __shared__ float s_red[16];
    __shared__ float s_dw[TPR < 256 ? 256 * 8 : 1];
    constexpr int ROWS = threads_of(TPR) / TPR;
    constexpr bool AHEAD = TPR < 1024;
    const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR, width = p.width;
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + group;
    float dw[NV][8];
    Raw8<TW> w[NV];
    Raw8<T> x[NV], y[NV], a[NV];
    float inv_next = 0.f;
    auto fetch = [&](int64_t row) {
        const size_t at = (size_t)row * width;
        inv_next = p.inv_rms[row];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const Place<EXACT> v(lane + TPR * n, width);
            v.load(x[n], static_cast<const T *>(p.x) + at);
            v.load(y[n], static_cast<const T *>(p.d_y) + at);
            if (p.d_residual) v.load(a[n], static_cast<const T *>(p.d_residual) + at);
        }
    };
    if (AHEAD && row < p.rows) fetch(row);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        if (p.weight) Place<EXACT>(lane + TPR * n, width).load(w[n], static_cast<const TW *>(p.weight));
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[n][i] = 0.f;
    }
    for (; row < p.rows; row += stride) {
        if (!AHEAD) fetch(row);
        const size_t at = (size_t)row * width;
        const float inv = inv_next;
        float sum = 0.f;
        Raw8<T> xr[NV], yr[NV], ar[NV];  // widened again where they are used: a row in fp32 would take twice the registers
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const Place<EXACT> v(lane + TPR * n, width);
            xr[n] = x[n];
            yr[n] = y[n];
            ar[n] = a[n];
            float h[8], t[8];
            v.widen(xr[n], h);
            v.widen(yr[n], t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] *= inv;
                dw[n][i] += t[i] * h[i];
                sum += (p.weight ? t[i] * w[n].get(i) : t[i]) * h[i];
            }
        }
        if (AHEAD) fetch(row + stride < p.rows ? row + stride : row);
        sum = row_reduce<TPR>(sum, Add(), s_red) / (float)width;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            xr[n].again();
            yr[n].again();
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = p.weight ? yr[n].get(i) * w[n].get(i) : yr[n].get(i);
                d[i] = inv * (t - xr[n].get(i) * inv * sum);
                if (p.d_residual) d[i] += ar[n].get(i);
            }
            Place<EXACT>(lane + TPR * n, width).store(static_cast<T *>(p.d_x) + at, d);
        }
    }
    if (!p.partial) return;
    float *out = p.partial + (size_t)blockIdx.x * width;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
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
        if (group == 0) Place<EXACT>(lane + TPR * n, width).store(out, dw[n]);
    }
}

// Workgroup: 16 columns, 16 threads a column, each every 16th partial row.
__global__ __launch_bounds__(256) void k_norm_back_sums(const NormBackParams p, int blocks)
{
    __shared__ float s[16][17];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    float sum = 0.f;
    if (col < p.width) {
#pragma unroll 8
        for (int b = r; b < blocks; b += 16) sum += p.partial[(size_t)b * p.width + col];
    }
    s[r][c] = sum;
    __syncthreads();
    if (r == 0 && col < p.width) {
        for (int n = 1; n < 16; ++n) sum += s[n][c];
        p.d_weight[col] = sum;
    }
}

// Threads and vectors of a row: up to 64 vectors the power of two of lanes
// that covers it, then one wave up to WAVE vectors a lane, which spares the
// barriers; past that a workgroup.  At 29,273 rows of 2,048 in bf16 the forward
// pass takes 92 us with a row a wave (four vectors a lane); the backward pass
// 100 us so and 88 us with a row a workgroup, as its lanes then hold a quarter
// of the three rows and the weight's gradient.  The widest rows (above 16,384)
// do not fit a workgroup's registers: 60 to 144 bytes a lane lie in scratch
// memory forwards (3,000 rows of 32,768 in bf16: 159 us) and 324 to 520 backwards
// (642 us, 4 times the copy rate's 152, where 6,000 rows of 16,384 take 145); rows of
// 8,193 to 16,384 backwards put 12 bytes there in bf16 and 52 to 68 in fp32.
template <int WAVE, typename F>
hipError_t by_width(int64_t width, F &&f)
{
    using std::integral_constant;
    const int64_t v = (width + 7) / 8;
    if (v <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (v <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (v <= 64) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (v <= 128) return f(integral_constant<int, 64>(), integral_constant<int, 2>());
    if (v <= 256) {
        if constexpr (WAVE >= 4) return f(integral_constant<int, 64>(), integral_constant<int, 4>());
        else return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    }
    if (v <= 512) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (v <= 1024) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
    if (v <= 2048) return f(integral_constant<int, 1024>(), integral_constant<int, 2>());
    return f(integral_constant<int, 1024>(), integral_constant<int, 4>());
}

template <typename T, typename TW>
hipError_t norm_typed(const NormParams &p, hipStream_t s)
{
    return by_width<4>(p.width, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, ROWS = threads_of(TPR) / TPR;
        const int64_t need = (p.rows + ROWS - 1) / ROWS;
        const dim3 blocks((unsigned)(need < NORM_BLOCKS ? need : NORM_BLOCKS)), threads(threads_of(TPR));
        if (p.width % 8 == 0) hipLaunchKernelGGL((k_norm<T, TW, TPR, NV, true>), blocks, threads, 0, s, p);
        else hipLaunchKernelGGL((k_norm<T, TW, TPR, NV, false>), blocks, threads, 0, s, p);
        return hipGetLastError();
    });
}

template <typename T, typename TW>
hipError_t norm_back_typed(const NormBackParams &p, hipStream_t s)
{
    return by_width<2>(p.width, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        const int blocks = norm_back_blocks(p.rows, p.width);
        if (p.width % 8 == 0)
            hipLaunchKernelGGL((k_norm_back<T, TW, TPR, NV, true>), dim3((unsigned)blocks), dim3(threads_of(TPR)), 0, s, p);
        else
            hipLaunchKernelGGL((k_norm_back<T, TW, TPR, NV, false>), dim3((unsigned)blocks), dim3(threads_of(TPR)), 0, s, p);
        if (p.partial)
            hipLaunchKernelGGL(k_norm_back_sums, dim3((unsigned)((p.width + 15) / 16)), dim3(256), 0, s, p, blocks);
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
    // 16,384 elements a workgroup, up to two workgroups a CU (29,273 rows of
    // 2,048 in bf16: 88 us; with four, whose partial rows are twice as many, 97 us).
    // 8,192, 16,384 and 32,768 elements, on the device (a graph's replay): 1,217 rows of
    // 1,001 in fp32 10.9, 14.0 and 18.9 us, 256 of 2,048 in bf16 8.7, 11.7 and
    // 18.9, 300 of 8,192 in fp32 21.5, 15.4 and 16.8, 1,000 of 4,096 in bf16 17.1,
    // 16.9 and 21.6.  Calls one by one take 16.7 to 17.0 us in all of the first two
    // forms, the host's time, but for the 300 rows (20.0 and 16.7), and up to 21
    // in the third.
    const int64_t n = rows * width / 16384;
    return n < 1 ? 1 : n > 512 ? 512 : (int)n;
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
