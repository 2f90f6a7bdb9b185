// gdr_packed.hip -- fp32 states written into the slots of a state cache in 16
// or 8 bits, and read back (the formats: gdr_packed.hpp).
//
// Bound by memory: each state is read once and written once.  A workgroup takes
// 32 rows of one state, 32 lanes a row and eight rows at a time, so that a row's
// largest value is a reduction over lanes; vectors of four values where rows
// consist of whole ones.
#include "gdr_packed.hpp"

namespace gdr {
namespace {

constexpr int ROWS = 32;  // of a workgroup

struct Where {
    size_t state, cache;  // first rows of the states and of the cache
    int rows;             // 0: nothing to do
    bool valid;           // false: a slot id out of range
};

// This workgroup's rows; request b's id for the unpacked states.
__device__ __forceinline__ Where rows_of(const PackedParams &a, bool skip_empty)
{
    const Params &p = a.p;
    const int parts = (p.dv + ROWS - 1) / ROWS;
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % p.HV, b = blockIdx.x / (parts * p.HV);
    const int slot = p.slot_ids[b];
    const bool valid = slot >= 0 && slot < p.num_slots;
    if (a.ids && part == 0 && h == 0 && threadIdx.x == 0) a.ids[b] = valid ? b : -1;
    Where w{((size_t)b * p.HV + h) * p.dv + part * ROWS, ((size_t)slot * p.HV + h) * p.dv + part * ROWS,
            p.dv - part * ROWS < ROWS ? p.dv - part * ROWS : ROWS, valid};
    if (valid && skip_empty) {
        int64_t s, e;
        request_range(p, b, s, e);
        if (e <= s) w.rows = 0;
    }
    return w;
}

// Lane l of a row holds columns (l + 32 n) VEC .. + VEC - 1.
template <int TYPE, int VEC>
__global__ __launch_bounds__(256) void k_pack(const PackedParams a)
{
    constexpr int NV = 256 / 32 / VEC, PASSES = ROWS / 8;
    const Where w = rows_of(a, a.skip_empty);
    if (!w.valid) return;
    const int l = threadIdx.x % 32, r = threadIdx.x / 32, dk = a.p.dk;
    float x[PASSES][NV][VEC];
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int row = r + 8 * i, col = (l + 32 * n) * VEC;
            const bool on = row < w.rows && col < dk;
            const float *src = a.states + (w.state + row) * dk + col;
#pragma unroll
            for (int c = 0; c < VEC; ++c) x[i][n][c] = 0.f;
            if (!on) continue;
            if constexpr (VEC == 4) {
                const w4 v = __builtin_nontemporal_load(reinterpret_cast<const w4 *>(src));
#pragma unroll
                for (int c = 0; c < 4; ++c) x[i][n][c] = as_float(v[c]);
            } else {
                x[i][n][0] = src[0];
            }
        }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int row = r + 8 * i;
        uint32_t ex = 0;
        if constexpr (TYPE == CACHE_E4M3) {
            float top = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int c = 0; c < VEC; ++c) top = fmaxf(top, fabsf(x[i][n][c]));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
            ex = scale_byte(top);
            if (row < w.rows && l == 0) a.scale[w.cache + row] = (uint8_t)ex;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (l + 32 * n) * VEC;
            if (row >= w.rows || col >= dk) continue;
            const size_t at = (w.cache + row) * dk + col;
            if constexpr (TYPE == CACHE_E4M3) {
                if constexpr (VEC == 4) {
                    reinterpret_cast<uint32_t *>(static_cast<char *>(a.data) + at)[0] = to_codes(x[i][n], scale_of(ex));
                } else {
                    const float v[4] = {x[i][n][0], 0.f, 0.f, 0.f};
                    static_cast<uint8_t *>(a.data)[at] = (uint8_t)to_codes(v, scale_of(ex));
                }
            } else {
                using T = typename CacheType<TYPE>::T;
                if constexpr (VEC == 4) {
                    const uint2 v = {two_halves<T>(x[i][n][0], x[i][n][1]), two_halves<T>(x[i][n][2], x[i][n][3])};
                    *reinterpret_cast<uint2 *>(static_cast<T *>(a.data) + at) = v;
                } else {
                    static_cast<T *>(a.data)[at] = from_f32<T>(x[i][n][0]);
                }
            }
        }
    }
}

template <int TYPE, int VEC>
__global__ __launch_bounds__(256) void k_unpack(const PackedParams a)
{
    constexpr int NV = 256 / 32 / VEC, PASSES = ROWS / 8;
    const Where w = rows_of(a, false);
    const int l = threadIdx.x % 32, r = threadIdx.x / 32, dk = a.p.dk;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int row = r + 8 * i;
        if (row >= w.rows) continue;
        const float scale = TYPE == CACHE_E4M3 && w.valid ? scale_of(a.scale[w.cache + row]) : 1.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = (l + 32 * n) * VEC;
            if (col >= dk) continue;
            const size_t at = (w.cache + row) * dk + col;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (!w.valid) {
                // zeros
            } else if constexpr (TYPE == CACHE_E4M3) {
                if constexpr (VEC == 4) from_codes(reinterpret_cast<const uint32_t *>(static_cast<const char *>(a.data) + at)[0], scale, x);
                else from_codes(static_cast<const uint8_t *>(a.data)[at], scale, x);
            } else {
                using T = typename CacheType<TYPE>::T;
                if constexpr (VEC == 4) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const T *>(a.data) + at);
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[c] = half_of<T>(c < 2 ? v.x : v.y, c % 2);
                } else {
                    x[0] = to_f32(static_cast<const T *>(a.data)[at]);
                }
            }
            float *dst = a.states + (w.state + row) * dk + col;
            if constexpr (VEC == 4) *reinterpret_cast<float4 *>(dst) = float4{x[0], x[1], x[2], x[3]};
            else dst[0] = x[0];
        }
    }
}

template <typename F>
hipError_t by_type(const PackedParams &a, F &&f)
{
    using std::integral_constant;
    const auto go = [&](auto type) {
        return a.p.dk % 4 == 0 ? f(type, integral_constant<int, 4>()) : f(type, integral_constant<int, 1>());
    };
    if (a.type == CACHE_F16) return go(integral_constant<int, CACHE_F16>());
    if (a.type == CACHE_BF16) return go(integral_constant<int, CACHE_BF16>());
    return go(integral_constant<int, CACHE_E4M3>());
}

}  // namespace

int64_t pack_blocks(int batch, int heads, int dv) { return (int64_t)batch * heads * ((dv + ROWS - 1) / ROWS); }

hipError_t launch_pack(const PackedParams &a, hipStream_t s)
{
    const int64_t blocks = pack_blocks(a.p.B, a.p.HV, a.p.dv);
    if (blocks == 0) return hipSuccess;
    return by_type(a, [&](auto type, auto vec) {
        hipLaunchKernelGGL((k_pack<decltype(type)::value, decltype(vec)::value>), dim3((unsigned)blocks), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_unpack(const PackedParams &a, hipStream_t s)
{
    const int64_t blocks = pack_blocks(a.p.B, a.p.HV, a.p.dv);
    if (blocks == 0) return hipSuccess;
    return by_type(a, [&](auto type, auto vec) {
        hipLaunchKernelGGL((k_unpack<decltype(type)::value, decltype(vec)::value>), dim3((unsigned)blocks), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_packed_step(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s)
{
    if (a.type == CACHE_F16) return launch_packed_step_f16(a, rule, per_key, act, s);
    if (a.type == CACHE_BF16) return launch_packed_step_bf16(a, rule, per_key, act, s);
    return launch_packed_step_e4m3(a, rule, per_key, act, s);
}

}  // namespace gdr
