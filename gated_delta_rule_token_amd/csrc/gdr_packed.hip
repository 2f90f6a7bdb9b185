// gdr_packed.hip -- fp32 states written into the slots of a state cache in 16
// or 8 bits, and read back (the formats: gdr_packed.hpp).
//
// Bound by memory: each state is read once and written once.  A workgroup takes
// 32 rows of one state, 32 lanes a row and eight rows at a time (to 64 and 32 keys
// 16 and 8 lanes, and as many more rows), so that a row's largest value is a
// reduction over lanes; vectors of four values, of which a
// row's last may start earlier and share columns with the one before: both write
// the same bytes.  67 x 26 states of 256 x 30 and of 256 x 97 into 8 bits take 14
// and 40 us; value by value, with 32 lanes for any row, they took 37 and 50.
#include "gdr_packed.hpp"

namespace gdr {
namespace {

constexpr int PASSES = 4;  // of a workgroup over its rows
constexpr int rows_at(int lanes) { return 256 / lanes * PASSES; }

// 16, 8 and 4 bytes at any value's address.
typedef uint32_t V16 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t V8 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t V4 __attribute__((aligned(1)));

// First column of vector `i` of a row, or -1: past its end.
template <int VEC> __device__ __forceinline__ int column(int i, int dk)
{
    const int at = i * VEC;
    return at >= dk ? -1 : at + VEC <= dk ? at : dk - VEC;
}

struct Where {
    size_t state, cache;  // first rows of the states and of the cache
    int rows;             // 0: nothing to do
    bool valid;           // false: a slot id out of range
};

// This workgroup's rows; request b's id for the unpacked states.
template <int ROWS> __device__ __forceinline__ Where rows_of(const PackedParams &a, bool skip_empty)
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

// Lane l of a row holds its vectors l + LANES n.
template <int TYPE, int VEC, int LANES, int NV>
__global__ __launch_bounds__(256) void k_pack(const PackedParams a)
{
    const Where w = rows_of<rows_at(LANES)>(a, a.skip_empty);
    if (!w.valid) return;
    constexpr int STEP = 256 / LANES;
    const int l = threadIdx.x % LANES, r = threadIdx.x / LANES, dk = a.p.dk;
    float x[PASSES][NV][VEC];
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int row = r + STEP * i, col = column<VEC>(l + LANES * n, dk);
            const bool on = row < w.rows && col >= 0;
            const float *src = a.states + (w.state + row) * dk + col;
#pragma unroll
            for (int c = 0; c < VEC; ++c) x[i][n][c] = 0.f;
            if (!on) continue;
            if constexpr (VEC == 4) {
                const V16 v = __builtin_nontemporal_load(reinterpret_cast<const V16 *>(src));
#pragma unroll
                for (int c = 0; c < 4; ++c) x[i][n][c] = as_float(v[c]);
            } else {
                x[i][n][0] = src[0];
            }
        }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int row = r + STEP * i;
        uint32_t ex = 0;
        if constexpr (TYPE == CACHE_E4M3) {
            ex = scale_byte_of(reinterpret_cast<const float (&)[NV * VEC]>(x[i]), [](float top) {
#pragma unroll
                for (int o = 1; o < LANES; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
                return top;
            });
            if (row < w.rows && l == 0) a.scale[w.cache + row] = (uint8_t)ex;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = column<VEC>(l + LANES * n, dk);
            if (row >= w.rows || col < 0) continue;
            const size_t at = (w.cache + row) * dk + col;
            if constexpr (TYPE == CACHE_E4M3) {
                if constexpr (VEC == 4) {
                    *reinterpret_cast<V4 *>(static_cast<char *>(a.data) + at) = to_codes(x[i][n], scale_of(ex));
                } else {
                    const float v[4] = {x[i][n][0], 0.f, 0.f, 0.f};
                    static_cast<uint8_t *>(a.data)[at] = (uint8_t)to_codes(v, scale_of(ex));
                }
            } else {
                using T = typename CacheType<TYPE>::T;
                if constexpr (VEC == 4) {
                    const V8 v = {two_halves<T>(x[i][n][0], x[i][n][1]), two_halves<T>(x[i][n][2], x[i][n][3])};
                    *reinterpret_cast<V8 *>(static_cast<T *>(a.data) + at) = v;
                } else {
                    static_cast<T *>(a.data)[at] = from_f32<T>(x[i][n][0]);
                }
            }
        }
    }
}

template <int TYPE, int VEC, int LANES, int NV>
__global__ __launch_bounds__(256) void k_unpack(const PackedParams a)
{
    const Where w = rows_of<rows_at(LANES)>(a, false);
    constexpr int STEP = 256 / LANES;
    const int l = threadIdx.x % LANES, r = threadIdx.x / LANES, dk = a.p.dk;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int row = r + STEP * i;
        if (row >= w.rows) continue;
        const float scale = TYPE == CACHE_E4M3 && w.valid ? scale_of(a.scale[w.cache + row]) : 1.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int col = column<VEC>(l + LANES * n, dk);
            if (col < 0) continue;
            const size_t at = (w.cache + row) * dk + col;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            if (!w.valid) {
                // zeros
            } else if constexpr (TYPE == CACHE_E4M3) {
                if constexpr (VEC == 4) from_codes(*reinterpret_cast<const V4 *>(static_cast<const char *>(a.data) + at), scale, x);
                else from_codes(static_cast<const uint8_t *>(a.data)[at], scale, x);
            } else {
                using T = typename CacheType<TYPE>::T;
                if constexpr (VEC == 4) {
                    const V8 v = *reinterpret_cast<const V8 *>(static_cast<const T *>(a.data) + at);
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[c] = half_of<T>(v[c / 2], c % 2);
                } else {
                    x[0] = to_f32(static_cast<const T *>(a.data)[at]);
                }
            }
            float *dst = a.states + (w.state + row) * dk + col;
            if constexpr (VEC == 4) {
                V16 v;
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = __builtin_bit_cast(uint32_t, x[c]);
                *reinterpret_cast<V16 *>(dst) = v;
            } else {
                dst[0] = x[0];
            }
        }
    }
}

// f with the type, the vectors, the lanes of a row and the vectors of a lane.
template <typename F>
hipError_t by_form(const PackedParams &a, F &&f)
{
    using std::integral_constant;
    using one = integral_constant<int, 1>;
    using four = integral_constant<int, 4>;
    const auto go = [&](auto type) {
        if (a.p.dk < 4) return f(type, one(), integral_constant<int, 8>(), one());
        if (a.p.dk <= 32) return f(type, four(), integral_constant<int, 8>(), one());
        if (a.p.dk <= 64) return f(type, four(), integral_constant<int, 16>(), one());
        if (a.p.dk <= 128) return f(type, four(), integral_constant<int, 32>(), one());
        return f(type, four(), integral_constant<int, 32>(), integral_constant<int, 2>());
    };
    if (a.type == CACHE_F16) return go(integral_constant<int, CACHE_F16>());
    if (a.type == CACHE_BF16) return go(integral_constant<int, CACHE_BF16>());
    return go(integral_constant<int, CACHE_E4M3>());
}

int64_t blocks_of(const PackedParams &a, int rows) { return (int64_t)a.p.B * a.p.HV * ((a.p.dv + rows - 1) / rows); }

}  // namespace

int64_t pack_blocks(int batch, int heads, int dv) { return (int64_t)batch * heads * ((dv + 31) / 32); }

hipError_t launch_pack(const PackedParams &a, hipStream_t s)
{
    if (a.p.B == 0) return hipSuccess;
    return by_form(a, [&](auto type, auto vec, auto lanes, auto nv) {
        hipLaunchKernelGGL((k_pack<decltype(type)::value, decltype(vec)::value, decltype(lanes)::value, decltype(nv)::value>),
                           dim3((unsigned)blocks_of(a, rows_at(lanes()))), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_unpack(const PackedParams &a, hipStream_t s)
{
    if (a.p.B == 0) return hipSuccess;
    return by_form(a, [&](auto type, auto vec, auto lanes, auto nv) {
        hipLaunchKernelGGL((k_unpack<decltype(type)::value, decltype(vec)::value, decltype(lanes)::value, decltype(nv)::value>),
                           dim3((unsigned)blocks_of(a, rows_at(lanes()))), dim3(256), 0, s, a);
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
