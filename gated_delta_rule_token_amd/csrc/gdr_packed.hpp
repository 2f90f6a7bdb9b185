// gdr_packed.hpp -- the state cache's number formats, and the step of the
// recurrence on it: one to a few tokens of each request, the states read from
// the cache, updated in registers and written back rounded.
//
// Formats.  fp16 and bf16 hold a state's values as they are.  With e4m3 a row
// (a value channel's dk keys) has a power of two 2^e of its own, the least with
// max |row| <= 448 2^e, and holds the values over 2^e, rounded to nearest even.
// A power of two costs the rounding nothing (e4m3's steps are relative) and is
// part of gfx950's conversions, so neither scaling is an instruction; it is a
// byte a row.  The rows of a state evolve separately (gdr_device.hpp), so the
// lanes that hold a row form its scale with one more reduction.  e is at least
// -100: rows below 448 2^-100 lose their bits, and a row of zeros has a scale.
// A NaN stays one and an infinity becomes one (e4m3 has none); the rest of the
// row is held as ever.
#pragma once

#include "gdr_packed_launch.hpp"

namespace gdr {

typedef uint32_t w4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef short s2 __attribute__((ext_vector_type(2)));

// By value: __builtin_bit_cast of a vector's element itself reads element 0.
__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }

constexpr uint32_t SCALE_MIN = 27;  // 2^-100

// 2^(byte - 127): the conversions read the exponent's bits alone.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The scale's byte for a row whose largest magnitude is `top`: 448 is 1.75
// 2^8, so a significand above 1.75 carries into the next power.
__device__ __forceinline__ uint32_t scale_byte(float top)
{
    const uint32_t e = (__builtin_bit_cast(uint32_t, top) + 0x1FFFFFu) >> 23;
    return e < SCALE_MIN + 8 ? SCALE_MIN : e - 8;
}

// Four values in one word of codes, and back.
__device__ __forceinline__ void from_codes(uint32_t w, float scale, float *v)
{
    const f2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, false);
    const f2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale, true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
}

__device__ __forceinline__ uint32_t to_codes(const float *v, float scale)
{
    s2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[0], v[1], scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[2], v[3], scale, true);
    return __builtin_bit_cast(uint32_t, w);
}

// The 16-bit types, two values a word.
template <typename T> __device__ __forceinline__ float half_of(uint32_t w, int i)
{
    return to_f32(__builtin_bit_cast(T, (uint16_t)(i ? w >> 16 : w)));
}
template <typename T> __device__ __forceinline__ uint32_t two_halves(float a, float b)
{
    return __builtin_bit_cast(uint16_t, from_f32<T>(a)) | (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(b)) << 16;
}

// Over the LANES (4, 8 or 16) neighbours that hold a row.
template <int LANES, typename Op>
__device__ __forceinline__ float row_reduce(float x, Op op)
{
    x = op(x, dpp_mov<0xB1>(x));                            // lane ^ 1
    x = op(x, dpp_mov<0x4E>(x));                            // lane ^ 2
    if constexpr (LANES > 4) x = op(x, dpp_mov<0x141>(x));  // i <-> 7 - i within 8
    if constexpr (LANES > 8) x = op(x, dpp_mov<0x140>(x));  // i <-> 15 - i within 16
    return x;
}

template <int TYPE> struct CacheType { using T = half_t; };
template <> struct CacheType<CACHE_BF16> { using T = bf16_t; };

// A workgroup (4 waves) holds packed_step_rows(DK) rows of one (request, value
// head) state.  LANES lanes hold a row, 16 values each: with e4m3 16
// neighbouring bytes, with 16 bits 8 values of each half of the row, so that
// every access is a 16-byte vector and a wave's vectors are contiguous.
template <typename TA, int TYPE, int DK, bool VD>
__global__ __launch_bounds__(256) void k_packed_step(const PackedParams a, int rule, int per_key)
{
    constexpr bool EIGHT = TYPE == CACHE_E4M3;
    using TC = typename CacheType<TYPE>::T;
    constexpr int C = 16, LANES = DK / C, RPW = 64 / LANES, G = packed_step_rows(DK) / (4 * RPW), V = EIGHT ? 1 : 2;
    const Params &p = a.p;
    const int parts = (p.dv + packed_step_rows(DK) - 1) / packed_step_rows(DK);
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % p.HV, b = blockIdx.x / (parts * p.HV);
    const int slot = p.slot_ids[b];
    if (slot < 0 || slot >= p.num_slots) return;
    int64_t s, e;
    request_range(p, b, s, e);
    if (e <= s) return;  // the states stay as they are, to the bit
    const int lane = threadIdx.x & 63, l = lane % LANES, r = lane / LANES, wave = threadIdx.x >> 6;
    const int row0 = part * packed_step_rows(DK) + wave * G * RPW + r;  // + RPW for each row group
    const int qh = (int)(((int64_t)h * p.H) / p.HV);
    const bool retrieves = rule_retrieves(rule), decays = rule_decays(rule), rate = rule_has_beta(rule);
    const auto column = [&](int c) { return EIGHT ? l * C + c : (c < 8 ? 0 : DK / 2) + l * 8 + c % 8; };
    const TA *q = static_cast<const TA *>(p.q), *k = static_cast<const TA *>(p.k), *v = static_cast<const TA *>(p.v);
    TA *o = static_cast<TA *>(p.o);

    // Eight neighbouring values of q or k as they lie in memory.
    struct Eight { w4 w[sizeof(TA) / 2]; };
    const auto load8 = [](const TA *src) {
        Eight x;
#pragma unroll
        for (unsigned i = 0; i < sizeof(TA) / 2; ++i) x.w[i] = reinterpret_cast<const w4 *>(src)[i];
        return x;
    };
    const auto get8 = [](const Eight &x, int i) {
        if constexpr (sizeof(TA) == 4) return as_float(x.w[i / 4][i % 4]);
        else return half_of<TA>(x.w[0][i / 2], i % 2);
    };
    Eight qw[2], kw[2];
    float vw[G];
    const auto fetch = [&](int64_t t) {
        const TA *qr = q + (t * p.H + qh) * DK, *kr = k + (t * p.H + qh) * DK;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            qw[n] = load8(qr + column(8 * n));
            kw[n] = load8(kr + column(8 * n));
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int row = row0 + g * RPW;
            vw[g] = to_f32(v[(t * p.HV + h) * p.dv + (row < p.dv ? row : p.dv - 1)]);
        }
    };
    fetch(s);

    const size_t head = ((size_t)slot * p.HV + h) * p.dv;
    w4 raw[G][V];
    uint32_t ex[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int row = row0 + g * RPW, at = row < p.dv ? row : p.dv - 1;
        const char *src = static_cast<const char *>(a.data) + (head + at) * DK * (EIGHT ? 1 : 2) + l * 16;
#pragma unroll
        for (int n = 0; n < V; ++n) raw[g][n] = __builtin_nontemporal_load(reinterpret_cast<const w4 *>(src + n * DK));
        ex[g] = EIGHT ? a.scale[head + at] : 0;
    }
    float S[G][C];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if constexpr (EIGHT) {
#pragma unroll
            for (int n = 0; n < 4; ++n) from_codes(raw[g][0][n], scale_of(ex[g]), &S[g][4 * n]);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) S[g][c] = half_of<TC>(raw[g][c / 8][c % 8 / 2], c % 2);
        }
    }

    for (int64_t t = s; t < e; ++t) {
        const size_t th = (size_t)t * p.HV + h;
        float qv[C], kv[C], vi[G], qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            qv[c] = get8(qw[c / 8], c % 8);
            kv[c] = get8(kw[c / 8], c % 8);
            qq = fmaf(qv[c], qv[c], qq);
            kk = fmaf(kv[c], kv[c], kk);
            qk = fmaf(qv[c], kv[c], qk);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) vi[g] = vw[g];
        if (t + 1 < e) fetch(t + 1);
        const auto add = [](float x, float y) { return x + y; };
        qk = row_reduce<LANES>(qk, add);
        if (p.qk_l2_norm) {
            const float inq = 1.f / sqrtf(row_reduce<LANES>(qq, add) + 1e-12f);
            const float ink = 1.f / sqrtf(row_reduce<LANES>(kk, add) + 1e-12f);
            qk *= inq * ink;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                qv[c] *= inq;
                kv[c] *= ink;
            }
        }
        float alpha = 1.f, av[C], kb[C];  // decay: one, or for each key
        if (decays && !per_key) alpha = expf(log_decay(p, th, h));
        const float bt = rate ? update_rate(p, th) : 1.f;
        if constexpr (VD) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                av[c] = per_key ? expf(log_decay_key(p, th, h, column(c))) : alpha;
                kb[c] = av[c] * kv[c] * (p.erase ? p.erase[th * DK + column(c)] : 1.f);
                qv[c] *= av[c];
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float get = 0.f, u = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                get = fmaf(S[g][c], VD ? kb[c] : kv[c], get);
                u = fmaf(S[g][c], qv[c], u);
            }
            get = row_reduce<LANES>(get, add);
            u = row_reduce<LANES>(u, add);
            if constexpr (!VD) {
                get *= alpha;
                u *= alpha;
            }
            const float put = retrieves ? bt * (vi[g] - get) : vi[g];
#pragma unroll
            for (int c = 0; c < C; ++c) S[g][c] = fmaf(VD ? av[c] : alpha, S[g][c], put * kv[c]);
            const int row = row0 + g * RPW;
            if (l == 0 && row < p.dv) o[th * p.dv + row] = from_f32<TA>(p.scale * (u + qk * put));
        }
    }

#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int row = row0 + g * RPW;
        if constexpr (EIGHT) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) top = fmaxf(top, fabsf(S[g][c]));
            top = row_reduce<LANES>(top, [](float x, float y) { return fmaxf(x, y); });
            ex[g] = scale_byte(top);
#pragma unroll
            for (int n = 0; n < 4; ++n) raw[g][0][n] = to_codes(&S[g][4 * n], scale_of(ex[g]));
        } else {
#pragma unroll
            for (int c = 0; c < C; c += 2) raw[g][c / 8][c % 8 / 2] = two_halves<TC>(S[g][c], S[g][c + 1]);
        }
        if (row >= p.dv) continue;
        char *dst = static_cast<char *>(a.data) + (head + row) * DK * (EIGHT ? 1 : 2) + l * 16;
#pragma unroll
        for (int n = 0; n < V; ++n) __builtin_nontemporal_store(raw[g][n], reinterpret_cast<w4 *>(dst + n * DK));
        if (EIGHT && l == 0) a.scale[head + row] = (uint8_t)ex[g];
    }
}

template <typename TA, int TYPE, int DK>
hipError_t packed_step_at(const PackedParams &a, int rule, bool per_key, hipStream_t s)
{
    const int64_t blocks = (int64_t)a.p.B * a.p.HV * ((a.p.dv + packed_step_rows(DK) - 1) / packed_step_rows(DK));
    const dim3 grid((unsigned)blocks), threads(256);
    if (per_key || rule == GATED_DELTA_V2)
        hipLaunchKernelGGL((k_packed_step<TA, TYPE, DK, true>), grid, threads, 0, s, a, rule, (int)per_key);
    else
        hipLaunchKernelGGL((k_packed_step<TA, TYPE, DK, false>), grid, threads, 0, s, a, rule, 0);
    return hipGetLastError();
}

template <typename TA, int TYPE>
hipError_t packed_step_by_dk(const PackedParams &a, int rule, bool per_key, hipStream_t s)
{
    if (a.p.dk == 64) return packed_step_at<TA, TYPE, 64>(a, rule, per_key, s);
    if (a.p.dk == 128) return packed_step_at<TA, TYPE, 128>(a, rule, per_key, s);
    return packed_step_at<TA, TYPE, 256>(a, rule, per_key, s);
}

template <int TYPE>
hipError_t packed_step_typed(const PackedParams &a, int rule, bool per_key, int act, hipStream_t s)
{
    if (act == 1) return packed_step_by_dk<half_t, TYPE>(a, rule, per_key, s);
    if (act == 2) return packed_step_by_dk<bf16_t, TYPE>(a, rule, per_key, s);
    return packed_step_by_dk<float, TYPE>(a, rule, per_key, s);
}

}  // namespace gdr
