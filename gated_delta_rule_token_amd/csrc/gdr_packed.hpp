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
// A NaN stays one and an infinity becomes one (e4m3 has none); neither counts in
// the largest value, so the rest of the row is held as ever.
#pragma once

#include "gdr_packed_launch.hpp"

#include <type_traits>
#include <utility>

namespace gdr {

typedef uint32_t w4 __attribute__((ext_vector_type(4)));
typedef uint32_t Any4 __attribute__((ext_vector_type(4), aligned(1)));  // 16 bytes from any address
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

// The same for a lane's part of a row; reduce: the largest over the row's lanes.  An
// infinite largest value, which would leave the others no bits, is formed again of
// the finite ones (fmaxf leaves NaN out by itself).
template <int N, typename Reduce>
__device__ __forceinline__ uint32_t scale_byte_of(const float (&v)[N], Reduce reduce)
{
    constexpr float INF = __builtin_inff();
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(v[i]));
    top = reduce(top);
    if (top == INF) {
        top = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(v[i]) < INF ? fabsf(v[i]) : 0.f);
        top = reduce(top);
    }
    return scale_byte(top);
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

// Over the LANES (1, 4, 8 or 16) neighbours that hold a row.
template <int LANES, typename Op>
__device__ __forceinline__ float row_reduce(float x, Op op)
{
    if constexpr (LANES > 1) x = op(x, dpp_mov<0xB1>(x));   // lane ^ 1
    if constexpr (LANES > 1) x = op(x, dpp_mov<0x4E>(x));   // lane ^ 2
    if constexpr (LANES > 4) x = op(x, dpp_mov<0x141>(x));  // i <-> 7 - i within 8
    if constexpr (LANES > 8) x = op(x, dpp_mov<0x140>(x));  // i <-> 15 - i within 16
    return x;
}

template <int TYPE> struct CacheType { using T = half_t; };
template <> struct CacheType<CACHE_BF16> { using T = bf16_t; };

// ---------------------------------------------------------------- any tokens, on the vector units
// LANES lanes hold a row, 16 values each: with e4m3 16 neighbouring bytes, with
// 16 bits 8 values of each half of the row, so that every access is a 16-byte
// vector and a wave's vectors are contiguous.  To 16 keys that is a lane a row
// (142 requests x 32 heads of 15 by 256 in 8 bits 49 us; 117 in the form of 64
// keys).  A wave holds G times 64 / LANES rows.  With single tokens (ONE) each row
// group is widened, stepped and rounded by itself, so few registers are live beside
// the packed values; more tokens keep all groups in fp32 between them.
// Bound by memory for single tokens (256 requests x 32 heads of 128): 8 bits 57
// to 60 us for 277 MB, 16 bits 97 us for 543 MB, fp32 activations the same.  Waves
// and rows, in us for 8 and 16 bits: 2 waves of 64 rows 60 and 109, 4 of 32 rows 63
// and 104, 4 of 16 rows 73 and 96; as the form for more tokens 68 and 102.
template <int TYPE, int DK, bool ONE> struct StepForm {
    static constexpr bool EIGHT = TYPE == CACHE_E4M3;
    static constexpr int WAVES = DK == 16 ? 1 : ONE && EIGHT ? 2 : 4;
    static constexpr int ROWS = DK == 128 && (EIGHT || !ONE) ? 128 : 64;  // of a workgroup
};

// EXACT: p.dk is DK; else it is less, and a lane's vector that would pass the
// row's end starts earlier: the columns that it then shares with another lane
// count in that lane's sums only, and both write the same bytes.  Such rows share
// cache lines, which plain accesses keep for their next use (without: 256
// requests x 32 heads of 56, 63 and 150 in 16 bits 37, 49 and 189 us instead of
// 30, 40 and 167).  Rows of under 16 values have a lane each, which takes them
// value by value.
// Requests of fewer than `least` tokens are left alone.
template <typename TA, int TYPE, int DK, bool VD, bool ONE, bool EXACT>
__global__ __launch_bounds__((64 * StepForm<TYPE, DK, ONE>::WAVES)) void k_packed_step(const PackedParams a, int rule,
                                                                                       int per_key, int least)
{
    using Form = StepForm<TYPE, DK, ONE>;
    constexpr bool EIGHT = TYPE == CACHE_E4M3;
    using TC = typename CacheType<TYPE>::T;
    constexpr int C = 16, LANES = DK / C, RPW = 64 / LANES, G = Form::ROWS / (Form::WAVES * RPW), V = EIGHT ? 1 : 2;
    constexpr int VC = EIGHT ? 16 : 8;  // values of a vector
    const Params &p = a.p;
    const int dk = EXACT ? DK : p.dk, ROW = dk * (EIGHT ? 1 : 2);  // values and bytes of a row
    const int parts = (p.dv + Form::ROWS - 1) / Form::ROWS;
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % p.HV, b = blockIdx.x / (parts * p.HV);
    const int slot = p.slot_ids[b];
    if (slot < 0 || slot >= p.num_slots) return;
    int64_t s, e;
    request_range(p, b, s, e);
    if (e - s < least) return;  // without tokens the states stay as they are, to the bit
    const int lane = threadIdx.x & 63, l = lane % LANES, r = lane / LANES, wave = threadIdx.x >> 6;
    const int row0 = part * Form::ROWS + wave * G * RPW + r;  // + RPW for each row group
    const int qh = (int)(((int64_t)h * p.H) / p.HV);
    const bool retrieves = rule_retrieves(rule), decays = rule_decays(rule), rate = rule_has_beta(rule);
    // this lane's vectors: the first column, and how many of the columns are another lane's
    constexpr bool narrow = !EXACT && DK == 16;
    int at[V], others[V];
#pragma unroll
    for (int n = 0; n < V; ++n) {
        const int want = n * (DK / 2) + l * VC;
        at[n] = EXACT || narrow || want + VC <= dk ? want : dk - VC;
        others[n] = EXACT ? 0 : want - at[n];
    }
    const auto column = [&](int c) { return at[c / VC] + c % VC; };
    const auto own = [&](int c) { return EXACT || (narrow ? column(c) < dk : c % VC >= others[c / VC]); };
    const auto add = [](float x, float y) { return x + y; };
    const TA *q = static_cast<const TA *>(p.q), *k = static_cast<const TA *>(p.k), *v = static_cast<const TA *>(p.v);
    TA *o = static_cast<TA *>(p.o);

    // Eight neighbouring values of q or k as they lie in memory.
    struct Eight { w4 w[sizeof(TA) / 2]; };
    const auto load8 = [&](const TA *row, int col) {
        Eight x;
        if constexpr (narrow) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const TA v = col + i < dk ? row[col + i] : from_f32<TA>(0.f);
                if constexpr (sizeof(TA) == 4) x.w[i / 4][i % 4] = __builtin_bit_cast(uint32_t, v);
                else x.w[0][i / 2] = (i % 2 ? x.w[0][i / 2] : 0) | (uint32_t)__builtin_bit_cast(uint16_t, v) << (16 * (i % 2));
            }
        } else {
#pragma unroll
            for (unsigned i = 0; i < sizeof(TA) / 2; ++i) x.w[i] = reinterpret_cast<const Any4 *>(row + col)[i];
        }
        return x;
    };
    const auto get8 = [](const Eight &x, int i) {
        if constexpr (sizeof(TA) == 4) return as_float(x.w[i / 4][i % 4]);
        else return half_of<TA>(x.w[0][i / 2], i % 2);
    };
    Eight qw[2], kw[2];
    float vw[G];
    const auto fetch = [&](int64_t t) {
        const TA *qr = q + (t * p.H + qh) * dk, *kr = k + (t * p.H + qh) * dk;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            qw[n] = load8(qr, column(8 * n));
            kw[n] = load8(kr, column(8 * n));
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int row = row0 + g * RPW;
            vw[g] = to_f32(v[(t * p.HV + h) * p.dv + (row < p.dv ? row : p.dv - 1)]);
        }
    };
    fetch(s);  // before the states, so that waiting for it does not wait for them

    const size_t head = ((size_t)slot * p.HV + h) * p.dv;
    w4 raw[G][V];
    uint32_t ex[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int row = row0 + g * RPW, from = row < p.dv ? row : p.dv - 1;
        const char *src = static_cast<const char *>(a.data) + (head + from) * ROW;
#pragma unroll
        for (int n = 0; n < V; ++n) {
            if constexpr (narrow) {
                using Code = typename std::conditional<EIGHT, uint8_t, uint16_t>::type;
                constexpr int PER = 4 / sizeof(Code);  // values of a word
#pragma unroll
                for (int i = 0; i < VC; ++i) {
                    const uint32_t v = at[n] + i < dk ? reinterpret_cast<const Code *>(src)[at[n] + i] : 0;
                    raw[g][n][i / PER] = (i % PER ? raw[g][n][i / PER] : 0) | v << (32 / PER * (i % PER));
                }
            } else {
                const Any4 *from = reinterpret_cast<const Any4 *>(src + at[n] * (16 / VC));
                if constexpr (EXACT) raw[g][n] = __builtin_nontemporal_load(from);
                else raw[g][n] = *from;
            }
        }
        ex[g] = EIGHT ? a.scale[head + from] : 0;
    }
    const auto widen = [&](int g, float (&S)[C]) {
        if constexpr (EIGHT) {
#pragma unroll
            for (int n = 0; n < 4; ++n) from_codes(raw[g][0][n], scale_of(ex[g]), &S[4 * n]);
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) S[c] = half_of<TC>(raw[g][c / 8][c % 8 / 2], c % 2);
        }
    };
    const auto put_back = [&](int g, const float (&S)[C]) {
        const int row = row0 + g * RPW;
        w4 out[V];
        uint32_t eo = 0;
        if constexpr (EIGHT) {
            eo = scale_byte_of(S, [](float top) { return row_reduce<LANES>(top, [](float x, float y) { return fmaxf(x, y); }); });
#pragma unroll
            for (int n = 0; n < 4; ++n) out[0][n] = to_codes(&S[4 * n], scale_of(eo));
        } else {
#pragma unroll
            for (int c = 0; c < C; c += 2) out[c / 8][c % 8 / 2] = two_halves<TC>(S[c], S[c + 1]);
        }
        if (row >= p.dv) return;
        char *dst = static_cast<char *>(a.data) + (head + row) * ROW;
#pragma unroll
        for (int n = 0; n < V; ++n) {
            if constexpr (narrow) {
                using Code = typename std::conditional<EIGHT, uint8_t, uint16_t>::type;
                constexpr int PER = 4 / sizeof(Code);
#pragma unroll
                for (int i = 0; i < VC; ++i)
                    if (at[n] + i < dk) reinterpret_cast<Code *>(dst)[at[n] + i] = (Code)(out[n][i / PER] >> (32 / PER * (i % PER)));
            } else if (EXACT || others[n] < VC) {
                Any4 *to = reinterpret_cast<Any4 *>(dst + at[n] * (16 / VC));
                if constexpr (EXACT) __builtin_nontemporal_store(out[n], to);
                else *to = out[n];
            }
        }
        if (EIGHT && l == 0) a.scale[head + row] = (uint8_t)eo;
    };

    // A decay for each key or the erase gate: the workgroup forms a token's
    // factors once, for all its rows, a token ahead of their use.  (Formed by the
    // lanes for themselves, 256 requests x 32 heads of 128 on 16-bit states took
    // 316 us for a token and 830 for four.)
    __shared__ __align__(16) float s_decay[VD ? 2 : 1][VD ? DK : 1], s_erase[VD ? 2 : 1][VD ? DK : 1];
    const auto stage = [&](int64_t t) {
        const size_t th = (size_t)t * p.HV + h;
        for (int j = threadIdx.x; j < dk; j += 64 * Form::WAVES) {
            s_decay[(t - s) & 1][j] = expf(per_key ? log_decay_key(p, th, h, j) : decays ? log_decay(p, th, h) : 0.f);
            s_erase[(t - s) & 1][j] = p.erase ? p.erase[th * dk + j] : 1.f;
        }
    };
    // One token: its vectors and scalars, then each row group's step.
    float qv[C], kv[C], av[C], kb[C], vi[G], qk, alpha, bt;  // qv and kb: for dots
    const auto token = [&](int64_t t) {
        const size_t th = (size_t)t * p.HV + h;
        float qq = 0.f, kk = 0.f;
        qk = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float qc = get8(qw[c / 8], c % 8);
            kv[c] = get8(kw[c / 8], c % 8);
            qv[c] = own(c) ? qc : 0.f;
            kb[c] = own(c) ? kv[c] : 0.f;
            qq = fmaf(qv[c], qv[c], qq);
            kk = fmaf(kb[c], kb[c], kk);
            qk = fmaf(qv[c], kb[c], qk);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) vi[g] = vw[g];
        if (!ONE && t + 1 < e) fetch(t + 1);
        qk = row_reduce<LANES>(qk, add);
        if (p.qk_l2_norm) {
            const float inq = 1.f / sqrtf(row_reduce<LANES>(qq, add) + 1e-12f);
            const float ink = 1.f / sqrtf(row_reduce<LANES>(kk, add) + 1e-12f);
            qk *= inq * ink;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                qv[c] *= inq;
                kv[c] *= ink;
                kb[c] *= ink;
            }
        }
        alpha = !VD && decays ? expf(log_decay(p, th, h)) : 1.f;
        bt = rate ? update_rate(p, th) : 1.f;
        if constexpr (VD) {
            lds_barrier();
            if (!ONE && t + 1 < e) stage(t + 1);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int j = EXACT || column(c) < dk ? column(c) : 0;
                av[c] = s_decay[(t - s) & 1][j];
                kb[c] = av[c] * kb[c] * s_erase[(t - s) & 1][j];
                qv[c] *= av[c];
            }
        }
    };
    const auto step = [&](int64_t t, int g, float (&S)[C]) {
        float get = 0.f, u = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            get = fmaf(S[c], kb[c], get);
            u = fmaf(S[c], qv[c], u);
        }
        get = row_reduce<LANES>(get, add);
        u = row_reduce<LANES>(u, add);
        if constexpr (!VD) {
            get *= alpha;
            u *= alpha;
        }
        const float put = retrieves ? bt * (vi[g] - get) : vi[g];
#pragma unroll
        for (int c = 0; c < C; ++c) S[c] = fmaf(VD ? av[c] : alpha, S[c], put * kv[c]);
        const int row = row0 + g * RPW;
        if (l == 0 && row < p.dv) o[((size_t)t * p.HV + h) * p.dv + row] = from_f32<TA>(p.scale * (u + qk * put));
    };
    if constexpr (VD) stage(s);
    if constexpr (ONE) {
        token(s);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float S[C];
            widen(g, S);
            step(s, g, S);
            put_back(g, S);
        }
    } else {
        float S[G][C];
#pragma unroll
        for (int g = 0; g < G; ++g) widen(g, S[g]);
        for (int64_t t = s; t < e; ++t) {
            token(t);
#pragma unroll
            for (int g = 0; g < G; ++g) step(t, g, S[g]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) put_back(g, S[g]);
    }
}

// ---------------------------------------------------------------- 1 to 8 tokens, on the matrix cores
// A request's tokens together.  First for 16-bit activations and one decay a head.
// With S the packed states, x_n the vectors k_0 .. k_7, q_0 .. q_7 and
// a_t the decays, per row
//   z_n = S . x_n for all 16 n                         (matrix product)
//   for each token t:  z <- a_t z,  d_t = beta_t (v_t - z_t),  z <- z + d_t (k_t . x_n)
// so that z_n is at every step the dot of x_n with the state of the moment, d_t
// the new value that token t writes, and z of q_t after step t its output; then
//   S <- (prod a) S + sum_t (prod of the later a) d_t k_t       (matrix product)
// (the norms of q and k are factors of z and d).  So the states are read once
// from registers, whatever the number of tokens: on the vector units each
// token takes 3 operations a value, which at 4 tokens is 1.5 times the memory's
// time.  256 requests x 32 heads of 128, vector units and this, in us: 16 bits
// 2 tokens 115 and 104, 4 tokens 157 and 108 (562 MB), 7 tokens 237 and 116;
// 8 bits, 4 tokens 143 and 76; 64 requests x 32 heads of 256, 4 tokens, 159 and 116
// in 16 bits, 146 and 68 in 8; but single tokens 60 and 67 in 8 bits, 96 and 102
// in 16, which the vector units take where every request has one.
//
// Operands.  The states are an operand as they are: 16-bit values, or codes
// as fp16 or bf16 (either holds every code), with the row's scale a factor of
// z.  Vectors of the other 16-bit type go in as two planes, exact for fp16 in
// bf16; bf16 in fp16 is scaled by a power of two that brings the largest to
// [2^14, 2^15), where two planes hold 2^-39 of it.  d (fp32) goes into the
// second product as three bf16 planes, all 24 bits: where a token replaces values,
// d k takes away what is there, and what it is off by stays (with two planes, under
// 2^-17, values 2^12 times smaller than those before them were off by several of fp16's
// steps).  An fp16 k takes two planes.  The 32 inner places of a product hold 8 tokens of
// four plane pairs: one product beside a bf16 k, two beside others, of which the second,
// of the small pairs, has the same operand k (fp16 activations, 4 tokens: 117 us on
// 16 bits with and without it, 84 and 87 on 8).
//
// Any other call (GEN: fp32 activations, a decay for each key, the erase gate)
// takes the decays into the vectors.  With D_t the product of the decays up to
// token t (a vector over the keys), x_n is D_n o e_n o k_n and D_n o q_n, token
// t's write enters a later x_n's dot by sum_j k_t (D_n / D_t) e_n k_n, and S by
// d_t (D_T / D_t) o k_t: a lane forms these for its two keys, the quotients as
// running products of the later decays, which do not overflow.  x_n in fp32 goes
// in as planes (two of fp16 scaled as above, 2^-22 of its largest value; a third
// would take 32 registers of 256 keys; three of bf16 beside a bf16 cache), k_t and
// d_t as three of bf16 each.  256 requests x 32 heads of 128, 4 tokens, vector
// units and this, in us: a decay for each key on 16 and 8 bits 229 and 118, 210 and
// 96; fp32 activations 211 and 112, 205 and 90; 64 requests x 32 heads of 256, a
// decay for each key, 243 and 123, 224 and 79.  8 bits wait for the vectors' own
// work: 7 tokens take 119 us, 53 of them with 16 rows a state.
//
// A tile is 16 rows: lane (c, kb) of a wave holds row c, 8 keys of every 32 (with
// codes 16 of 64) at the kb-th place, which is the first product's operand; the
// second product is transposed (keys by rows), with the keys in the order that
// gives each lane the values it holds.  So a row's 64-byte pieces lie with 4
// lanes; whole 128-byte lines come from loading an even and an odd row's line
// with 8 lanes each and exchanging pieces between lanes c and c ^ 1 (without it
// 4 tokens on 16 bits take 129 us).
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float Any4f __attribute__((ext_vector_type(4), aligned(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

// Lane N's value, in each 16 neighbours.
template <int N> __device__ __forceinline__ float lane_of(float x) { return dpp_mov<0x150 + N>(x); }

__device__ __forceinline__ f4v mfma(h8 a, h8 b, f4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4v mfma(b8 a, b8 b, f4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
template <typename T> struct Vec8 { using V = h8; };
template <> struct Vec8<bf16_t> { using V = b8; };

// Sixteen values over a wave: lane (c, any) gets the c-th.  At each step a lane
// keeps half of its values, those that its place in 16 names, and gives its
// partner the others: 45 operations where 16 reductions take 128.
template <int N, int CTRL, typename Op> __device__ __forceinline__ void fold(float (&v)[16], bool upper, Op op)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float keep = upper ? v[N + i] : v[i], give = upper ? v[i] : v[N + i];
        v[i] = op(keep, dpp_mov<CTRL>(give));
    }
}

template <typename Op> __device__ __forceinline__ float sixteen(float (&v)[16], int c, Op op)
{
    fold<8, 0x128>(v, c & 8, op);  // c ^ 8
    fold<4, 0x141>(v, c & 4, op);  // i <-> 7 - i within 8
    fold<2, 0x4E>(v, c & 2, op);   // c ^ 2
    fold<1, 0xB1>(v, c & 1, op);   // c ^ 1
    float x = v[0];
    x = op(x, __shfl_xor(x, 16));
    return op(x, __shfl_xor(x, 32));
}

// The power of two that brings `top` to [2^14, 2^15), and its inverse.
__device__ __forceinline__ void half_scale(float top, float &up, float &back)
{
    int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127 - 14;
    e = top > 0.f ? (e < -120 ? -120 : e > 120 ? 120 : e) : 0;
    up = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
    back = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}

// Planes of 8 bits: the upper half of an fp32 value is a bf16, what lies below it is
// exact, and so three planes hold all 24 bits.  below: x without its bits in `mask`
// (UPPER; 0: x; all: 0; NaN and infinities give NaN); uppers: two upper halves in a word.
constexpr uint32_t UPPER = 0xFFFF0000u;
__device__ __forceinline__ float below(float x, uint32_t mask) { return x - as_float(__builtin_bit_cast(uint32_t, x) & mask); }
__device__ __forceinline__ uint32_t uppers(float a, float b)
{
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302);
}

// Orders a wave's own LDS accesses: writes of other lanes before it, reads after.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename F, int... I> __device__ __forceinline__ void each(F &&f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}

// Own row's two 64-byte pieces (of 16 bytes a lane) from the lines of an even
// and of an odd row, and back: lanes c and c ^ 1 exchange one vector.
__device__ __forceinline__ void exchange(w4 &x, w4 &y, bool odd)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(odd ? x[i] : y[i]), 0xB1, 0xF, 0xF, false);
        x[i] = odd ? got : x[i];
        y[i] = odd ? y[i] : got;
    }
}

// A wave takes the tiles of 16 rows wave, wave + `waves`, ... of one state, by
// itself (its LDS is its own), the next PRE of them on their way.  (At least two
// waves a SIMD asked for: with one, products would accumulate in registers that
// the vector units do not reach, 64 moves a tile.)
// EXACT: p.dk is DK; else (GEN) it is over 16 and less, and a lane's 16 bytes of a
// row that would pass its end start earlier: keys that they share with another
// lane's count there in the dots (x is 0 here), and both write the same bytes, by
// plain accesses as above.  256 requests x 32 heads, 2 and 4 tokens, vector units
// and this, in us: heads of 56 in 16 bits 71, 111 and 31, 36, in 8 bits 55, 88 and
// 32, 37; of 96 in 16 bits 128, 202 and 82, 90; of 150 361, 589 and 188, 202; of
// 224 513, 840 and 387, 430.  (Of 255 in 16 bits, odd rows across each other's
// lines, 622, 941 and 820, 895: behind at 2 tokens, ahead from 4.)
template <typename TA, int TYPE, int DK, int PRE, bool GEN, bool EXACT>
__global__ __launch_bounds__(256, 2) void k_packed_few(const PackedParams a, int rule, int per_key, int waves)
{
    constexpr bool EIGHT = TYPE == CACHE_E4M3, BF = !GEN && std::is_same<TA, bf16_t>::value;
    constexpr int KS = DK / 32, NV = EIGHT ? KS / 2 : KS, T = 8;
    constexpr bool LINES = EXACT && NV > 1;
    // type of the dots' operands, and planes of x
    using TE = typename std::conditional<GEN, half_t, TA>::type;
    using TC = typename std::conditional<EIGHT, TE, typename CacheType<TYPE>::T>::type;
    constexpr bool CB = std::is_same<TC, bf16_t>::value, SAME = !GEN && std::is_same<TC, TA>::value;
    constexpr int PX = GEN ? (CB ? 3 : 2) : SAME ? 1 : 2, PK = GEN ? 3 : BF ? 1 : 2;
    using VA = typename Vec8<TA>::V;
    using VC = typename Vec8<TC>::V;
    // a wave's k by keys (and before it, where x does not come from memory, x)
    constexpr int K_BYTES = PK * DK * T * 2, XR = DK + 8, X_BYTES = GEN ? PX * 16 * XR * 2 : 0;  // (rows of x in different banks)
    __shared__ __align__(16) char s_kx4[4][K_BYTES > X_BYTES ? K_BYTES : X_BYTES];
    __shared__ __align__(16) float s_d4[4][T][16], s_all4[4][GEN ? DK : 4];
    const Params &p = a.p;
    const int dk = EXACT ? DK : p.dk, ROW = dk * (EIGHT ? 1 : 2);  // values and bytes of a row
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), gw = blockIdx.x * 4 + wid;
    const int bh = gw / waves, wave = gw - bh * waves;
    if (bh >= p.B * p.HV) return;
    const int b = bh / p.HV, h = bh - b * p.HV;
    auto &s_k = *reinterpret_cast<bf16_t (*)[PK][DK][T]>(s_kx4[wid]);
    auto &s_x = *reinterpret_cast<TC (*)[PX][16][XR]>(s_kx4[wid]);
    auto &s_d = s_d4[wid];
    auto &s_all = s_all4[wid];
    const int slot = p.slot_ids[b];
    if (slot < 0 || slot >= p.num_slots) return;
    int64_t s, e;
    request_range(p, b, s, e);
    if (e <= s || e - s > T) return;
    const int n = (int)(e - s);
    const int lane = threadIdx.x & 63, c = lane & 15, kb = lane >> 4;
    const int tiles = (p.dv + 15) / 16;
    const int qh = (int)(((int64_t)h * p.H) / p.HV);
    constexpr int VK = EIGHT ? 16 : 8;  // keys of 16 bytes
    const auto wanted = [](int m, int kb) { return m * 4 * VK + kb * VK; };
    const auto piece = [&](int m, int kb) {
        const int at = wanted(m, kb);
        return EXACT || at + VK <= dk ? at : dk - VK;
    };
    const auto key = [&](int f, int kb) { return EIGHT ? piece(f / 2, kb) + 8 * (f % 2) : piece(f, kb); };

    // vector c: k of token c, q of token c - 8
    const int own = c & 7, tt = own < n ? own : n - 1;
    const size_t th = (size_t)(s + tt) * p.HV + h;
    w4 xr[KS];
    if constexpr (!GEN) {
        const TA *x = static_cast<const TA *>(c < 8 ? p.k : p.q) + ((size_t)(s + tt) * p.H + qh) * DK;
#pragma unroll
        for (int f = 0; f < KS; ++f) xr[f] = *reinterpret_cast<const w4 *>(x + key(f, kb));
    }
    const size_t head = ((size_t)slot * p.HV + h) * p.dv;
    char *const mat = static_cast<char *>(a.data) + head * ROW;
    uint8_t *const scales = EIGHT ? a.scale + head : nullptr;
    const TA *const vv = static_cast<const TA *>(p.v) + th * p.dv;
    w4 raw[PRE][NV];
    uint32_t ex[PRE], exr[PRE][4];
    TA vr[PRE][4];
    const auto fetch = [&](int j, int tile) {
        if (tile >= tiles) return;
        const int row = 16 * tile + c, at = row < p.dv ? row : p.dv - 1;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            if constexpr (EXACT) {
                const int r = LINES ? 16 * tile + (c & ~1) + m % 2 : row, rr = r < p.dv ? r : p.dv - 1;
                raw[j][m] = __builtin_nontemporal_load(reinterpret_cast<const w4 *>(mat + rr * ROW + m / 2 * 128 + (LINES ? (c & 1) * 64 : 0) + kb * 16));
            } else {
                raw[j][m] = *reinterpret_cast<const Any4 *>(mat + at * ROW + piece(m, kb) * (16 / VK));
            }
        }
        if (EIGHT) ex[j] = scales[at];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int r = 16 * tile + 4 * kb + m, rr = r < p.dv ? r : p.dv - 1;
            if (EIGHT) exr[j][m] = scales[rr];
            vr[j][m] = vv[rr];
        }
    };
#pragma unroll
    for (int j = 0; j < PRE; ++j) fetch(j, wave + j * waves);
    const bool decays = rule_decays(rule), retrieves = rule_retrieves(rule);
    const float beta = rule_has_beta(rule) ? update_rate(p, th) : 1.f;
    // x as operands; what z, d and the states are multiplied by
    VC y[PX][KS];
    float back = 1.f, al[T], cl[T], put[T], all = 1.f, oscale = p.scale, binv = retrieves ? beta : 0.f;
    s_d[lane / 16][lane % 16] = 0.f;
    s_d[4 + lane / 16][lane % 16] = 0.f;

    if constexpr (GEN) {
        // Lane: keys KL lane + m.  With D_t the product of the decays up to token t,
        // x_n is D_n o (e_n o k_n), D_n o q_n, and the rest is relative to a token.
        constexpr int KL = DK / 64;
        const auto plus = [](float x, float y) { return x + y; };
        const int j0 = KL * lane;
        // every token's values as they lie in memory, none waited for before the last is asked for
        using Bits = typename std::conditional<sizeof(TA) == 4, uint32_t, uint16_t>::type;
        const auto value = [](uint32_t x) {
            if constexpr (sizeof(TA) == 4) return as_float(x);
            else return to_f32(__builtin_bit_cast(TA, (uint16_t)x));
        };
        const bool wide_gate = p.gate_dt == 0;
        uint32_t kw[T][KL], qw[T][KL], gw_[T][KL], ew[T][KL];
        each([&](auto t_) {
            constexpr int t = decltype(t_)::value;
            if (t < n) {
                const size_t tq = ((size_t)(s + t) * p.H + qh) * dk + j0, tv = ((size_t)(s + t) * p.HV + h) * dk + j0;
#pragma unroll
                for (int m = 0; m < KL; ++m) {
                    kw[t][m] = qw[t][m] = gw_[t][m] = ew[t][m] = 0;  // past the row's end
                    if (!EXACT && j0 + m >= dk) continue;
                    kw[t][m] = static_cast<const Bits *>(p.k)[tq + m];
                    qw[t][m] = static_cast<const Bits *>(p.q)[tq + m];
                    if (per_key) gw_[t][m] = wide_gate ? static_cast<const uint32_t *>(p.gate)[tv + m] : static_cast<const Bits *>(p.gate)[tv + m];
                    if (p.erase) ew[t][m] = reinterpret_cast<const uint32_t *>(p.erase)[tv + m];
                }
            }
        }, std::make_integer_sequence<int, T>());
        const bool raw_gate = per_key && p.gate_qwen;
        float bias[KL];
#pragma unroll
        for (int m = 0; m < KL; ++m) bias[m] = raw_gate && (EXACT || j0 + m < dk) ? p.dt_bias[(size_t)h * dk + j0 + m] : 0.f;
        const float slope = raw_gate ? gate_scale(p, h) : 1.f;
        const float alpha = decays && !per_key ? expf(log_decay(p, th, h)) : 1.f;  // of vector c's token
        float kv[T][KL], rv[T][KL], qv[T][KL], av[T][KL], norm[16];
        each([&](auto t_) {
            constexpr int t = decltype(t_)::value;
            norm[t] = norm[8 + t] = 0.f;
            if (t < n) {
                const float at = lane_of<t>(alpha);
#pragma unroll
                for (int m = 0; m < KL; ++m) {
                    kv[t][m] = value(kw[t][m]);
                    qv[t][m] = value(qw[t][m]);
                    av[t][m] = at;
                    if (per_key && (EXACT || j0 + m < dk)) {  // (past the row's end a decay of 1: no 0 x infinity)
                        const float x = wide_gate ? as_float(gw_[t][m]) : value(gw_[t][m]);
                        av[t][m] = expf(raw_gate ? slope * softplus_f32(x + bias[m]) : x);
                    }
                    rv[t][m] = p.erase ? as_float(ew[t][m]) : 1.f;
                    norm[t] = fmaf(kv[t][m], kv[t][m], norm[t]);
                    norm[8 + t] = fmaf(qv[t][m], qv[t][m], norm[8 + t]);
                }
            }
        }, std::make_integer_sequence<int, T>());
        const float inv = p.qk_l2_norm ? 1.f / sqrtf(sixteen(norm, c, plus) + 1e-12f) : 1.f;
        // the columns of x in the order of the lanes' pieces: in the one that starts earlier, its own come last
        int place[KL];
#pragma unroll
        for (int m = 0; m < KL; ++m) {
            const int j = j0 + m, rest = dk % VK, last = dk - rest;
            place[m] = EXACT || rest == 0 || j < last || j >= last + VK ? j : j < dk ? j + VK - rest : j - rest;
        }
        float gone[KL], top[16];  // gone: decays up to a token
#pragma unroll
        for (int m = 0; m < KL; ++m) gone[m] = 1.f;
        each([&](auto t_) {
            constexpr int t = decltype(t_)::value;
            top[t] = top[8 + t] = 0.f;
            if (t < n) {
                const float ink = lane_of<t>(inv), inq = lane_of<8 + t>(inv);
#pragma unroll
                for (int m = 0; m < KL; ++m) {
                    kv[t][m] *= ink;
                    qv[t][m] *= inq;
                    rv[t][m] *= kv[t][m];
                    gone[m] *= av[t][m];
                    top[t] = fmaxf(top[t], fabsf(gone[m] * rv[t][m]));
                    top[8 + t] = fmaxf(top[8 + t], fabsf(gone[m] * qv[t][m]));
                }
            }
        }, std::make_integer_sequence<int, T>());
        float up = 1.f;
        if constexpr (!CB) half_scale(sixteen(top, c, [](float x, float y) { return fmaxf(x, y); }), up, back);
#pragma unroll
        for (int m = 0; m < KL; ++m) gone[m] = 1.f;
        each([&](auto t_) {
            constexpr int t = decltype(t_)::value;
            if (t < n) {
                float r[KL], w[KL];
                const float upr = lane_of<t>(up), upq = lane_of<8 + t>(up);
#pragma unroll
                for (int m = 0; m < KL; ++m) {
                    gone[m] *= av[t][m];
                    r[m] = gone[m] * rv[t][m] * upr;
                    w[m] = gone[m] * qv[t][m] * upq;
                }
#pragma unroll
                for (int x = 0; x < PX; ++x) {
                    TC hr[KL], hq[KL];
#pragma unroll
                    for (int m = 0; m < KL; ++m) {
                        hr[m] = from_f32<TC>(r[m]);
                        hq[m] = from_f32<TC>(w[m]);
                        r[m] -= to_f32(hr[m]);
                        w[m] -= to_f32(hq[m]);
                    }
                    if constexpr (EXACT) {
                        __builtin_memcpy(__builtin_assume_aligned(&s_x[x][t][j0], 2 * KL), hr, sizeof(hr));
                        __builtin_memcpy(__builtin_assume_aligned(&s_x[x][8 + t][j0], 2 * KL), hq, sizeof(hq));
                    } else {
#pragma unroll
                        for (int m = 0; m < KL; ++m) {
                            s_x[x][t][place[m]] = hr[m];
                            s_x[x][8 + t][place[m]] = hq[m];
                        }
                    }
                }
                // what token t's write adds to the later dots
                float since[KL], dots[16];  // since: decays after token t
#pragma unroll
                for (int m = 0; m < KL; ++m) since[m] = kv[t][m];
                each([&](auto u_) {
                    constexpr int u = decltype(u_)::value;
                    dots[u] = dots[8 + u] = 0.f;
                    if (u >= t && u < n) {
#pragma unroll
                        for (int m = 0; m < KL; ++m) {
                            if (u > t) since[m] *= av[u][m];
                            if (u > t) dots[u] = fmaf(since[m], rv[u][m], dots[u]);
                            dots[8 + u] = fmaf(since[m], qv[u][m], dots[8 + u]);
                        }
                    }
                }, std::make_integer_sequence<int, T>());
                cl[t] = sixteen(dots, c, plus);
#pragma unroll
                for (int m = 0; m < KL; ++m) kv[t][m] = since[m];
            }
        }, std::make_integer_sequence<int, T>());
#pragma unroll
        for (int m = 0; m < KL; ++m) s_all[j0 + m] = gone[m];
        wave_sync();
#pragma unroll
        for (int x = 0; x < PX; ++x)
#pragma unroll
            for (int f = 0; f < KS; ++f)
                y[x][f] = *reinterpret_cast<const VC *>(&s_x[x][c][EIGHT ? wanted(f / 2, kb) + 8 * (f % 2) : wanted(f, kb)]);
        wave_sync();
#pragma unroll
        for (int m = 0; m < KL; ++m) {
            w4 planes[3];
#pragma unroll
            for (int t = 0; t < T; t += 2) {
                float v0 = t < n ? kv[t][m] : 0.f, v1 = t + 1 < n ? kv[t + 1][m] : 0.f;
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    planes[x][t / 2] = uppers(v0, v1);
                    v0 = below(v0, UPPER);
                    v1 = below(v1, UPPER);
                }
            }
#pragma unroll
            for (int x = 0; x < PK; ++x) *reinterpret_cast<w4 *>(&s_k[x][j0 + m][0]) = planes[x];
        }
        wave_sync();
    } else {
        const float alpha = decays ? expf(log_decay(p, th, h)) : 1.f;

        VA x[KS];
#pragma unroll
        for (int f = 0; f < KS; ++f) x[f] = __builtin_bit_cast(VA, xr[f]);
        // k by keys, tokens together
        if (c < 8) {
#pragma unroll
            for (int f = 0; f < KS; ++f)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float kf = c < n ? to_f32((TA)x[f][j]) : 0.f;
                    const bf16_t hi = from_f32<bf16_t>(kf);
                    s_k[0][key(f, kb) + j][c] = hi;
                    if constexpr (!BF) s_k[1][key(f, kb) + j][c] = from_f32<bf16_t>(kf - to_f32(hi));
                }
        }
        f4v gram = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < KS; ++f) gram = mfma(x[f], x[f], gram);
        // x as operands of the cache's type
        if constexpr (SAME) {
#pragma unroll
            for (int f = 0; f < KS; ++f) y[0][f] = __builtin_bit_cast(VC, xr[f]);
        } else {
            float up = 1.f;
            if constexpr (BF) {  // bf16 in two fp16 planes: scaled to fp16's upper range
                float top = 0.f;
#pragma unroll
                for (int f = 0; f < KS; ++f)
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(to_f32((TA)x[f][j])));
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                half_scale(top, up, back);
            }
#pragma unroll
            for (int f = 0; f < KS; ++f)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = to_f32((TA)x[f][j]) * up;
                    const TC hi = from_f32<TC>(v);
                    y[0][f][j] = hi;
                    y[1][f][j] = from_f32<TC>(v - to_f32(hi));
                }
        }
        // norms and the products of the tokens' vectors
        float inv = 1.f;
        if (p.qk_l2_norm) {
            const float mine = c % 4 == 0 ? gram[0] : c % 4 == 1 ? gram[1] : c % 4 == 2 ? gram[2] : gram[3];
            inv = 1.f / sqrtf(__shfl(mine, 16 * (c / 4) + c) + 1e-12f);
        }
        float later = 1.f;
        each([&](auto t_) {
            constexpr int t = decltype(t_)::value;
            if (t < n) {
                const float at = lane_of<t>(alpha), kt = lane_of<t>(inv), g = __shfl(gram[t % 4], 16 * (t / 4) + c);
                const bool past = c >= 8 && t > c - 8;  // q of a token before t
                al[t] = past ? 1.f : at;
                cl[t] = past ? 0.f : kt * g;
                all *= at;
                if (t > own) later *= at;
            }
        }, std::make_integer_sequence<int, T>());
        const float put_own = later * inv;
        oscale = p.scale * inv;
        binv = retrieves ? beta * inv : 0.f;
        each([&](auto t_) {
            constexpr int t = decltype(t_)::value;
            if (t < n) put[t] = lane_of<t>(put_own);
        }, std::make_integer_sequence<int, T>());
        wave_sync();
    }

    for (int t0 = wave; t0 < tiles; t0 += PRE * waves)
#pragma unroll
        for (int i = 0; i < PRE; ++i) {
            const int tile = t0 + i * waves;
            if (tile >= tiles) break;
            if constexpr (LINES)
#pragma unroll
                for (int m = 0; m < NV; m += 2) exchange(raw[i][m], raw[i][m + 1], c & 1);
            // dots of the states with every vector: rows 4 kb + j, column c
            f4v z = {0.f, 0.f, 0.f, 0.f}, z1 = z;
#pragma unroll
            for (int f = 0; f < KS; ++f) {
                VC sv;
                if constexpr (EIGHT) {
                    const uint32_t w0 = raw[i][f / 2][f % 2 * 2], w1 = raw[i][f / 2][f % 2 * 2 + 1];
                    w4 o;
                    if constexpr (CB) {
                        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, false));
                        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, true));
                        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, false));
                        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, true));
                    } else {
                        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false));
                        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true));
                        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false));
                        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true));
                    }
                    sv = __builtin_bit_cast(VC, o);
                } else {
                    const w4 o = raw[i][f];
                    sv = __builtin_bit_cast(VC, o);
                }
                if constexpr (PX == 1) {
                    if (f % 2) z1 = mfma(sv, y[0][f], z1);
                    else z = mfma(sv, y[0][f], z);
                } else {
                    z = mfma(sv, y[0][f], z);
                    z1 = mfma(sv, y[1][f], z1);
                    if constexpr (PX == 3) z1 = mfma(sv, y[2][f], z1);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] += z1[j];
            // decayed states, to which the update is added
            float S[KS][8];
#pragma unroll
            for (int f = 0; f < KS; ++f) {
                f4v each_all[2];
                if constexpr (GEN) {
                    using V = typename std::conditional<EXACT, f4v, Any4f>::type;
                    each_all[0] = *reinterpret_cast<const V *>(&s_all[key(f, kb)]);
                    each_all[1] = *reinterpret_cast<const V *>(&s_all[key(f, kb) + 4]);
                }
                if constexpr (EIGHT) {
                    from_codes(raw[i][f / 2][f % 2 * 2], scale_of(ex[i]), &S[f][0]);
                    from_codes(raw[i][f / 2][f % 2 * 2 + 1], scale_of(ex[i]), &S[f][4]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) S[f][j] *= GEN ? each_all[j / 4][j % 4] : all;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        S[f][j] = fmaf(half_of<TC>(raw[i][f][j / 2], j % 2), GEN ? each_all[j / 4][j % 4] : all, 0.f);
                }
            }
            float vj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[j] *= EIGHT ? scale_of(exr[i][j]) * back : back;
                vj[j] = beta * to_f32(vr[i][j]);
            }
            fetch(i, tile + PRE * waves);
            // the tokens in order: the new values d, and the dots with the states after them
            each([&](auto t_) {
                constexpr int t = decltype(t_)::value;
                if (t < n) {
                    float d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (!GEN) z[j] *= al[t];
                        d[j] = retrieves ? fmaf(-binv, z[j], vj[j]) : vj[j];
                    }
                    if (c == t) *reinterpret_cast<f4v *>(&s_d[t][4 * kb]) = f4v{d[0], d[1], d[2], d[3]};
                    // (not into a q of a token before t: nothing of t, a NaN neither, reaches that output)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float dt = lane_of<t>(d[j]);
                        z[j] = t > 0 && c >= 8 && c < 8 + t ? z[j] : fmaf(dt, cl[t], z[j]);
                    }
                }
            }, std::make_integer_sequence<int, T>());
            if (c >= 8 && c - 8 < n) {
                TA *o = static_cast<TA *>(p.o) + th * p.dv + 16 * tile + 4 * kb;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (16 * tile + 4 * kb + j < p.dv) o[j] = from_f32<TA>(oscale * z[j]);
            }
            wave_sync();
            // d of row c in planes hi, mid, lo, beside k's at the same inner places: by kb, hi
            // mid lo - (k is exact), or lo - lo - and then hi mid hi mid beside k's hi hi mid mid, or
            // lo - mid - and then hi mid hi hi beside hi hi mid lo
            float d[T];
#pragma unroll
            for (int t = 0; t < T; ++t) d[t] = GEN ? s_d[t][c] : t < n ? s_d[t][c] * put[t] : 0.f;  // 0 past the tokens
            wave_sync();
            const auto planes = [&](uint32_t first, uint32_t second) {
                w4 d8;
#pragma unroll
                for (int t = 0; t < T; t += 2)
                    d8[t / 2] = uppers(below(below(d[t], first), second), below(below(d[t + 1], first), second));
                return __builtin_bit_cast(b8, d8);
            };
            b8 d8, low8;
            if constexpr (BF) {
                d8 = planes(kb == 0 ? 0 : UPPER, kb < 2 ? 0 : kb == 2 ? UPPER : ~0u);
            } else {
                d8 = planes(kb == 1 || (!GEN && kb == 3) ? UPPER : 0, 0);
                low8 = planes(UPPER, kb & 1 ? ~0u : GEN && kb == 2 ? 0 : UPPER);
            }
            const int k_plane = BF || kb == 0 ? 0 : GEN ? kb - 1 : kb >> 1;
#pragma unroll
            for (int f = 0; f < KS; ++f)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const b8 k8 = *reinterpret_cast<const b8 *>(&s_k[k_plane][key(f, c / 4) + 4 * j + c % 4][0]);
                    f4v acc = {S[f][4 * j], S[f][4 * j + 1], S[f][4 * j + 2], S[f][4 * j + 3]};
                    if constexpr (!BF) acc = mfma(k8, low8, acc);
                    acc = mfma(k8, d8, acc);
#pragma unroll
                    for (int m = 0; m < 4; ++m) S[f][4 * j + m] = acc[m];
                }
            const int row = 16 * tile + c;
            w4 out[NV];
            uint32_t eo = 0;
            if constexpr (EIGHT) {
                eo = scale_byte_of(reinterpret_cast<const float (&)[8 * KS]>(S), [](float top) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    return fmaxf(top, __shfl_xor(top, 32));
                });
#pragma unroll
                for (int f = 0; f < KS; ++f) {
                    out[f / 2][f % 2 * 2] = to_codes(&S[f][0], scale_of(eo));
                    out[f / 2][f % 2 * 2 + 1] = to_codes(&S[f][4], scale_of(eo));
                }
            } else {
#pragma unroll
                for (int f = 0; f < KS; ++f)
#pragma unroll
                    for (int j = 0; j < 4; ++j) out[f][j] = two_halves<TC>(S[f][2 * j], S[f][2 * j + 1]);
            }
            if constexpr (LINES)
#pragma unroll
                for (int m = 0; m < NV; m += 2) exchange(out[m], out[m + 1], c & 1);
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                if constexpr (EXACT) {
                    const int r = LINES ? 16 * tile + (c & ~1) + m % 2 : row;
                    if (r < p.dv) __builtin_nontemporal_store(out[m], reinterpret_cast<w4 *>(mat + r * ROW + m / 2 * 128 + (LINES ? (c & 1) * 64 : 0) + kb * 16));
                } else if (row < p.dv && wanted(m, kb) < dk) {
                    *reinterpret_cast<Any4 *>(mat + row * ROW + piece(m, kb) * (16 / VK)) = out[m];
                }
            }
            if (EIGHT && kb == 0 && row < p.dv) scales[row] = (uint8_t)eo;
        }
}

template <typename TA, int TYPE, int DK, bool VD, bool ONE>
hipError_t launch_step(const PackedParams &a, int rule, bool per_key, int least, hipStream_t s)
{
    using Form = StepForm<TYPE, DK, ONE>;
    const dim3 blocks((unsigned)((int64_t)a.p.B * a.p.HV * ((a.p.dv + Form::ROWS - 1) / Form::ROWS)));
    const dim3 threads(64 * Form::WAVES);
    if (a.p.dk == DK)
        hipLaunchKernelGGL((k_packed_step<TA, TYPE, DK, VD, ONE, true>), blocks, threads, 0, s, a, rule, (int)per_key, least);
    else
        hipLaunchKernelGGL((k_packed_step<TA, TYPE, DK, VD, ONE, false>), blocks, threads, 0, s, a, rule, (int)per_key, least);
    return hipGetLastError();
}

template <typename TA, int TYPE, int DK>
hipError_t packed_step_at(const PackedParams &a, int rule, bool per_key, hipStream_t s)
{
    const Params &p = a.p;
    const bool keyed = per_key || rule == GATED_DELTA_V2;  // per-key vectors
    const bool one = !p.cu_seqlens && p.L == 1;            // no request has more than a token
    if (one)
        return keyed ? launch_step<TA, TYPE, DK, true, true>(a, rule, per_key, 1, s)
                     : launch_step<TA, TYPE, DK, false, true>(a, rule, per_key, 1, s);
    // Up to 8 tokens on the matrix cores: 16-bit activations with one decay a head, or any.
    if constexpr (DK >= 64) {
        // Waves of a state: one, which spares the tokens' own work, until too few
        // states leave SIMDs idle: 2,048 waves, two a SIMD.  4 tokens, 32 heads of
        // 128, in us with 1,024, 2,048, 4,096 and 8,192 waves at least: 8-bit states of
        // 32 requests 19.4, 16.0, 18.8 and 22.2, of 64 25.3, 25.5, 26.8 and 30.7;
        // 16-bit ones 21.1, 20.8, 23.9 and 26.2, 32.1, 32.2, 36.5 and 37.2.
        const int64_t states = (int64_t)p.B * p.HV;
        int waves = 1;
        while (waves < 8 && waves * 16 < p.dv && states * waves < 2048) waves *= 2;
        const dim3 blocks((unsigned)((states * waves + 3) / 4)), threads(256);
        // Tiles ahead: two in 8 bits, but one where two would spill (GEN, 256 keys) or leave two
        // waves a SIMD instead of three (other dims: 4 tokens, heads of 96 in 8 bits 83 and 68 us).
        constexpr int PRE = TYPE == CACHE_E4M3 ? 2 : 1, PRE_GEN = DK > 192 ? 1 : PRE;
        const bool exact = p.dk == DK;
        if constexpr (sizeof(TA) == 2) {
            if (exact && !keyed)
                hipLaunchKernelGGL((k_packed_few<TA, TYPE, DK, PRE, false, true>), blocks, threads, 0, s, a, rule, 0, waves);
        }
        if (exact && (keyed || sizeof(TA) == 4))
            hipLaunchKernelGGL((k_packed_few<TA, TYPE, DK, PRE_GEN, true, true>), blocks, threads, 0, s, a, rule, (int)per_key, waves);
        // (to 192 keys with products over 192: 256 requests x 32 heads of 192, 2 tokens,
        // 446 -> 313 us in 16 bits and 228 -> 188 in 8)
        if (DK == 256 && p.dk <= 192)
            hipLaunchKernelGGL((k_packed_few<TA, TYPE, DK == 256 ? 192 : DK, PRE, true, false>), blocks, threads, 0, s, a, rule, (int)per_key, waves);
        else if (!exact)
            hipLaunchKernelGGL((k_packed_few<TA, TYPE, DK, 1, true, false>), blocks, threads, 0, s, a, rule, (int)per_key, waves);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess || (p.cu_seqlens ? p.T : p.L) <= 8) return err;
    }
    // requests of more than 8 tokens, or any of up to 16 keys
    const int least = DK >= 64 ? 9 : 1;
    return keyed ? launch_step<TA, TYPE, DK, true, false>(a, rule, per_key, least, s)
                 : launch_step<TA, TYPE, DK, false, false>(a, rule, false, least, s);
}

template <typename TA, int TYPE>
hipError_t packed_step_by_dk(const PackedParams &a, int rule, bool per_key, hipStream_t s)
{
    if (a.p.dk <= 16) return packed_step_at<TA, TYPE, 16>(a, rule, per_key, s);
    if (a.p.dk <= 64) return packed_step_at<TA, TYPE, 64>(a, rule, per_key, s);
    if (a.p.dk <= 128) return packed_step_at<TA, TYPE, 128>(a, rule, per_key, s);
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
