// gdr_rotary.hip -- root-mean-square norm of every head of q and k and the
// rotation by the tokens' positions in one pass, and its backward pass.
//
//   h = x inv w,  inv = 1 / sqrt(mean x^2 + eps)      (inv = 1 without the norm)
//   a = position[axis_i] freq_i;  pair i of h turned by a:
//   (y_0, y_1) = (h_0 cos a - h_1 sin a, h_1 cos a + h_0 sin a)
// and backwards, with g the pairs of dy turned by -a, t = w g and n = x inv,
//   dx = inv (t - n mean(t n)),   dw = sum over tokens and heads of g n
// (dx = t without the norm; its statistics are formed again: a sum more, nothing
// kept).
//
// Bound by memory: a head's row lies in the registers of LPR lanes between its
// load and its store.  A lane holds both values of its pairs: VEC elements
// from each half of the turned columns, or 2 VEC neighbours.  The angles of a
// workgroup's tokens are formed once, by all its threads, and lie in LDS for
// every head.  An angle is the product of an int32 and an fp32 value, taken in
// turns and in 64 bits: at position 10^6 an fp32 product is off by 0.03.
#include "gdr_rotary_launch.hpp"

namespace gdr {
namespace {

constexpr int THREADS = 256;
constexpr int ANGLES = 2048;  // pairs of (token, frequency) whose cos and sin LDS holds

// 16, 8 and 4 bytes from any even address.
typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t v2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t v1 __attribute__((aligned(2)));

// VEC elements as they lie in memory.
template <typename T, int VEC> struct Raw {
    static constexpr int BYTES = VEC * sizeof(T), WORDS = (BYTES + 3) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *src)
    {
        if constexpr (BYTES == 16) {
            const v4 x = *reinterpret_cast<const v4 *>(src);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = x[i];
        } else if constexpr (BYTES == 8) {
            const v2 x = *reinterpret_cast<const v2 *>(src);
            w[0] = x[0];
            w[1] = x[1];
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const v1 *>(src);
        } else {
            w[0] = __builtin_bit_cast(uint16_t, src[0]);
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[i]);
        else return to_f32(__builtin_bit_cast(T, (uint16_t)(w[i / 2] >> (16 * (i % 2)))));
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void store(T *dst, const float *v)
{
    constexpr int BYTES = VEC * sizeof(T), WORDS = (BYTES + 3) / 4;
    if constexpr (BYTES == 2) {
        dst[0] = from_f32<T>(v[0]);
    } else {
        uint32_t o[WORDS];
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) o[i] = __builtin_bit_cast(uint32_t, v[i]);
            else o[i] = __builtin_bit_cast(uint16_t, from_f32<T>(v[2 * i])) |
                        (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(v[2 * i + 1])) << 16;
        }
        if constexpr (BYTES == 16) *reinterpret_cast<v4 *>(dst) = v4{o[0], o[1], o[2], o[3]};
        else if constexpr (BYTES == 8) *reinterpret_cast<v2 *>(dst) = v2{o[0], o[1]};
        else *reinterpret_cast<v1 *>(dst) = o[0];
    }
}

// Where a lane's vector lies in a head: `at` the columns of its two parts of
// VEC elements, `pair` its first turned pair (or -1: not turned).
template <int VEC> struct Place {
    int at[2], pair;
    bool on, second;  // second: the second part lies inside the head
    __device__ __forceinline__ Place(const RotaryParams &p, int vector)
    {
        const int base = vector * VEC;
        const bool turned = base < p.half;
        on = 2 * base < p.dim;
        at[0] = turned && !p.neighbours ? base : 2 * base;
        at[1] = turned && !p.neighbours ? p.half + base : 2 * base + VEC;
        second = VEC > 1 || at[1] < p.dim;
        pair = turned ? base : -1;
        if (!on) at[0] = 0;
        if (!on || !second) at[1] = VEC > 1 ? VEC : at[0];  // its values count for nothing
    }
};

// VEC neighbouring values in LDS, their address a multiple of VEC.
template <int VEC>
__device__ __forceinline__ void read(const float *src, float *v)
{
    __builtin_memcpy(v, __builtin_assume_aligned(src, VEC < 4 ? 4 * VEC : 16), 4 * VEC);
}

// Pair i of a lane's 2 VEC values: both halves' i-th, or two neighbours.
template <int VEC>
__device__ __forceinline__ void turn(float (&x)[2 * VEC], const float *cs, const float *sn, bool neighbours, float sign)
{
    float c[VEC], s[VEC];
    read<VEC>(cs, c);
    read<VEC>(sn, s);
    const auto pair = [&](float &a, float &b, int i) {
        const float a0 = a, b0 = b, t = sign * s[i];
        a = a0 * c[i] - b0 * t;
        b = b0 * c[i] + a0 * t;
    };
    if (neighbours) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) pair(x[2 * i], x[2 * i + 1], i);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) pair(x[i], x[VEC + i], i);
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor(x, o);
    return x;
}

// Sine and cosine of `turns` whole turns, by the Taylor series within an eighth
// of a turn (their first terms left out are under 3e-8).
__device__ __forceinline__ void sincos_turns(double turns, float &sn, float &cs)
{
    const double f = turns - rint(turns);
    const float n = rintf(4.f * (float)f);
    const float r = (float)fma((double)n, -0.25, f), y = r * r;  // (rounded before the quarters are off, it would lose two bits)
    const float s = r * fmaf(y, fmaf(y, fmaf(y, fmaf(y, 42.058693944897653f, -76.705859753061386f), 81.605249276075054f),
                                     -41.341702240399755f), 6.2831853071795865f);
    const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 60.244641371876664f, -85.456817206693732f), 64.939394022668291f),
                                 -19.739208802178716f), 1.f);
    const int quarter = (int)n & 3;
    const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
    sn = quarter & 2 ? -a : a;
    cs = (quarter + 1) & 2 ? -b : b;
}

// cos and sin of the angles of a workgroup's tokens: a thread takes one
// frequency, and every groups-th token.  (With both found by division in a loop
// over all pairs, and the library's sincospi, gradients of 40,021 tokens and one
// head of q and k took 41 us.)
struct Angles {
    double turn;  // of a position
    const int32_t *positions;
    int f, group, groups;
    __device__ __forceinline__ Angles(const RotaryParams &p)
    {
        groups = THREADS / p.half;
        group = threadIdx.x / p.half;
        f = threadIdx.x - group * p.half;
        int axis = p.axis_of ? p.axis_of[f] : 0;
        axis = axis < 0 ? 0 : axis < p.axes ? axis : p.axes - 1;
        positions = p.positions + axis * p.tokens;
        turn = (double)p.freq[f] * 0.15915494309189535;
    }
    // tokens t0 .. t0 + n - 1
    __device__ __forceinline__ void fill(const RotaryParams &p, int64_t t0, int n, float *cs, float *sn) const
    {
        if (group >= groups) return;
        for (int token = group; token < n; token += groups)
            sincos_turns((double)positions[t0 + token] * turn, sn[token * p.half + f], cs[token * p.half + f]);
    }
};

// A workgroup takes p.block tokens, all heads of q and then of k for each.
template <typename T, typename TW, int VEC, int LPR, int NV>
__global__ __launch_bounds__(THREADS) void k_rotary(const RotaryParams p)
{
    __shared__ __align__(16) float s_cos[ANGLES], s_sin[ANGLES], s_w[2][ROTARY_MAX_DIM];
    constexpr int ROWS = THREADS / LPR;
    const int lane = threadIdx.x % LPR;
    const int heads = p.part[0].heads + p.part[1].heads;
    const int64_t t0 = p.first + (int64_t)blockIdx.x * p.block;
    const int n = (int)(p.tokens - t0 < p.block ? p.tokens - t0 : p.block);
    const int step_t = ROWS / heads, step_h = ROWS - step_t * heads;
    int token = threadIdx.x / LPR / heads, head = threadIdx.x / LPR - token * heads;
    Raw<T, VEC> x[NV][2] = {};  // 0 in lanes that hold nothing
    auto fetch = [&](int token, int head) {
        const int z = head >= p.part[0].heads;
        const RotaryPart &part = p.part[z];
        const T *row = static_cast<const T *>(part.x) + (t0 + token) * part.stride +
                       (int64_t)(z ? head - p.part[0].heads : head) * p.dim;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Place<VEC> at(p, lane + LPR * v);
            if (!at.on) continue;
            x[v][0].load(row + at.at[0]);
            if (at.second) x[v][1].load(row + at.at[1]);
        }
    };
    const Angles angles(p);
    if (token < n) fetch(token, head);
    angles.fill(p, t0, n, s_cos, s_sin);
    for (int i = threadIdx.x; i < 2 * p.dim; i += THREADS) {
        const int z = i >= p.dim, c = z ? i - p.dim : i;
        s_w[z][c] = p.part[z].weight ? to_f32(static_cast<const TW *>(p.part[z].weight)[c]) : 1.f;
    }
    lds_barrier();
    while (token < n) {
        const int z = head >= p.part[0].heads;
        const RotaryPart &part = p.part[z];
        float h[NV][2 * VEC], sum = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                h[v][i] = x[v][0].get(i);
                h[v][VEC + i] = x[v][1].get(i);
                sum += h[v][i] * h[v][i] + h[v][VEC + i] * h[v][VEC + i];
            }
        }
        T *row = static_cast<T *>(part.y) + (t0 + token) * part.out_stride +
                 (int64_t)(z ? head - p.part[0].heads : head) * p.dim;
        const int now = token;
        token += step_t;
        head += step_h;
        if (head >= heads) {
            head -= heads;
            ++token;
        }
        if (token < n) fetch(token, head);
        const float inv = p.norm ? 1.f / sqrtf(row_sum<LPR>(sum) / (float)p.dim + p.eps) : 1.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Place<VEC> at(p, lane + LPR * v);
            float w[2 * VEC];
            read<VEC>(&s_w[z][at.at[0]], &w[0]);
            read<VEC>(&s_w[z][at.at[1]], &w[VEC]);
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) h[v][i] *= inv * w[i];
            if (!at.on) continue;
            if (at.pair >= 0)
                turn<VEC>(h[v], &s_cos[now * p.half + at.pair], &s_sin[now * p.half + at.pair], p.neighbours, 1.f);
            store<T, VEC>(row + at.at[0], &h[v][0]);
            if (at.second) store<T, VEC>(row + at.at[1], &h[v][VEC]);
        }
    }
}

// blockIdx.y: q or k.  A workgroup takes part.block tokens at a time; the
// weight's gradient stays in a lane's registers, as its columns are the same for
// every row, and its sums over the workgroup's rows and then over the workgroups
// have a fixed order.  (Four waves a SIMD asked for: with three, and the
// weights kept in registers, 29,273 tokens x 16 + 16 heads of 128 in bf16 took 163
// instead of 143 us.  A row's work has few branches: with one for every value of
// lanes that hold nothing, a workgroup's two turns took 18 us, and 1,500 tokens 26
// instead of 20.  NORM is the call's: chosen value by value it took 58,000 tokens x
// 32 heads of 64 from 140 to 149 us.)
template <typename T, typename TW, int VEC, int LPR, int NV, bool NORM>
__global__ __launch_bounds__(THREADS, 4) void k_rotary_back(const RotaryParams p)
{
    __shared__ __align__(16) float s_cos[ANGLES], s_sin[ANGLES], s_w[ROTARY_MAX_DIM];
    __shared__ float s_dw[THREADS][2 * VEC + 1];
    constexpr int ROWS = THREADS / LPR;
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const RotaryPart &part = p.part[blockIdx.y];
    const int heads = part.heads;
    if ((int)blockIdx.x >= part.blocks) return;
    float dw[NV][2 * VEC] = {};
    const Angles angles(p);
    for (int i = threadIdx.x; i < p.dim; i += THREADS)
        s_w[i] = part.weight ? to_f32(static_cast<const TW *>(part.weight)[i]) : 1.f;
    const auto weights = [&](const Place<VEC> &at, float (&w)[2 * VEC]) {
        read<VEC>(&s_w[at.at[0]], &w[0]);
        read<VEC>(&s_w[at.at[1]], &w[VEC]);
    };
    Raw<T, VEC> x[NV][2] = {}, y[NV][2] = {};  // 0 in lanes that hold nothing
    const int step_t = ROWS / heads, step_h = ROWS - step_t * heads;
    for (int64_t t0 = (int64_t)blockIdx.x * part.block; t0 < p.tokens; t0 += (int64_t)part.blocks * part.block) {
        const int n = (int)(p.tokens - t0 < part.block ? p.tokens - t0 : part.block);
        int token = group / heads, head = group - token * heads;
        auto fetch = [&](int token, int head) {
            const T *row = static_cast<const T *>(part.x) + (t0 + token) * part.stride + (int64_t)head * p.dim;
            const T *dy = static_cast<const T *>(part.d_y) + ((t0 + token) * heads + head) * p.dim;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const Place<VEC> at(p, lane + LPR * v);
                if (!at.on) continue;
                x[v][0].load(row + at.at[0]);
                y[v][0].load(dy + at.at[0]);
                if (at.second) {
                    x[v][1].load(row + at.at[1]);
                    y[v][1].load(dy + at.at[1]);
                }
            }
        };
        if (token < n) fetch(token, head);
        lds_barrier();  // the last tokens' angles have been used
        angles.fill(p, t0, n, s_cos, s_sin);
        lds_barrier();
        while (token < n) {
            float h[NV][2 * VEC], g[NV][2 * VEC], sum = 0.f, dot = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const Place<VEC> at(p, lane + LPR * v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    h[v][i] = x[v][0].get(i);
                    h[v][VEC + i] = x[v][1].get(i);
                    g[v][i] = y[v][0].get(i);
                    g[v][VEC + i] = y[v][1].get(i);
                }
                float w[2 * VEC];
                weights(at, w);
                if (at.pair >= 0)
                    turn<VEC>(g[v], &s_cos[token * p.half + at.pair], &s_sin[token * p.half + at.pair], p.neighbours, -1.f);
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) {
                    sum += h[v][i] * h[v][i];
                    dot += g[v][i] * w[i] * h[v][i];
                }
            }
            T *row = static_cast<T *>(part.y) + (t0 + token) * part.out_stride + (int64_t)head * p.dim;
            token += step_t;
            head += step_h;
            if (head >= heads) {
                head -= heads;
                ++token;
            }
            if (token < n) fetch(token, head);
            float inv = 1.f, mean = 0.f;
            __builtin_amdgcn_sched_barrier(0);  // (the row's two halves mixed hold more than the registers)
            if constexpr (NORM) {
                inv = 1.f / sqrtf(row_sum<LPR>(sum) / (float)p.dim + p.eps);
                mean = row_sum<LPR>(dot) * inv / (float)p.dim;
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const Place<VEC> at(p, lane + LPR * v);
                float w[2 * VEC];
                weights(at, w);
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) {
                    const float nx = h[v][i] * inv, t = g[v][i] * w[i];
                    dw[v][i] += g[v][i] * nx;
                    g[v][i] = NORM ? inv * (t - nx * mean) : t;  // (without: x, be it an infinity, has no part in it)
                }
                if (!at.on) continue;
                store<T, VEC>(row + at.at[0], &g[v][0]);
                if (at.second) store<T, VEC>(row + at.at[1], &g[v][VEC]);
            }
        }
    }
    if (!part.partial) return;
    float *out = part.partial + (size_t)blockIdx.x * p.dim;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) s_dw[threadIdx.x][i] = dw[v][i];
        __syncthreads();
        // value i of lane l of this vector: one thread each
        for (int e = threadIdx.x; e < LPR * 2 * VEC; e += THREADS) {
            const int l = e / (2 * VEC), i = e % (2 * VEC);
            const Place<VEC> at(p, l + LPR * v);
            if (!at.on || (i >= VEC && !at.second)) continue;
            float sum = 0.f;
            for (int r = 0; r < ROWS; ++r) sum += s_dw[r * LPR + l][i];
            out[(i < VEC ? at.at[0] : at.at[1]) + i % VEC] = sum;
        }
    }
}

// Workgroup: 16 columns, 64 threads a column, each every 64th partial row.
__global__ __launch_bounds__(1024) void k_rotary_back_sums(const RotaryParams p)
{
    __shared__ float s[64][17];
    const RotaryPart &part = p.part[blockIdx.y];
    if (!part.d_weight) return;
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    float sum = 0.f;
    if (col < p.dim) {
        for (int b = r; b < part.blocks; b += 512) {  // eight loads at once
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = b + 64 * i < part.blocks ? part.partial[(size_t)(b + 64 * i) * p.dim + col] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x[i];
        }
    }
    s[r][c] = sum;
    __syncthreads();
    if (r < 4) {
        for (int n = r + 4; n < 64; n += 4) sum += s[n][c];
        s[r][c] = sum;
    }
    __syncthreads();
    if (r == 0 && col < p.dim) part.d_weight[col] = s[0][c] + s[1][c] + s[2][c] + s[3][c];
}

// Vectors, lanes and vectors a lane of a head: vectors of 16, 8 or 4 bytes (16
// and 8 in fp32) where the head and its turned part consist of whole pairs of
// them, else single pairs.
template <typename T, bool BACK, typename F>
hipError_t by_form(const RotaryParams &p, F &&f)
{
    using std::integral_constant;
    constexpr int V = 16 / sizeof(T);
    const auto fits = [&](int v) { return p.dim % (2 * v) == 0 && p.half % v == 0; };
    const auto lanes = [&](auto vec) {
        const int vectors = p.dim / (2 * vec());
        // Three vectors a lane where they fill more lanes (29,273 tokens, 32 heads of 72,
        // 72 and 36 columns turned, in fp16 86 -> 71 and 114 -> 80 us; of 80 with 20
        // 117 -> 97, gradients 198 -> 142; but gradients of 72 with 72 114 -> 253).
        if constexpr (vec() < V && (!BACK || vec() <= 2)) {
            if (vectors > 8 && vectors <= 12) return f(vec, integral_constant<int, 4>(), integral_constant<int, 3>());
            if (vectors > 16 && vectors <= 24) return f(vec, integral_constant<int, 8>(), integral_constant<int, 3>());
        }
        if (vectors <= 4) return f(vec, integral_constant<int, 4>(), integral_constant<int, 1>());
        if (vectors <= 8) return f(vec, integral_constant<int, 8>(), integral_constant<int, 1>());
        if (vectors <= 16) return f(vec, integral_constant<int, 16>(), integral_constant<int, 1>());
        if constexpr (vec() < 8) {
            if (vec() == 4 || vectors <= 32) return f(vec, integral_constant<int, 32>(), integral_constant<int, 1>());
        }
        return f(vec, integral_constant<int, vec() < 4 ? 64 : 16>(), integral_constant<int, 1>());
    };
    if (fits(V)) return lanes(integral_constant<int, V>());
    if (fits(V / 2)) return lanes(integral_constant<int, V / 2>());
    if constexpr (V == 8) {
        if (fits(2)) return lanes(integral_constant<int, 2>());
    }
    using one = integral_constant<int, 1>;
    if (p.dim <= 32) return f(one(), integral_constant<int, 16>(), one());
    if (p.dim <= 64) return f(one(), integral_constant<int, 32>(), one());
    if (p.dim <= 128) return f(one(), integral_constant<int, 32>(), integral_constant<int, 2>());
    return f(one(), integral_constant<int, 64>(), integral_constant<int, 2>());
}

template <typename F>
hipError_t by_types(const RotaryParams &p, F &&f)
{
    if (p.dt == 1) return p.weight_dt == 1 ? f(half_t(), half_t()) : f(half_t(), float());
    if (p.dt == 2) return p.weight_dt == 2 ? f(bf16_t(), bf16_t()) : f(bf16_t(), float());
    return f(float(), float());
}

// Tokens a workgroup takes at a time: about `rows` heads, and no more angles
// than LDS holds.
int token_block(const RotaryParams &p, int64_t heads, int64_t rows)
{
    int64_t n = (rows + heads - 1) / heads;
    if (n * p.half > ANGLES) n = ANGLES / p.half;
    return (int)(n < 1 ? 1 : n);
}

}  // namespace

int rotary_back_blocks(int64_t tokens, int64_t heads, int64_t all_heads, int64_t dim)
{
    // 4,096 elements a workgroup, up to four workgroups a CU for q and k together.
    // 16,384, 8,192, 4,096 and 2,048: 1,217 tokens x 9 and 3 heads of 72 in fp32 26,
    // 21, 20 and 20 us (19 of them the host's); 29,273 x 16 + 16 heads of 128 in bf16
    // 142 each, 143 with twice as many workgroups.
    const int64_t n = tokens * heads * dim / 4096;
    // A part of few heads still forms every token's angles: 29,273 tokens x 16 and 1
    // heads of 128 with 128, 256 and 512 workgroups for the one 101, 91 and 86 us.
    const int64_t most = std::max<int64_t>(512, 1024 * heads / std::max<int64_t>(all_heads, 1));
    return n < 1 ? 1 : n > most ? (int)most : (int)n;
}

hipError_t launch_rotary(const RotaryParams &params, hipStream_t s)
{
    RotaryParams p = params;
    const int64_t heads = (int64_t)p.part[0].heads + p.part[1].heads;
    if (p.tokens == 0 || heads == 0) return hipSuccess;
    return by_types(p, [&](auto t, auto w) {
        using T = decltype(t);
        using TW = decltype(w);
        return by_form<T, false>(p, [&](auto vec, auto lpr, auto nv) {
            // 16 KB of rows a workgroup: 29,273 tokens x 32 heads of 128 in fp16 with 8, 16,
            // 32 and 64 KB 103, 94, 96 and 100 us; 14,000 in fp32 with 16, 32 and 64 87, 92
            // and 92; and at most 8 heads for each of its places (97,069 tokens x 4 heads of
            // 13 in fp16 with 4, 8, 16 and 40 28, 27, 28 and 40).
            p.block = token_block(p, heads, std::min(16384 / (p.dim * (int)sizeof(T)), 8 * THREADS / lpr()));
            const int64_t spread = (p.tokens + 511) / 512;  // few tokens: a workgroup each
            if (p.block > spread) p.block = (int)spread;
            // a launch has fewer than 2^32 threads: further tokens take another
            const int64_t most = (int64_t)((1 << 24) - 1) * p.block;
            for (; p.first < p.tokens; p.first += most) {
                const dim3 blocks((unsigned)((std::min(most, p.tokens - p.first) + p.block - 1) / p.block));
                hipLaunchKernelGGL((k_rotary<T, TW, decltype(vec)::value, decltype(lpr)::value, decltype(nv)::value>),
                                   blocks, dim3(THREADS), 0, s, p);
                hipError_t err = hipGetLastError();
                if (err != hipSuccess) return err;
            }
            return hipSuccess;
        });
    });
}

hipError_t launch_rotary_backward(const RotaryParams &params, hipStream_t s)
{
    RotaryParams p = params;
    const int64_t heads = (int64_t)p.part[0].heads + p.part[1].heads;
    bool single = false;
    if (p.tokens > 0 && heads > 0) {
        hipError_t err = by_types(p, [&](auto t, auto w) {
            using T = decltype(t);
            using TW = decltype(w);
            return by_form<T, true>(p, [&](auto vec, auto lpr, auto nv) {
                for (RotaryPart &part : p.part) {
                    part.blocks = 0;
                    if (!part.heads) continue;
                    // 64 heads at a time (as fast as 128, 2 % faster than 32); fewer, to two for
                    // each place of the workgroup, or up to 80 where every workgroup then has
                    // one turn (without: 613 tokens x 4 + 20 heads of 256 in fp32 24 instead of
                    // 20 us, 3,597 x 10 + 10 of 128 in bf16 30 instead of 26).
                    const int64_t most = rotary_back_blocks(p.tokens, part.heads, heads, p.dim);
                    const int64_t share = (p.tokens + most - 1) / most, full = token_block(p, part.heads, 64);
                    const int64_t least = std::min<int64_t>(full, token_block(p, part.heads, 2 * THREADS / lpr()));
                    const int64_t block = share * 4 <= full * 5 ? std::max(share, least) : full;
                    part.block = (int)std::min<int64_t>(block, ANGLES / p.half);
                    part.blocks = (int)std::min(most, (p.tokens + part.block - 1) / part.block);
                }
                if (p.part[0].blocks <= 1 && p.part[1].blocks <= 1) {  // one workgroup's sums are the result
                    single = true;
                    for (RotaryPart &part : p.part) part.partial = part.heads ? part.d_weight : nullptr;
                }
                const dim3 blocks((unsigned)std::max(p.part[0].blocks, p.part[1].blocks), 2);
                const auto kernel = p.norm ? k_rotary_back<T, TW, decltype(vec)::value, decltype(lpr)::value, decltype(nv)::value, true>
                                           : k_rotary_back<T, TW, decltype(vec)::value, decltype(lpr)::value, decltype(nv)::value, false>;
                hipLaunchKernelGGL(kernel, blocks, dim3(THREADS), 0, s, p);
                return hipGetLastError();
            });
        });
        if (err != hipSuccess) return err;
    }
    if (!single && (p.part[0].d_weight || p.part[1].d_weight))
        hipLaunchKernelGGL(k_rotary_back_sums, dim3((unsigned)((p.dim + 15) / 16), 2), dim3(1024), 0, s, p);
    return hipGetLastError();
}

}  // namespace gdr
