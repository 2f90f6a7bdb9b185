// gdr_backward.hpp -- the backward pass of the gated delta rule (gfx950), for
// the rules with one log decay per value head (linear, gated, delta,
// gated_delta).  Included once per activation type (gdr_backward_*.hip).
//
// Mathematics.  A request's tokens are cut into chunks of C (64; 32 at a key
// width above 128).  Per value head and chunk, with S0 (dv x dk) the state
// before it, q^ = scale q / |q|, k^ = k / |k| (norms only with qk_l2_norm), G
// the cumulative log decay in the chunk, Gamma its last value, b the update
// rate and L_ts = e^(G_t - G_s) k^_t . k^_s (s < t), the forward recurrence
// unrolls to
//   E  = (I + L diag(b))^-1 (V - e^G K S0^T),   D = diag(b) E      (D = V without retrieval)
//   O  = e^G Q S0^T + P D,                      P_ts = e^(G_t - G_s) q^_t . k^_s  (s <= t)
//   S1 = e^Gamma S0 + (e^(Gamma - G) D)^T K
// and its reverse, given dO and dS1, to
//   dD = P^T dO + e^(Gamma - G) K dS1^T
//   Y  = (I + diag(b) L)^-T dD,   dV = diag(b) Y,   db_t = Y_t . E_t   (dV = dD without retrieval)
//   dS0 = e^Gamma dS1 + (e^G dO)^T Q - (b e^G Y)^T K
//   F = dO D^T (s <= t),  X = Y D^T (s < t),  W_ts = b_t e^(G_t - G_s) X_ts
//   dQ = e^G dO S0 + (F e^(G_t - G_s)) K
//   dK = e^(Gamma - G) D dS1 + (F e^(G_t - G_s))^T Q - b e^G Y S0 - (W + W^T) K
// The log decay g_s scales everything that crosses from before token s to s
// or after it, and nothing else:
//   dg_s = e^Gamma <dS1, S0> + sum_{t<s} u_t + sum_{t>=s} w_t + sum_{t>=s>r} M_tr
//   u_t = k^_t . (e^(Gamma - G_t) dS1^T d_t),  w_t = e^(G_t) (q^_t . S0^T dO_t - b_t k^_t . S0^T Y_t),
//   M = F o P - X o diag(b) L
// (sums of the terms themselves: a difference of two suffix sums over a
// chunk would lose the small gradients of strongly decayed tokens).
//
// Kernels, in order:
//   k_back_table   chunk table (one workgroup)
//   k_back_prep    per chunk and value head: the two triangular inverses, P, decay factors
//   k_back_states  per request, head and 64 state rows: forward chain, keeps S0 and E of every chunk
//   k_back_chain   the same backwards: dS1, Y, dV
//   k_back_chains  both of them in one launch; by themselves only where that is
//                  faster (fp16 and fp32 rows of 65 to 128, many chains)
//   k_back_join    between the segments of a chain, where it is cut (see there)
//   k_back_grad    per chunk and q/k head: dQ, dK (summed over the value heads that share them)
//   k_back_gate    per chunk and value head: dg, db
// and the sums over chunks or heads (k_back_gate_sums, k_back_rate_sums).
//
// Figures at the kernels are of a ragged batch of 8 requests, 29,273 tokens, 16
// q/k and 32 value heads, dk = dv = 128, bf16: 2.93 ms, of which 0.23 ms are the
// floor of its inputs and outputs at the copy rate (5.2 TB/s) and 1.0 ms that of
// its products, in planes, at the rate of a large bf16 product (1234 TFLOP/s).
// What the kernels hand on (S0 and dS1 64 KB each, E and Y 32 KB each, the
// triangular operands 54 KB a chunk and head) is 3.6 GB, written and read once.
//
// Planes.  The products run on v_mfma_f32_16x16x32_bf16 at fp32's precision
// and range: an fp32 operand is cut into three bf16 planes of 8 significant
// bits each, whose sum is the operand exactly, and of the nine products of
// two such operands the six of up to 2^-16 relative size are formed (the
// others are below 2^-24 of the product).  A bf16 activation is one plane, an
// fp16 one two, so that a product with q, k or d_o takes three or five.  The
// rate of the instruction is 16 times the fp32 matrix instruction's, so six
// products are 2.7 times as fast as the fp32 one and three 5.3 times; unlike
// a split into fp16 pairs it needs no scaling, whatever the size of the
// incoming gradient.
//
// Fragments.  Of a 16x16 fp32 accumulator lane l = 16 j + c holds rows 4 j + i
// (i = 0..3) of column c.  Two accumulators over rows 32 x + 0..15 and + 16..31
// are, element by element, the B operand over those 32 rows if operand slot e
// of lane group j stands for row 32 x + 16 (e / 4) + 4 j + e % 4, the order
// used for every operand here: a wave that holds S^T (dk x 16 state rows)
// feeds it to K S^T, that result to (I + ..)^-1, and that one to the state
// update, with no move between lanes.  What a kernel leaves for the next one
// lies as such fragments: 512 bf16 a block and plane (lane l's eight at 8 l),
// or fp32 blocks of 16x16 (lane l's four at 4 l, holding row c, columns 4 j + i).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "gdr_backward_launch.hpp"
#include "gdr_device.hpp"

namespace gdr {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef unsigned int u2 __attribute__((ext_vector_type(2)));
typedef unsigned int u4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int FRAG = 256;    // floats of an fp32 fragment block
constexpr int BLOCK = 512;   // bf16 of a plane's fragment block

template <typename TA> constexpr int planes_of = sizeof(TA) == 4 ? 3 : 1;
template <> constexpr int planes_of<half_t> = 2;

template <int DK> struct Geo {
    static constexpr int C = back_chunk(DK);
    static constexpr int MB = C / 16, KB = DK / 16, MX = MB / 2, KX = KB / 2, TRI = MB * (MB + 1) / 2;
    static constexpr int LC = C + 4;           // floats of a chunk x chunk row in LDS
    static constexpr int ACT = MB * KX;        // blocks of a plane of a chunk's q or k
    static constexpr int NT = back_tri_blocks(C);
};

// Blocks of a triangular chunk x chunk operand, 32 columns each.  Lower: row
// block m, columns of block pair y <= m / 2.  Upper: row block m, y >= m / 2.
template <int MB> __device__ __forceinline__ constexpr int lower_block(int m, int y) { return m < 2 ? m : 2 * m - 2 + y; }
template <int MB> __device__ __forceinline__ constexpr int upper_block(int m, int y)
{
    return MB == 2 ? m : m < 2 ? 2 * m + y : m + 2;
}

// A value that every lane of the wave has alike, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A value that the compiler knows nothing of.
__device__ __forceinline__ int opaque(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

__device__ __forceinline__ constexpr int tri(int m, int k) { return m * (m + 1) / 2 + k; }

__device__ __forceinline__ f4 mfma1(float a, float b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f4 mfma4(f4 a, f4 b, f4 c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma1(a[i], b[i], c);
    return c;
}

__device__ __forceinline__ f4 mfma(b8 a, b8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// a b over the products of planes i + j <= 2, smallest first
template <int NA, int NB>
__device__ __forceinline__ f4 mm(const b8 (&a)[NA], const b8 (&b)[NB], f4 c)
{
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < NA && s - i < NB) c = mfma(a[i], b[s - i], c);
    return c;
}

// The top 16 bits of two words.
__device__ __forceinline__ unsigned int top_halves(unsigned int lo, unsigned int hi)
{
    return __builtin_amdgcn_perm(hi, lo, 0x07060302);
}

// Two floats as N bf16 planes, one word each: each plane is the top 8
// significant bits of what the planes before it leave.
template <int N>
__device__ __forceinline__ void split_pair(float x, float y, unsigned int (&w)[N])
{
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const unsigned int a = __builtin_bit_cast(unsigned int, x), b = __builtin_bit_cast(unsigned int, y);
        w[p] = top_halves(a, b);
        if (p + 1 < N) {
            x -= __builtin_bit_cast(float, a & 0xffff0000u);
            y -= __builtin_bit_cast(float, b & 0xffff0000u);
        }
    }
}

template <int N>
__device__ __forceinline__ void split4(f4 v, u2 (&w)[N])
{
    unsigned int lo[N], hi[N];
    split_pair<N>(v[0], v[1], lo);
    split_pair<N>(v[2], v[3], hi);
#pragma unroll
    for (int p = 0; p < N; ++p) w[p] = u2{lo[p], hi[p]};
}

// Two accumulators (rows 0..15 and 16..31 of a 32-row step) as an operand.
template <int N>
__device__ __forceinline__ void split8(f4 a, f4 b, b8 (&out)[N])
{
    u2 lo[N], hi[N];
    split4<N>(a, lo);
    split4<N>(b, hi);
#pragma unroll
    for (int p = 0; p < N; ++p) out[p] = __builtin_bit_cast(b8, u4{lo[p][0], lo[p][1], hi[p][0], hi[p][1]});
}

__device__ __forceinline__ b8 get_block(const uint16_t *blk)
{
    return __builtin_bit_cast(b8, *reinterpret_cast<const u4 *>(blk + (threadIdx.x & 63) * 8));
}

__device__ __forceinline__ void put_block(uint16_t *blk, b8 v)
{
    *reinterpret_cast<u4 *>(blk + (threadIdx.x & 63) * 8) = __builtin_bit_cast(u4, v);
}

// Half (of 16 columns) `half` of a block of each of three planes, `stride`
// apart: lane `at`'s four.
__device__ __forceinline__ void put_half(uint16_t *blk, size_t stride, int at, int half, f4 v)
{
    u2 w[3];
    split4<3>(v, w);
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<u2 *>(blk + p * stride + at * 8 + half * 4) = w[p];
}

// e^(hi + lo), |lo| below |hi| or so: the sum's rounding error enters as a factor
__device__ __forceinline__ float exp_split(float hi, float lo)
{
    const float s = hi + lo;
    return expf(s) * (1.f + ((hi - s) + lo));
}

__device__ __forceinline__ float exp_of(double x)
{
    const float hi = (float)x;
    return expf(hi) * (1.f + (float)(x - (double)hi));
}

// x of another lane of the quad (every lane is written: no value to keep, and
// no move to set one)
template <int CTRL> __device__ __forceinline__ float quad_move(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// 4x4 transpose within each quad of lanes: element p of lane q <- element q of lane p
__device__ __forceinline__ f4 quad_transpose(f4 v)
{
    const bool odd = threadIdx.x & 1, up = threadIdx.x & 2;
    f4 g;  // the other lane's, moved by every lane before any choice
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = quad_move<0xB1>(v[i ^ 1]);  // lane ^ 1
    v = f4{odd ? g[0] : v[0], odd ? v[1] : g[1], odd ? g[2] : v[2], odd ? v[3] : g[3]};
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = quad_move<0x4E>(v[i ^ 2]);  // lane ^ 2
    return f4{up ? g[0] : v[0], up ? g[1] : v[1], up ? v[2] : g[2], up ? v[3] : g[3]};
}

// Where a lane's four lie in a fragment whose rows are an accumulator tile's rows, after quad_transpose.
__device__ __forceinline__ int quad_lane()
{
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    return (4 * j + (c & 3)) + 16 * (c >> 2);
}

// Accumulator tile -> fragment block whose rows are the tile's rows.
__device__ __forceinline__ void put_frag_rows(float *blk, f4 v)
{
    *reinterpret_cast<f4 *>(blk + quad_lane() * 4) = quad_transpose(v);
}

// Accumulator tile -> fragment block whose rows are the tile's columns: as it lies.
__device__ __forceinline__ void put_frag_cols(float *blk, f4 v)
{
    *reinterpret_cast<f4 *>(blk + (threadIdx.x & 63) * 4) = v;
}

__device__ __forceinline__ f4 get_frag(const float *blk) { return *reinterpret_cast<const f4 *>(blk + (threadIdx.x & 63) * 4); }

// ---- rows of a chunk in memory
// A chunk's `cnt` valid rows of `width` elements, `step` elements apart, as a
// buffer: a load past the last valid row gives zero and a store there does
// nothing, by the bounds check of the buffer instructions, so that a lane's
// offset is the same for every chunk and no load stands under a condition
// (one would be waited for where it is issued).  Lanes whose column lies past
// the width use offset NOWHERE.  VEC: both widths are multiples of 4 (four
// elements from a column that is one lie all within the row or all past it);
// without it elements go one by one.
template <typename TA> struct Raw4 { TA x[4]; };

constexpr unsigned NOWHERE = 0x80000000u;

struct ChunkRows {
    __amdgpu_buffer_rsrc_t buf;
    template <typename TA>
    __device__ __forceinline__ ChunkRows(const TA *first, int cnt, int step, int width, bool live = true)
    {
        const unsigned bytes = live ? ((unsigned)(cnt - 1) * (unsigned)step + (unsigned)width) * (unsigned)sizeof(TA) : 0;  // < 2^31
        buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<TA *>(first), 0, (int)bytes, 0x00027000);
    }
};

// fp32 fragment blocks as a buffer, `blocks` of them (none: every load gives zero)
struct Frags {
    __amdgpu_buffer_rsrc_t buf;
    __device__ __forceinline__ Frags(const float *first, int blocks)
    {
        buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(first), 0, blocks * FRAG * 4, 0x00027000);
    }
    __device__ __forceinline__ f4 get(int block) const
    {
        return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(buf, (threadIdx.x & 63) * 16, block * FRAG * 4, 0));
    }
};

// byte offsets of elements c .. c + 3 of row `row`
template <bool VEC, typename TA> struct At4 {
    unsigned x[VEC ? 1 : 4];
    __device__ __forceinline__ At4(int row, int step, int c, int width)
    {
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : 4); ++i)
            x[i] = c + i < width ? ((unsigned)row * (unsigned)step + (unsigned)(c + i)) * (unsigned)sizeof(TA) : NOWHERE;
    }
    // `rows` rows of `step` elements further (NOWHERE stays past every buffer)
    __device__ __forceinline__ At4 down(int rows, int step) const
    {
        // formed anew at each use (one addition): kept over a chain's steps the
        // offsets would take registers that its operands need
        asm volatile("" : "+s"(step));
        At4 a = *this;
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : 4); ++i) a.x[i] += (unsigned)rows * (unsigned)step * (unsigned)sizeof(TA);
        return a;
    }
};

template <bool VEC, typename TA>
__device__ __forceinline__ Raw4<TA> load_raw4(const ChunkRows &rows, const At4<VEC, TA> &at)
{
    if constexpr (VEC && sizeof(TA) == 4)
        return __builtin_bit_cast(Raw4<TA>, __builtin_amdgcn_raw_buffer_load_b128(rows.buf, at.x[0], 0, 0));
    else if constexpr (VEC)
        return __builtin_bit_cast(Raw4<TA>, __builtin_amdgcn_raw_buffer_load_b64(rows.buf, at.x[0], 0, 0));
    else {
        Raw4<TA> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TA) == 4) r.x[i] = __builtin_bit_cast(TA, __builtin_amdgcn_raw_buffer_load_b32(rows.buf, at.x[i], 0, 0));
            else r.x[i] = __builtin_bit_cast(TA, __builtin_amdgcn_raw_buffer_load_b16(rows.buf, at.x[i], 0, 0));
        }
        return r;
    }
}

template <bool VEC, typename TA>
__device__ __forceinline__ void store4(const ChunkRows &rows, const At4<VEC, TA> &at, f4 v)
{
    Raw4<TA> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.x[i] = from_f32<TA>(v[i]);
    if constexpr (VEC && sizeof(TA) == 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, r), rows.buf, at.x[0], 0, 0);
    else if constexpr (VEC)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, r), rows.buf, at.x[0], 0, 0);
    else
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TA) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned int, r.x[i]), rows.buf, at.x[i], 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, r.x[i]), rows.buf, at.x[i], 0, 0);
        }
}

template <typename TA> __device__ __forceinline__ f4 widen(const Raw4<TA> &r)
{
    return f4{to_f32(r.x[0]), to_f32(r.x[1]), to_f32(r.x[2]), to_f32(r.x[3])};
}

// Values loaded a step ahead, taken up here: without this the compiler moves
// their conversion up to the load, and the wait for memory with it.
template <typename T> __device__ __forceinline__ void arrive(T &v)
{
    static_assert(sizeof(T) % 4 == 0, "whole registers");
    unsigned int w[sizeof(T) / 4];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (unsigned n = 0; n < sizeof(T) / 4; ++n) asm volatile("" : "+v"(w[n]));
    __builtin_memcpy(&v, w, sizeof(T));
}

__device__ __forceinline__ float dot4(f4 a, f4 b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }

// Sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float sum_j(float x)
{
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// Chunk `ci`'s first token and how many of C tokens it has, by its request
// (k_back_prep, which leaves them in a.where for the kernels after it).
__device__ __forceinline__ void chunk_tokens(const BackParams &a, int ci, int C, int64_t &t0, int &cnt)
{
    int lo = 0, hi = a.p.B - 1;  // largest b with off[b] <= ci (ci < off[B])
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.off[mid] <= ci) lo = mid;
        else hi = mid - 1;
    }
    const int skip = uniform(ci - a.off[lo]) * C;
    t0 = (int64_t)uniform(a.tok[2 * lo]) + skip;
    cnt = min(uniform(a.tok[2 * lo + 1]) - skip, C);
}

// Rows of q or k in LDS as planes: C rows of LD bf16, plane after plane.  The
// pad of 16 makes consecutive rows start 8 banks apart, so that the 8-byte
// reads of 16 rows (row_operand) and the transposing reads of 4 rows (col_operand)
// go over all banks evenly.
template <int DK> struct Rows {
    using G = Geo<DK>;
    static constexpr int LD = DK + 16, PLANE = G::C * LD;
    // channels 32 x + .. of row `row`
    template <int NP> static __device__ __forceinline__ void row_operand(const uint16_t *rows, int row, int x, b8 (&out)[NP])
    {
        const int j = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const uint16_t *at = rows + q * PLANE + row * LD + 32 * x + 4 * j;
            const u2 lo = *reinterpret_cast<const u2 *>(at), hi = *reinterpret_cast<const u2 *>(at + 16);
            out[q] = __builtin_bit_cast(b8, u4{lo[0], lo[1], hi[0], hi[1]});
        }
    }
    // tokens 32 y + .. of channel 16 kb + c: the transposing read hands lane c
    // of a group of 16 column c of the 4 rows by 16 columns that the group addresses
    template <int NP> static __device__ __forceinline__ void col_operand(const uint16_t *rows, int kb, int y, b8 (&out)[NP])
    {
        const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const uint16_t *at = rows + q * PLANE + (32 * y + 4 * j + (c >> 2)) * LD + 16 * kb + (c & 3) * 4;
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 lds_s4;
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)at);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(at + 16 * LD));
            const u2 l = __builtin_bit_cast(u2, lo), h = __builtin_bit_cast(u2, hi);
            out[q] = __builtin_bit_cast(b8, u4{l[0], l[1], h[0], h[1]});
        }
    }
};

// The same rows as the 16-bit activations themselves, cut into planes as they are read.
template <int DK, typename TA> struct RawRows {
    static __device__ __forceinline__ void planes(const b8 (&raw)[1], b8 (&out)[planes_of<TA>])
    {
        if constexpr (planes_of<TA> == 1) {
            out[0] = raw[0];
        } else {
            const u4 w = __builtin_bit_cast(u4, raw[0]);
            split8<planes_of<TA>>(widen(__builtin_bit_cast(Raw4<TA>, u2{w[0], w[1]})),
                                  widen(__builtin_bit_cast(Raw4<TA>, u2{w[2], w[3]})), out);
        }
    }
    static __device__ __forceinline__ void row_operand(const uint16_t *rows, int row, int x, b8 (&out)[planes_of<TA>])
    {
        b8 raw[1];
        Rows<DK>::row_operand(rows, row, x, raw);
        planes(raw, out);
    }
    static __device__ __forceinline__ void col_operand(const uint16_t *rows, int kb, int y, b8 (&out)[planes_of<TA>])
    {
        b8 raw[1];
        Rows<DK>::col_operand(rows, kb, y, raw);
        planes(raw, out);
    }
};

// A chunk's rows of q or k on their way from memory to LDS planes, four
// elements at a time, in the registers of NT threads.
template <int DK, typename TA, int NT, bool VEC> struct StageRows {
    using G = Geo<DK>;
    static constexpr int LPR = DK / 4, N = G::C * LPR / NT, NP = planes_of<TA>;
    Raw4<TA> x[N];
    // the thread's place in the first NT / LPR rows
    static __device__ __forceinline__ At4<VEC, TA> place(int step, int dk)
    {
        return At4<VEC, TA>(threadIdx.x / LPR, step, threadIdx.x % LPR * 4, dk);
    }
    __device__ __forceinline__ void load(const TA *first, int cnt, int step, int dk, const At4<VEC, TA> &at)
    {
        const ChunkRows rows(first, cnt, step, dk);
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = load_raw4(rows, at.down(n * (NT / LPR), step));
    }
    // as they are (16-bit activations)
    __device__ __forceinline__ void store_raw(uint16_t *rows) const
    {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int g = threadIdx.x + NT * n;
            *reinterpret_cast<u2 *>(rows + g / LPR * Rows<DK>::LD + g % LPR * 4) = __builtin_bit_cast(u2, x[n]);
        }
    }
    __device__ __forceinline__ void store(uint16_t *rows) const
    {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int g = threadIdx.x + NT * n;
            u2 w[NP];
            if constexpr (NP == 1) w[0] = __builtin_bit_cast(u2, x[n]);
            else split4<NP>(widen(x[n]), w);
#pragma unroll
            for (int q = 0; q < NP; ++q)
                *reinterpret_cast<u2 *>(rows + q * Rows<DK>::PLANE + g / LPR * Rows<DK>::LD + g % LPR * 4) = w[q];
        }
    }
};

// Zero in the gradient rows of tokens that no request covers: those before the
// first and after the last one of cu_seqlens, and those past seq_lens[b].  Run
// by the workgroups `n` of `of` that have no chunk, of which there is always
// one (a request leaves part of its last chunk or the budget's spare one), and
// the more the fewer tokens are covered.
__device__ __forceinline__ void zero_rest(const BackParams &a, int64_t n, int64_t of, int act)
{
    const Params &p = a.p;
    const int64_t first = p.B > 0 ? a.tok[0] : 0;
    const int64_t last = p.B > 0 ? (int64_t)a.tok[2 * p.B - 2] + a.tok[2 * p.B - 1] : 0;
    auto clear = [&](void *base, size_t row, size_t bytes) {  // an even number of bytes a row
        char *at = static_cast<char *>(base) + row * bytes;
        if (bytes % 16 == 0)
            for (size_t i = threadIdx.x; i < bytes / 16; i += 256) reinterpret_cast<u4 *>(at)[i] = u4{0, 0, 0, 0};
        else
            for (size_t i = threadIdx.x; i < bytes / 2; i += 256) reinterpret_cast<uint16_t *>(at)[i] = 0;
    };
    for (int64_t t = n; t < p.T; t += of) {
        int64_t from = first, end = last;  // of the covered tokens that t may be one of
        if (!p.cu_seqlens && p.B > 0) {
            from = t / p.L * p.L;
            end = from + a.tok[2 * (t / p.L) + 1];
        }
        if (t >= from && t < end) {  // on to this workgroup's last token before their end
            t += (end - 1 - t) / of * of;
            continue;
        }
        clear(a.dq, t, (size_t)p.H * p.dk * act);
        clear(a.dk, t, (size_t)p.H * p.dk * act);
        clear(a.dv, t, (size_t)p.HV * p.dv * act);
        if (a.decays) clear(a.d_gate, t, (size_t)p.HV * (p.gate_dt ? 2 : 4));
        if (a.d_rate) clear(a.d_rate, t, 4);
        else if (a.d_beta) clear(a.d_beta, t, (size_t)p.HV * 4);
    }
}

// ---------------------------------------------------------------- prologue
// One workgroup per (chunk, value head).  Value heads that share a q/k head
// each form its K K^T and Q K^T: one workgroup for all of them, the heads in
// turn, took 28 us of the smallest call against 19 us, and gained 5 % of the
// kernel on a long batch of two heads a group (372 and 392 us).  Of fp32 rows it
// leaves k and q as operand fragments with channels as rows (once a q/k head)
// for k_back_grad, whose LDS has no room for them.  Both inverses come from
// one solve: with U = -(I + L diag(b))^-1 L,
//   (I + L diag(b))^-1 = I + U diag(b),   (I + diag(b) L)^-1 = I + diag(b) U
// (two solves: 390 us).  It goes by 16x16 blocks on the fp32 matrix instruction:
// the diagonal ones by forward substitution, a thread a column; then wave j
// takes block column j down, U_ij = -(I + U_ii diag(b)) (L_ij + sum_k L_ik diag(b) U_kj)
// over j <= k < i, its U_kj staying in the accumulators' layout.  360 us: 0.85 GB
// written and 0.5 GB read, 3.8 TB/s; bound by the solve's dependent steps, hidden
// behind other workgroups' (4 a CU).
template <int DK, typename TA, bool RETR, bool VEC>
__global__ __launch_bounds__(256) void k_back_prep(const BackParams a)
{
    using G = Geo<DK>;
    using RW = Rows<DK>;
    constexpr int C = G::C, MB = G::MB, MX = G::MX, KX = G::KX, LC = G::LC, TRI = G::TRI, ACT = G::ACT, NT = G::NT;
    constexpr int NP = planes_of<TA>, SLOTS = (TRI + 3) / 4, INV = 16 * 20;
    constexpr int STAGE = 2 * NP * RW::PLANE * 2, SOLVE = (C * LC + MB * INV) * 4;
    __shared__ __align__(16) char mem[STAGE > SOLVE ? STAGE : SOLVE];
    __shared__ double s_G[C];
    __shared__ __align__(16) float s_b[C];
    __shared__ float s_rq[C], s_rk[C];

    const Params &p = a.p;
    const int ci = blockIdx.x / p.HV, h = blockIdx.x % p.HV, R = p.HV / p.H, hq = h / R, used = a.off[p.B];
    if (ci >= used) {
        if (a.zero_rest) zero_rest(a, blockIdx.x - used * p.HV, (a.chunks - used) * p.HV, sizeof(TA));
        return;
    }
    int64_t t0;
    int cnt;
    chunk_tokens(a, ci, C, t0, cnt);

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), c = lane & 15, j = lane >> 4;
    if (h == 0 && tid == 0) {
        a.where[2 * ci] = (int32_t)t0;
        a.where[2 * ci + 1] = cnt;
    }
    uint16_t *Kr = reinterpret_cast<uint16_t *>(mem), *Qr = Kr + NP * RW::PLANE;

    // decays and rates, a lane a token
    if (wave == 0) {
        double g = 0.0;
        float b = 0.f;
        if (lane < cnt) {
            const size_t th = (size_t)(t0 + lane) * p.HV + h;
            if (a.decays) {
                // a decay of -inf (a reset) would make differences of G undefined; e^-1e5 is 0 too
                const float x = log_decay(p, th, h);
                g = x < -1e5f ? -1e5 : (double)x;
            }
            b = RETR ? update_rate(p, th) : 1.f;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double x = __shfl_up(g, o);
            if (lane >= o) g += x;
        }
        const double end = __shfl(g, C - 1);
        if (lane < C) {
            s_G[lane] = g;
            s_b[lane] = b;
            float *sc = a.sc + (size_t)blockIdx.x * (BACK_SC * C);
            const float hi = (float)g;
            sc[SC_EG * C + lane] = exp_of(g);
            sc[SC_KD * C + lane] = exp_of(end - g);
            sc[SC_B * C + lane] = b;
            sc[SC_GH * C + lane] = hi;
            sc[SC_GL * C + lane] = (float)(g - (double)hi);
        }
    }
    // rows of q and k, and the reciprocals of their norms
    {
        StageRows<DK, TA, 256, VEC> k, q;
        constexpr int LPR = DK / 4;  // lanes of a row
        const size_t first = ((size_t)t0 * p.H + hq) * p.dk;
        const auto at = k.place(p.H * p.dk, p.dk);
        k.load(static_cast<const TA *>(p.k) + first, cnt, p.H * p.dk, p.dk, at);
        q.load(static_cast<const TA *>(p.q) + first, cnt, p.H * p.dk, p.dk, at);
#pragma unroll
        for (int n = 0; n < k.N; ++n) {
            const int g = tid + 256 * n;
            float rq = 1.f, rk = 1.f;
            if (p.qk_l2_norm) {
                const f4 qv = widen(q.x[n]), kv = widen(k.x[n]);
                float sq = dot4(qv, qv), sk = dot4(kv, kv);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) {
                    sq += __shfl_xor(sq, o);
                    sk += __shfl_xor(sk, o);
                }
                rq = 1.f / sqrtf(sq + 1e-12f);
                rk = 1.f / sqrtf(sk + 1e-12f);
            }
            if (g % LPR == 0) {
                s_rq[g / LPR] = rq * p.scale;
                s_rk[g / LPR] = rk;
            }
        }
        k.store(Kr);
        q.store(Qr);
    }
    __syncthreads();

    if constexpr (NP == 3) {
        uint16_t *act = a.act + ((size_t)ci * p.H + hq) * 2 * NP * ACT * BLOCK;
        for (int n = h % R == 0 ? wave : 2 * ACT; n < 2 * ACT; n += 4) {
            const int kind = n / ACT, blk = n % ACT;
            b8 v[NP];
            RW::col_operand(kind == 0 ? Kr : Qr, blk / MX, blk % MX, v);
#pragma unroll
            for (int q = 0; q < NP; ++q) put_block(act + (size_t)((kind * NP + q) * ACT + blk) * BLOCK, v[q]);
        }
    }

    // lower triangle of Q K^T and K K^T, tile (m, kb): rows t of block m, columns s of block kb
    f4 qk[SLOTS], kk[SLOTS];
    int tm[SLOTS], tk[SLOTS];
#pragma unroll
    for (int n = 0; n < SLOTS; ++n) {
        const int id = wave + 4 * n;
        int m = 0;
        while (m + 1 < MB && tri(m + 1, 0) <= id) ++m;
        tm[n] = id < TRI ? m : -1;
        tk[n] = id - tri(m, 0);
        qk[n] = kk[n] = f4{0.f, 0.f, 0.f, 0.f};
        if (id < TRI) {
#pragma unroll
            for (int x = 0; x < KX; ++x) {
                b8 s[NP], q[NP], k[NP];
                RW::row_operand(Kr, 16 * tk[n] + c, x, s);
                RW::row_operand(Qr, 16 * tm[n] + c, x, q);
                qk[n] = mm(q, s, qk[n]);
                if (RETR) {
                    RW::row_operand(Kr, 16 * tm[n] + c, x, k);
                    kk[n] = mm(k, s, kk[n]);
                }
            }
            const float rs = s_rk[16 * tk[n] + c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * tm[n] + 4 * j + i;
                qk[n][i] *= rs * s_rq[t];
                kk[n][i] *= rs * s_rk[t];
            }
        }
    }
    __syncthreads();  // the staged rows give way to L and the diagonal inverses

    float *Lm = reinterpret_cast<float *>(mem), *inv = Lm + C * LC;
    const f4 zero = {0.f, 0.f, 0.f, 0.f};
    {
        const size_t rec = blockIdx.x;
        constexpr size_t STRIDE = (size_t)NT * BLOCK;
        uint16_t *pt = a.tri + rec * 3 * (RETR ? 3 : 1) * STRIDE;  // P^T; (I + diag(b) L)^-T; (I + L diag(b))^-1
        if (tid < C) {
            float *sc = a.sc + rec * (BACK_SC * C);
            sc[SC_RQ * C + tid] = s_rq[tid];
            sc[SC_RK * C + tid] = s_rk[tid];
        }
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) {
            const int m = tm[n], kb = tk[n];
            if (m >= 0) {
                const int s = 16 * kb + c;
                const double gs = s_G[s];
                f4 P;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * m + 4 * j + i;
                    const float e = s <= t ? exp_of(s_G[t] - gs) : 0.f;
                    P[i] = e * qk[n][i];
                    if (RETR) Lm[t * LC + s] = s < t ? e * kk[n][i] : 0.f;
                }
                uint16_t *blk = pt + upper_block<MB>(kb, m / 2) * BLOCK;
                put_half(blk, STRIDE, lane, m & 1, P);
                if (m == kb && (m & 1)) put_half(blk, STRIDE, lane, 0, zero);
            }
        }
        if constexpr (RETR) {
            uint16_t *t2 = pt + 3 * STRIDE, *t1 = t2 + 3 * STRIDE;
            __syncthreads();
            if (tid < MB * 16) {
                const int d = tid / 16, col = tid & 15;
                float x[16];
#pragma unroll
                for (int row = 0; row < 16; ++row) {
                    float acc = -Lm[(16 * d + row) * LC + 16 * d + col];
#pragma unroll
                    for (int s = 0; s < row; ++s) acc -= Lm[(16 * d + row) * LC + 16 * d + s] * s_b[16 * d + s] * x[s];
                    x[row] = acc;
                    inv[d * INV + row * 20 + col] = acc;
                }
            }
            __syncthreads();
            if (wave < MB) {
                const float b = s_b[16 * wave + c];
                f4 U[MB];
#pragma unroll
                for (int i = 0; i < MB; ++i) U[i] = zero;
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    if (i == wave) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) U[i][e] = inv[i * INV + (4 * j + e) * 20 + c];
                    } else if (i > wave) {
                        f4 acc;
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[e] = Lm[(16 * i + 4 * j + e) * LC + 16 * wave + c];
#pragma unroll
                        for (int k = 0; k < i; ++k) {
                            if (k < wave) continue;
                            acc = mfma4(*reinterpret_cast<const f4 *>(Lm + (16 * i + c) * LC + 16 * k + 4 * j) *
                                            *reinterpret_cast<const f4 *>(s_b + 16 * k + 4 * j), U[k], acc);
                        }
                        f4 T = *reinterpret_cast<const f4 *>(inv + i * INV + c * 20 + 4 * j) * *reinterpret_cast<const f4 *>(s_b + 16 * i + 4 * j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) T[e] += c == 4 * j + e ? 1.f : 0.f;
                        U[i] = -mfma4(T, acc, zero);
                    }
                    if (i >= wave) {  // tile: rows t of block i, columns s of block `wave`
                        f4 one = zero;
#pragma unroll
                        for (int e = 0; e < 4; ++e) one[e] = i == wave && c == 4 * j + e ? 1.f : 0.f;
                        uint16_t *blk = t1 + lower_block<MB>(i, wave / 2) * BLOCK;
                        put_half(blk, STRIDE, quad_lane(), wave & 1, quad_transpose(U[i] * b + one));
                        if (i == wave && !(i & 1)) put_half(blk, STRIDE, lane, 1, zero);
                        blk = t2 + upper_block<MB>(wave, i / 2) * BLOCK;
                        put_half(blk, STRIDE, lane, i & 1, *reinterpret_cast<const f4 *>(s_b + 16 * i + 4 * j) * U[i] + one);
                        if (i == wave && (i & 1)) put_half(blk, STRIDE, lane, 0, zero);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------- pieces of the chains
// BLOCKS consecutive fragment blocks on their way from memory to LDS, in the
// registers of 256 threads.
template <int BLOCKS> struct Copy {
    static constexpr int WORDS = BLOCKS * 64, N = (WORDS + 255) / 256;
    u4 x[N];
    __device__ __forceinline__ void load(const uint16_t *src)
    {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + 256 * n;
            x[n] = reinterpret_cast<const u4 *>(src)[at < WORDS ? at : 0];
        }
    }
    __device__ __forceinline__ void store(uint16_t *dst) const
    {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int at = threadIdx.x + 256 * n;
            if (at < WORDS) reinterpret_cast<u4 *>(dst)[at] = x[n];
        }
    }
};

// Columns 16 vb .. + 15 (of `width`) of the chunk's rows: a lane loads four
// columns of row 16 m + 4 j + c % 4, and a transpose within quads of lanes
// gives the accumulators' layout.
template <int MB, typename TA, bool VEC> struct Cols {
    Raw4<TA> x[MB];
    static __device__ __forceinline__ At4<VEC, TA> place(int vb, int step, int width)
    {
        const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
        return At4<VEC, TA>(4 * j + (c & 3), step, 16 * vb + 4 * (c >> 2), width);
    }
    __device__ __forceinline__ void load(const TA *first, int cnt, int step, int width, const At4<VEC, TA> &at)
    {
        const ChunkRows rows(first, cnt, step, width);
#pragma unroll
        for (int m = 0; m < MB; ++m) x[m] = load_raw4(rows, at.down(16 * m, step));
    }
    __device__ __forceinline__ void get(f4 (&out)[MB]) const
    {
#pragma unroll
        for (int m = 0; m < MB; ++m) out[m] = quad_transpose(widen(x[m]));
    }
};

// Row `row` of a (request, head)'s dv state rows as S^T tiles: dk = 16 kb + 4 j + i.
template <bool VEC, int KB>
__device__ __forceinline__ void load_state(f4 (&S)[KB], const float *head, int row, int dv, int dk, int j)
{
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        S[kb] = f4{0.f, 0.f, 0.f, 0.f};
        if (head) S[kb] = widen(load_raw4(ChunkRows(head, dv, dk, dk), At4<VEC, float>(row, dk, 16 * kb + 4 * j, dk)));
    }
}

// acc[m] += K S^T, K's planes in LDS
template <int DK, int NP>
__device__ __forceinline__ void rows_times_state(f4 (&acc)[Geo<DK>::MB], const uint16_t *rows, const f4 (&S)[Geo<DK>::KB], int c)
{
    using G = Geo<DK>;
#pragma unroll
    for (int x = 0; x < G::KX; ++x) {
        b8 s[3];
        split8<3>(S[2 * x], S[2 * x + 1], s);
        b8 k[G::MB][NP];
#pragma unroll
        for (int m = 0; m < G::MB; ++m) Rows<DK>::row_operand(rows, 16 * m + c, x, k[m]);
#pragma unroll
        for (int n = 2; n >= 0; --n)
#pragma unroll
            for (int i = 0; i <= n; ++i)
                if (i < NP)
#pragma unroll
                    for (int m = 0; m < G::MB; ++m) acc[m] = mfma(k[m][i], s[n - i], acc[m]);
    }
}

// S = gamma S + rows^T X (+ rows2^T X2), the rows' (k's or q's) planes in LDS, X
// by token blocks.  The products are summed by themselves and reach S in one
// rounding: added to it plane by plane they would round it six times a chunk,
// and over a long chain without decay that error adds up.
template <int DK, int NP, bool TWO>
__device__ __forceinline__ void state_update(f4 (&S)[Geo<DK>::KB], float gamma, const uint16_t *rows, const f4 (&X)[Geo<DK>::MB],
                                             const uint16_t *rows2, const f4 (&X2)[Geo<DK>::MB])
{
    using G = Geo<DK>;
    b8 x[TWO ? 2 : 1][G::MX][3];
#pragma unroll
    for (int y = 0; y < G::MX; ++y) {
        split8<3>(X[2 * y], X[2 * y + 1], x[0][y]);
        if (TWO) split8<3>(X2[2 * y], X2[2 * y + 1], x[TWO ? 1 : 0][y]);
    }
#pragma unroll
    for (int k0 = 0; k0 < G::KB; k0 += 4) {
        f4 sum[4];
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) sum[kb] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int y = 0; y < G::MX; ++y)
#pragma unroll
            for (int two = 0; two < (TWO ? 2 : 1); ++two) {
                b8 k[4][NP];
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) Rows<DK>::col_operand(two ? rows2 : rows, k0 + kb, y, k[kb]);
#pragma unroll
                for (int n = 2; n >= 0; --n)
#pragma unroll
                    for (int i = 0; i <= n; ++i)
                        if (i < NP)
#pragma unroll
                            for (int kb = 0; kb < 4; ++kb) sum[kb] = mfma(k[kb][i], x[two][y][n - i], sum[kb]);
            }
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[k0 + kb][i] = fmaf(gamma, S[k0 + kb][i], sum[kb][i]);
    }
}

// acc[m] += T X over token blocks 2 y and 2 y + 1 for a triangular operand's planes in LDS
template <int MB, bool UPPER, int NB>
__device__ __forceinline__ void tri_times(f4 (&acc)[MB], const uint16_t *T, int y, const b8 (&x)[NB])
{
    constexpr int NT = back_tri_blocks(16 * MB);
#pragma unroll
    for (int i = 2; i >= 0; --i) {  // planes of T, smallest first
        b8 t[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m)
            if (UPPER ? 2 * y + 1 >= m : 2 * y <= m)
                t[m] = get_block(T + (i * NT + (UPPER ? upper_block<MB>(m, y) : lower_block<MB>(m, y))) * BLOCK);
#pragma unroll
        for (int n = 2 - i; n >= 0; --n)
            if (n < NB)
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    if (UPPER ? 2 * y + 1 >= m : 2 * y <= m) acc[m] = mfma(t[m], x[n], acc[m]);
    }
}

// Scalars of a chunk on their way to LDS: thread t < C holds token t's.
struct ChunkScalars {
    float eg, kd, b, rq, rk;
    __device__ __forceinline__ void load(const float *sc, int C, int t)
    {
        t = t < C ? t : C - 1;
        eg = sc[SC_EG * C + t];
        kd = sc[SC_KD * C + t];
        b = sc[SC_B * C + t];
        rq = sc[SC_RQ * C + t];
        rk = sc[SC_RK * C + t];
    }
};

// ---------------------------------------------------------------- segments
// A chain step maps every state row s affinely and alike, s <- s M_c + c_c.
// With few (request, head) pairs a chain is cut into a.nseg segments (the rule is
// at back_segments): a first pass
// (CARRY) gives each segment's M (rows of the identity as start, values left
// out) and its c (zero start, nothing kept), k_back_join hands the true states
// from segment to segment, and the pass that keeps its results runs all
// segments side by side.  Backwards a row of dS takes M^T, so M is formed once.
// States between kernels are accumulators as they lie: [pair][segment][row
// block][kb][lane] float4.
struct Segment {
    int first, count, len;  // chunks; tokens
    int64_t start;
    // segment `seg` of a.nseg of request b
    template <int C> static __device__ __forceinline__ Segment of(const BackParams &a, int b, int seg)
    {
        const int f0 = uniform(a.off[b]), n0 = uniform(a.off[b + 1]) - f0;
        const int lo = (int)((int64_t)n0 * seg / a.nseg), hi = (int)((int64_t)n0 * (seg + 1) / a.nseg);
        return Segment{f0 + lo, hi - lo, min(uniform(a.tok[2 * b + 1]) - lo * C, (hi - lo) * C), (int64_t)uniform(a.tok[2 * b]) + lo * C};
    }
};

__device__ __forceinline__ size_t seg_at(const BackParams &a, int bh, int seg, int blocks, int block, int KB)
{
    return ((((size_t)bh * a.nseg + seg) * blocks + block) * KB) * FRAG;
}

template <int KB> __device__ __forceinline__ void put_state(float *at, const f4 (&S)[KB])
{
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) put_frag_cols(at + kb * FRAG, S[kb]);
}

template <int KB> __device__ __forceinline__ void get_state(f4 (&S)[KB], const float *at)
{
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) S[kb] = get_frag(at + kb * FRAG);
}

// One workgroup per (request, value head, 16 state rows): the states at the
// segments' starts (backwards: at their ends), one after the other.  A wave
// forms two 16-channel blocks of each state from all of the one before, which
// goes round the waves through LDS as planes; its rows of M and its carry are
// loaded a segment ahead.  65,536 tokens x 16 heads: 14 us for 8 segments; with
// 64 state rows a workgroup, each wave all channels of 16 of them, 65 us.
template <int DK, bool REVERSE, bool VEC>
__device__ __forceinline__ void join_segments(const BackParams &a, int block, uint16_t (&s_x)[2][3 * Geo<DK>::KX * BLOCK])
{
    using G = Geo<DK>;
    constexpr int KB = G::KB, KX = G::KX;
    const Params &p = a.p;
    const int vb = block % a.VB, bh = block / a.VB;
    float *seg_carry = REVERSE ? a.seg_dcarry : a.seg_carry, *seg_state = REVERSE ? a.seg_dstate : a.seg_state;
    const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    const float *init = REVERSE ? a.d_final : p.init;
    f4 m[2][KB], carry[2];
    auto rows = [&](int seg) { return (REVERSE ? a.seg_m : a.seg_mt) + seg_at(a, bh, seg, KB, 2 * wave, KB); };
    auto add = [&](int seg) { return seg_carry + seg_at(a, bh, seg, a.VB, vb, KB) + 2 * wave * FRAG; };
    auto fetch = [&](const float *M, int kb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) m[h][kb] = get_frag(M + (h * KB + kb) * FRAG);
    };
    {
        const int seg = REVERSE ? a.nseg - 1 : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) carry[h] = get_frag(add(seg) + h * FRAG);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) fetch(rows(seg), kb);
    }
    f4 S[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        S[x] = f4{0.f, 0.f, 0.f, 0.f};
        if (init)
            S[x] = widen(load_raw4(ChunkRows(init + (size_t)bh * p.dv * p.dk, p.dv, p.dk, p.dk),
                                   At4<VEC, float>(16 * vb + c, p.dk, 16 * (2 * wave + x) + 4 * j, p.dk)));
    }
    for (int n = 0; n < a.nseg; ++n) {
        const int seg = REVERSE ? a.nseg - 1 - n : n;
        float *out = seg_state + seg_at(a, bh, seg, a.VB, vb, KB) + 2 * wave * FRAG;
        uint16_t *x = s_x[n & 1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            put_frag_cols(out + h * FRAG, S[h]);
            put_half(x + wave * BLOCK, KX * BLOCK, lane, h, S[h]);
        }
        if (n + 1 == a.nseg) break;
        lds_barrier();  // one a segment: the other buffer's readers have passed the last one
        const int ahead = min(n + 1, a.nseg - 2), to = REVERSE ? a.nseg - 1 - ahead : ahead;
        arrive(carry);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            S[h] = carry[h];
            carry[h] = get_frag(add(to) + h * FRAG);
        }
#pragma unroll
        for (int y = 0; y < KX; ++y) {
            b8 r[2][3], v[3];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                arrive(m[h][2 * y]);
                arrive(m[h][2 * y + 1]);
                split8<3>(m[h][2 * y], m[h][2 * y + 1], r[h]);
            }
            fetch(rows(to), 2 * y);
            fetch(rows(to), 2 * y + 1);
#pragma unroll
            for (int q = 0; q < 3; ++q) v[q] = get_block(x + (q * KX + y) * BLOCK);
#pragma unroll
            for (int h = 0; h < 2; ++h) S[h] = mm(r[h], v, S[h]);
        }
    }
}

template <int DK, bool VEC>
__global__ __launch_bounds__(DK * 2) void k_back_join(const BackParams a)
{
    __shared__ __align__(16) uint16_t s_x[2][3 * Geo<DK>::KX * BLOCK];
    const int n = gridDim.x / 2;
    if ((int)blockIdx.x < n) join_segments<DK, false, VEC>(a, blockIdx.x, s_x);
    else join_segments<DK, true, VEC>(a, blockIdx.x - n, s_x);
}

// ---------------------------------------------------------------- forward chain
// One workgroup per (segment, request, value head, 64 state rows); wave w keeps S^T of
// 16 rows in its accumulators over the whole chain.  Everything that a step
// reads from memory is loaded one step ahead: within the step there are only
// LDS reads, and stores that nothing waits for.  Two workgroups a CU where
// registers allow.  656 us by itself: 1.45 GB written and 1.3 GB read, 4.2 TB/s
// over all, but the longest request's 109 steps, 6 us each, are what it waits
// for: while all 512 chains run it is bound by memory and VALU, at the end by
// latency (beside the other chain: see k_back_chains).
template <int DK, typename TA, bool RETR> struct StatesLds {
    __align__(16) uint16_t Kr[planes_of<TA> * Rows<DK>::PLANE];
    __align__(16) uint16_t T[RETR ? 3 * Geo<DK>::NT * BLOCK : 8];
    __align__(16) float s_eg[Geo<DK>::C], s_x[Geo<DK>::C];
    float s_gamma;
};

template <int DK, typename TA, bool RETR, bool VEC, bool CARRY>
__device__ __forceinline__ void states_chain(const BackParams &a, int block, StatesLds<DK, TA, RETR> &lds)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, MX = G::MX, KB = G::KB, NT = G::NT, NP = planes_of<TA>;
    constexpr int TRIS = RETR ? 3 : 1;  // triangular operands of a record
    uint16_t *Kr = lds.Kr, *T = lds.T;
    float *s_eg = lds.s_eg, *s_x = lds.s_x, &s_gamma = lds.s_gamma;
    const Params &p = a.p;
    const int tiles = a.VB / 4 + (CARRY ? KB / 4 : 0);
    const int tile = block % tiles, pair = block / tiles, seg = pair / (p.B * p.HV);
    const int h = pair % p.HV, b = uniform(a.order[pair / p.HV % p.B]), bh = b * p.HV + h;
    const Segment sg = Segment::of<C>(a, b, seg);
    const int first = sg.first, count = sg.count, len = sg.len;
    const int64_t start = sg.start;
    if (!CARRY && count == 0) return;
    const int hq = h / (p.HV / p.H);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), c = lane & 15, j = lane >> 4;
    const bool map = CARRY && tile >= a.VB / 4;  // rows of M
    const int vb = tile * 4 + wave - (map ? a.VB : 0), col = vb * 16 + c;

    f4 S[KB], E[MB];
    if constexpr (CARRY) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[kb][i] = map && 16 * kb + 4 * j + i == col ? 1.f : 0.f;
    } else if (a.nseg > 1) {
        get_state<KB>(S, a.seg_state + seg_at(a, bh, seg, a.VB, vb, KB));
    } else {
        load_state<VEC>(S, p.init ? p.init + (size_t)bh * p.dv * p.dk : nullptr, col, p.dv, p.dk, j);
    }
    StageRows<DK, TA, 256, VEC> k;
    Copy<RETR ? 3 * NT : 0> tri_next;
    ChunkScalars x;
    Cols<MB, TA, VEC> v;
    const int kstep = p.H * p.dk, vstep = p.HV * p.dv;
    const auto kat = k.place(kstep, p.dk);
    const auto vat = v.place(vb, vstep, p.dv);
    auto fetch = [&](int n) {
        const int cnt = min(len - n * C, C);
        const size_t t0 = (size_t)start + (size_t)n * C, rec = (size_t)(first + n) * p.HV + h;
        k.load(static_cast<const TA *>(p.k) + t0 * kstep + hq * p.dk, cnt, kstep, p.dk, kat);
        tri_next.load(a.tri + (rec * TRIS + TRIS - 1) * 3 * NT * BLOCK);
        x.load(a.sc + rec * (BACK_SC * C), C, tid);
        v.load(static_cast<const TA *>(p.v) + t0 * vstep + h * p.dv, cnt, vstep, p.dv, vat);
    };
    auto stage = [&](int n) {  // chunk n's operands into LDS, the next chunk's on their way
        lds_barrier();  // the previous step's reads
        arrive(k.x);
        arrive(x);
        arrive(v.x);
        k.store(Kr);
        tri_next.store(T);
        if (tid < C) {
            s_eg[tid] = x.eg * x.rk;
            s_x[tid] = x.kd * x.b * x.rk;
            if (tid == C - 1) s_gamma = x.eg;
        }
        v.get(E);
        fetch(min(n + 1, count - 1));
        lds_barrier();
    };
    if (count > 0) fetch(0);
    for (int n = 0; n < count; ++n) {
        const size_t rec = (size_t)(first + n) * p.HV + h;
        stage(n);
        if constexpr (CARRY) {
            if (map)
#pragma unroll
                for (int m = 0; m < MB; ++m) E[m] = f4{0.f, 0.f, 0.f, 0.f};
        } else {
            float *Sw = a.s + (rec * KB * a.VB + vb) * FRAG;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) put_frag_rows(Sw + (size_t)kb * a.VB * FRAG, S[kb]);
        }
        if constexpr (RETR) {
            f4 Y[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) Y[m] = f4{0.f, 0.f, 0.f, 0.f};
            rows_times_state<DK, NP>(Y, Kr, S, c);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                Y[m] = E[m] - *reinterpret_cast<const f4 *>(s_eg + 16 * m + 4 * j) * Y[m];
                E[m] = f4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int y = 0; y < MX; ++y) {
                b8 z[3];
                split8<3>(Y[2 * y], Y[2 * y + 1], z);
                tri_times<MB, false>(E, T, y, z);
            }
        }
        float *Ew = a.e + (rec * MB * a.VB + vb) * FRAG;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (!CARRY) put_frag_rows(Ew + (size_t)m * a.VB * FRAG, E[m]);
            E[m] *= *reinterpret_cast<const f4 *>(s_x + 16 * m + 4 * j);
        }
        state_update<DK, NP, false>(S, s_gamma, Kr, E, Kr, E);
    }
    if constexpr (CARRY) {
        if (map) {  // M as fragment blocks of its rows (for M) and of its columns (for M^T)
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                put_frag_cols(a.seg_m + seg_at(a, bh, seg, KB, vb, KB) + kb * FRAG, S[kb]);
                put_frag_rows(a.seg_mt + seg_at(a, bh, seg, KB, kb, KB) + vb * FRAG, S[kb]);
            }
        } else {
            put_state<KB>(a.seg_carry + seg_at(a, bh, seg, a.VB, vb, KB), S);
        }
    }
}

// ---------------------------------------------------------------- backward chain
// As the forward chain; a step has two triangular products and the update of
// dS by q and by k.  1.03 ms by itself: 1.7 GB written and 2.4 GB read, 3.9 TB/s; 109 steps
// of 9.4 us, of which a wave's 198 matrix instructions take 1.3 us and its 1100
// VALU instructions (planes, transposes) 2 us: 56 % of the waves' time is waiting
// for LDS, memory and the step before.  By itself it gained nothing from
// transposes across banks instead of quads, which spared 300 of the latter, nor
// from one XCD for the workgroups that share operands (1041 us against 1047);
// neither was tried in the joint launch, which memory bounds.
// fp16 rows lie in LDS as two planes: 112 KB and one workgroup a CU, where bf16
// has 75 KB and two.
template <int DK, typename TA, bool RETR> struct ChainLds {
    __align__(16) uint16_t Kr[planes_of<TA> * Rows<DK>::PLANE], Qr[planes_of<TA> * Rows<DK>::PLANE];
    __align__(16) uint16_t T[(RETR ? 6 : 3) * Geo<DK>::NT * BLOCK];  // P^T, then (I + diag(b) L)^-T
    __align__(16) float s_kd[Geo<DK>::C], s_b[Geo<DK>::C], s_q[Geo<DK>::C], s_k[Geo<DK>::C];
    float s_gamma;
};

template <int DK, typename TA, bool RETR, bool VEC, bool CARRY>
__device__ __forceinline__ void gradient_chain(const BackParams &a, int block, ChainLds<DK, TA, RETR> &lds)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, MX = G::MX, KB = G::KB, NT = G::NT, NP = planes_of<TA>;
    constexpr int TRIS = RETR ? 3 : 1;
    uint16_t *Kr = lds.Kr, *Qr = lds.Qr, *T = lds.T;
    float *s_kd = lds.s_kd, *s_b = lds.s_b, *s_q = lds.s_q, *s_k = lds.s_k, &s_gamma = lds.s_gamma;
    const Params &p = a.p;
    const int tiles = a.VB / 4;
    const int tile = block % tiles, pair = block / tiles, seg = pair / (p.B * p.HV);
    const int h = pair % p.HV, b = uniform(a.order[pair / p.HV % p.B]), bh = b * p.HV + h;
    const Segment sg = Segment::of<C>(a, b, seg);
    const int first = sg.first, count = sg.count, len = sg.len;
    const int64_t start = sg.start;
    const int hq = h / (p.HV / p.H);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), c = lane & 15, j = lane >> 4;
    const int vb = tile * 4 + wave, col = vb * 16 + c;

    f4 dS[KB];
    if constexpr (CARRY) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) dS[kb] = f4{0.f, 0.f, 0.f, 0.f};
    } else if (a.nseg > 1) {
        get_state<KB>(dS, a.seg_dstate + seg_at(a, bh, seg, a.VB, vb, KB));
    } else {
        load_state<VEC>(dS, a.d_final ? a.d_final + (size_t)bh * p.dv * p.dk : nullptr, col, p.dv, p.dk, j);
    }
    StageRows<DK, TA, 256, VEC> k, q;
    Copy<(RETR ? 6 : 3) * NT> tri_next;
    ChunkScalars x;
    Cols<MB, TA, VEC> o;
    const int kstep = p.H * p.dk, vstep = p.HV * p.dv;
    const auto kat = k.place(kstep, p.dk);
    const auto vat = o.place(vb, vstep, p.dv);
    auto fetch = [&](int n) {
        const int cnt = min(len - n * C, C);
        const size_t t0 = (size_t)start + (size_t)n * C, rec = (size_t)(first + n) * p.HV + h;
        k.load(static_cast<const TA *>(p.k) + t0 * kstep + hq * p.dk, cnt, kstep, p.dk, kat);
        q.load(static_cast<const TA *>(p.q) + t0 * kstep + hq * p.dk, cnt, kstep, p.dk, kat);
        tri_next.load(a.tri + rec * TRIS * 3 * NT * BLOCK);
        x.load(a.sc + rec * (BACK_SC * C), C, tid);
        o.load(static_cast<const TA *>(a.d_o) + t0 * vstep + h * p.dv, cnt, vstep, p.dv, vat);
    };
    f4 dO[MB];
    auto stage = [&](int n) {
        lds_barrier();
        arrive(k.x);
        arrive(q.x);
        arrive(x);
        arrive(o.x);
        k.store(Kr);
        q.store(Qr);
        tri_next.store(T);
        if (tid < C) {
            s_kd[tid] = x.kd * x.rk;
            s_b[tid] = x.b;
            s_q[tid] = x.eg * x.rq;
            s_k[tid] = -x.eg * x.rk;
            if (tid == C - 1) s_gamma = x.eg;
        }
        o.get(dO);
        fetch(max(n - 1, 0));
        lds_barrier();
    };
    if (count > 0) fetch(count - 1);
    for (int n = count - 1; n >= 0; --n) {
        const size_t rec = (size_t)(first + n) * p.HV + h;
        const int cnt = min(len - n * C, C);
        stage(n);
        if constexpr (!CARRY) {
            float *Sw = a.ds + (rec * KB * a.VB + vb) * FRAG;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) put_frag_rows(Sw + (size_t)kb * a.VB * FRAG, dS[kb]);
        }
        f4 D[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) D[m] = f4{0.f, 0.f, 0.f, 0.f};
        rows_times_state<DK, NP>(D, Kr, dS, c);
#pragma unroll
        for (int m = 0; m < MB; ++m) D[m] *= *reinterpret_cast<const f4 *>(s_kd + 16 * m + 4 * j);
#pragma unroll
        for (int y = 0; y < MX; ++y) {
            b8 g[NP];
            split8<NP>(dO[2 * y], dO[2 * y + 1], g);
            tri_times<MB, true>(D, T, y, g);
        }
        if constexpr (RETR) {
            f4 Y[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) Y[m] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int y = 0; y < MX; ++y) {
                b8 d[3];
                split8<3>(D[2 * y], D[2 * y + 1], d);
                tri_times<MB, true>(Y, T + 3 * NT * BLOCK, y, d);
            }
            float *Yw = a.y + (rec * MB * a.VB + vb) * FRAG;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (!CARRY) put_frag_rows(Yw + (size_t)m * a.VB * FRAG, Y[m]);
                D[m] = Y[m] * *reinterpret_cast<const f4 *>(s_b + 16 * m + 4 * j);
            }
        }
        const ChunkRows dvrows(static_cast<const TA *>(a.dv) + ((size_t)start + (size_t)n * C) * vstep + h * p.dv, cnt, vstep, p.dv);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (!CARRY) store4(dvrows, vat.down(16 * m, vstep), quad_transpose(D[m]));
            dO[m] *= *reinterpret_cast<const f4 *>(s_q + 16 * m + 4 * j);
            D[m] *= *reinterpret_cast<const f4 *>(s_k + 16 * m + 4 * j);
        }
        state_update<DK, NP, RETR>(dS, s_gamma, Qr, dO, Kr, D);
    }
    if constexpr (CARRY) {
        put_state<KB>(a.seg_dcarry + seg_at(a, bh, seg, a.VB, vb, KB), dS);
    } else if (a.d_init && seg == 0) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
            store4(ChunkRows(a.d_init + (size_t)bh * p.dv * p.dk, p.dv, p.dk, p.dk), At4<VEC, float>(col, p.dk, 16 * kb + 4 * j, p.dk), dS[kb]);
    }
}

// ---------------------------------------------------------------- the chains' kernels
// Neither chain reads what the other writes, so one launch may hold both: the
// long requests of one run while the other's end.  Ragged batch: 1.41 ms for both
// (one after the other 1.69; in the requests' own order 1.54), 3.7 GB read and
// 3.2 GB written: 4.9 TB/s, bound by memory at 95 % of a copy's rate.  16 tokens
// 9.8 us (17.4).  252 registers of bf16 rows of 128, 256 and 8 bytes of scratch
// in the first pass of segments; odd widths 8 to 32 bytes.
template <int DK, typename TA, bool RETR, bool VEC, bool CARRY>
__global__ __launch_bounds__(256, planes_of<TA> <= 2 && DK <= 128 ? 2 : 1) void k_back_states(const BackParams a)
{
    __shared__ StatesLds<DK, TA, RETR> lds;
    states_chain<DK, TA, RETR, VEC, CARRY>(a, blockIdx.x, lds);
}

template <int DK, typename TA, bool RETR, bool VEC, bool CARRY>
__global__ __launch_bounds__(256, planes_of<TA> == 1 && DK <= 128 ? 2 : 1) void k_back_chain(const BackParams a)
{
    __shared__ ChainLds<DK, TA, RETR> lds;
    gradient_chain<DK, TA, RETR, VEC, CARRY>(a, blockIdx.x, lds);
}

// Workgroup 2 n: the nth of the backward chain, 2 n + 1: of the forward one,
// which with CARRY has more.
template <int DK, typename TA, bool RETR, bool VEC, bool CARRY>
__global__ __launch_bounds__(256, planes_of<TA> == 1 && DK <= 128 ? 2 : 1) void k_back_chains(const BackParams a, int chains)
{
    __shared__ union {
        StatesLds<DK, TA, RETR> states;
        ChainLds<DK, TA, RETR> chain;
    } lds;
    const int n = blockIdx.x;
    if (n < 2 * chains && n % 2 == 0) gradient_chain<DK, TA, RETR, VEC, CARRY>(a, n / 2, lds.chain);
    else states_chain<DK, TA, RETR, VEC, CARRY>(a, n < 2 * chains ? n / 2 : n - chains, lds.states);
}

// ---------------------------------------------------------------- gradients of a chunk
// One workgroup (8 waves) per (chunk, q/k head), the value heads that share it
// in turn, dQ and dK summed over them in the accumulators.  A wave owns KW
// blocks of 16 key channels (accumulator rows) of TW blocks of 16 tokens
// (columns): the states' operands, which it alone uses, go from memory to its
// registers, those over tokens (d_o, Y, E) through LDS, cut into planes once
// for all waves, 32 state rows a step, double buffered.  Of the chunk x chunk
// products wave (ft, part) forms column blocks part * SBW .. of row block ft.
// 1.34 ms: 3.5 GB read and 0.3 GB written, 2.8 TB/s, one workgroup a CU (152 KB of
// LDS, 256 VGPRs); matrix and VALU instructions fill two thirds of the SIMDs'
// cycles, the rest is waiting between a head's phases.  Keeping the rows of q
// and k in LDS spared 0.4 ms against reading them again for each head.
// The registers do not hold everything: with retrieval, 16-bit rows of 65 to 128
// channels put 12 to 56 bytes a lane in scratch memory, fp32 ones (whose q and k
// stay in registers over all heads) 344 to 360 (160 to 200 without retrieval),
// and above 128 channels, where a wave has twice the accumulators, every type
// 240 to 736.  Up to 64 channels nothing spills.  That and the chunks of 32 are
// what those widths pay for (the batch's lengths, whole calls: 8 heads of 256 in
// bf16 4.4 ms and fp32 6.4, 32 heads of 128 in fp32 5.7).
template <int DK, typename TA, bool RETR, bool VEC>
__global__ __launch_bounds__(512, 2) void k_back_grad(const BackParams a)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, MX = G::MX, KB = G::KB, KX = G::KX, ACT = G::ACT, NT = G::NT, NP = planes_of<TA>;
    constexpr int KW = DK == 256 ? 2 : 1, TW = KB * MB / 8 / KW, SPAN = MB / TW, KWAVES = 8 / SPAN;
    constexpr int PARTS = 8 / MB, SBW = (MB + PARTS - 1) / PARTS;
    constexpr int NB = NP + 3 + (RETR ? 3 : 0);  // planes of a token block: d_o, E, Y
    constexpr int SETS = RETR ? 4 : 2;           // chunk x chunk operands: F by rows and columns, W likewise
    constexpr int IN = NB * MB * BLOCK, TRI_SET = 3 * NT * BLOCK;
    // the token blocks' planes, two steps of them, and then the chunk x chunk operands
    __shared__ __align__(16) uint16_t s_mem[2 * IN > SETS * TRI_SET ? 2 * IN : SETS * TRI_SET];
    __shared__ __align__(16) float s_sc[BACK_SC * C];
    __shared__ float s_u[KWAVES][C], s_w[KWAVES][C], s_db[C], s_row[C][MB], s_col[MB][C], s_dot[KWAVES];
    // the chunk's rows of k and q; fp32 rows do not fit beside the rest
    constexpr bool PARK = sizeof(TA) == 2;
    __shared__ __align__(16) uint16_t s_k[PARK ? Rows<DK>::PLANE : 8], s_q[PARK ? Rows<DK>::PLANE : 8];
    __shared__ f4 s_gram[RETR ? 2 : 1][SBW][512];  // each thread's elements of its tiles of K Q^T and K K^T

    const Params &p = a.p;
    const int ci = blockIdx.x / p.H, hq = blockIdx.x % p.H;
    if (ci >= a.off[p.B]) return;
    const int64_t t0 = uniform(a.where[2 * ci]);
    const int cnt = uniform(a.where[2 * ci + 1]);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), c = lane & 15, j = lane >> 4;
    const int kw = wave / SPAN, kb0 = kw * KW, tb0 = wave % SPAN * TW;
    const int ft = wave / PARTS, part = wave % PARTS;
    const int R = p.HV / p.H;
    const f4 zero = {0.f, 0.f, 0.f, 0.f};
    const uint16_t *act = a.act + (size_t)blockIdx.x * 2 * NP * ACT * BLOCK;

    const size_t first = ((size_t)t0 * p.H + hq) * p.dk;  // the chunk's first element of q and k
    const int kstep = p.H * p.dk, vstep = p.HV * p.dv;
    const ChunkRows qrows(static_cast<const TA *>(p.q) + first, cnt, kstep, p.dk), krows(static_cast<const TA *>(p.k) + first, cnt, kstep, p.dk);
    // q and k of the wave's channels and tokens
    Raw4<TA> qr[PARK ? 1 : KW][PARK ? 1 : TW], kr[PARK ? 1 : KW][PARK ? 1 : TW];
    if constexpr (PARK) {
        StageRows<DK, TA, 512, VEC> k, q;
        const auto at = k.place(kstep, p.dk);
        k.load(static_cast<const TA *>(p.k) + first, cnt, kstep, p.dk, at);
        q.load(static_cast<const TA *>(p.q) + first, cnt, kstep, p.dk, at);
        k.store_raw(s_k);
        q.store_raw(s_q);
        __syncthreads();
    } else {
#pragma unroll
        for (int x = 0; x < KW; ++x)
#pragma unroll
            for (int w = 0; w < TW; ++w) {
                const At4<VEC, TA> at(16 * (tb0 + w) + c, kstep, 16 * (kb0 + x) + 4 * j, p.dk);
                qr[x][w] = load_raw4(qrows, at);
                kr[x][w] = load_raw4(krows, at);
            }
    }
    auto row_of = [&](const uint16_t *rows, int x, int w) {
        return widen(*reinterpret_cast<const Raw4<TA> *>(rows + (16 * (tb0 + w) + (opaque(threadIdx.x) & 15)) * Rows<DK>::LD +
                                                         16 * (kb0 + x) + 4 * ((threadIdx.x & 63) >> 4)));
    };
    auto q_of = [&](int x, int w) {
        if constexpr (PARK) return row_of(s_q, x, w);
        else return widen(qr[x][w]);
    };
    auto k_of = [&](int x, int w) {
        if constexpr (PARK) return row_of(s_k, x, w);
        else return widen(kr[x][w]);
    };
    // tiles of (K Q^T, K K^T), rows s of block sb, columns t of block ft, of the normalised rows
    bool use[SBW];
    {
        const float *sc = a.sc + ((size_t)ci * p.HV + (size_t)hq * R) * (BACK_SC * C);
        const int t = 16 * ft + c;
        auto operand = [&](const ChunkRows &rows, const uint16_t *lds, int block, int y, b8 (&out)[NP]) {
            if constexpr (PARK) {
                RawRows<DK, TA>::row_operand(lds, 16 * block + c, y, out);
                return;
            }
            const int lo = 32 * y + 4 * j;
            split8<NP>(widen(load_raw4(rows, At4<VEC, TA>(16 * block + c, kstep, lo, p.dk))),
                       widen(load_raw4(rows, At4<VEC, TA>(16 * block + c, kstep, lo + 16, p.dk))), out);
        };
#pragma unroll
        for (int x = 0; x < SBW; ++x) {
            const int sb = part * SBW + x;
            use[x] = sb <= ft;
            if (use[x]) {
                f4 qk = zero, kk = zero;
#pragma unroll 2
                for (int y = 0; y < KX; ++y) {
                    b8 s[NP], q[NP], k[NP];
                    operand(krows, s_k, sb, y, s);
                    operand(qrows, s_q, ft, y, q);
                    qk = mm(s, q, qk);
                    if (RETR) {
                        operand(krows, s_k, ft, y, k);
                        kk = mm(s, k, kk);
                    }
                }
                const float rq = sc[SC_RQ * C + t], rk = sc[SC_RK * C + t];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float rs = sc[SC_RK * C + 16 * sb + 4 * j + i];
                    qk[i] *= rs * rq;
                    kk[i] *= rs * rk;
                }
                s_gram[0][x][tid] = qk;
                if (RETR) s_gram[1][x][tid] = kk;
            }
        }
    }
    f4 dq[KW][TW], dk[KW][TW];
#pragma unroll
    for (int x = 0; x < KW; ++x)
#pragma unroll
        for (int w = 0; w < TW; ++w) dq[x][w] = dk[x][w] = zero;

    // What a step over 32 state rows takes from memory, loaded two steps ahead:
    // the wave's blocks of S0 and dS1, and the token block that it cuts into
    // planes for all waves (E: waves 0 .., Y: waves 4 .., d_o: waves o_blk).
    const int VX = a.VB / 2;
    const int y_blk = wave - 4, o_blk = MB == 4 ? wave : wave - 2;
    const bool is_e = wave < MB, is_y = RETR && y_blk >= 0 && y_blk < MB, is_o = o_blk >= 0 && o_blk < MB;
    const int z_blk = is_e ? wave : is_y ? y_blk : 0;
    struct In {
        f4 z[2], s[KW][2], d[KW][2];
        Raw4<TA> o[2];
    } ahead[2];
    auto fetch = [&](In &f, int r, int vx) {
        const bool live = r < R;
        const int h = hq * R + min(r, R - 1);
        const size_t rec = (size_t)ci * p.HV + h;
        const Frags S(a.s + (rec * KB + kb0) * a.VB * FRAG, live ? KW * a.VB : 0), D(a.ds + (rec * KB + kb0) * a.VB * FRAG, live ? KW * a.VB : 0);
        const Frags Z((is_y ? a.y : a.e) + (rec * MB + z_blk) * a.VB * FRAG, live ? a.VB : 0);
        const ChunkRows orows(static_cast<const TA *>(a.d_o) + ((size_t)t0 * p.HV + h) * p.dv, cnt, vstep, p.dv, live);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int vb = 2 * vx + n;
            f.z[n] = Z.get(vb);
            f.o[n] = load_raw4(orows, At4<VEC, TA>(16 * (is_o ? o_blk : 0) + c, vstep, 16 * vb + 4 * j, p.dv));
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                f.s[x][n] = S.get(x * a.VB + vb);
                f.d[x][n] = D.get(x * a.VB + vb);
            }
        }
    };
    // block m's planes: d_o at [0, NP), E at [NP, NP + 3), Y after
    auto stage = [&](const In &f, uint16_t *dst) {
        if (is_e || is_y) {
            b8 v[3];
            uint16_t *at = dst + (size_t)(z_blk * NB + NP + (is_y ? 3 : 0)) * BLOCK;
            split8<3>(f.z[0], f.z[1], v);
#pragma unroll
            for (int n = 0; n < 3; ++n) put_block(at + n * BLOCK, v[n]);
        }
        if (is_o) {
            b8 v[NP];
            split8<NP>(widen(f.o[0]), widen(f.o[1]), v);
#pragma unroll
            for (int n = 0; n < NP; ++n) put_block(dst + (size_t)(o_blk * NB + n) * BLOCK, v[n]);
        }
    };
    // The loads stand under no condition: past the last step of the last head
    // they are of buffers with nothing in them (a load that may not have been
    // issued would make the wait for the one before it a wait for all).
    float sc_next;  // a thread's word of the chunk's scalars, a head ahead
    auto fetch_scalars = [&](int r) {
        const int n = tid < BACK_SC * C ? tid : 0;
        sc_next = a.sc[((size_t)ci * p.HV + (size_t)hq * R + r) * (BACK_SC * C) + n];
    };
    fetch_scalars(0);
    fetch(ahead[0], 0, 0);
    fetch(ahead[1], 0, 1);
    for (int r = 0; r < R; ++r) {
        const int h = hq * R + r;
        const size_t rec = (size_t)ci * p.HV + h;
        static_assert(BACK_SC * C <= 512, "a word a thread");
        // the lane's numbers anew for each head: what is derived from them would
        // else be formed once, ahead of the loop, and kept in scratch memory
        const int tid = opaque(threadIdx.x), lane = tid & 63, c = lane & 15, j = lane >> 4;
        arrive(sc_next);
        if (tid < BACK_SC * C) s_sc[tid] = sc_next;
        fetch_scalars(min(r + 1, R - 1));
        const float *s_eg = s_sc + SC_EG * C, *s_kd = s_sc + SC_KD * C, *s_b = s_sc + SC_B * C, *s_gh = s_sc + SC_GH * C,
                    *s_gl = s_sc + SC_GL * C, *s_rq = s_sc + SC_RQ * C, *s_rk = s_sc + SC_RK * C;

        // ---- products over the state rows
        f4 A1[KW][TW], A2[KW][TW], A3[KW][TW], F[SBW], X[SBW];
#pragma unroll
        for (int x = 0; x < KW; ++x)
#pragma unroll
            for (int w = 0; w < TW; ++w) A1[x][w] = A2[x][w] = A3[x][w] = zero;
#pragma unroll
        for (int x = 0; x < SBW; ++x) F[x] = X[x] = zero;
        float dot = 0.f;
        auto step = [&](In &f, int vx) {
            uint16_t *in = s_mem + (vx & 1) * IN;
            arrive(f);
            stage(f, in);
            b8 sp[KW][3], dp[KW][3];
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                if (tb0 == 0) dot += dot4(f.s[x][0], f.d[x][0]) + dot4(f.s[x][1], f.d[x][1]);
                split8<3>(f.s[x][0], f.s[x][1], sp[x]);
                split8<3>(f.d[x][0], f.d[x][1], dp[x]);
            }
            const bool wrap = vx + 2 >= VX;
            fetch(f, wrap ? r + 1 : r, wrap ? vx + 2 - VX : vx + 2);
            lds_barrier();  // one a step: the other buffer's readers have passed the last one
#pragma unroll
            for (int w = 0; w < TW; ++w) {
                __builtin_amdgcn_sched_barrier(0);  // one block's operands in registers at a time
                const uint16_t *at = in + (size_t)(tb0 + w) * NB * BLOCK;
                b8 ob[NP], eb[3], yb[3];
#pragma unroll
                for (int n = 0; n < NP; ++n) ob[n] = get_block(at + n * BLOCK);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    eb[n] = get_block(at + (NP + n) * BLOCK);
                    if (RETR) yb[n] = get_block(at + (NP + 3 + n) * BLOCK);
                }
#pragma unroll
                for (int x = 0; x < KW; ++x) {
#pragma unroll
                    for (int n = 2; n >= 0; --n)
#pragma unroll
                        for (int i = 0; i <= n; ++i) {  // three accumulators side by side
                            if (n - i < NP) A1[x][w] = mfma(sp[x][i], ob[n - i], A1[x][w]);
                            A3[x][w] = mfma(dp[x][i], eb[n - i], A3[x][w]);
                            if (RETR) A2[x][w] = mfma(sp[x][i], yb[n - i], A2[x][w]);
                        }
                }
            }
#pragma unroll
            for (int x = 0; x < SBW; ++x)
                if (use[x]) {
                    const uint16_t *rs = in + (size_t)((part * SBW + x) * NB + NP) * BLOCK, *ct = in + (size_t)ft * NB * BLOCK;
                    b8 es[3], ob[NP], yb[3];
#pragma unroll
                    for (int n = 0; n < 3; ++n) es[n] = get_block(rs + n * BLOCK);
#pragma unroll
                    for (int n = 0; n < NP; ++n) ob[n] = get_block(ct + n * BLOCK);
                    F[x] = mm(es, ob, F[x]);
                    if (RETR) {
#pragma unroll
                        for (int n = 0; n < 3; ++n) yb[n] = get_block(ct + (NP + 3 + n) * BLOCK);
                        X[x] = mm(es, yb, X[x]);
                    }
                }
        };
        for (int vx = 0; vx < VX; vx += 2) {
            step(ahead[0], vx);
            step(ahead[1], vx + 1);
        }

        // ---- per token: what crosses the token from the state
#pragma unroll
        for (int w = 0; w < TW; ++w) {
            const int t = 16 * (tb0 + w) + c;
            const float eg = s_eg[t], kd = s_kd[t] * s_b[t], be = -s_b[t] * eg;
            float u = 0.f, v = 0.f;
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                const f4 qh = q_of(x, w) * s_rq[t], kh = k_of(x, w) * s_rk[t];
                A1[x][w] *= eg;
                A3[x][w] *= kd;
                v += dot4(qh, A1[x][w]);
                u += dot4(kh, A3[x][w]);
                dq[x][w] += A1[x][w];
                dk[x][w] += A3[x][w];
                if (RETR) {
                    A2[x][w] *= be;
                    v += dot4(kh, A2[x][w]);
                    dk[x][w] += A2[x][w];
                }
            }
            u = sum_j(u);
            v = sum_j(v);
            if (j == 0) {
                s_u[kw][t] = u;
                s_w[kw][t] = v;
            }
        }
        if (tb0 == 0) {
#pragma unroll
            for (int n = 1; n < 64; n <<= 1) dot += __shfl_xor(dot, n);
            if (lane == 0) s_dot[kw] = dot;
        }

        lds_barrier();  // the last step's operands give way to the tiles'
        // ---- the chunk x chunk tiles: factors, M's part of dg, operands by rows and by columns
#pragma unroll
        for (int x = 0; x < SBW; ++x)
            if (use[x]) {
                const int sb = part * SBW + x, s0 = 16 * sb + 4 * j, t = 16 * ft + c;
                const float gh = s_gh[t], gl = s_gl[t], bt = s_b[t];
                const f4 rks = *reinterpret_cast<const f4 *>(s_rk + s0);
                const f4 qk = s_gram[0][x][tid], kk = RETR ? s_gram[1][x][tid] : zero;
                f4 f, wv = zero, M;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = s0 + i;
                    const float ex = n <= t ? exp_split(gh - s_gh[n], gl - s_gl[n]) * s_b[n] : 0.f;
                    f[i] = F[x][i] * ex;
                    M[i] = n < t ? f[i] * qk[i] : 0.f;
                    if (RETR) {
                        wv[i] = n < t ? -bt * ex * X[x][i] : 0.f;
                        M[i] += wv[i] * kk[i];
                        if (n == t) s_db[t] = X[x][i];  // Y_t . E_t
                    }
                }
                constexpr size_t STRIDE = (size_t)NT * BLOCK;
                const int lo = lower_block<MB>(ft, sb / 2) * BLOCK, up = upper_block<MB>(sb, ft / 2) * BLOCK;
                put_half(s_mem + lo, STRIDE, lane, sb & 1, f * rks);
                put_half(s_mem + TRI_SET + up, STRIDE, quad_lane(), ft & 1, quad_transpose(f * s_rq[t]));
                if (RETR) {
                    put_half(s_mem + (SETS - 2) * TRI_SET + lo, STRIDE, lane, sb & 1, wv * rks);
                    put_half(s_mem + (SETS - 1) * TRI_SET + up, STRIDE, quad_lane(), ft & 1, quad_transpose(wv * s_rk[t]));
                }
                if (sb == ft) {  // the half of a diagonal block pair that lies outside the triangle
#pragma unroll
                    for (int n = 0; n < SETS; ++n)
                        if ((n & 1) == (sb & 1)) put_half(s_mem + n * TRI_SET + (n & 1 ? up : lo), STRIDE, lane, n & 1 ? 0 : 1, zero);
                }
                // sums over the columns before each one, within the tile's row t ...
                const float four = (M[0] + M[1]) + (M[2] + M[3]);
                const float a1 = __shfl_up(four, 16), a2 = __shfl_up(four, 32), a3 = __shfl_up(four, 48);
                float pre = (j > 0 ? a1 : 0.f) + (j > 1 ? a2 : 0.f) + (j > 2 ? a3 : 0.f);
                if (j == 3) s_row[t][sb] = pre + four;
                // ... then over the rows t >= s
                f4 sum;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[i] = sum16(s0 + i <= t ? pre : 0.f);
                    pre += M[i];
                }
                if (c == 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s_col[ft][s0 + i] = sum[i];
            }
        __syncthreads();

        // ---- products over the chunk's tokens
#pragma unroll
        for (int yy = 0; yy < MX; ++yy) {
            b8 kt[KW][NP], qt[KW][NP];
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                if constexpr (PARK) {
                    RawRows<DK, TA>::col_operand(s_k, kb0 + x, yy, kt[x]);
                    RawRows<DK, TA>::col_operand(s_q, kb0 + x, yy, qt[x]);
                } else {
#pragma unroll
                    for (int n = 0; n < NP; ++n) {
                        kt[x][n] = get_block(act + (size_t)(n * ACT + (kb0 + x) * MX + yy) * BLOCK);
                        qt[x][n] = get_block(act + (size_t)((NP + n) * ACT + (kb0 + x) * MX + yy) * BLOCK);
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < TW; ++w) {
                const int tb = tb0 + w;
                b8 v[3];
                auto get = [&](int set, int blk) {
#pragma unroll
                    for (int n = 0; n < 3; ++n) v[n] = get_block(s_mem + set * TRI_SET + (n * NT + blk) * BLOCK);
                };
                if (2 * yy <= tb) {  // row t: columns s <= t
                    const int blk = lower_block<MB>(tb, yy);
                    get(0, blk);
#pragma unroll
                    for (int x = 0; x < KW; ++x) dq[x][w] = mm(kt[x], v, dq[x][w]);
                    if (RETR) {
                        get(SETS - 2, blk);
#pragma unroll
                        for (int x = 0; x < KW; ++x) dk[x][w] = mm(kt[x], v, dk[x][w]);
                    }
                }
                if (2 * yy + 1 >= tb) {  // column t: rows >= t
                    const int blk = upper_block<MB>(tb, yy);
                    get(1, blk);
#pragma unroll
                    for (int x = 0; x < KW; ++x) dk[x][w] = mm(qt[x], v, dk[x][w]);
                    if (RETR) {
                        get(SETS - 1, blk);
#pragma unroll
                        for (int x = 0; x < KW; ++x) dk[x][w] = mm(kt[x], v, dk[x][w]);
                    }
                }
            }
        }

        // ---- what k_back_gate joins to dg and db, a row of the record a wave
        if (lane < C) {
            float x = 0.f;
            if (wave == GX_U || wave == GX_W) {
#pragma unroll
                for (int n = 0; n < KWAVES; ++n) x += wave == GX_U ? s_u[n][lane] : s_w[n][lane];
            } else if (wave == GX_DB) {
                x = RETR ? s_db[lane] : 0.f;
            } else if (wave == GX_COL) {
#pragma unroll
                for (int m = 0; m < MB; ++m) x += m >= lane / 16 ? s_col[m][lane] : 0.f;
            } else if (wave == GX_STATE) {
#pragma unroll
                for (int n = 0; n < KWAVES; ++n) x += s_dot[n];
                x *= s_eg[C - 1];
            } else {  // columns of the blocks before block wave - GX_ROW + 1
#pragma unroll
                for (int m = 0; m < MB - 1; ++m) x += m <= wave - GX_ROW && m <= lane / 16 ? s_row[lane][m] : 0.f;
            }
            a.gx[(rec * GX + wave) * C + lane] = x;
        }
        __syncthreads();
    }

    // through the L2 norm: d x = r (d x^ - x^ (x^ . d x^)), x^ = r x
    const float *s_rq = s_sc + SC_RQ * C, *s_rk = s_sc + SC_RK * C;
    const float inv = 1.f / p.scale;
    if (p.qk_l2_norm) {
#pragma unroll
        for (int w = 0; w < TW; ++w) {
            float nq = 0.f, nk = 0.f;
#pragma unroll
            for (int x = 0; x < KW; ++x) {
                nq += dot4(q_of(x, w), dq[x][w]);
                nk += dot4(k_of(x, w), dk[x][w]);
            }
            nq = sum_j(nq);
            nk = sum_j(nk);
            if (j == 0) {
                s_u[kw][16 * (tb0 + w) + c] = nq;
                s_w[kw][16 * (tb0 + w) + c] = nk;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int w = 0; w < TW; ++w) {
        const int t = 16 * (tb0 + w) + c;
        const float rq = s_rq[t], rk = s_rk[t];
        float nq = 0.f, nk = 0.f;
        if (p.qk_l2_norm) {
#pragma unroll
            for (int n = 0; n < KWAVES; ++n) {
                nq += s_u[n][t];
                nk += s_w[n][t];
            }
            nq *= rq * inv * rq * inv;  // rq holds the scale too
            nk *= rk * rk;
        }
#pragma unroll
        for (int x = 0; x < KW; ++x) {
            const At4<VEC, TA> at(t, kstep, 16 * (kb0 + x) + 4 * j, p.dk);
            f4 gq = dq[x][w], gk = dk[x][w];
            if (p.qk_l2_norm) {
                gq -= q_of(x, w) * nq;
                gk -= k_of(x, w) * nk;
            }
            store4(ChunkRows(static_cast<const TA *>(a.dq) + first, cnt, kstep, p.dk), at, gq * rq);
            store4(ChunkRows(static_cast<const TA *>(a.dk) + first, cnt, kstep, p.dk), at, gk * rk);
        }
    }
}

// ---------------------------------------------------------------- dg and db
// A wave per (chunk, value head), a lane a token (28 us):
//   dg_s = e^Gamma <dS1, S0> + sum_{t<s} u_t + sum_{t>=s} w_t + sum_{t>=s>r} M_tr
// the last from the sums over r of whole blocks before s's own (rows) and
// within it (col); then the raw gate's and the rate's activation.
template <int C, bool RETR>
__global__ __launch_bounds__(256) void k_back_gate(const BackParams a)
{
    constexpr int MB = C / 16;
    const Params &p = a.p;
    const int64_t rec = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int ci = (int)(rec / p.HV), h = (int)(rec % p.HV);
    if (ci >= a.off[p.B]) return;
    const int64_t t0 = uniform(a.where[2 * ci]);
    const int cnt = uniform(a.where[2 * ci + 1]);
    const float *x = a.gx + (size_t)rec * GX * C;
    const int n0 = lane < C ? lane : C - 1;
    const bool mine = lane < C;
    const size_t th = (size_t)(t0 + (lane < cnt ? lane : cnt - 1)) * p.HV + h;
    const float raw = a.decays && p.gate_qwen ? load_gate(p, th) + p.dt_bias[h] : 0.f;
    // e^-|x| of the rate's logit x: the sigmoid's derivative is t / (1 + t)^2,
    // formed so because 1 - rate loses all its digits where the rate is near 1
    const float t = RETR && p.beta_sigmoid ? expf(-fabsf(p.beta[beta_index(p, th)])) : 0.f;
    const float col = x[GX_COL * C + n0], state = x[GX_STATE * C], db = x[GX_DB * C + n0];
    float pre = mine ? x[GX_U * C + n0] : 0.f, suf = mine ? x[GX_W * C + n0] : 0.f;
    float rows[MB];
    rows[0] = 0.f;
#pragma unroll
    for (int m = 1; m < MB; ++m) rows[m] = mine ? x[(GX_ROW + m - 1) * C + n0] : 0.f;
#pragma unroll
    for (int n = 1; n < 64; n <<= 1) {
        const float v = __shfl_up(pre, n), w = __shfl_down(suf, n);
        if (lane >= n) pre += v;
        if (lane + n < 64) suf += w;
#pragma unroll
        for (int m = 1; m < MB; ++m) {
            const float z = __shfl_down(rows[m], n);
            if (lane + n < 64) rows[m] += z;
        }
    }
    pre = __shfl_up(pre, 1);
    float g = (lane > 0 ? pre : 0.f) + suf + col + state;
#pragma unroll
    for (int m = 1; m < MB; ++m) g += m == n0 / 16 ? rows[m] : 0.f;
    float da = 0.f, ds = 0.f;  // raw-gate arm: d of the projection (and of the bias), d of the scale
    if (lane < cnt) {
        if (a.decays) {
            if (p.gate_qwen) {
                da = g * gate_scale(p, h) * sigmoid_f32(raw);
                ds = g * softplus_f32(raw);
                g = da;
            }
            if (p.gate_dt == 1) static_cast<half_t *>(a.d_gate)[th] = from_f32<half_t>(g);
            else if (p.gate_dt == 2) static_cast<bf16_t *>(a.d_gate)[th] = from_f32<bf16_t>(g);
            else static_cast<float *>(a.d_gate)[th] = g;
        }
        if (RETR) {
            const float r = 1.f / (1.f + t);
            a.d_beta[th] = p.beta_sigmoid ? db * (t * r * r) : db;
        }
    }
    if (a.decays && p.gate_qwen) {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            da += __shfl_xor(da, o);
            ds += __shfl_xor(ds, o);
        }
        if (lane == 0) {
            a.gate_sums[2 * rec] = da;
            a.gate_sums[2 * rec + 1] = ds;
        }
    }
}

// ---------------------------------------------------------------- launches
template <int DK, typename TA, bool RETR, bool VEC>
hipError_t launch_back_typed(const BackParams &a, hipStream_t s)
{
    const Params &p = a.p;
    const unsigned per_chunk = (unsigned)a.chunks * p.H, pairs = (unsigned)p.B * p.HV, tiles = a.VB / 4;
    const unsigned chains = pairs * a.nseg * tiles, carry = pairs * a.nseg * (tiles + Geo<DK>::KB / 4);
    const dim3 block(256);
    hipLaunchKernelGGL((k_back_prep<DK, TA, RETR, VEC>), dim3((unsigned)a.chunks * p.HV), block, 0, s, a);
    if (p.B == 0) return hipGetLastError();
    // One launch for both, but for many chains of fp16 and fp32 rows of 128: their
    // forward chain has two workgroups a CU (fp32: leaves room for a second) by
    // itself, and one in the joint kernel.  The ragged batch's lengths, one launch
    // against two: 32 heads of 128 fp16 3.96 / 3.80 ms, fp32 6.05 / 5.75; of 64
    // fp16 1.91 / 2.23, fp32 2.34 / 2.69; 8 heads of 256 bf16 4.42 / 4.91.
    constexpr bool SPLITS = planes_of<TA> > 1 && DK == 128;
    const auto launch_chains = [&](auto first_pass, unsigned backward, unsigned forward) {
        constexpr bool CARRY = decltype(first_pass)::value;
        if constexpr (SPLITS) {
            if (2 * chains > 256) {
                hipLaunchKernelGGL((k_back_states<DK, TA, RETR, VEC, CARRY>), dim3(forward), block, 0, s, a);
                hipLaunchKernelGGL((k_back_chain<DK, TA, RETR, VEC, CARRY>), dim3(backward), block, 0, s, a);
                return;
            }
        }
        hipLaunchKernelGGL((k_back_chains<DK, TA, RETR, VEC, CARRY>), dim3(backward + forward), block, 0, s, a, (int)backward);
    };
    if (a.nseg > 1) {
        launch_chains(std::true_type(), chains, carry);
        hipLaunchKernelGGL((k_back_join<DK, VEC>), dim3(2 * pairs * a.VB), dim3(DK * 2), 0, s, a);
    }
    launch_chains(std::false_type(), chains, chains);
    hipLaunchKernelGGL((k_back_grad<DK, TA, RETR, VEC>), dim3(per_chunk), dim3(512), 0, s, a);
    if (RETR || a.decays)
        hipLaunchKernelGGL((k_back_gate<Geo<DK>::C, RETR>), dim3(((unsigned)a.chunks * p.HV + 3) / 4), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <int DK, typename TA>
hipError_t launch_back_dk(const BackParams &a, bool retrieves, hipStream_t s)
{
    const bool vec = a.p.dk % 4 == 0 && a.p.dv % 4 == 0;
    if (retrieves) return vec ? launch_back_typed<DK, TA, true, true>(a, s) : launch_back_typed<DK, TA, true, false>(a, s);
    return vec ? launch_back_typed<DK, TA, false, true>(a, s) : launch_back_typed<DK, TA, false, false>(a, s);
}

template <typename TA>
hipError_t launch_back_act(const BackParams &a, bool retrieves, hipStream_t s)
{
    const int dk = a.p.dk;
    return dk <= 64 ? launch_back_dk<64, TA>(a, retrieves, s)
           : dk <= 128 ? launch_back_dk<128, TA>(a, retrieves, s)
                       : launch_back_dk<256, TA>(a, retrieves, s);
}

}  // namespace
}  // namespace gdr
