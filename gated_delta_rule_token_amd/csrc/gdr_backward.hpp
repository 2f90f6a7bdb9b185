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
//   k_back_prep    per chunk and q/k head: the two triangular inverses, P, decay factors
//   k_back_states  per request, head and 64 state rows: forward chain, keeps S0 and E of every chunk
//   k_back_chain   the same backwards: dS1, Y, dV
//   k_back_grad    per chunk and q/k head: dQ, dK (summed over the value heads that share them), dg, db
// Every product runs on v_mfma_f32_16x16x4_f32: fp32 operands, so that fp32
// gradients keep fp32's precision at any scale of the incoming gradient.
//
// Fragments.  The 16x16 fp32 accumulator of that instruction (lane l = 16 j +
// c, element i: row 4 j + i, column c) is, element by element, also its B
// operand with k = 4 j + i: a wave that holds S^T (dk x 16 state rows) feeds
// it to K S^T, and the result to (I + ..)^-1, and that result to the state
// update, with no move between lanes.  The A operand then takes k = 4 j + i
// too, four consecutive elements of a row.  What one kernel leaves for the
// next is stored as such blocks ("fragment blocks"): 256 floats, lane l's
// four at 4 l, holding row c, columns 4 j + i.
#pragma once

#include <hip/hip_runtime.h>

#include "gdr_backward_launch.hpp"
#include "gdr_device.hpp"

namespace gdr {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int FRAG = 256;  // floats of a fragment block

template <int DK> struct Geo {
    static constexpr int C = back_chunk(DK);
    static constexpr int MB = C / 16, KB = DK / 16, TRI = MB * (MB + 1) / 2;
    static constexpr int LD = DK + 4;   // floats of a staged q/k row
    static constexpr int LC = C + 4;    // floats of a staged chunk x chunk row
};

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

// 4x4 transpose within each quad of lanes: element p of lane q <- element q of lane p
__device__ __forceinline__ f4 quad_transpose(f4 v)
{
    const int lane = threadIdx.x;
    const bool odd = lane & 1, up = lane & 2;
    float g = dpp_mov<0xB1>(odd ? v[0] : v[1]);  // lane ^ 1
    v = odd ? f4{g, v[1], v[2], v[3]} : f4{v[0], g, v[2], v[3]};
    g = dpp_mov<0xB1>(odd ? v[2] : v[3]);
    v = odd ? f4{v[0], v[1], g, v[3]} : f4{v[0], v[1], v[2], g};
    g = dpp_mov<0x4E>(up ? v[0] : v[2]);         // lane ^ 2
    v = up ? f4{g, v[1], v[2], v[3]} : f4{v[0], v[1], g, v[3]};
    g = dpp_mov<0x4E>(up ? v[1] : v[3]);
    v = up ? f4{v[0], g, v[2], v[3]} : f4{v[0], v[1], v[2], g};
    return v;
}

// Accumulator tile -> fragment block whose rows are the tile's columns.
__device__ __forceinline__ void put_frag_cols(float *blk, f4 v)
{
    *reinterpret_cast<f4 *>(blk + (threadIdx.x & 63) * 4) = v;
}

// Accumulator tile -> fragment block whose rows are the tile's rows.
__device__ __forceinline__ void put_frag_rows(float *blk, f4 v)
{
    const int lane = threadIdx.x & 63, c = lane & 15, j = lane >> 4;
    *reinterpret_cast<f4 *>(blk + ((4 * j + (c & 3)) + 16 * (c >> 2)) * 4) = quad_transpose(v);
}

__device__ __forceinline__ f4 get_frag(const float *blk) { return *reinterpret_cast<const f4 *>(blk + (threadIdx.x & 63) * 4); }

// Four consecutive elements of a row of `width` (from column c), as they lie
// in memory; columns past the width are zero.  Rows start 16-byte aligned
// arrays whose width is a multiple of 4 when vec.
template <typename TA> struct Raw4 { TA x[4]; };

template <typename TA>
__device__ __forceinline__ Raw4<TA> load_raw4(const TA *row, int c, int width, bool vec)
{
    Raw4<TA> r;
    if (vec) {
        if (c < width) {
            if constexpr (sizeof(TA) == 4) *reinterpret_cast<uint4 *>(&r) = *reinterpret_cast<const uint4 *>(row + c);
            else *reinterpret_cast<uint2 *>(&r) = *reinterpret_cast<const uint2 *>(row + c);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.x[i] = from_f32<TA>(0.f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.x[i] = c + i < width ? row[c + i] : from_f32<TA>(0.f);
    }
    return r;
}

template <typename TA> __device__ __forceinline__ Raw4<TA> zero_raw4()
{
    Raw4<TA> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.x[i] = from_f32<TA>(0.f);
    return r;
}

template <typename TA> __device__ __forceinline__ f4 widen(const Raw4<TA> &r)
{
    return f4{to_f32(r.x[0]), to_f32(r.x[1]), to_f32(r.x[2]), to_f32(r.x[3])};
}

template <typename TA>
__device__ __forceinline__ void store4(TA *row, int c, int width, bool vec, f4 v)
{
    if (vec) {
        if (c >= width) return;
        Raw4<TA> r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.x[i] = from_f32<TA>(v[i]);
        if constexpr (sizeof(TA) == 4) *reinterpret_cast<uint4 *>(row + c) = *reinterpret_cast<const uint4 *>(&r);
        else *reinterpret_cast<uint2 *>(row + c) = *reinterpret_cast<const uint2 *>(&r);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < width) row[c + i] = from_f32<TA>(v[i]);
    }
}

__device__ __forceinline__ float dot4(f4 a, f4 b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }

// Sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float sum_j(float x)
{
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// The request of chunk `ci`, its first token and how many of C tokens it has.
__device__ __forceinline__ void chunk_tokens(const BackParams &a, int ci, int C, int64_t &t0, int &cnt)
{
    int lo = 0, hi = a.p.B - 1;  // largest b with off[b] <= ci (ci < off[B])
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.off[mid] <= ci) lo = mid;
        else hi = mid - 1;
    }
    const int64_t skip = (int64_t)(ci - a.off[lo]) * C;
    t0 = (int64_t)a.tok[2 * lo] + skip;
    const int64_t left = (int64_t)a.tok[2 * lo + 1] - skip;
    cnt = left < C ? (int)left : C;
}

// ---------------------------------------------------------------- prologue
// One workgroup per (chunk, q/k head); the value heads that share the head in
// turn.  The products K K^T and Q K^T are formed once for them.  Each unit
// lower triangular inverse goes by 16x16 blocks: the diagonal ones by forward
// substitution, a thread a column; then wave j takes block column j down,
// T_ij = -T_ii sum_k N_ik T_kj, its T_kj staying in the accumulators' layout.
template <int DK, typename TA, bool RETR>
__global__ __launch_bounds__(256) void k_back_prep(const BackParams a)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, KB = G::KB, LD = G::LD, LC = G::LC, TRI = G::TRI;
    constexpr int SLOTS = (TRI + 3) / 4, INV = 16 * 20;
    constexpr int STAGE = 2 * C * LD, SOLVE = C * LC + 2 * MB * INV;
    __shared__ __align__(16) float mem[STAGE > SOLVE ? STAGE : SOLVE];
    __shared__ double s_G[C];
    __shared__ __align__(16) float s_b[C];
    __shared__ float s_rq[C], s_rk[C];

    const Params &p = a.p;
    const int ci = blockIdx.x / p.H, hq = blockIdx.x % p.H;
    if (ci >= a.off[p.B]) return;
    int64_t t0;
    int cnt;
    chunk_tokens(a, ci, C, t0, cnt);

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, j = lane >> 4;
    float *Kh = mem, *Qh = mem + C * LD;

    // rows of q and k, normalised
    constexpr int LPR = DK / 4;  // lanes of a row
    const bool vec = p.dk % 4 == 0;
#pragma unroll
    for (int n = 0; n < C * LPR / 256; ++n) {
        const int g = tid + 256 * n, t = g / LPR, col = g % LPR * 4;
        f4 q = {0.f, 0.f, 0.f, 0.f}, k = q;
        if (t < cnt) {
            const size_t row = ((size_t)(t0 + t) * p.H + hq) * p.dk;
            q = widen(load_raw4(static_cast<const TA *>(p.q) + row, col, p.dk, vec));
            k = widen(load_raw4(static_cast<const TA *>(p.k) + row, col, p.dk, vec));
        }
        float rq = 1.f, rk = 1.f;
        if (p.qk_l2_norm) {
            float sq = dot4(q, q), sk = dot4(k, k);
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) {
                sq += __shfl_xor(sq, o);
                sk += __shfl_xor(sk, o);
            }
            rq = 1.f / sqrtf(sq + 1e-12f);
            rk = 1.f / sqrtf(sk + 1e-12f);
        }
        rq *= p.scale;
        *reinterpret_cast<f4 *>(Kh + t * LD + col) = k * rk;
        *reinterpret_cast<f4 *>(Qh + t * LD + col) = q * rq;
        if (col == 0) {
            s_rq[t] = rq;
            s_rk[t] = rk;
        }
    }
    __syncthreads();

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
            const float *qr = Qh + (16 * tm[n] + c) * LD + 4 * j, *kr = Kh + (16 * tm[n] + c) * LD + 4 * j,
                        *sr = Kh + (16 * tk[n] + c) * LD + 4 * j;
#pragma unroll 4
            for (int x = 0; x < KB; ++x) {
                const f4 s = *reinterpret_cast<const f4 *>(sr + 16 * x);
                qk[n] = mfma4(*reinterpret_cast<const f4 *>(qr + 16 * x), s, qk[n]);
                if (RETR) kk[n] = mfma4(*reinterpret_cast<const f4 *>(kr + 16 * x), s, kk[n]);
            }
        }
    }
    __syncthreads();  // the staged rows give way to L and the diagonal inverses

    float *Lm = mem, *inv = mem + C * LC;
    const int R = p.HV / p.H;
    for (int r = 0; r < R; ++r) {
        const int h = hq * R + r;
        const size_t rec = (size_t)ci * p.HV + h;
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
                float *sc = a.sc + rec * (BACK_SC * C);
                const float hi = (float)g;
                sc[SC_EG * C + lane] = exp_of(g);
                sc[SC_KD * C + lane] = exp_of(end - g);
                sc[SC_B * C + lane] = b;
                sc[SC_GH * C + lane] = hi;
                sc[SC_GL * C + lane] = (float)(g - (double)hi);
                sc[SC_RQ * C + lane] = s_rq[lane];
                sc[SC_RK * C + lane] = s_rk[lane];
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) {
            if (tm[n] >= 0) {
                const int s = 16 * tk[n] + c;
                const double gs = s_G[s];
                f4 P;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * tm[n] + 4 * j + i;
                    const float e = s <= t ? exp_of(s_G[t] - gs) : 0.f;
                    P[i] = e * qk[n][i];
                    if (RETR) Lm[t * LC + s] = s < t ? e * kk[n][i] : 0.f;
                }
                put_frag_cols(a.pt + (rec * TRI + tri(tm[n], tk[n])) * FRAG, P);
            }
        }
        if constexpr (RETR) {
            __syncthreads();
            // z = 0: I + L diag(b);  z = 1: I + diag(b) L
            if (tid < 2 * MB * 16) {
                const int z = tid / (MB * 16), d = tid / 16 % MB, col = tid & 15;
                float x[16];
#pragma unroll
                for (int row = 0; row < 16; ++row) {
                    const float bt = s_b[16 * d + row];
                    float acc = row == col ? 1.f : 0.f;
#pragma unroll
                    for (int s = 0; s < row; ++s)
                        acc -= Lm[(16 * d + row) * LC + 16 * d + s] * (z ? bt : s_b[16 * d + s]) * x[s];
                    x[row] = acc;
                    inv[(z * MB + d) * INV + row * 20 + col] = acc;
                }
            }
            __syncthreads();
            if (wave < MB) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    f4 T[MB];
#pragma unroll
                    for (int i = 0; i < MB; ++i) T[i] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < MB; ++i) {
                        if (i == wave) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) T[i][e] = inv[(z * MB + i) * INV + (4 * j + e) * 20 + c];
                        } else if (i > wave) {
                            f4 acc = {0.f, 0.f, 0.f, 0.f};
                            const float bt = s_b[16 * i + c];
#pragma unroll
                            for (int k = 0; k < i; ++k) {
                                if (k < wave) continue;
                                f4 N = *reinterpret_cast<const f4 *>(Lm + (16 * i + c) * LC + 16 * k + 4 * j);
                                N *= z ? f4{bt, bt, bt, bt} : *reinterpret_cast<const f4 *>(s_b + 16 * k + 4 * j);
                                acc = mfma4(N, T[k], acc);
                            }
                            const f4 Ti = *reinterpret_cast<const f4 *>(inv + (z * MB + i) * INV + c * 20 + 4 * j);
                            T[i] = -mfma4(Ti, acc, f4{0.f, 0.f, 0.f, 0.f});
                        }
                        if (i >= wave) {
                            if (z == 0) put_frag_rows(a.t1 + (rec * TRI + tri(i, wave)) * FRAG, T[i]);
                            else put_frag_cols(a.t2 + (rec * TRI + tri(i, wave)) * FRAG, T[i]);
                        }
                    }
                }
            }
        }
        __syncthreads();  // before the next head overwrites s_G, s_b, L
    }
}

// ---------------------------------------------------------------- staging of a chunk's q or k rows
// Each of NT threads holds C * DK / 4 / NT groups of four elements between
// the global load (stage_load) and the LDS store (stage_store).
template <int DK, typename TA, int NT> struct Stage {
    using G = Geo<DK>;
    static constexpr int LPR = DK / 4, N = G::C * LPR / NT;
    Raw4<TA> x[N];
    float r[N];

    __device__ __forceinline__ void load(const TA *src, const float *scale, int64_t t0, int cnt, int heads, int head,
                                         int dk, bool vec)
    {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int g = threadIdx.x + NT * n, t = g / LPR, col = g % LPR * 4;
            x[n] = t < cnt ? load_raw4(src + ((size_t)(t0 + t) * heads + head) * dk, col, dk, vec) : zero_raw4<TA>();
            r[n] = scale[t];
        }
    }
    __device__ __forceinline__ void store(float *dst) const
    {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int g = threadIdx.x + NT * n, t = g / LPR, col = g % LPR * 4;
            *reinterpret_cast<f4 *>(dst + t * G::LD + col) = widen(x[n]) * r[n];
        }
    }
};

// Column `col` (of `width`) of the chunk's rows in the accumulators' layout.
template <int MB, typename TA>
__device__ __forceinline__ void load_cols(f4 (&out)[MB], const TA *src, int64_t t0, int cnt, int heads, int head, int width,
                                          int col, int j)
{
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * m + 4 * j + i;
            out[m][i] = t < cnt && col < width ? to_f32(src[((size_t)(t0 + t) * heads + head) * width + col]) : 0.f;
        }
}

// One (request, head)'s state rows `col` as S^T tiles: dk = 16 kb + 4 j + i.
template <int KB>
__device__ __forceinline__ void load_state(f4 (&S)[KB], const float *row, int dk, bool ok, int j)
{
    const bool vec = dk % 4 == 0;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
        S[kb] = ok ? widen(load_raw4(row, 16 * kb + 4 * j, dk, vec)) : f4{0.f, 0.f, 0.f, 0.f};
}

// rows (token) x dk times the state: acc[m] += K[16 m ..][:] S^T
template <int DK>
__device__ __forceinline__ void rows_times_state(f4 (&acc)[Geo<DK>::MB], const float *rows, const f4 (&S)[Geo<DK>::KB], int c, int j)
{
    using G = Geo<DK>;
#pragma unroll
    for (int kb = 0; kb < G::KB; ++kb) {
        f4 x[G::MB];
#pragma unroll
        for (int m = 0; m < G::MB; ++m) x[m] = *reinterpret_cast<const f4 *>(rows + (16 * m + c) * G::LD + 16 * kb + 4 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < G::MB; ++m) acc[m] = mfma1(x[m][i], S[kb][i], acc[m]);
    }
}

// state update: S[kb] += rows^T X
template <int DK>
__device__ __forceinline__ void state_update(f4 (&S)[Geo<DK>::KB], const float *rows, const f4 (&X)[Geo<DK>::MB], int c, int j)
{
    using G = Geo<DK>;
#pragma unroll
    for (int m = 0; m < G::MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *row = rows + (16 * m + 4 * j + i) * G::LD + c;
#pragma unroll
            for (int kb = 0; kb < G::KB; ++kb) S[kb] = mfma1(row[16 * kb], X[m][i], S[kb]);
        }
}

// ---------------------------------------------------------------- forward chain
// One workgroup per (request, value head, 64 state rows); wave w keeps S^T of
// 16 rows in its accumulators over the whole chain.
template <int DK, typename TA, bool RETR>
__global__ __launch_bounds__(256, 2) void k_back_states(const BackParams a)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, KB = G::KB, TRI = G::TRI;
    __shared__ __align__(16) float Kh[C * G::LD];
    __shared__ __align__(16) float s_eg[C], s_x[C];
    const Params &p = a.p;
    const int tiles = (a.VB + 3) / 4;
    const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, h = bh % p.HV, b = bh / p.HV;
    const int first = a.off[b], count = a.off[b + 1] - first;
    if (count == 0) return;
    const int hq = h / (p.HV / p.H);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, j = lane >> 4;
    const int vb = tile * 4 + wave, col = vb * 16 + c;
    const bool on = vb < a.VB, vec = p.dk % 4 == 0;
    const int64_t start = a.tok[2 * b];
    const int64_t len = a.tok[2 * b + 1];

    f4 S[KB];
    load_state(S, p.init ? p.init + (((size_t)b * p.HV + h) * p.dv + col) * p.dk : nullptr, p.dk,
               p.init != nullptr && col < p.dv, j);
    Stage<DK, TA, 256> k;
    {
        const float *sc = a.sc + ((size_t)first * p.HV + h) * (BACK_SC * C);
        k.load(static_cast<const TA *>(p.k), sc + SC_RK * C, start, len < C ? (int)len : C, p.H, hq, p.dk, vec);
    }
    for (int n = 0; n < count; ++n) {
        const size_t rec = (size_t)(first + n) * p.HV + h;
        const int64_t t0 = start + (int64_t)n * C;
        const int64_t left = len - (int64_t)n * C;
        const int cnt = left < C ? (int)left : C;
        const float *sc = a.sc + rec * (BACK_SC * C);
        lds_barrier();  // the previous step's reads of Kh, s_*
        k.store(Kh);
        if (tid < C) {
            s_eg[tid] = sc[SC_EG * C + tid];
            s_x[tid] = sc[SC_KD * C + tid] * sc[SC_B * C + tid];
        }
        const float gamma = sc[SC_EG * C + C - 1];
        if (n + 1 < count) {
            const int64_t rest = left - C;
            k.load(static_cast<const TA *>(p.k), sc + (size_t)p.HV * (BACK_SC * C) + SC_RK * C, t0 + C,
                   rest < C ? (int)rest : C, p.H, hq, p.dk, vec);
        }
        lds_barrier();
        if (!on) continue;
        f4 E[MB];
        load_cols<MB>(E, static_cast<const TA *>(p.v), t0, cnt, p.HV, h, p.dv, col, j);
        float *Sw = a.s + (rec * KB * a.VB + vb) * FRAG;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) put_frag_rows(Sw + (size_t)kb * a.VB * FRAG, S[kb]);
        if constexpr (RETR) {
            f4 Y[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) Y[m] = f4{0.f, 0.f, 0.f, 0.f};
            rows_times_state<DK>(Y, Kh, S, c, j);
            f4 Z[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                Z[m] = E[m] - *reinterpret_cast<const f4 *>(s_eg + 16 * m + 4 * j) * Y[m];
                E[m] = f4{0.f, 0.f, 0.f, 0.f};
            }
            const float *T = a.t1 + rec * TRI * FRAG;
#pragma unroll
            for (int kb = 0; kb < MB; ++kb)
#pragma unroll
                for (int m = kb; m < MB; ++m) E[m] = mfma4(get_frag(T + tri(m, kb) * FRAG), Z[kb], E[m]);
        }
        float *Ew = a.e + (rec * MB * a.VB + vb) * FRAG;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            put_frag_rows(Ew + (size_t)m * a.VB * FRAG, E[m]);
            E[m] *= *reinterpret_cast<const f4 *>(s_x + 16 * m + 4 * j);
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) S[kb] *= gamma;
        state_update<DK>(S, Kh, E, c, j);
    }
}

// ---------------------------------------------------------------- backward chain
template <int DK, typename TA, bool RETR>
__global__ __launch_bounds__(256, 2) void k_back_chain(const BackParams a)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, KB = G::KB, TRI = G::TRI;
    __shared__ __align__(16) float Kh[C * G::LD], Qh[C * G::LD];
    __shared__ __align__(16) float s_eg[C], s_kd[C], s_b[C];
    const Params &p = a.p;
    const int tiles = (a.VB + 3) / 4;
    const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, h = bh % p.HV, b = bh / p.HV;
    const int first = a.off[b], count = a.off[b + 1] - first;
    const int hq = h / (p.HV / p.H);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, j = lane >> 4;
    const int vb = tile * 4 + wave, col = vb * 16 + c;
    const bool on = vb < a.VB, vec = p.dk % 4 == 0;
    const int64_t start = a.tok[2 * b];
    const int64_t len = a.tok[2 * b + 1];
    const TA *kp = static_cast<const TA *>(p.k), *qp = static_cast<const TA *>(p.q);

    f4 dS[KB];
    const size_t srow = (((size_t)b * p.HV + h) * p.dv + col) * p.dk;
    load_state(dS, a.d_final ? a.d_final + srow : nullptr, p.dk, a.d_final != nullptr && col < p.dv, j);
    Stage<DK, TA, 256> k, q;
    auto fetch = [&](int n) {
        const float *sc = a.sc + ((size_t)(first + n) * p.HV + h) * (BACK_SC * C);
        const int64_t left = len - (int64_t)n * C;
        const int cnt = left < C ? (int)left : C;
        k.load(kp, sc + SC_RK * C, start + (int64_t)n * C, cnt, p.H, hq, p.dk, vec);
        q.load(qp, sc + SC_RQ * C, start + (int64_t)n * C, cnt, p.H, hq, p.dk, vec);
    };
    if (count > 0) fetch(count - 1);
    for (int n = count - 1; n >= 0; --n) {
        const size_t rec = (size_t)(first + n) * p.HV + h;
        const int64_t t0 = start + (int64_t)n * C;
        const int64_t left = len - (int64_t)n * C;
        const int cnt = left < C ? (int)left : C;
        const float *sc = a.sc + rec * (BACK_SC * C);
        lds_barrier();
        k.store(Kh);
        q.store(Qh);
        if (tid < C) {
            s_eg[tid] = sc[SC_EG * C + tid];
            s_kd[tid] = sc[SC_KD * C + tid];
            s_b[tid] = sc[SC_B * C + tid];
        }
        const float gamma = sc[SC_EG * C + C - 1];
        if (n > 0) fetch(n - 1);
        lds_barrier();
        if (!on) continue;
        f4 dO[MB];
        load_cols<MB>(dO, static_cast<const TA *>(a.d_o), t0, cnt, p.HV, h, p.dv, col, j);
        float *Sw = a.ds + (rec * KB * a.VB + vb) * FRAG;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) put_frag_rows(Sw + (size_t)kb * a.VB * FRAG, dS[kb]);
        f4 D[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) D[m] = f4{0.f, 0.f, 0.f, 0.f};
        rows_times_state<DK>(D, Kh, dS, c, j);
#pragma unroll
        for (int m = 0; m < MB; ++m) D[m] *= *reinterpret_cast<const f4 *>(s_kd + 16 * m + 4 * j);
        const float *P = a.pt + rec * TRI * FRAG;
#pragma unroll
        for (int kb = 0; kb < MB; ++kb)
#pragma unroll
            for (int m = 0; m <= kb; ++m) D[m] = mfma4(get_frag(P + tri(kb, m) * FRAG), dO[kb], D[m]);
        if constexpr (RETR) {
            f4 Y[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) Y[m] = f4{0.f, 0.f, 0.f, 0.f};
            const float *T = a.t2 + rec * TRI * FRAG;
#pragma unroll
            for (int kb = 0; kb < MB; ++kb)
#pragma unroll
                for (int m = 0; m <= kb; ++m) Y[m] = mfma4(get_frag(T + tri(kb, m) * FRAG), D[kb], Y[m]);
            float *Yw = a.y + (rec * MB * a.VB + vb) * FRAG;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                put_frag_rows(Yw + (size_t)m * a.VB * FRAG, Y[m]);
                D[m] = Y[m] * *reinterpret_cast<const f4 *>(s_b + 16 * m + 4 * j);
            }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const f4 eg = *reinterpret_cast<const f4 *>(s_eg + 16 * m + 4 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * m + 4 * j + i;
                if (t < cnt && col < p.dv)
                    static_cast<TA *>(a.dv)[((size_t)(t0 + t) * p.HV + h) * p.dv + col] = from_f32<TA>(D[m][i]);
            }
            dO[m] *= eg;
            D[m] *= -eg;
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) dS[kb] *= gamma;
        state_update<DK>(dS, Qh, dO, c, j);
        if constexpr (RETR) state_update<DK>(dS, Kh, D, c, j);
    }
    if (a.d_init && on && col < p.dv) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) store4(a.d_init + srow, 16 * kb + 4 * j, p.dk, vec, dS[kb]);
    }
}

// ---------------------------------------------------------------- gradients of a chunk
// One workgroup (8 waves) per (chunk, q/k head), the value heads that share it
// in turn, dQ and dK summed over them in the accumulators.  Wave (tb, part)
// owns the 16 tokens of block tb as accumulator columns and 1/PARTS of the key
// channels as rows; of the chunk x chunk products it forms SBW column blocks.
template <int DK, typename TA, bool RETR>
__global__ __launch_bounds__(512, 2) void k_back_grad(const BackParams a)
{
    using G = Geo<DK>;
    constexpr int C = G::C, MB = G::MB, KB = G::KB, LD = G::LD, LC = G::LC;
    constexpr int PARTS = 8 / MB, KBW = KB / PARTS, SBW = (MB + PARTS - 1) / PARTS;
    __shared__ __align__(16) float Kh[C * LD], Qh[C * LD], Fe[C * LC], Wm[C * LC];
    __shared__ __align__(16) float s_sc[5 * C];
    __shared__ float s_u[PARTS][C], s_w[PARTS][C], s_db[C], s_row[C][MB], s_col[MB][C], s_dot[8];

    const Params &p = a.p;
    const int ci = blockIdx.x / p.H, hq = blockIdx.x % p.H;
    if (ci >= a.off[p.B]) return;
    int64_t t0;
    int cnt;
    chunk_tokens(a, ci, C, t0, cnt);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, j = lane >> 4;
    const int tb = wave / PARTS, part = wave % PARTS, kb0 = part * KBW;
    const int t = 16 * tb + c;
    const bool live = t < cnt, veck = p.dk % 4 == 0, vecv = p.dv % 4 == 0;
    const int R = p.HV / p.H;
    {
        const float *sc = a.sc + ((size_t)ci * p.HV + (size_t)hq * R) * (BACK_SC * C);
        Stage<DK, TA, 512> k, q;
        k.load(static_cast<const TA *>(p.k), sc + SC_RK * C, t0, cnt, p.H, hq, p.dk, veck);
        q.load(static_cast<const TA *>(p.q), sc + SC_RQ * C, t0, cnt, p.H, hq, p.dk, veck);
        k.store(Kh);
        q.store(Qh);
    }
    __syncthreads();
    const f4 zero = {0.f, 0.f, 0.f, 0.f};
    // tiles of (K Q^T, K K^T): rows s of block sb, columns t
    f4 qk[SBW], kk[SBW];
    bool use[SBW];
#pragma unroll
    for (int x = 0; x < SBW; ++x) {
        const int sb = part * SBW + x;
        use[x] = sb <= tb;
        qk[x] = kk[x] = zero;
        if (use[x]) {
#pragma unroll 4
            for (int kb = 0; kb < KB; ++kb) {
                const f4 s = *reinterpret_cast<const f4 *>(Kh + (16 * sb + c) * LD + 16 * kb + 4 * j);
                qk[x] = mfma4(s, *reinterpret_cast<const f4 *>(Qh + t * LD + 16 * kb + 4 * j), qk[x]);
                if (RETR) kk[x] = mfma4(s, *reinterpret_cast<const f4 *>(Kh + t * LD + 16 * kb + 4 * j), kk[x]);
            }
        }
    }
    f4 dq[KBW], dk[KBW];
#pragma unroll
    for (int kb = 0; kb < KBW; ++kb) dq[kb] = dk[kb] = zero;

    for (int r = 0; r < R; ++r) {
        const int h = hq * R + r;
        const size_t rec = (size_t)ci * p.HV + h;
        for (int n = tid; n < 5 * C; n += 512) s_sc[n] = a.sc[rec * (BACK_SC * C) + n];
        __syncthreads();
        const float *s_b = s_sc + SC_B * C, *s_gh = s_sc + SC_GH * C, *s_gl = s_sc + SC_GL * C;
        const float eg = s_sc[SC_EG * C + t], kd = s_sc[SC_KD * C + t], bt = s_b[t];

        // products over the state rows
        f4 A1[KBW], A2[KBW], A3[KBW], F[SBW], X[SBW];
#pragma unroll
        for (int kb = 0; kb < KBW; ++kb) A1[kb] = A2[kb] = A3[kb] = zero;
#pragma unroll
        for (int x = 0; x < SBW; ++x) F[x] = X[x] = zero;
        float db = 0.f, dot = 0.f;
        const TA *orow = static_cast<const TA *>(a.d_o) + ((size_t)(t0 + t) * p.HV + h) * p.dv;
        const float *Sp = a.s + rec * KB * a.VB * FRAG, *Dp = a.ds + rec * KB * a.VB * FRAG;
        const float *Ep = a.e + rec * MB * a.VB * FRAG, *Yp = RETR ? a.y + rec * MB * a.VB * FRAG : nullptr;
        for (int vb = 0; vb < a.VB; ++vb) {
            const f4 o = live ? widen(load_raw4(orow, 16 * vb + 4 * j, p.dv, vecv)) : zero;
            const f4 e = get_frag(Ep + ((size_t)tb * a.VB + vb) * FRAG);
            const f4 y = RETR ? get_frag(Yp + ((size_t)tb * a.VB + vb) * FRAG) : zero;
            f4 s[KBW], d[KBW];
#pragma unroll
            for (int kb = 0; kb < KBW; ++kb) {
                s[kb] = get_frag(Sp + ((size_t)(kb0 + kb) * a.VB + vb) * FRAG);
                d[kb] = get_frag(Dp + ((size_t)(kb0 + kb) * a.VB + vb) * FRAG);
            }
#pragma unroll
            for (int x = 0; x < SBW; ++x)
                if (use[x]) {
                    const f4 es = get_frag(Ep + ((size_t)(part * SBW + x) * a.VB + vb) * FRAG);
                    F[x] = mfma4(es, o, F[x]);
                    if (RETR) X[x] = mfma4(es, y, X[x]);
                }
            if (RETR) db += dot4(y, e);
            const f4 bd = RETR ? e * bt : e;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int kb = 0; kb < KBW; ++kb) {
                    A1[kb] = mfma1(s[kb][i], o[i], A1[kb]);
                    A3[kb] = mfma1(d[kb][i], bd[i], A3[kb]);
                    if (RETR) A2[kb] = mfma1(s[kb][i], y[i], A2[kb]);
                }
            if (tb == 0)
#pragma unroll
                for (int kb = 0; kb < KBW; ++kb) dot += dot4(s[kb], d[kb]);
        }

        // per token: what crosses the token from the state
        float u = 0.f, w = 0.f;
#pragma unroll
        for (int kb = 0; kb < KBW; ++kb) {
            const f4 qh = *reinterpret_cast<const f4 *>(Qh + t * LD + 16 * (kb0 + kb) + 4 * j);
            const f4 kh = *reinterpret_cast<const f4 *>(Kh + t * LD + 16 * (kb0 + kb) + 4 * j);
            A1[kb] *= eg;
            A3[kb] *= kd;
            w += dot4(qh, A1[kb]);
            u += dot4(kh, A3[kb]);
            dq[kb] += A1[kb];
            dk[kb] += A3[kb];
            if (RETR) {
                A2[kb] *= -bt * eg;
                w += dot4(kh, A2[kb]);
                dk[kb] += A2[kb];
            }
        }
        u = sum_j(u);
        w = sum_j(w);
        db = sum_j(db);
        if (j == 0) {
            s_u[part][t] = u;
            s_w[part][t] = w;
            if (part == 0) s_db[t] = db;
        }
        if (tb == 0) {
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o);
            if (lane == 0) s_dot[part] = dot;
        }

        // the chunk x chunk tiles: factors, and M's part of dg
#pragma unroll
        for (int x = 0; x < SBW; ++x)
            if (use[x]) {
                const int s0 = 16 * (part * SBW + x) + 4 * j;
                const float gh = s_gh[t], gl = s_gl[t];
                f4 f, wv = zero, M;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = s0 + i;
                    const float e = s <= t ? exp_split(gh - s_gh[s], gl - s_gl[s]) * (RETR ? s_b[s] : 1.f) : 0.f;
                    f[i] = F[x][i] * e;
                    M[i] = s < t ? f[i] * qk[x][i] : 0.f;
                    if (RETR) {
                        wv[i] = s < t ? bt * e * X[x][i] : 0.f;
                        M[i] -= wv[i] * kk[x][i];
                    }
                }
                *reinterpret_cast<f4 *>(Fe + t * LC + s0) = f;
                if (RETR) *reinterpret_cast<f4 *>(Wm + t * LC + s0) = wv;
                // sums over the columns before each one, within the tile's row t ...
                const float four = (M[0] + M[1]) + (M[2] + M[3]);
                const float a1 = __shfl_up(four, 16), a2 = __shfl_up(four, 32), a3 = __shfl_up(four, 48);
                float pre = (j > 0 ? a1 : 0.f) + (j > 1 ? a2 : 0.f) + (j > 2 ? a3 : 0.f);
                if (j == 3) s_row[t][part * SBW + x] = pre + four;
                // ... then over the rows t >= s
                f4 sum;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum[i] = sum16(s0 + i <= t ? pre : 0.f);
                    pre += M[i];
                }
                if (c == 0)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s_col[tb][s0 + i] = sum[i];
            }
        __syncthreads();

        // products over the chunk's tokens
#pragma unroll
        for (int sb = 0; sb < MB; ++sb) {
            if (sb <= tb) {  // row t: columns s <= t
                const f4 f = *reinterpret_cast<const f4 *>(Fe + t * LC + 16 * sb + 4 * j);
                const f4 wv = RETR ? *reinterpret_cast<const f4 *>(Wm + t * LC + 16 * sb + 4 * j) : zero;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int kb = 0; kb < KBW; ++kb) {
                        const float x = Kh[(16 * sb + 4 * j + i) * LD + 16 * (kb0 + kb) + c];
                        dq[kb] = mfma1(x, f[i], dq[kb]);
                        if (RETR) dk[kb] = mfma1(x, -wv[i], dk[kb]);
                    }
            }
            if (sb >= tb) {  // column t: rows >= t
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * sb + 4 * j + i;
                    const float f = Fe[row * LC + t], wv = RETR ? -Wm[row * LC + t] : 0.f;
#pragma unroll
                    for (int kb = 0; kb < KBW; ++kb) {
                        dk[kb] = mfma1(Qh[row * LD + 16 * (kb0 + kb) + c], f, dk[kb]);
                        if (RETR) dk[kb] = mfma1(Kh[row * LD + 16 * (kb0 + kb) + c], wv, dk[kb]);
                    }
                }
            }
        }

        // wave 0, a lane a token: dg and db
        if (wave == 0) {
            const int s = lane < C ? lane : C - 1;
            const bool mine = lane < C;
            float us = 0.f, ws = 0.f;
#pragma unroll
            for (int n = 0; n < PARTS; ++n) {
                us += s_u[n][s];
                ws += s_w[n][s];
            }
            us = mine ? us : 0.f;
            ws = mine ? ws : 0.f;
            float rows[MB];  // rows[m]: suffix sums over t of the sums over columns of blocks before m
            rows[0] = 0.f;
#pragma unroll
            for (int m = 1; m < MB; ++m) rows[m] = rows[m - 1] + (mine && m - 1 <= lane / 16 ? s_row[s][m - 1] : 0.f);
            float pre = us, suf = ws;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const float x = __shfl_up(pre, o), y = __shfl_down(suf, o);
                if (lane >= o) pre += x;
                if (lane + o < 64) suf += y;
#pragma unroll
                for (int m = 1; m < MB; ++m) {
                    const float z = __shfl_down(rows[m], o);
                    if (lane + o < 64) rows[m] += z;
                }
            }
            pre = __shfl_up(pre, 1);
            float g = lane > 0 ? pre : 0.f;
            g += suf;
            const int blk = s / 16;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (m == blk) g += rows[m];
                if (m >= blk) g += s_col[m][s];
            }
            float d = 0.f;
#pragma unroll
            for (int n = 0; n < PARTS; ++n) d += s_dot[n];
            g += s_sc[SC_EG * C + C - 1] * d;
            float da = 0.f, ds = 0.f;  // raw-gate arm: d of the projection (and of the bias), d of the scale
            if (lane < cnt) {
                const size_t th = (size_t)(t0 + lane) * p.HV + h;
                if (a.decays) {
                    if (p.gate_qwen) {
                        const float x = load_gate(p, th) + p.dt_bias[h];
                        da = g * gate_scale(p, h) * sigmoid_f32(x);
                        ds = g * softplus_f32(x);
                        g = da;
                    }
                    if (p.gate_dt == 1) static_cast<half_t *>(a.d_gate)[th] = from_f32<half_t>(g);
                    else if (p.gate_dt == 2) static_cast<bf16_t *>(a.d_gate)[th] = from_f32<bf16_t>(g);
                    else static_cast<float *>(a.d_gate)[th] = g;
                }
                if (RETR) {
                    const float rate = s_b[lane];
                    a.d_beta[th] = p.beta_sigmoid ? s_db[lane] * rate * (1.f - rate) : s_db[lane];
                }
            }
            if (p.gate_qwen) {
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
        __syncthreads();
    }

    // through the L2 norm: d x = r (d x^ - x^ (x^ . d x^)), x^ = r x
    float nq = 0.f, nk = 0.f;
    const float *sc = a.sc + ((size_t)ci * p.HV + (size_t)hq * R) * (BACK_SC * C);
    const float rq = sc[SC_RQ * C + t], rk = sc[SC_RK * C + t], inv = 1.f / p.scale;
    if (p.qk_l2_norm) {
#pragma unroll
        for (int kb = 0; kb < KBW; ++kb) {
            nq += dot4(*reinterpret_cast<const f4 *>(Qh + t * LD + 16 * (kb0 + kb) + 4 * j), dq[kb]);
            nk += dot4(*reinterpret_cast<const f4 *>(Kh + t * LD + 16 * (kb0 + kb) + 4 * j), dk[kb]);
        }
        nq = sum_j(nq);
        nk = sum_j(nk);
        if (j == 0) {
            s_u[part][t] = nq;
            s_w[part][t] = nk;
        }
        __syncthreads();
        nq = nk = 0.f;
#pragma unroll
        for (int n = 0; n < PARTS; ++n) {
            nq += s_u[n][t];
            nk += s_w[n][t];
        }
        nq *= inv * inv;
    }
    if (live) {
        const size_t row = ((size_t)(t0 + t) * p.H + hq) * p.dk;
#pragma unroll
        for (int kb = 0; kb < KBW; ++kb) {
            const int col = 16 * (kb0 + kb) + 4 * j;
            f4 gq = dq[kb], gk = dk[kb];
            if (p.qk_l2_norm) {
                gq -= *reinterpret_cast<const f4 *>(Qh + t * LD + col) * nq;
                gk -= *reinterpret_cast<const f4 *>(Kh + t * LD + col) * nk;
            }
            store4(static_cast<TA *>(a.dq) + row, col, p.dk, veck, gq * rq);
            store4(static_cast<TA *>(a.dk) + row, col, p.dk, veck, gk * rk);
        }
    }
}

// ---------------------------------------------------------------- launches
template <int DK, typename TA, bool RETR>
hipError_t launch_back_typed(const BackParams &a, hipStream_t s)
{
    const Params &p = a.p;
    const unsigned per_chunk = (unsigned)a.chunks * p.H, chains = (unsigned)p.B * p.HV * ((a.VB + 3) / 4);
    if (a.chunks > 0) {
        hipLaunchKernelGGL((k_back_prep<DK, TA, RETR>), dim3(per_chunk), dim3(256), 0, s, a);
        hipLaunchKernelGGL((k_back_states<DK, TA, RETR>), dim3(chains), dim3(256), 0, s, a);
    }
    hipLaunchKernelGGL((k_back_chain<DK, TA, RETR>), dim3(chains), dim3(256), 0, s, a);
    if (a.chunks > 0) hipLaunchKernelGGL((k_back_grad<DK, TA, RETR>), dim3(per_chunk), dim3(512), 0, s, a);
    return hipGetLastError();
}

template <typename TA>
hipError_t launch_back_act(const BackParams &a, bool retrieves, hipStream_t s)
{
    const int dk = a.p.dk;
    if (dk <= 64) return retrieves ? launch_back_typed<64, TA, true>(a, s) : launch_back_typed<64, TA, false>(a, s);
    if (dk <= 128) return retrieves ? launch_back_typed<128, TA, true>(a, s) : launch_back_typed<128, TA, false>(a, s);
    return retrieves ? launch_back_typed<256, TA, true>(a, s) : launch_back_typed<256, TA, false>(a, s);
}

}  // namespace
}  // namespace gdr
