// gdr_backward_launch.hpp -- the backward pass's argument block, workspace
// layout and launchers (internal to libgdr).
#pragma once

#include <hip/hip_runtime.h>

#include "gdr_device.hpp"

namespace gdr {

// Tokens of a chunk: 64, or 32 where a chunk's q and k rows of up to 256
// channels would not fit twice in LDS beside the chunk x chunk tiles.
__host__ __device__ constexpr int back_chunk(int dk) { return dk > 128 ? 32 : 64; }
__host__ __device__ constexpr int back_dk_tile(int dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }

// 16 x 32 blocks of a triangular chunk x chunk operand
__host__ __device__ constexpr int back_tri_blocks(int C) { return C == 64 ? 6 : 2; }

// Per (chunk, value head) scalars, a row of back_chunk floats each: e^G,
// e^(Gamma - G), update rate, G as (hi, lo), and the factors of q (with the
// scale) and k.
enum BackScalar : int { SC_EG = 0, SC_KD, SC_B, SC_GH, SC_GL, SC_RQ, SC_RK, BACK_SC };

// Rows (of back_chunk floats) of what k_back_grad leaves for dg and db, per
// (chunk, value head): u, w, Y . E, M's sums within the column's own block,
// the state's part, and M's sums over the column blocks before each block.
enum BackGateRow : int { GX_U = 0, GX_W, GX_DB, GX_COL, GX_STATE, GX_ROW, GX = GX_ROW + 3 };

struct BackParams {
    Params p;                   // q, k, v, gate, beta, requests, initial state
    const void *d_o;
    const float *d_final;       // (B, HV, dv, dk) or nullptr (zeros)
    void *dq, *dk, *dv, *d_gate;
    float *d_beta;              // (T, HV): the output, or workspace when it is summed over the heads
    float *d_rate;              // (T, 1) when d_beta is summed over the heads, or nullptr
    float *gate_sums;           // raw-gate arm: per (chunk, value head) sums of d_a and of d_scale
    float *d_a_log, *d_dt_bias, *d_gate_scale;
    float *d_init;              // or nullptr
    // workspace
    int32_t *off;               // (B + 1) first chunk of each request; off[B] = chunks in use
    int32_t *tok;               // (B, 2) first token and length of each request
    int32_t *order;             // (B) requests, the longest first
    int32_t *where;             // (chunks, 2) first token and length of each chunk
    uint16_t *act;              // fp32 activations, per (chunk, q/k head): operand fragments of k^T, q^T
    uint16_t *tri;              // per (chunk, value head): P^T, and with retrieval (I + diag(b) L)^-T, (I + L diag(b))^-1
    float *sc, *s, *ds, *e, *y; // scalars; S0, dS1, E, Y as fp32 fragments
    float *gx;                  // see BackGateRow
    // between the segments of the chains (nseg > 1): M by rows and by columns,
    // carries, states at their starts, and the same of the backward chain
    float *seg_m, *seg_mt, *seg_carry, *seg_state, *seg_dcarry, *seg_dstate;
    int32_t nseg;
    int32_t chunks;             // chunk budget: ceil(T / C) + B
    int32_t VB;                 // 16-row blocks of dv, a multiple of 4
    int32_t decays;
    int32_t zero_rest;          // zero in the gradient rows of tokens that no request covers
};

// Chunk table: request b covers [m_b, m_(b+1)) where m is the running maximum
// of the clamped cu_seqlens (so ranges never overlap), or its part of a
// uniform batch.
hipError_t launch_back_table(const BackParams &a, hipStream_t s);
hipError_t launch_back_f32(const BackParams &a, bool retrieves, hipStream_t s);
hipError_t launch_back_f16(const BackParams &a, bool retrieves, hipStream_t s);
hipError_t launch_back_bf16(const BackParams &a, bool retrieves, hipStream_t s);
// After the gradients: parameters of the raw-gate arm and a rate shared by the heads.
hipError_t launch_back_sums(const BackParams &a, hipStream_t s);

// Gradients of the gate fusion (gdr_gate_backward); dt: 0 fp32, 1 fp16, 2 bf16.
struct GateBackParams {
    int64_t rows;
    int32_t heads, dt;
    const void *a, *d_decay, *b, *d_beta;
    const float *dt_bias, *decay_scale;
    void *d_a, *d_b;
    float *d_dt_bias, *d_scale;
    float *partial;             // gate_back_blocks x 2 x heads floats
};
int gate_back_blocks(int64_t rows, int heads);
hipError_t launch_gate_backward(const GateBackParams &g, hipStream_t s);

}  // namespace gdr
