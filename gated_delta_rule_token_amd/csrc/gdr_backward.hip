// gdr_backward.hip -- the backward pass's chunk table, its sums over tokens
// and heads, and the gradients of the standalone gate fusion.
#include "gdr_backward_launch.hpp"

namespace gdr {

// ---------------------------------------------------------------- chunk table
// One workgroup.  Request b covers [m_b, m_(b+1)), m_b the largest of the
// clamped cu_seqlens entries up to b: for a non-decreasing cu_seqlens its own
// range, and in any case ranges that do not overlap, so two requests never
// write one gradient row and the chunk counts sum to at most
// ceil(T / C) + B.  off[] is the exclusive prefix sum of the chunk counts, and
// order[] the requests from the longest to the shortest, up to RANKED of them
// (each is compared with every other: 256 take 6 us, 1024 would take 100):
// the chains start in that order.
constexpr int RANKED = 256;

__global__ __launch_bounds__(256) void k_back_table(const BackParams a, int C)
{
    __shared__ int64_t s_m[256], s_n[256];
    __shared__ int64_t carry_m, carry_n;
    __shared__ int32_t s_len[RANKED];
    const Params &p = a.p;
    const int tid = threadIdx.x;
    if (tid == 0) {
        int64_t x = p.cu_seqlens ? p.cu_seqlens[0] : 0;
        carry_m = x < 0 ? 0 : (x > p.T ? p.T : x);
        carry_n = 0;
    }
    __syncthreads();
    for (int base = 0; base < p.B; base += 256) {
        const int b = base + tid;
        int64_t start = 0, end = 0;
        if (p.cu_seqlens) {
            int64_t x = b < p.B ? p.cu_seqlens[b + 1] : 0;
            s_m[tid] = x < 0 ? 0 : (x > p.T ? p.T : x);
            __syncthreads();
            for (int o = 1; o < 256; o <<= 1) {
                const int64_t v = tid >= o ? s_m[tid - o] : 0;
                __syncthreads();
                if (v > s_m[tid]) s_m[tid] = v;
                __syncthreads();
            }
            const int64_t m = carry_m;
            start = tid > 0 && s_m[tid - 1] > m ? s_m[tid - 1] : m;
            end = s_m[tid] > m ? s_m[tid] : m;
        } else if (b < p.B) {
            request_range(p, b, start, end);
        }
        const int64_t n = b < p.B ? (end - start + C - 1) / C : 0;
        s_n[tid] = n;
        __syncthreads();
        for (int o = 1; o < 256; o <<= 1) {
            const int64_t v = tid >= o ? s_n[tid - o] : 0;
            __syncthreads();
            s_n[tid] += v;
            __syncthreads();
        }
        if (b < p.B) {
            a.off[b] = (int32_t)(carry_n + s_n[tid] - n);
            a.tok[2 * b] = (int32_t)start;
            a.tok[2 * b + 1] = (int32_t)(end - start);
            if (p.B <= RANKED) s_len[b] = (int32_t)n;
            else a.order[b] = b;
        }
        __syncthreads();
        if (tid == 255) {
            carry_n += s_n[255];
            if (p.cu_seqlens && s_m[255] > carry_m) carry_m = s_m[255];
        }
        __syncthreads();
    }
    if (tid == 0) a.off[p.B] = (int32_t)carry_n;
    if (p.B <= RANKED)
        for (int b = tid; b < p.B; b += 256) {
            const int32_t n = s_len[b];
            int rank = 0;
#pragma unroll 8
            for (int i = 0; i < p.B; ++i) rank += s_len[i] > n || (s_len[i] == n && i < b);
            a.order[rank] = b;
        }
}

hipError_t launch_back_table(const BackParams &a, hipStream_t s)
{
    hipLaunchKernelGGL(k_back_table, dim3(1), dim3(256), 0, s, a, back_chunk(a.p.dk));
    return hipGetLastError();
}

// ---------------------------------------------------------------- sums over chunks and heads
// Block (256) sum in a fixed order.
__device__ __forceinline__ float block_sum(float x, float *s)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
    __syncthreads();
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Workgroup h: the chunks' sums of head h, always added in the same order.
__global__ __launch_bounds__(256) void k_back_gate_sums(const BackParams a)
{
    __shared__ float s[4];
    const int h = blockIdx.x, n = a.off[a.p.B];
    float da = 0.f, ds = 0.f;
    for (int ci = threadIdx.x; ci < n; ci += 256) {
        const float *x = a.gate_sums + 2 * ((size_t)ci * a.p.HV + h);
        da += x[0];
        ds += x[1];
    }
    da = block_sum(da, s);
    ds = block_sum(ds, s);
    if (threadIdx.x == 0) {
        a.d_dt_bias[h] = da;
        if (a.d_gate_scale) a.d_gate_scale[h] = ds;
        if (a.d_a_log) a.d_a_log[h] = ds * gate_scale(a.p, h);  // scale = -exp(a_log)
    }
}

// One rate per token: the sum over the value heads, for the tokens of each request.
__global__ __launch_bounds__(256) void k_back_rate_sums(const BackParams a)
{
    const int b = blockIdx.x;
    const int64_t t0 = a.tok[2 * b];
    const int32_t len = a.tok[2 * b + 1];
    for (int64_t t = (int64_t)blockIdx.y * 256 + threadIdx.x; t < len; t += (int64_t)gridDim.y * 256) {
        const float *x = a.d_beta + (size_t)(t0 + t) * a.p.HV;
        float sum = 0.f;
        for (int h = 0; h < a.p.HV; ++h) sum += x[h];
        a.d_rate[t0 + t] = sum;
    }
}

hipError_t launch_back_sums(const BackParams &a, hipStream_t s)
{
    if (a.p.gate_qwen && a.decays) hipLaunchKernelGGL(k_back_gate_sums, dim3(a.p.HV), dim3(256), 0, s, a);
    if (a.d_rate && a.p.B > 0) {
        const int64_t most = (a.p.T + 255) / 256;
        hipLaunchKernelGGL(k_back_rate_sums, dim3(a.p.B, (unsigned)(most < 1 ? 1 : most > 64 ? 64 : most)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- gate fusion
// x = a + dt_bias, decay = scale softplus(x), beta = sigmoid(b):
//   d_a = d_decay scale sigmoid(x),  d_b = d_beta beta (1 - beta)
//   d_dt_bias = sum over rows of d_a,  d_scale = sum over rows of d_decay softplus(x)
// Memory-bound and elementwise but for the sums.  A thread keeps V columns
// (heads) and walks down the rows of its workgroup's slice, so that the sums
// stay in registers; the sums of several slices are joined in a fixed order by
// a second kernel.  V = 8 where a row is a whole number of 16-byte vectors.
// The elementwise functions are the hardware's 2^x and 1/x (an ulp each) with
// short series of their own, good to a few ulps: with expf, log1pf and IEEE
// divisions the kernel was bound by its 200 VALU instructions an element
// (262,144 x 32 in bf16 with the rate: 33.7 us; now 26.6, and 19.5 at the copy
// rate).  Small calls are bound by the launches and the call itself, 14 us.
template <typename T, int V> struct __align__(sizeof(T) * V) Pack { T x[V]; };

// e^-x for x >= 0: x log2(e) in two parts, the small one as a factor.  The
// product's rounding error comes exactly from an fma with the rounded product
// taken off (Dekker's two-product, by fma); the constants are log2(e) rounded to
// fp32 and what that leaves of it.
__device__ __forceinline__ float exp_minus(float x)
{
    x = x > 128.f ? 128.f : x;
    const float t = x * -1.44269502e+0f;
    const float lo = fmaf(x, -1.92596303e-8f, fmaf(x, -1.44269502e+0f, -t));
    return __builtin_amdgcn_exp2f(t) * fmaf(lo, 0.69314718f, 1.f);
}

// log(1 + e) for 0 <= e <= 1: 2 atanh(s), s = e / (2 + e) <= 1/3, to s^15
__device__ __forceinline__ float log_one_plus(float e)
{
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), s2 = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, s2, 1.f / 13.f);
    p = fmaf(p, s2, 1.f / 11.f);
    p = fmaf(p, s2, 1.f / 9.f);
    p = fmaf(p, s2, 1.f / 7.f);
    p = fmaf(p, s2, 1.f / 5.f);
    p = fmaf(p, s2, 1.f / 3.f);
    p = fmaf(p, s2, 1.f);
    return 2.f * s * p;
}

constexpr int GATE_THREADS = 256;

// columns a workgroup covers, in threads: all of them, or 256 at a time
__host__ __device__ __forceinline__ int gate_cols(int heads, int V) { return heads / V < GATE_THREADS ? heads / V : GATE_THREADS; }

template <typename T, int V>
__global__ __launch_bounds__(GATE_THREADS) void k_gate_back(const GateBackParams g)
{
    __shared__ float s_sum[2 * GATE_THREADS * V];
    const int cols = gate_cols(g.heads, V), lanes = GATE_THREADS / cols;  // rows side by side
    const int cx = threadIdx.x % cols, ry = threadIdx.x / cols;
    const int col = (blockIdx.y * cols + cx) * V;
    const bool on = ry < lanes && col < g.heads;
    const int64_t per = (g.rows + gridDim.x - 1) / gridDim.x;
    const int64_t r0 = (int64_t)blockIdx.x * per, r1 = r0 + per < g.rows ? r0 + per : g.rows;
    float sa[V], ss[V], bias[V], scale[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sa[v] = ss[v] = 0.f;
        bias[v] = on ? g.dt_bias[col + v] : 0.f;
        scale[v] = on ? g.decay_scale[col + v] : 0.f;
    }
    typedef Pack<T, V> P;
    const bool rate = g.d_b != nullptr;
    for (int64_t r = r0 + ry; on && r < r1; r += lanes) {
        const size_t at = (size_t)r * g.heads + col;
        const P a = *reinterpret_cast<const P *>(static_cast<const T *>(g.a) + at);
        const P d = *reinterpret_cast<const P *>(static_cast<const T *>(g.d_decay) + at);
        P b, e, out;
        if (rate) {
            b = *reinterpret_cast<const P *>(static_cast<const T *>(g.b) + at);
            e = *reinterpret_cast<const P *>(static_cast<const T *>(g.d_beta) + at);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            // from the smaller side: nothing overflows or cancels
            const float x = to_f32(a.x[v]) + bias[v], dd = to_f32(d.x[v]);
            const float ex = exp_minus(fabsf(x)), u = __builtin_amdgcn_rcpf(1.f + ex);
            const float da = dd * scale[v] * (x > 0.f ? u : ex * u);
            out.x[v] = from_f32<T>(da);
            sa[v] += da;
            ss[v] += dd * ((x > 0.f ? x : 0.f) + log_one_plus(ex));
        }
        *reinterpret_cast<P *>(static_cast<T *>(g.d_a) + at) = out;
        if (rate) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // beta (1 - beta) likewise
                const float x = exp_minus(fabsf(to_f32(b.x[v]))), y = __builtin_amdgcn_rcpf(1.f + x);
                out.x[v] = from_f32<T>(to_f32(e.x[v]) * (x * y * y));
            }
            *reinterpret_cast<P *>(static_cast<T *>(g.d_b) + at) = out;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s_sum[threadIdx.x * V + v] = sa[v];
        s_sum[(GATE_THREADS + threadIdx.x) * V + v] = ss[v];
    }
    __syncthreads();
    // sums over the rows side by side: thread (which, column), and where these
    // are few, several threads of every nth row
    const int outs = 2 * cols * V, parts = outs < GATE_THREADS ? GATE_THREADS / outs : 1;
    for (int n0 = 0; n0 < outs; n0 += GATE_THREADS) {
        const int n = n0 + (int)threadIdx.x % (outs < GATE_THREADS ? outs : GATE_THREADS), part = parts > 1 ? (int)threadIdx.x / outs : 0;
        const int which = n / (cols * V), c = n % (cols * V), at = (int)blockIdx.y * cols * V + c;
        float sum = 0.f;
        if (n < outs && part < parts) {
#pragma unroll 4
            for (int r = part; r < lanes; r += parts) sum += s_sum[(which * GATE_THREADS + r * cols) * V + c];
        }
        if (parts > 1) {
            __syncthreads();  // every row has been read
            s_sum[threadIdx.x] = sum;
            __syncthreads();
            if ((int)threadIdx.x < outs)
                for (int q = 1; q < parts; ++q) sum += s_sum[q * outs + threadIdx.x];
        }
        if (n < outs && part == 0 && at < g.heads)
            (gridDim.x > 1 ? g.partial + ((size_t)blockIdx.x * 2 + which) * g.heads : which ? g.d_scale : g.d_dt_bias)[at] = sum;
    }
}

// Workgroup (head, which): the slices' sums.
__global__ __launch_bounds__(256) void k_gate_back_sums(const GateBackParams g, int slices)
{
    __shared__ float s[4];
    const int h = blockIdx.x, which = blockIdx.y;
    float sum = 0.f;
    for (int n = threadIdx.x; n < slices; n += 256) sum += g.partial[((size_t)n * 2 + which) * g.heads + h];
    sum = block_sum(sum, s);
    if (threadIdx.x == 0) (which ? g.d_scale : g.d_dt_bias)[h] = sum;
}

// Slices of 4096 elements, up to two workgroups per CU.  Up to 8192 elements
// of whole vectors are one slice, whose sums need no second launch.  One slice
// against several, on the device (a graph's replay): 8,192 elements 6.0 / 6.8 us in
// fp16 and 7.6 / 7.6 with the rate in bf16, 12,288 7.4 / 6.9, 16,384 8.8 / 6.9,
// 32,768 14 / 6.9.  (Calls one by one wait for the host, not for this: 13.5 us
// against 15.7 up to 32,768 elements.)  Slices of 2048, 4096 and 8192: 65,536
// elements 6.4, 6.9 and 8.2 us; 2 million with the rate 11.5, 11.4 and 11.2.
int gate_back_blocks(int64_t rows, int heads)
{
    const int64_t n = rows * heads <= 8192 && heads % 8 == 0 ? 1 : rows * heads / 4096;
    return n < 1 ? 1 : n > 512 ? 512 : (int)n;
}

template <typename T>
static void launch_gate_typed(const GateBackParams &g, int slices, hipStream_t s)
{
    const bool vec = g.heads % 8 == 0;
    const int V = vec ? 8 : 1, cols = gate_cols(g.heads, V);
    const dim3 grid((unsigned)slices, (unsigned)((g.heads / V + cols - 1) / cols));
    if (vec) hipLaunchKernelGGL((k_gate_back<T, 8>), grid, dim3(GATE_THREADS), 0, s, g);
    else hipLaunchKernelGGL((k_gate_back<T, 1>), grid, dim3(GATE_THREADS), 0, s, g);
}

hipError_t launch_gate_backward(const GateBackParams &g, hipStream_t s)
{
    const int slices = gate_back_blocks(g.rows, g.heads);
    if (g.dt == 1) launch_gate_typed<half_t>(g, slices, s);
    else if (g.dt == 2) launch_gate_typed<bf16_t>(g, slices, s);
    else launch_gate_typed<float>(g, slices, s);
    if (slices > 1) hipLaunchKernelGGL(k_gate_back_sums, dim3(g.heads, 2), dim3(256), 0, s, g, slices);
    return hipGetLastError();
}

}  // namespace gdr
