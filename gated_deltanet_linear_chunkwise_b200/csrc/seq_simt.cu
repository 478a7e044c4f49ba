// seq_simt.cu -- gradients of the gated delta rule over packed sequences, CUDA cores, fp32.
//
// Per sequence and head, chunks of 64 tokens, Sig = S^T entering a chunk, D the gradient of the
// one leaving it (d_k x d_v), G the prefix sums of log alpha inside the chunk, Gam_ij = e^{G_i - G_j}:
//
//   Y = V - e^G K Sig,  U = T (beta Y),  T = (I + tril(beta Gam o K K^T, -1))^-1
//   O = e^G Q Sig + P U,  P = tril(Gam o Q K^T),   Sig' = e^{G_L} Sig + (e^{G_L - G} K)^T U
//
// and backwards
//
//   dU = P^T dO + e^{G_L - G} K D,  dR = T^T dU,  D' = e^{G_L} D + (e^G Q)^T dO - (beta e^G K)^T dR
//   dV = beta dR,  dP = tril(Gam o dO U^T),  dA = -tril(Gam o dR U^T, -1)
//   dQ = e^G dO Sig^T + dP K
//   dK = -beta e^G dR Sig^T + e^{G_L - G} U D^T + dP^T Q + (beta dA) K + (beta dA)^T K
//   dbeta = rowsum(dR o Y) + rowsum(dA o K K^T)
//
// Every term holds one decay over a range of tokens, and d/dlog alpha_t is the sum of the terms
// whose range holds t: sums over ranges only, no differences of large sums.
//
// Four kernels: prep (T, P, decays; every chunk by itself), the chain forwards (Sig, Y, U; 16 columns of
// Sig a block, they are independent), the chain backwards (D, dR, dV, dS_in) and the gradients of
// a chunk.  This file serves fp32 inputs (and calls without tokens); its bound is the fp32 pipe.
#include <cuda_bf16.h>

#include "seq_gates.cuh"

namespace gdn {
namespace {

constexpr int C = kSeqChunk;
constexpr int LC = C + 4;  // row pitch of a 64 x 64 matrix in shared memory
constexpr int NC = 16;     // columns of Sig that a chain block holds

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// rows x cols values of a token-major tensor into dst [64][pitch], zeros behind the chunk's end
// (cols a multiple of 4, rows 16-byte aligned), four pieces a thread on their way together.
__device__ __forceinline__ void load_rows(float *dst, int pitch, const float *src, long long stride, int rows, int cols) {
    const int pieces = cols / 4;
    for (int i0 = threadIdx.x; i0 < C * pieces; i0 += 4 * blockDim.x) {
        float4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * blockDim.x, r = i / pieces, c = i % pieces * 4;
            x[k] = i < C * pieces && r < rows ? *reinterpret_cast<const float4 *>(src + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * blockDim.x, r = i / pieces, c = i % pieces * 4;
            if (i >= C * pieces) break;
            float *to = dst + r * pitch + c;  // odd pitches: rows spread over the banks
            to[0] = x[k].x;
            to[1] = x[k].y;
            to[2] = x[k].z;
            to[3] = x[k].w;
        }
    }
}

// acc[4][4] += sum_k a(i, k) b(k, j) over this thread's rows i0 .. i0+3 and columns j0 .. j0+3
template <typename FA, typename FB>
__device__ __forceinline__ void mm44(float (&acc)[4][4], int K, FA a, FB b) {
    for (int k = 0; k < K; ++k) {
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = a(i, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = b(k, j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
}

__global__ void __launch_bounds__(256) k_prep(const __grid_constant__ SeqProblem p, const __grid_constant__ SeqWork w) {
    extern __shared__ float sm[];
    const long long c = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk), tid = threadIdx.x, pk = p.dk + 1;
    const SeqChunk ch = seq_chunk(p, c);
    if (ch.rows == 0) return;
    float *sK = sm, *sQ = sK + C * pk, *sA = sQ + C * pk, *sT = sA + C * LC, *sBeta = sT + C * LC;
    double *sG = reinterpret_cast<double *>(sBeta + C);
    load_rows(sK, pk, (const float *)p.k + ch.first * p.k_stride + (size_t)hk * p.dk, p.k_stride, ch.rows, p.dk);
    load_rows(sQ, pk, (const float *)p.q + ch.first * p.q_stride + (size_t)hk * p.dk, p.q_stride, ch.rows, p.dk);
    if (tid < C) {
        const bool on = tid < ch.rows;
        const size_t g = (size_t)(ch.first + tid) * p.H + h;
        sG[tid] = on ? seq_log_gate(p.alpha[g], kSeqBwdLogFloor) : 0.0;
        sBeta[tid] = on ? p.beta[g] : 0.f;
    }
    __syncthreads();
    if (tid == 0)
        for (int i = 1; i < C; ++i) sG[i] += sG[i - 1];
    __syncthreads();
    const size_t idx = (size_t)c * p.H + h;
    if (tid < C) {
        w.eg[idx * C + tid] = expf((float)sG[tid]);
        w.el[idx * C + tid] = expf((float)(sG[C - 1] - sG[tid]));
    }
    const int i0 = tid / 16 * 4, j0 = tid % 16 * 4;
    float qk[4][4] = {}, kk[4][4] = {};
    mm44(qk, p.dk, [&](int i, int k) { return sQ[(i0 + i) * pk + k]; }, [&](int k, int j) { return sK[(j0 + j) * pk + k]; });
    mm44(kk, p.dk, [&](int i, int k) { return sK[(i0 + i) * pk + k]; }, [&](int k, int j) { return sK[(j0 + j) * pk + k]; });
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int i = i0 + a, j = j0 + b;
            const float gam = j <= i ? expf((float)(sG[i] - sG[j])) : 0.f;
            w.P[idx * C * C + i * C + j] = gam * qk[a][b];
            sA[i * LC + j] = j < i ? sBeta[i] * gam * kk[a][b] : 0.f;
        }
    __syncthreads();
    // column tid of T by forward substitution
    if (tid < C) {
        for (int i = 0; i < C; ++i) sT[i * LC + tid] = 0.f;
        for (int i = 0; i < C; ++i) {
            float x[4] = {i == tid ? 1.f : 0.f, 0.f, 0.f, 0.f};  // rows above the diagonal are zeros: whole fours
            for (int j = tid & ~3; j < i; j += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&sA[i * LC + j]);  // zeros from column i on
                x[0] = fmaf(-a.x, sT[j * LC + tid], x[0]);
                x[1] = fmaf(-a.y, sT[(j + 1) * LC + tid], x[1]);
                x[2] = fmaf(-a.z, sT[(j + 2) * LC + tid], x[2]);
                x[3] = fmaf(-a.w, sT[(j + 3) * LC + tid], x[3]);
            }
            sT[i * LC + tid] = i < tid ? 0.f : (x[0] + x[1]) + (x[2] + x[3]);
        }
    }
    __syncthreads();
    for (int i = tid; i < C * C; i += blockDim.x) w.T[idx * C * C + i] = sT[i / C * LC + i % C];
}

// The chains.  A block holds NC columns of Sig (d_v); 256 threads.
struct ChainTile {
    float *K, *Q, *V, *T, *P, *S, *X, *R, *eg, *el, *beta;
};
__device__ __forceinline__ ChainTile chain_tile(float *sm, int dk) {
    ChainTile t;
    const int pk = dk + 1;
    t.K = sm;
    t.Q = t.K + C * pk;
    t.T = t.Q + C * pk;
    t.P = t.T + C * LC;
    t.S = t.P + C * LC;      // [NC][pk]
    t.V = t.S + NC * pk;     // [C][NC]
    t.X = t.V + C * NC;
    t.R = t.X + C * NC;
    t.eg = t.R + C * NC;
    t.el = t.eg + C;
    t.beta = t.el + C;
    return t;
}
size_t chain_bytes(int dk) { return sizeof(float) * (size_t)(2 * C * (dk + 1) + 2 * C * LC + NC * (dk + 1) + 3 * C * NC + 3 * C); }

__device__ __forceinline__ void chain_load(const SeqProblem &p, const SeqWork &w, const ChainTile &t, long long row, int rows,
                                           size_t idx, int h, int c0, bool with_qp, const float *v, long long v_stride) {
    const int hk = h / (p.H / p.Hk), pk = p.dk + 1;
    load_rows(t.K, pk, (const float *)p.k + row * p.k_stride + (size_t)hk * p.dk, p.k_stride, rows, p.dk);
    if (with_qp) load_rows(t.Q, pk, (const float *)p.q + row * p.q_stride + (size_t)hk * p.dk, p.q_stride, rows, p.dk);
    load_rows(t.V, NC, v + row * v_stride + (size_t)h * p.dv + c0, v_stride, rows, NC);
    load_rows(t.T, LC, w.T + idx * C * C, C, C, C);
    if (with_qp) load_rows(t.P, LC, w.P + idx * C * C, C, C, C);
    if (threadIdx.x < C) {
        t.eg[threadIdx.x] = w.eg[idx * C + threadIdx.x];
        t.el[threadIdx.x] = w.el[idx * C + threadIdx.x];
        t.beta[threadIdx.x] = threadIdx.x < rows ? p.beta[(size_t)(row + threadIdx.x) * p.H + h] : 0.f;
    }
}

__global__ void __launch_bounds__(256) k_chain_fwd(const __grid_constant__ SeqProblem p, const __grid_constant__ SeqWork w) {
    extern __shared__ float sm[];
    const int groups = p.dv / NC, s = blockIdx.x / (p.H * groups), h = blockIdx.x / groups % p.H, c0 = blockIdx.x % groups * NC;
    const int tid = threadIdx.x, pk = p.dk + 1, dv = p.dv;
    const SeqRange r = seq_rows_in_order(p, s);
    seq_report(p, r.bad, h == 0 && c0 == 0 && tid == 0);
    if (r.slot < 0) return;
    const ChainTile t = chain_tile(sm, p.dk);
    for (int i = tid; i < NC * p.dk; i += blockDim.x)
        t.S[i / p.dk * pk + i % p.dk] = p.S_in ? p.S_in[(((size_t)s * p.H + h) * dv + c0) * p.dk + i] : 0.f;
    const long long base = seq_chunk_base(p, s, r.first);
    const int i = tid / 4, j0 = tid % 4 * 4;  // a row of the chunk, four columns
    for (long long c = 0; c < seq_chunks_of(r.len); ++c) {
        const size_t idx = (size_t)(base + c) * p.H + h;
        const long long row = r.first + c * C;
        __syncthreads();
        chain_load(p, w, t, row, (int)min((long long)C, r.len - c * C), idx, h, c0, false, (const float *)p.v, p.v_stride);
        __syncthreads();
        for (int e = tid; e < NC * p.dk; e += blockDim.x) w.Sig[(idx * dv + c0) * p.dk + e] = t.S[e / p.dk * pk + e % p.dk];
        float x[4] = {};
        for (int k = 0; k < p.dk; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fmaf(t.K[i * pk + k], t.S[(j0 + j) * pk + k], x[j]);
        for (int j = 0; j < 4; ++j) {
            const float y = t.V[i * NC + j0 + j] - t.eg[i] * x[j];
            w.Y[(idx * C + i) * dv + c0 + j0 + j] = y;
            t.R[i * NC + j0 + j] = t.beta[i] * y;
        }
        __syncthreads();
        float u[4] = {};
        for (int m = 0; m <= i; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = fmaf(t.T[i * LC + m], t.R[m * NC + j0 + j], u[j]);
        for (int j = 0; j < 4; ++j) {
            w.U[(idx * C + i) * dv + c0 + j0 + j] = u[j];
            t.X[i * NC + j0 + j] = t.el[i] * u[j];
        }
        __syncthreads();
        for (int e = tid; e < NC * p.dk; e += blockDim.x) {
            const int n = e / p.dk, k = e % p.dk;
            float a = t.eg[C - 1] * t.S[n * pk + k];
            for (int m = 0; m < C; ++m) a = fmaf(t.X[m * NC + n], t.K[m * pk + k], a);
            t.S[n * pk + k] = a;
        }
    }
}

__global__ void __launch_bounds__(256) k_chain_bwd(const __grid_constant__ SeqProblem p, const __grid_constant__ SeqWork w) {
    extern __shared__ float sm[];
    const int groups = p.dv / NC, s = blockIdx.x / (p.H * groups), h = blockIdx.x / groups % p.H, c0 = blockIdx.x % groups * NC;
    const int tid = threadIdx.x, pk = p.dk + 1, dv = p.dv;
    const SeqRange r = seq_rows_in_order(p, s);
    const ChainTile t = chain_tile(sm, p.dk);
    const size_t soff = (((size_t)s * p.H + h) * dv + c0) * p.dk;
    if (r.slot < 0) {
        for (int i = tid; p.dS_in && i < NC * p.dk; i += blockDim.x) p.dS_in[soff + i] = 0.f;
        return;
    }
    for (int i = tid; i < NC * p.dk; i += blockDim.x) t.S[i / p.dk * pk + i % p.dk] = p.dS_out ? p.dS_out[soff + i] : 0.f;
    const long long base = seq_chunk_base(p, s, r.first);
    const int i = tid / 4, j0 = tid % 4 * 4;
    for (long long c = seq_chunks_of(r.len) - 1; c >= 0; --c) {
        const size_t idx = (size_t)(base + c) * p.H + h;
        const long long row = r.first + c * C;
        const int rows = (int)min((long long)C, r.len - c * C);
        __syncthreads();
        chain_load(p, w, t, row, rows, idx, h, c0, true, (const float *)p.d_o, (long long)p.H * dv);
        __syncthreads();
        for (int e = tid; e < NC * p.dk; e += blockDim.x) w.D[(idx * dv + c0) * p.dk + e] = t.S[e / p.dk * pk + e % p.dk];
        float x[4] = {};
        for (int k = 0; k < p.dk; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fmaf(t.K[i * pk + k], t.S[(j0 + j) * pk + k], x[j]);
        for (int j = 0; j < 4; ++j) x[j] *= t.el[i];
        for (int m = i; m < C; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fmaf(t.P[m * LC + i], t.V[m * NC + j0 + j], x[j]);
        for (int j = 0; j < 4; ++j) t.X[i * NC + j0 + j] = x[j];  // dU
        __syncthreads();
        float y[4] = {};
        for (int m = i; m < C; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fmaf(t.T[m * LC + i], t.X[m * NC + j0 + j], y[j]);
        for (int j = 0; j < 4; ++j) {
            w.dR[(idx * C + i) * dv + c0 + j0 + j] = y[j];
            if (i < rows) ((float *)p.dv_out)[((row + i) * p.H + h) * dv + c0 + j0 + j] = t.beta[i] * y[j];
            t.R[i * NC + j0 + j] = t.beta[i] * t.eg[i] * y[j];
            t.V[i * NC + j0 + j] *= t.eg[i];  // this thread's own entries; others read them only behind the barrier
        }
        __syncthreads();
        for (int e = tid; e < NC * p.dk; e += blockDim.x) {
            const int n = e / p.dk, k = e % p.dk;
            float a = t.eg[C - 1] * t.S[n * pk + k];
            for (int m = 0; m < C; ++m)
                a += t.V[m * NC + n] * t.Q[m * pk + k] - t.R[m * NC + n] * t.K[m * pk + k];
            t.S[n * pk + k] = a;
        }
    }
    __syncthreads();
    for (int i = tid; p.dS_in && i < NC * p.dk; i += blockDim.x) p.dS_in[soff + i] = t.S[i / p.dk * pk + i % p.dk];
}

// Sum over the 16 lanes that share a thread tile's rows.
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

struct GradTile {
    float *K, *Q, *dO, *U, *dR, *P, *A, *eg, *el, *beta, *into, *past, *red;
};
__device__ __forceinline__ GradTile grad_tile(float *sm, int dk, int dv) {
    GradTile t;
    t.K = sm;
    t.Q = t.K + C * (dk + 1);
    t.dO = t.Q + C * (dk + 1);
    t.U = t.dO + C * (dv + 1);
    t.dR = t.U + C * (dv + 1);
    t.P = t.dR + C * (dv + 1);
    t.A = t.P + C * LC;
    t.eg = t.A + C * LC;
    t.el = t.eg + C;
    t.beta = t.el + C;
    t.into = t.beta + C;
    t.past = t.into + C;
    t.red = t.past + C;
    return t;
}
size_t grad_bytes(int dk, int dv) { return sizeof(float) * (size_t)(2 * C * (dk + 1) + 3 * C * (dv + 1) + 2 * C * LC + 5 * C + 8) + sizeof(double) * C; }

__global__ void __launch_bounds__(256) k_grads(const __grid_constant__ SeqProblem p, const __grid_constant__ SeqWork w) {
    extern __shared__ float sm[];
    const long long c = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk), tid = threadIdx.x, dk = p.dk, dv = p.dv, pk = dk + 1, pv = dv + 1;
    const SeqChunk ch = seq_chunk(p, c);
    if (ch.rows == 0) return;
    const size_t idx = (size_t)c * p.H + h;
    const GradTile t = grad_tile(sm, dk, dv);
    double *sG = reinterpret_cast<double *>(t.red + 8);
    load_rows(t.K, pk, (const float *)p.k + ch.first * p.k_stride + (size_t)hk * dk, p.k_stride, ch.rows, dk);
    load_rows(t.Q, pk, (const float *)p.q + ch.first * p.q_stride + (size_t)hk * dk, p.q_stride, ch.rows, dk);
    load_rows(t.dO, pv, (const float *)p.d_o + (ch.first * p.H + h) * dv, (long long)p.H * dv, ch.rows, dv);
    load_rows(t.U, pv, w.U + idx * C * dv, (long long)dv, C, dv);
    load_rows(t.dR, pv, w.dR + idx * C * dv, (long long)dv, C, dv);
    if (tid < C) {
        const bool on = tid < ch.rows;
        const size_t g = (size_t)(ch.first + tid) * p.H + h;
        t.eg[tid] = w.eg[idx * C + tid];
        t.el[tid] = w.el[idx * C + tid];
        t.beta[tid] = on ? p.beta[g] : 0.f;
        sG[tid] = on ? seq_log_gate(p.alpha[g], kSeqBwdLogFloor) : 0.0;
    }
    __syncthreads();
    if (tid == 0)
        for (int i = 1; i < C; ++i) sG[i] += sG[i - 1];
    __syncthreads();
    const int i0 = tid / 16 * 4, cg = tid % 16, j0 = cg * 4;
    float M[4][4] = {};
    {
        float qk[4][4] = {}, kk[4][4] = {}, dP[4][4] = {}, dA[4][4] = {};
        mm44(qk, dk, [&](int i, int k) { return t.Q[(i0 + i) * pk + k]; }, [&](int k, int j) { return t.K[(j0 + j) * pk + k]; });
        mm44(kk, dk, [&](int i, int k) { return t.K[(i0 + i) * pk + k]; }, [&](int k, int j) { return t.K[(j0 + j) * pk + k]; });
        mm44(dP, dv, [&](int i, int k) { return t.dO[(i0 + i) * pv + k]; }, [&](int k, int j) { return t.U[(j0 + j) * pv + k]; });
        mm44(dA, dv, [&](int i, int k) { return t.dR[(i0 + i) * pv + k]; }, [&](int k, int j) { return t.U[(j0 + j) * pv + k]; });
        for (int a = 0; a < 4; ++a)
            for (int b = 0; b < 4; ++b) {
                const int i = i0 + a, j = j0 + b;
                const float gam = j <= i ? expf((float)(sG[i] - sG[j])) : 0.f;
                const float x = gam * dP[a][b], y = j < i ? -gam * dA[a][b] : 0.f;
                t.P[i * LC + j] = x;
                t.A[i * LC + j] = y;
                M[a][b] = x * qk[a][b] + t.beta[i] * y * kk[a][b];
            }
    }
    __syncthreads();
    const float *Sig = w.Sig + idx * dv * dk, *D = w.D + idx * dv * dk;
    float into[4] = {}, past[4] = {}, db[4] = {}, all = 0.f;
    for (int n0 = 0; n0 < dk; n0 += 64) {
        const int col = n0 + j0;
        const bool on = col < dk;  // dk is a multiple of 16: a thread's four columns are all in or all out
        float dq[4][4] = {}, kin[4][4] = {}, kout[4][4] = {}, kA[4][4] = {}, kT[4][4] = {};
        if (on) {
            mm44(dq, dv, [&](int i, int k) { return t.dO[(i0 + i) * pv + k]; }, [&](int k, int j) { return Sig[(size_t)k * dk + col + j]; });
            mm44(kin, dv, [&](int i, int k) { return t.dR[(i0 + i) * pv + k]; }, [&](int k, int j) { return Sig[(size_t)k * dk + col + j]; });
            mm44(kout, dv, [&](int i, int k) { return t.U[(i0 + i) * pv + k]; }, [&](int k, int j) { return D[(size_t)k * dk + col + j]; });
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b) {
                    const int i = i0 + a;
                    const float qv = t.Q[i * pk + col + b], kv = t.K[i * pk + col + b];
                    dq[a][b] *= t.eg[i];
                    kin[a][b] *= -t.beta[i] * t.eg[i];
                    kout[a][b] *= t.el[i];
                    into[a] += qv * dq[a][b] + kv * kin[a][b];
                    past[a] += kv * kout[a][b];
                }
            mm44(dq, C, [&](int i, int k) { return t.P[(i0 + i) * LC + k]; }, [&](int k, int j) { return t.K[k * pk + col + j]; });
            mm44(kA, C, [&](int i, int k) { return t.A[(i0 + i) * LC + k]; }, [&](int k, int j) { return t.K[k * pk + col + j]; });
            mm44(kT, C, [&](int i, int k) { return t.P[k * LC + i0 + i]; }, [&](int k, int j) { return t.Q[k * pk + col + j]; });
            mm44(kT, C, [&](int i, int k) { return t.A[k * LC + i0 + i] * t.beta[k]; }, [&](int k, int j) { return t.K[k * pk + col + j]; });
            for (int a = 0; a < 4; ++a) {
                const int i = i0 + a;
                const size_t g = (size_t)(ch.first + i);
                for (int b = 0; b < 4; ++b) {
                    db[a] += t.K[i * pk + col + b] * kA[a][b];
                    const float dkv = kin[a][b] + kout[a][b] + t.beta[i] * kA[a][b] + kT[a][b];
                    if (i >= ch.rows) continue;
                    if (w.dqh) {
                        w.dqh[(g * p.H + h) * dk + col + b] = dq[a][b];
                        w.dkh[(g * p.H + h) * dk + col + b] = dkv;
                    } else {
                        ((float *)p.dq)[(g * p.H + h) * dk + col + b] = dq[a][b];
                        ((float *)p.dk_out)[(g * p.H + h) * dk + col + b] = dkv;
                    }
                }
            }
        }
    }
    for (int a = 0; a < 4; ++a)
        for (int n = cg; n < dv; n += 16)
            db[a] += t.dR[(i0 + a) * pv + n] * w.Y[(idx * C + i0 + a) * dv + n];
    for (int e = tid; e < dk * dv; e += blockDim.x) all += Sig[e] * D[e];
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (tid % 32 == 0) t.red[tid / 32] = all;
    for (int a = 0; a < 4; ++a) {
        const float x = sum16(into[a]), y = sum16(past[a]), z = sum16(db[a]);
        if (cg == 0) {
            t.into[i0 + a] = x;
            t.past[i0 + a] = y;
            if (i0 + a < ch.rows) p.dbeta[(size_t)(ch.first + i0 + a) * p.H + h] = z;
        }
    }
    __syncthreads();  // dP has been read: M takes its place
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) t.P[(i0 + a) * LC + j0 + b] = M[a][b];
    __syncthreads();
    if (tid < C)  // column sums over the rows from each row on
        for (int i = C - 2; i >= 0; --i) t.P[i * LC + tid] += t.P[(i + 1) * LC + tid];
    __syncthreads();
    if (tid < ch.rows) {
        float g = 0.f;
        for (int i = 0; i < 8; ++i) g += t.red[i];
        g *= t.eg[C - 1];
        for (int j = 0; j < tid; ++j) g += t.P[tid * LC + j] + t.past[j];
        for (int i = tid; i < C; ++i) g += t.into[i];
        const size_t at = (size_t)(ch.first + tid) * p.H + h;
        p.dalpha[at] = g / fmaxf(p.alpha[at], expf(kSeqBwdLogFloor));
    }
}

template <typename T>
__global__ void k_share(const __grid_constant__ SeqProblem p, const float *dqh, const float *dkh) {
    const long long n = p.n_tokens * p.Hk * p.dk;
    const int per = p.H / p.Hk;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const long long tok = i / (p.Hk * p.dk);
        const int hk = (int)(i / p.dk % p.Hk), e = (int)(i % p.dk);
        float a = 0.f, b = 0.f;
        for (int g = 0; g < per; ++g) {
            const long long at = (tok * p.H + hk * per + g) * p.dk + e;
            a += dqh[at];
            b += dkh[at];
        }
        put((T *)p.dq + i, a);
        put((T *)p.dk_out + i, b);
    }
}

// 64 rows a block; a row is covered where a range that is in order holds it.
__global__ void __launch_bounds__(256) k_zero_rows(const __grid_constant__ SeqProblem p, float *dqh, float *dkh) {
    __shared__ unsigned char covered[64];
    const long long r0 = blockIdx.x * 64ll;
    if (threadIdx.x < 64) covered[threadIdx.x] = 0;
    seq_each_in_order<256>(p, p.n_seqs, [&](int, const SeqRange &r, bool late) {
        if (late) return;
        const long long a = max(r.first, r0), b = min(r.first + r.len, r0 + 64);
        for (long long i = a; i < b; ++i) covered[i - r0] = 1;
    });
    __syncthreads();
    const int es = p.dtype == GDN_DTYPE_BF16 ? 2 : 4;
    auto zero = [&](void *base, long long row, long long bytes) {  // 4-byte words: bytes is a multiple of 4
        if (!base) return;
        unsigned *w = reinterpret_cast<unsigned *>((char *)base + row * bytes);
        for (long long i = threadIdx.x; i < bytes / 4; i += blockDim.x) w[i] = 0;
    };
    for (int i = 0; i < 64 && r0 + i < p.n_tokens; ++i) {
        if (covered[i]) continue;
        const long long row = r0 + i;
        zero(p.dq, row, (long long)p.Hk * p.dk * es);
        zero(p.dk_out, row, (long long)p.Hk * p.dk * es);
        zero(p.dv_out, row, (long long)p.H * p.dv * es);
        zero(p.dalpha, row, (long long)p.H * 4);
        zero(p.dbeta, row, (long long)p.H * 4);
        zero(dqh, row, (long long)p.H * p.dk * 4);
        zero(dkh, row, (long long)p.H * p.dk * 4);
    }
}

cudaError_t run(const SeqProblem &p, const SeqWork &w, cudaStream_t s) {
    const unsigned chunks = (unsigned)(seq_max_chunks(p) * p.H), chains = (unsigned)(p.n_seqs * p.H * (p.dv / NC));
    const size_t prep = sizeof(float) * (size_t)(2 * C * (p.dk + 1) + 2 * C * LC + C) + sizeof(double) * C;
    const size_t chain = chain_bytes(p.dk), grad = grad_bytes(p.dk, p.dv);
    cudaError_t e;
    if ((e = cudaFuncSetAttribute(k_prep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep))) return e;
    if ((e = cudaFuncSetAttribute(k_chain_fwd, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)chain))) return e;
    if ((e = cudaFuncSetAttribute(k_chain_bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)chain))) return e;
    if ((e = cudaFuncSetAttribute(k_grads, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)grad))) return e;
    if (chunks) k_prep<<<chunks, 256, prep, s>>>(p, w);
    k_chain_fwd<<<chains, 256, chain, s>>>(p, w);
    k_chain_bwd<<<chains, 256, chain, s>>>(p, w);
    if (chunks) k_grads<<<chunks, 256, grad, s>>>(p, w);
    return cudaGetLastError();
}

}  // namespace

size_t seq_bwd_workspace(const SeqProblem &p, void *base, SeqWork *w) {
    const size_t n = (size_t)seq_max_chunks(p) * p.H, rows = (size_t)p.n_tokens * p.H;
    size_t at = 0;
    auto take = [&](size_t floats) {
        float *x = reinterpret_cast<float *>((char *)base + at);
        at += align256(floats * sizeof(float));
        return x;
    };
    SeqWork v;
    v.T = take(n * C * C);
    v.P = take(n * C * C);
    v.eg = take(n * C);
    v.el = take(n * C);
    v.Sig = take(n * p.dk * p.dv);
    v.D = take(n * p.dk * p.dv);
    v.U = take(n * C * p.dv);
    v.Y = take(n * C * p.dv);
    v.dR = take(n * C * p.dv);
    v.dqh = p.H > p.Hk ? take(rows * p.dk) : nullptr;
    v.dkh = p.H > p.Hk ? take(rows * p.dk) : nullptr;
    if (w) *w = v;
    return at;
}

cudaError_t launch_seq_zero_rows(const SeqProblem &p, float *dqh, float *dkh, cudaStream_t s) {
    if (!p.cu || p.n_tokens == 0) return cudaSuccess;
    k_zero_rows<<<(unsigned)((p.n_tokens + 63) / 64), 256, 0, s>>>(p, dqh, dkh);
    return cudaGetLastError();
}

cudaError_t launch_seq_share(const SeqProblem &p, const float *dqh, const float *dkh, cudaStream_t s) {
    if (!dqh || p.n_tokens == 0) return cudaSuccess;
    const long long n = p.n_tokens * p.Hk * p.dk;
    const unsigned blocks = (unsigned)min((n + 255) / 256, 148ll * 16);
    if (p.dtype == GDN_DTYPE_BF16) k_share<__nv_bfloat16><<<blocks, 256, 0, s>>>(p, dqh, dkh);
    else k_share<float><<<blocks, 256, 0, s>>>(p, dqh, dkh);
    return cudaGetLastError();
}

cudaError_t launch_seq_bwd_simt(const SeqProblem &p, void *ws, cudaStream_t s) {
    SeqWork w;
    seq_bwd_workspace(p, ws, &w);
    cudaError_t e = launch_seq_zero_rows(p, w.dqh, w.dkh, s);
    if (e == cudaSuccess && p.n_seqs) e = run(p, w, s);
    return e == cudaSuccess ? launch_seq_share(p, w.dqh, w.dkh, s) : e;
}

}  // namespace gdn
