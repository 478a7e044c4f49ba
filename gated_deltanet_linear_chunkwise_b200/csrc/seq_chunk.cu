// seq_chunk.cu -- the chunked gated delta rule over packed sequences on the tensor cores (bf16 q, k, v).
//
// Notation and formulas as in seq_simt.cu; chunks of 64 tokens.  Three kernels:
//
// k_prep       every (chunk, head) by itself: T, P and the decays.
// k_chunk_fwd  a block walks the chunks of one sequence and head with 16 columns of the state
//              (d_v columns are independent), S = Sig^T's 16 rows in registers:
//                X^T = S [K;Q]^T,  Y = V - e^G X_K,  U^T = (beta Y)^T T^T,
//                O^T = e^G X_Q^T + U^T P^T,  S <- e^{G_L} S + (e^{G_L-G} U)^T K
// k_chunk_bwd  the same walk backwards with 16 rows of D^T:
//                dU^T = e^{G_L-G} D^T K^T + dO^T P,  dR^T = dU^T T,
//                D^T <- e^{G_L} D^T + (e^G dO)^T Q - (beta e^G dR)^T K
//
// The state leaves in fp32 and has to be as exact as a fp32 recurrence, so its products are split ones
// (seq_mma.cuh); what only reaches a bf16 output (Q S, P U) takes two terms.  Every operand on the state's
// side has 16 rows and every other one is read as it lies (K, Q by ldmatrix; T and P are
// stored by k_prep in the order in which a lane needs them, and go to registers directly).
//
// Why warp-level products and not tcgen05: with 16 rows of the state a block, one sequence
// of 20 heads fills 140 of 148 SMs and its 64-token step is as short as it gets.  A tcgen05 product has 128 rows of
// K and Q against N = 16 here and is bound by its A operand's shared memory reads (128 rows x 16 x 2 bytes at
// 128 B/clk: 32 clk an instruction, as long as the 16 warp products that it replaces), and pays a
// round trip through tensor memory for each of three dependent products of a step.
#include <cuda.h>
#include <cuda_bf16.h>

#include "gates.cuh"
#include "seq_internal.h"
#include "seq_mma.cuh"

namespace gdn {

bool seq_row_map(CUtensorMap *m, const void *x, long long rows, long long row_stride, int heads, int d, int cols);  // gdn_tc.cu

namespace {

using namespace mma;
using sm100::cp_async16;

constexpr int C = kSeqChunk;
constexpr int NV = 16;       // rows of S (columns of d_v) that a block holds
constexpr int PC = C + 8;    // pitch of a [16][64] plane: 9 x 16 bytes, odd, so ldmatrix rows spread over the banks

// T and P lie in the order of the B operand's fragments, a term behind the other: unit (t, b) is the n-tile of 8
// tokens from 8t against the 16 tokens from 16b, a lane's two words of it.  Below the diagonal b <= t / 2 (20
// units), above it (the transposes) b >= t / 2.  P reaches O only and has two terms; T and the transposes have three.
__host__ __device__ constexpr int low_unit(int t) { return (t / 2) * (t / 2 + 1) + (t & 1) * (t / 2 + 1); }
__host__ __device__ constexpr int up_unit(int t) { return 20 - low_unit(8 - t) ; }
constexpr int kUnits = 20;

struct ChunkWork {
    uint2 *T, *P, *Tt, *Pt;  // [chunk x H][terms][20][32]; P or the transposes may be null
    float *gates;            // [chunk x H][3][64]: e^G, e^{G_L - G}, beta
    double *G;               // [chunk x H][64], or null
    float *Sig, *D;          // [chunk x H][dv][dk]
    float *U, *X, *dR;       // [chunk x H][dv][64]: X = e^G K Sig
    float *past, *into, *db; // [chunk x H][dv / 16][64]: a slice's part of the gates' gradients
    float *dqh, *dkh;        // as in SeqWork
    int *err;                // a bounded wait that gave up (k_prep clears it)
};

template <int NF>
__global__ void __launch_bounds__(128) k_prep(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                              const float floor_log) {
    constexpr int DK = 16 * NF, kTile = (DK + 63) / 64 * C * 64;
    // K and Q, and in their place, once they have been multiplied, A and its inverse
    constexpr int kRows = 2 * kTile * (int)sizeof(bf16), kMat = C * (C + 1) * (int)sizeof(float);
    __shared__ __align__(16) unsigned char room[kRows > kMat ? kRows : kMat];
    bf16 *const sK = reinterpret_cast<bf16 *>(room), *const sQ = sK + kTile;
    float(*const sA)[C + 1] = reinterpret_cast<float(*)[C + 1]>(room);
    __shared__ double sG[C];
    __shared__ float sB[C];
    const long long c = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk), tid = threadIdx.x, lane = tid & 31, warp = warp_number();
    if (blockIdx.x == 0 && tid == 0) *w.err = 0;
    const SeqChunk ch = seq_chunk(p, c);
    if (ch.rows == 0) return;
    for (int i = tid; i < C * (DK / 8); i += 128) {
        const int r = i / (DK / 8), col = i % (DK / 8) * 8, on = r < ch.rows ? 16 : 0;
        const long long row = ch.first + (on ? r : 0);
        cp_async16((char *)sK + sw_byte(C, r, col), (const bf16 *)p.k + row * p.k_stride + (size_t)hk * DK + col, on);
        cp_async16((char *)sQ + sw_byte(C, r, col), (const bf16 *)p.q + row * p.q_stride + (size_t)hk * DK + col, on);
    }
    sm100::cp_async_commit();
    const size_t idx = (size_t)c * p.H + h;
    if (warp == 0) {  // two tokens a lane: prefix sums of log alpha in 64 bits (decays are differences of them)
        double g[2];
        float b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const size_t at = (size_t)(ch.first + i) * p.H + h;
            g[e] = i < ch.rows ? fmax(log_gate<double>(p.alpha[at]), (double)floor_log) : 0.0;
            b[e] = i < ch.rows ? p.beta[at] : 0.f;
        }
        double run = g[0] + g[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += y;
        }
        const double total = __shfl_sync(0xffffffffu, run, 31);
        const double G[2] = {run - g[1], run};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            sG[i] = G[e];
            sB[i] = b[e];
            w.gates[idx * 3 * C + i] = expf((float)G[e]);
            w.gates[idx * 3 * C + C + i] = expf((float)(total - G[e]));
            w.gates[idx * 3 * C + 2 * C + i] = b[e];
            if (w.G) w.G[idx * C + i] = G[e];
        }
    }
    sm100::cp_async_wait_all();
    __syncthreads();
    // warp: rows 16 warp .. + 15; columns up to the diagonal
    float kk[8][4] = {}, qk[8][4] = {};
    const uint32_t aK = sm100::smem_u32(sK), aQ = sm100::smem_u32(sQ);
#pragma unroll
    for (int ks = 0; ks < NF; ++ks) {
        uint32_t a[4], q[4];
        const uint32_t at = sw_byte(C, 16 * warp + (lane & 15), 16 * ks + (lane >> 4) * 8);
        ldsm4(a, aK + at);
        ldsm4(q, aQ + at);
#pragma unroll
        for (int t = 0; t < 8; t += 2) {
            if (t > 2 * warp) continue;
            uint32_t b[4];
            ldsm4(b, aK + b_lane(8 * t, 8 * t + 8, ks & 3, lane) + (ks >> 2) * C * 128);
            mma::mma(kk[t], a, b[0], b[1]);
            mma::mma(kk[t + 1], a, b[2], b[3]);
            mma::mma(qk[t], q, b[0], b[1]);
            mma::mma(qk[t + 1], q, b[2], b[3]);
        }
    }
    // the decays; A to shared memory; P's terms to memory (Pt's pairs lie along the rows: it goes through shared memory)
    __syncthreads();
    const int i0 = 16 * warp + lane / 4, j0 = 2 * (lane & 3);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + (e >> 1) * 8, j = 8 * t + j0 + (e & 1);
            if (t / 2 > warp) {
                sA[i][j] = 0.f;
                continue;
            }
            const float gam = j <= i ? expf((float)(sG[i] - sG[j])) : 0.f;
            qk[t][e] *= gam;
            sA[i][j] = j < i ? sB[i] * gam * kk[t][e] : 0.f;
        }
    }
    auto put_unit = [&](uint2 *dst, int terms, int unit, float x0, float x1, float y0, float y1) {
        uint32_t a[3], b[3];
        split(x0, x1, a);
        split(y0, y1, b);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < terms) dst[((idx * terms + e) * kUnits + unit) * 32 + lane] = make_uint2(a[e], b[e]);
    };
    if (w.P) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (b > warp) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half)
                put_unit(w.P, 2, low_unit(2 * warp + half) + b, qk[2 * b][2 * half], qk[2 * b][2 * half + 1], qk[2 * b + 1][2 * half],
                         qk[2 * b + 1][2 * half + 1]);
        }
    }
    __syncthreads();
    // (I + A)^-1 in place, by halves: the four 16 x 16 diagonal blocks first, a column a thread
    if (tid < C) {
        const int o = tid & ~15, col = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == col ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) s = fmaf(-sA[o + i][o + j], x[j], s);
            x[i] = s;  // rows above the diagonal come out as zeros
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) sA[o + i][o + col] = x[i];
    }
    // T21 = -T22 (A21 T11), blocks of 16 then of 32.  A thread has 4 x W columns-rows of the product
    __syncthreads();
    {
        const int pair = tid >> 6, e = tid & 63, o = 32 * pair, r = e / 16 * 4, col = e % 16;
        float m[4] = {};
        for (int k = 0; k < 16; ++k) {
            const float b = sA[o + k][o + col];
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = fmaf(sA[o + 16 + r + i][o + k], b, m[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) sA[o + 16 + r + i][o + col] = m[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = 0.f;
        for (int k = 0; k < 16; ++k) {
            const float b = sA[o + 16 + k][o + col];
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = fmaf(-sA[o + 16 + r + i][o + 16 + k], b, m[i]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) sA[o + 16 + r + i][o + col] = m[i];
    }
    __syncthreads();
    {
        const int r = tid / 16 * 4, col = tid % 16 * 2;
        float m[4][2] = {};
        for (int k = 0; k < 32; ++k) {
            const float b0 = sA[k][col], b1 = sA[k][col + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = sA[32 + r + i][k];
                m[i][0] = fmaf(a, b0, m[i][0]);
                m[i][1] = fmaf(a, b1, m[i][1]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) sA[32 + r + i][col] = m[i][0], sA[32 + r + i][col + 1] = m[i][1];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i][0] = m[i][1] = 0.f;
        for (int k = 0; k < 32; ++k) {
            const float b0 = sA[32 + k][col], b1 = sA[32 + k][col + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = -sA[32 + r + i][32 + k];
                m[i][0] = fmaf(a, b0, m[i][0]);
                m[i][1] = fmaf(a, b1, m[i][1]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) sA[32 + r + i][col] = m[i][0], sA[32 + r + i][col + 1] = m[i][1];
    }
    __syncthreads();
    const int n = lane / 4, k2 = 2 * (lane & 3);
    for (int t = 2 * warp; t < 2 * warp + 2; ++t) {
        for (int b = 0; b <= t / 2; ++b) {
            const float *x = &sA[8 * t + n][16 * b + k2];
            put_unit(w.T, 3, low_unit(t) + b, x[0], x[1], x[8], x[9]);
        }
        if (w.Tt)
            for (int b = t / 2; b < 4; ++b) {
                const int i = 16 * b + k2, j = 8 * t + n;
                put_unit(w.Tt, 3, up_unit(t) + b - t / 2, sA[i][j], sA[i + 1][j], sA[i + 8][j], sA[i + 9][j]);
            }
    }
    if (w.Pt) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t / 2 > warp) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) sA[i0 + (e >> 1) * 8][8 * t + j0 + (e & 1)] = qk[t][e];
        }
        __syncthreads();
        for (int t = 2 * warp; t < 2 * warp + 2; ++t)
            for (int b = t / 2; b < 4; ++b) {
                const int i = 16 * b + k2, j = 8 * t + n;
                put_unit(w.Pt, 3, up_unit(t) + b - t / 2, sA[i][j], sA[i + 1][j], sA[i + 8][j], sA[i + 9][j]);
            }
    }
}

// Shared memory of a chain block, 1024-byte aligned.  Two blocks fit an SM: only K, which is read from a step's
// first product to its last, has two buffers; the others are fetched again as soon as they have been read.
template <int NF, bool BWD> struct ChainSmem {
    static constexpr int PK = 16 * NF + 8, kTile = (16 * NF + 63) / 64 * C * 64;
    static constexpr int kTermsP = BWD ? 3 : 2;
    bf16 K[2][kTile], Q[kTile];  // as the tensor maps leave them
    uint2 T[3][kUnits][32], P[kTermsP][kUnits][32];
    bf16 V[C][NV];               // v, or do
    float gates[2][3][C];
    bf16 S[3][NV][PK];           // the state's terms
    bf16 U[3][NV][PC];           // e^{G_L-G} U; backwards e^G dO
    bf16 R[3][NV][PC];           // beta Y; backwards dU, then -beta e^G dR
    bf16 W[BWD ? 1 : 2][NV][PC]; // U for O
    uint64_t bar[5];             // K and gates (two), Q, V, T, P
};
enum { kBarK = 0, kBarV = 2, kBarT = 3, kBarP = 4 };
// Four warps carry the state from chunk to chunk, four more (where O is wanted) compute it beside them, one fetches.
constexpr int chain_threads(bool with_o) { return with_o ? 288 : 160; }

struct ChainMaps {
    CUtensorMap q, k, v;  // v: v, or do
};

// One thread's fetches (a handful of copies a chunk; as 16-byte copies by the threads they were 900 address lookups a
// chunk in ldmatrix's way, and loads of T and P to registers made every ldmatrix wait for them: 6400 clocks a step).
template <int NF, bool BWD> struct ChainFetch {
    ChainSmem<NF, BWD> &sm;
    const ChainMaps &maps;
    const ChunkWork &w;
    int hk, h, c0;
    __device__ __forceinline__ void tile(bf16 *dst, const CUtensorMap *map, uint64_t *bar, int row) const {
#pragma unroll
        for (int c = 0; c < 16 * NF; c += 64) sm100::tma_load_3d(dst + c * C, map, bar, c, hk, row);
    }
    static constexpr uint32_t kTileBytes = ChainSmem<NF, BWD>::kTile * 2;
    __device__ __forceinline__ void k(int b, int row, size_t idx) const {  // and the gates
        uint64_t *bar = &sm.bar[kBarK + b];
        sm100::mbar_arrive_expect_tx(bar, kTileBytes + 3 * C * 4);
        tile(sm.K[b], &maps.k, bar, row);
        sm100::bulk_copy_g2s(&sm.gates[b][0][0], w.gates + idx * 3 * C, 3 * C * 4, bar);
    }
    __device__ __forceinline__ void v(int row, bool with_q) const {  // 16 columns of v (or do); forwards with Q
        uint64_t *bar = &sm.bar[kBarV];
        sm100::mbar_arrive_expect_tx(bar, C * NV * 2 + (with_q ? kTileBytes : 0));
        sm100::tma_load_3d(&sm.V[0][0], &maps.v, bar, c0, h, row);
        if (with_q) tile(sm.Q, &maps.q, bar, row);
    }
    __device__ __forceinline__ void t(const uint2 *src) const {
        sm100::mbar_arrive_expect_tx(&sm.bar[kBarT], sizeof(sm.T));
        sm100::bulk_copy_g2s(sm.T, src, sizeof(sm.T), &sm.bar[kBarT]);
    }
    __device__ __forceinline__ void p(const uint2 *src, int row, bool with_q) const {  // backwards with Q, read last
        sm100::mbar_arrive_expect_tx(&sm.bar[kBarP], sizeof(sm.P) + (with_q ? kTileBytes : 0));
        sm100::bulk_copy_g2s(sm.P, src, sizeof(sm.P), &sm.bar[kBarP]);
        if (with_q) tile(sm.Q, &maps.q, &sm.bar[kBarP], row);
    }
};

// The rows behind a sequence's end belong to the next one: zeros (what they hold may not be finite).
__device__ __forceinline__ void zero_tail(bf16 *tile, int slabs, int pieces, int rows) {  // pieces of 16 bytes a row
    for (int i = threadIdx.x; i < (C - rows) * slabs * pieces; i += blockDim.x)
        reinterpret_cast<uint4 *>(tile)[i / ((C - rows) * pieces) * C * pieces + rows * pieces + i % ((C - rows) * pieces)] =
            make_uint4(0, 0, 0, 0);
    sm100::fence_proxy_async_smem();  // later copies land here
}

// Before the first fetch.
template <int NF, bool BWD> __device__ __forceinline__ void chain_init(ChainSmem<NF, BWD> &sm) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 5; ++i) sm100::mbar_init(&sm.bar[i], 1);
        sm100::fence_barrier_init();
    }
    __syncthreads();
}
// A block that gave up leaves no copy in flight: the last copy of every barrier is waited for once more.
template <int NF, bool BWD>
__device__ __forceinline__ void chain_leave(ChainSmem<NF, BWD> &sm, const SeqProblem &p, long long turn, int p_turn, int *err) {
    const uint32_t now = (uint32_t)turn & 1;
    sm100::mbar_wait(&sm.bar[kBarK + now], (uint32_t)(turn >> 1) & 1, err, sm100::kWaitLimitNs, true);
    sm100::mbar_wait(&sm.bar[kBarV], now, err, sm100::kWaitLimitNs, true);
    sm100::mbar_wait(&sm.bar[kBarT], now, err, sm100::kWaitLimitNs, true);
    if (p_turn >= 0) sm100::mbar_wait(&sm.bar[kBarP], p_turn & 1, err, sm100::kWaitLimitNs, true);  // P's last fetch, if any
    if (p.status && threadIdx.x == 0) atomicOr(p.status, GDN_SEQ_TIMEOUT);
}

// hi += a0 b0; lo += the other products of the terms of a with those of b that are above 2^-24, for the
// shorter tile (while it lasts) and the longer one; lo's sums are two, to keep products of one apart.
template <int AT, int BT>
__device__ __forceinline__ void mma_split(float (&hi)[2][4], float (&lo)[2][2][4], const uint32_t (&a)[AT][4], const uint2 (&b0)[BT],
                                          const uint2 (&b1)[BT], bool both) {
#pragma unroll
    for (int k = 0; k < (AT > BT ? AT : BT); ++k)
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int j = k - i;
            if (j < 0 || j >= BT) continue;
            if (both) mma::mma(k ? lo[0][k - 1 & 1] : hi[0], a[i], b0[j].x, b0[j].y);
            mma::mma(k ? lo[1][k - 1 & 1] : hi[1], a[i], b1[j].x, b1[j].y);
        }
}
// Unit (t, b) of T or P in shared memory; the blocks of a tile are counted from the diagonal's far end: block m
// of a lower triangle is 16-token block m, of an upper one block 3 - m.
// `src`: the address of unit (t, 0) of a lower triangle, (t, 3) of an upper one.
template <bool LOW, int TERMS> __device__ __forceinline__ void tri_frag(uint2 (&f)[TERMS], uint32_t src, int m) {
#pragma unroll
    for (int e = 0; e < TERMS; ++e) f[e] = lds2(src + e * kUnits * 256 + (LOW ? m : -m) * 256);
}
template <bool LOW> __device__ __forceinline__ uint32_t tri_addr(uint32_t src, int t, int lane) {
    return src + (LOW ? low_unit(t) : up_unit(t) + 3 - t / 2) * 256 + lane * 8;
}

// Sum over the lanes that hold the other rows of the same columns.
__device__ __forceinline__ float rows_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// The S (or D^T) rows of a block: warp w has the column pairs (16 columns) w and w + 4.
template <int NF> struct StateRows {
    float x[2][2][4];
    template <typename F> __device__ __forceinline__ void each(int warp, int lane, F &&f) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (warp + 4 * m >= NF) continue;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    f(lane / 4 + 8 * half, 16 * (warp + 4 * m) + 8 * t + 2 * (lane & 3), x[m][t][2 * half], x[m][t][2 * half + 1]);
        }
    }
};
template <int NF> __device__ __forceinline__ void put_state(uint32_t planes, StateRows<NF> &st, int warp, int lane) {
    constexpr int PK = 16 * NF + 8;
    const uint32_t at = planes + (lane / 4 * PK + 16 * warp + 2 * (lane & 3)) * 2;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (warp + 4 * m >= NF) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[3];
            split(st.x[m][i / 2][2 * (i & 1)], st.x[m][i / 2][2 * (i & 1) + 1], t);
#pragma unroll
            for (int e = 0; e < 3; ++e) sts(at + (e * NV + (i & 1) * 8) * PK * 2 + 128 * m + 16 * (i / 2), t[e]);
        }
    }
}
// The address of a lane's pairs of tokens (tile t, rows n and n + 8) in a [16][64] plane.
__device__ __forceinline__ uint32_t pair_addr(uint32_t plane, int t, int lane) { return plane + (lane / 4 * PC + 8 * t + 2 * (lane & 3)) * 2; }
template <int N> __device__ __forceinline__ void put_pair(uint32_t at, int half, float x, float y) {
    uint32_t t[N];
    split(x, y, t);
#pragma unroll
    for (int e = 0; e < N; ++e) sts(at + (e * NV + half * 8) * PC * 2, t[e]);
}

// st = decay st + sum over the planes pl: (plane's 3 terms [16][64 tokens]) x (rows [64 tokens][dk]).
// Here and below the next step's fragments are loaded before a step's products: left to the compiler, each
// step waited for its own loads (840 clocks for 48 products a warp).
template <int NF, int SETS>
__device__ __forceinline__ void update_state(StateRows<NF> &st, float decay, const uint32_t (&planes)[SETS], const uint32_t (&rows)[SETS],
                                             int warp, int lane) {
    float hi[2][2][4], lo[2][2][4];
    uint32_t a[2][3][4], b[2][2][4];
    const uint32_t al = a_lane(PC, lane), b0 = bt_lane(C, 16 * warp, lane), b1 = bt_lane(C, 16 * (warp + 4), lane);
    auto load = [&](int i) {
        const int s = i / 4, kb = i % 4;
#pragma unroll
        for (int e = 0; e < 3; ++e) ldsm4(a[i & 1][e], planes[s] + al + e * NV * PC * 2 + 32 * kb);
        if (warp < NF) ldsm4_t(b[i & 1][0], rows[s] + b0 + kb * 16 * 128);
        if (warp + 4 < NF) ldsm4_t(b[i & 1][1], rows[s] + b1 + kb * 16 * 128);
    };
    load(0);
#pragma unroll
    for (int i = 0; i < 4 * SETS; ++i) {
        if (i + 1 < 4 * SETS) load(i + 1);
        const auto &x = a[i & 1];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (warp + 4 * m >= NF) continue;
            const auto &y = b[i & 1][m];
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(lo[m][t], x[2], y[2 * t], y[2 * t + 1], i == 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(hi[m][t], x[0], y[2 * t], y[2 * t + 1], i == 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(lo[m][t], x[1], y[2 * t], y[2 * t + 1]);
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (warp + 4 * m >= NF) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.x[m][t][e] = fmaf(decay, st.x[m][t][e], hi[m][t][e] + lo[m][t][e]);
    }
}

// hi + lo = S rows^T for the token tiles t0, t1 of rows [64 tokens][dk], with TERMS terms of S.
template <int NF, int TERMS>
__device__ __forceinline__ void state_times(float (&hi)[2][4], float (&lo)[2][4], uint32_t planes, uint32_t rows, int t0, int t1, int lane) {
    constexpr int PK = 16 * NF + 8;
    uint32_t a[2][TERMS][4], b[2][4], bl[4];
    planes += a_lane(PK, lane);
#pragma unroll
    for (int x = 0; x < 4; ++x) bl[x] = rows + b_lane(8 * t0, 8 * t1, x, lane);
    auto load = [&](int ks) {
#pragma unroll
        for (int e = 0; e < TERMS; ++e) ldsm4(a[ks & 1][e], planes + e * NV * PK * 2 + 32 * ks);
        ldsm4(b[ks & 1], bl[ks & 3] + (ks >> 2) * C * 128);
    };
    load(0);
#pragma unroll
    for (int ks = 0; ks < NF; ++ks) {
        if (ks + 1 < NF) load(ks + 1);
        const auto &x = a[ks & 1];
        const auto &y = b[ks & 1];
#pragma unroll
        for (int e = TERMS - 1; e > 1; --e)
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(lo[t], x[e], y[2 * t], y[2 * t + 1], ks == 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) mma::mma(hi[t], x[0], y[2 * t], y[2 * t + 1], ks == 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) mma::mma(lo[t], x[1], y[2 * t], y[2 * t + 1], ks == 0 && TERMS == 2);
    }
}

// hi + lo = planes [16][64 tokens] x T (or P) for the token tiles t0 (the shorter one) and t1, from shared memory.
// LOW: T as it is; else its transpose.  `planes`: A's address with the lane part; `step`: from 16 tokens to the next.
template <bool LOW, int AT, int BT, bool TRANS = false>
__device__ __forceinline__ void times_triangle(float (&hi)[2][4], float (&lo)[2][2][4], uint32_t planes, int term, int step, uint32_t tri,
                                               int t0, int t1, int lane) {
    const int n0 = LOW ? t0 / 2 + 1 : 4 - t0 / 2, n1 = LOW ? t1 / 2 + 1 : 4 - t1 / 2;  // n0 <= 2, n1 >= 3
    uint32_t a[2][AT][4];
    uint2 f0[2][BT], f1[2][BT];
    const uint32_t src0 = tri_addr<LOW>(tri, t0, lane), src1 = tri_addr<LOW>(tri, t1, lane);
    auto load = [&](int m) {
#pragma unroll
        for (int e = 0; e < AT; ++e) {
            const uint32_t at = planes + e * term + step * (LOW ? m : 3 - m);
            TRANS ? ldsm4_t(a[m & 1][e], at) : ldsm4(a[m & 1][e], at);
        }
        if (m < 2 && m < n0) tri_frag<LOW, BT>(f0[m & 1], src0, m);
        tri_frag<LOW, BT>(f1[m & 1], src1, m);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[t][e] = lo[t][0][e] = lo[t][1][e] = 0.f;
    load(0);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m >= n1) continue;
        if (m + 1 < 4 && m + 1 < n1) load(m + 1);
        mma_split<AT, BT>(hi, lo, a[m & 1], f0[m & 1], f1[m & 1], m < 2 && m < n0);
    }
}

// SAVE: the pass that gdn_bwd makes (no O; Sig, U and X of every chunk are kept).
template <int NF, bool SAVE>
__global__ void __launch_bounds__(chain_threads(!SAVE), 1) k_chunk_fwd(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                                                const __grid_constant__ ChainMaps maps) {
    constexpr int DK = 16 * NF, PK = DK + 8, kSlabs = (DK + 63) / 64;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<ChainSmem<NF, false> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const uint32_t aS = sm100::smem_u32(sm.S), aU = sm100::smem_u32(sm.U), aR = sm100::smem_u32(sm.R), aT = sm100::smem_u32(sm.T),
                   aP = sm100::smem_u32(sm.P);
    const int groups = p.dv / NV, s = blockIdx.x / (p.H * groups), h = blockIdx.x / groups % p.H, c0 = blockIdx.x % groups * NV;
    const int hk = h / (p.H / p.Hk), lane = threadIdx.x & 31, warp = warp_number();
    const SeqRange r = seq_range(p, s);
    seq_report(p, r, blockIdx.x % (p.H * groups) == 0 && threadIdx.x == 0);
    if (r.slot < 0) return;
    const long long n_chunks = seq_chunks_of(r.len), base = seq_chunk_base(p, s, r.first);
    const size_t soff = (((size_t)r.slot * p.H + h) * p.dv + c0) * DK;
    const ChainFetch<NF, false> fetch = {sm, maps, w, hk, h, c0};
    constexpr int kFetchWarp = SAVE ? 4 : 8;
    const bool fetcher = threadIdx.x == 32 * kFetchWarp;
    auto index = [&](long long c) { return (size_t)(base + c) * p.H + h; };
    auto first_row = [&](long long c) { return (int)(r.first + c * C); };
    chain_init(sm);
    if (fetcher && n_chunks > 0) {
        fetch.k(0, first_row(0), index(0));
        fetch.v(first_row(0), !SAVE);
        fetch.t(w.T + index(0) * 3 * kUnits * 32);
    }
    StateRows<NF> st = {};
    if (warp < 4) {
        if (!seq_starts_zero(p, s))
            st.each(warp, lane, [&](int n, int col, float &x, float &y) {
                const float2 t = *reinterpret_cast<const float2 *>(p.S_in + soff + (size_t)n * DK + col);
                x = t.x;
                y = t.y;
            });
        put_state(aS, st, warp, lane);
    }
    const int t0 = warp & 3, t1 = 7 - t0;  // this warp's token tiles (8 tokens each), the shorter one in T first
    bool ok = true;
    for (long long c = 0; c < n_chunks; ++c) {
        const int b = (int)(c & 1);
        const uint32_t parity = (uint32_t)c & 1;
        const size_t idx = index(c);
        const long long row = r.first + c * C;
        const int rows = (int)min((long long)C, r.len - c * C);
        ok = ok && sm100::mbar_wait(&sm.bar[kBarK + b], (uint32_t)(c >> 1) & 1, w.err) && sm100::mbar_wait(&sm.bar[kBarV], parity, w.err);
        // behind this barrier the state's terms are there and the last step's buffers have been read
        if (!__syncthreads_and(ok)) return chain_leave(sm, p, c, SAVE ? -1 : (int)c - 1, w.err);
        if (fetcher) {
            if (c + 1 < n_chunks) fetch.k(b ^ 1, first_row(c + 1), index(c + 1));
            if (!SAVE) fetch.p(w.P + idx * 2 * kUnits * 32, 0, false);
        }
        if (rows < C) {
            zero_tail(sm.K[b], kSlabs, 8, rows);
            if (!SAVE) zero_tail(sm.Q, kSlabs, 8, rows);
            zero_tail(&sm.V[0][0], 1, NV / 8, rows);
            __syncthreads();
        }
        if (warp == kFetchWarp) {  // it keeps the barriers' count
            __syncthreads();
            if (fetcher && c + 1 < n_chunks) fetch.v(first_row(c + 1), !SAVE);
            __syncthreads();
            if (fetcher && c + 1 < n_chunks) fetch.t(w.T + index(c + 1) * 3 * kUnits * 32);
            continue;
        }
        if (warp >= 4) {  // O^T = e^G S Q^T + U^T P^T
            float qh[2][4], ql[2][4], oh[2][4], ol[2][2][4];
            state_times<NF, 2>(qh, ql, aS, sm100::smem_u32(sm.Q), t0, t1, lane);
            ok = ok && sm100::mbar_wait(&sm.bar[kBarP], parity, w.err);
            __syncthreads();
            __syncthreads();
            times_triangle<true, 2, 2>(oh, ol, sm100::smem_u32(sm.W) + a_lane(PC, lane), NV * PC * 2, 32, aP, t0, t1, lane);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
                const float2 eg = *reinterpret_cast<const float2 *>(&sm.gates[b][0][tok]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    // the neighbour row's lane takes the second token of both rows, this one or it the first: pairs of columns
                    float x = fmaf(eg.x, qh[t][2 * half] + ql[t][2 * half], oh[t][2 * half] + ol[t][0][2 * half]);
                    float y = fmaf(eg.y, qh[t][2 * half + 1] + ql[t][2 * half + 1], oh[t][2 * half + 1] + ol[t][0][2 * half + 1]);
                    const bool odd = lane & 4;
                    const float other = __shfl_xor_sync(0xffffffffu, odd ? x : y, 4);
                    const int i = tok + odd, n = (lane / 4 & ~1) + 8 * half;
                    if (i < rows)
                        *reinterpret_cast<uint32_t *>((bf16 *)p.o + ((row + i) * p.H + h) * p.dv + c0 + n) =
                            odd ? pack(other, y) : pack(x, other);
                }
            }
            continue;
        }
        if (SAVE)
            st.each(warp, lane, [&](int n, int col, float &x, float &y) {
                *reinterpret_cast<float2 *>(w.Sig + (idx * p.dv + c0 + n) * DK + col) = make_float2(x, y);
            });
        // X^T = S K^T
        float kh[2][4], kl[2][4];
        state_times<NF, 3>(kh, kl, aS, sm100::smem_u32(sm.K[b]), t0, t1, lane);
        // beta Y's terms
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 eg = *reinterpret_cast<const float2 *>(&sm.gates[b][0][tok]);
            const float2 be = *reinterpret_cast<const float2 *>(&sm.gates[b][2][tok]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = lane / 4 + 8 * half;
                const float x = eg.x * (kh[t][2 * half] + kl[t][2 * half]), y = eg.y * (kh[t][2 * half + 1] + kl[t][2 * half + 1]);
                if (SAVE) *reinterpret_cast<float2 *>(w.X + (idx * p.dv + c0 + n) * C + tok) = make_float2(x, y);
                put_pair<3>(pair_addr(aR, t ? t1 : t0, lane), half, be.x * (__bfloat162float(sm.V[tok][n]) - x),
                            be.y * (__bfloat162float(sm.V[tok + 1][n]) - y));
            }
        }
        ok = ok && sm100::mbar_wait(&sm.bar[kBarT], parity, w.err);
        __syncthreads();
        // U^T = (beta Y)^T T^T
        float uh[2][4], ul[2][2][4];
        times_triangle<true, 3, 3>(uh, ul, aR + a_lane(PC, lane), NV * PC * 2, 32, aT, t0, t1, lane);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 el = *reinterpret_cast<const float2 *>(&sm.gates[b][1][tok]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = lane / 4 + 8 * half, i = 2 * half;
                const float x = uh[t][i] + (ul[t][0][i] + ul[t][1][i]), y = uh[t][i + 1] + (ul[t][0][i + 1] + ul[t][1][i + 1]);
                if (SAVE) *reinterpret_cast<float2 *>(w.U + (idx * p.dv + c0 + n) * C + tok) = make_float2(x, y);
                put_pair<3>(pair_addr(aU, t ? t1 : t0, lane), half, el.x * x, el.y * y);
                if (!SAVE) put_pair<2>(pair_addr(sm100::smem_u32(sm.W), t ? t1 : t0, lane), half, x, y);
            }
        }
        __syncthreads();
        const uint32_t planes[1] = {aU}, krows[1] = {sm100::smem_u32(sm.K[b])};
        update_state<NF, 1>(st, sm.gates[b][0][C - 1], planes, krows, warp, lane);
        put_state(aS, st, warp, lane);
    }
    if (!SAVE && p.S_out && warp < 4)
        st.each(warp, lane, [&](int n, int col, float &x, float &y) {
            *reinterpret_cast<float2 *>(p.S_out + soff + (size_t)n * DK + col) = make_float2(x, y);
        });
    // the last waits' answers: nobody reads buffers any more, so every thread may report for itself
    if (!ok && p.status) atomicOr(p.status, GDN_SEQ_TIMEOUT);
}

template <int NF>
__global__ void __launch_bounds__(chain_threads(false), 1) k_chunk_bwd(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                                                const __grid_constant__ ChainMaps maps) {
    constexpr int DK = 16 * NF, PK = DK + 8, kSlabs = (DK + 63) / 64;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<ChainSmem<NF, true> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const uint32_t aS = sm100::smem_u32(sm.S), aU = sm100::smem_u32(sm.U), aR = sm100::smem_u32(sm.R), aT = sm100::smem_u32(sm.T),
                   aP = sm100::smem_u32(sm.P);
    const int groups = p.dv / NV, s = blockIdx.x / (p.H * groups), h = blockIdx.x / groups % p.H, c0 = blockIdx.x % groups * NV;
    const int hk = h / (p.H / p.Hk), lane = threadIdx.x & 31, warp = warp_number();
    const SeqRange r = seq_rows(p, s);
    const size_t soff = (((size_t)s * p.H + h) * p.dv + c0) * DK;
    const long long n_chunks = seq_chunks_of(r.len), base = seq_chunk_base(p, s, r.first);  // 0 of a bad range
    const ChainFetch<NF, true> fetch = {sm, maps, w, hk, h, c0};
    const bool fetcher = threadIdx.x == 128;
    auto index = [&](long long c) { return (size_t)(base + c) * p.H + h; };
    auto first_row = [&](long long c) { return (int)(r.first + c * C); };
    chain_init(sm);
    if (fetcher && n_chunks > 0) {
        const long long c = n_chunks - 1;
        fetch.k(0, first_row(c), index(c));
        fetch.v(first_row(c), false);
        fetch.t(w.Tt + index(c) * 3 * kUnits * 32);
        fetch.p(w.Pt + index(c) * 3 * kUnits * 32, first_row(c), true);
    }
    StateRows<NF> st = {};
    if (warp < 4) {
        if (r.slot >= 0 && p.dS_out)
            st.each(warp, lane, [&](int n, int col, float &x, float &y) {
                const float2 t = *reinterpret_cast<const float2 *>(p.dS_out + soff + (size_t)n * DK + col);
                x = t.x;
                y = t.y;
            });
        put_state(aS, st, warp, lane);
    }
    const int t1 = warp & 3, t0 = 7 - t1;  // the shorter tile first, as in k_chunk_fwd
    bool ok = true;
    for (long long c = n_chunks - 1; c >= 0; --c) {
        const long long turn = n_chunks - 1 - c;
        const int b = (int)(turn & 1);
        const uint32_t parity = (uint32_t)turn & 1;
        const size_t idx = index(c);
        const long long row = r.first + c * C;
        const int rows = (int)min((long long)C, r.len - c * C);
        ok = ok && sm100::mbar_wait(&sm.bar[kBarK + b], (uint32_t)(turn >> 1) & 1, w.err) &&
             sm100::mbar_wait(&sm.bar[kBarV], parity, w.err) && sm100::mbar_wait(&sm.bar[kBarP], parity, w.err);
        if (!__syncthreads_and(ok)) return chain_leave(sm, p, turn, (int)turn, w.err);
        if (fetcher && c > 0) fetch.k(b ^ 1, first_row(c - 1), index(c - 1));
        if (rows < C) {
            zero_tail(sm.K[b], kSlabs, 8, rows);
            zero_tail(sm.Q, kSlabs, 8, rows);
            zero_tail(&sm.V[0][0], 1, NV / 8, rows);
            __syncthreads();
        }
        if (warp == 4) {
            __syncthreads();
            if (fetcher && c > 0) fetch.v(first_row(c - 1), false);
            __syncthreads();
            if (fetcher && c > 0) fetch.t(w.Tt + index(c - 1) * 3 * kUnits * 32);
            __syncthreads();
            __syncthreads();
            if (fetcher && c > 0) fetch.p(w.Pt + index(c - 1) * 3 * kUnits * 32, first_row(c - 1), true);
            continue;
        }
        st.each(warp, lane, [&](int n, int col, float &x, float &y) {
            *reinterpret_cast<float2 *>(w.D + (idx * p.dv + c0 + n) * DK + col) = make_float2(x, y);
        });
        // D^T K^T, and dO^T P
        float zh[2][4], zl[2][4], ph[2][4], pl[2][2][4];
        state_times<NF, 3>(zh, zl, aS, sm100::smem_u32(sm.K[b]), t0, t1, lane);
        times_triangle<false, 1, 3, true>(ph, pl, sm100::smem_u32(sm.V) + at_lane(NV, lane), 0, 16 * NV * 2, aP, t0, t1, lane);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 el = *reinterpret_cast<const float2 *>(&sm.gates[b][1][tok]);
            const float2 eg = *reinterpret_cast<const float2 *>(&sm.gates[b][0][tok]);
            float past0 = 0.f, past1 = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = lane / 4 + 8 * half, i = 2 * half;
                const float zx = el.x * (zh[t][i] + zl[t][i]), zy = el.y * (zh[t][i + 1] + zl[t][i + 1]);
                const float2 u = *reinterpret_cast<const float2 *>(w.U + (idx * p.dv + c0 + n) * C + tok);
                past0 = fmaf(u.x, zx, past0);
                past1 = fmaf(u.y, zy, past1);
                put_pair<3>(pair_addr(aR, t ? t1 : t0, lane), half, zx + (ph[t][i] + (pl[t][0][i] + pl[t][1][i])),
                            zy + (ph[t][i + 1] + (pl[t][0][i + 1] + pl[t][1][i + 1])));  // dU
                put_pair<3>(pair_addr(aU, t ? t1 : t0, lane), half, eg.x * __bfloat162float(sm.V[tok][n]),
                            eg.y * __bfloat162float(sm.V[tok + 1][n]));
            }
            past0 = rows_sum(past0);
            past1 = rows_sum(past1);
            if (lane < 4) *reinterpret_cast<float2 *>(w.past + (idx * groups + c0 / NV) * C + tok) = make_float2(past0, past1);
        }
        ok = ok && sm100::mbar_wait(&sm.bar[kBarT], parity, w.err);
        __syncthreads();
        // dR^T = dU^T T
        float rh[2][4], rl[2][2][4];
        times_triangle<false, 3, 3>(rh, rl, aR + a_lane(PC, lane), NV * PC * 2, 32, aT, t0, t1, lane);
        __syncthreads();  // dU has been read: -beta e^G dR takes its place
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 eg = *reinterpret_cast<const float2 *>(&sm.gates[b][0][tok]);
            const float2 be = *reinterpret_cast<const float2 *>(&sm.gates[b][2][tok]);
            float into0 = 0.f, into1 = 0.f, db0 = 0.f, db1 = 0.f;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = lane / 4 + 8 * half, i = 2 * half;
                const float x = rh[t][i] + (rl[t][0][i] + rl[t][1][i]), y = rh[t][i + 1] + (rl[t][0][i + 1] + rl[t][1][i + 1]);
                const size_t at = (idx * p.dv + c0 + n) * C + tok;
                *reinterpret_cast<float2 *>(w.dR + at) = make_float2(x, y);
                const float2 X = *reinterpret_cast<const float2 *>(w.X + at);
                const bf16 *vp = (const bf16 *)p.v + (row + tok) * p.v_stride + (size_t)h * p.dv + c0 + n;
                bf16 *dvp = (bf16 *)p.dv_out + ((row + tok) * p.H + h) * p.dv + c0 + n;
                const float bx = be.x * x, by = be.y * y;
                into0 = fmaf(-bx, X.x, into0);
                into1 = fmaf(-by, X.y, into1);
                if (tok < rows) {
                    db0 = fmaf(x, __bfloat162float(vp[0]) - X.x, db0);
                    dvp[0] = __float2bfloat16_rn(bx);
                }
                if (tok + 1 < rows) {
                    db1 = fmaf(y, __bfloat162float(vp[p.v_stride]) - X.y, db1);
                    dvp[(size_t)p.H * p.dv] = __float2bfloat16_rn(by);
                }
                put_pair<3>(pair_addr(aR, t ? t1 : t0, lane), half, -eg.x * bx, -eg.y * by);
            }
            into0 = rows_sum(into0);
            into1 = rows_sum(into1);
            db0 = rows_sum(db0);
            db1 = rows_sum(db1);
            if (lane < 4) {
                *reinterpret_cast<float2 *>(w.into + (idx * groups + c0 / NV) * C + tok) = make_float2(into0, into1);
                *reinterpret_cast<float2 *>(w.db + (idx * groups + c0 / NV) * C + tok) = make_float2(db0, db1);
            }
        }
        __syncthreads();
        const uint32_t planes[2] = {aU, aR}, mrows[2] = {sm100::smem_u32(sm.Q), sm100::smem_u32(sm.K[b])};
        update_state<NF, 2>(st, sm.gates[b][0][C - 1], planes, mrows, warp, lane);
        put_state(aS, st, warp, lane);
        __syncthreads();  // Q has been read
    }
    if (p.dS_in && warp < 4)
        st.each(warp, lane, [&](int n, int col, float &x, float &y) {
            *reinterpret_cast<float2 *>(p.dS_in + soff + (size_t)n * DK + col) = make_float2(x, y);
        });
    if (!ok && p.status) atomicOr(p.status, GDN_SEQ_TIMEOUT);
}

// The gradients of a chunk and head from what the chains left: 8 warps, warp w has the 16 tokens from 16 (w % 4).
// Warps 0-3 make dQ (and dK's part that sums over later tokens), warps 4-7 dK:
//   dQ = e^G dO Sig^T + dP K,  dK = -beta e^G dR Sig^T + e^{G_L-G} U D^T + (beta dA) K + [dP; beta dA]^T [Q; K]
// Products that reach the gates' fp32 gradients are at fp32 accuracy (dO Sig^T, dP, dA: every term); those that
// only reach the bf16 dQ and dK take two terms of each operand.
// Bound by the products: 6200 warp products at d = 112, 8 clocks each on a quarter of an SM.
template <int NF> struct GradSmem {  // 1024-byte aligned
    static constexpr int kTile = (16 * NF + 63) / 64 * C * 64;
    bf16 K[kTile], Q[kTile], dO[2 * C * 64];  // swizzled rows
    union {
        bf16 SD[5][128 * 64];                 // 64 columns of Sig (3 terms) and D (2), [dv][64] swizzled
        struct {
            bf16 U[3][128 * 64];              // [dv][64 tokens] swizzled
            bf16 PA[4][C][PC];                // dP and beta dA, 2 terms each
        };
        float kT[C][16 * NF + 4];
    };
    float M[C][C + 1];
    double G[C];
    float gates[3][C], into[C], past[C], db[C], red[8];
};

template <int NF>
__global__ void __launch_bounds__(256, 1) k_chunk_grads(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w) {
    constexpr int DK = 16 * NF;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<GradSmem<NF> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const long long c = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk), tid = threadIdx.x, lane = tid & 31, warp = warp_number();
    const int mt = warp & 3, role = warp >> 2, dv = p.dv, nvf = dv / 16;
    const SeqChunk ch = seq_chunk(p, c);
    if (ch.rows == 0) return;
    const size_t idx = (size_t)c * p.H + h;
    auto rows_in = [&](bf16 *dst, const bf16 *src, long long stride, int pieces) {
        for (int i = tid; i < C * pieces; i += 256) {
            const int r = i / pieces, col = i % pieces * 8, on = r < ch.rows ? 16 : 0;
            cp_async16((char *)dst + sw_byte(C, r, col), src + (ch.first + (on ? r : 0)) * stride + col, on);
        }
    };
    rows_in(sm.dO, (const bf16 *)p.d_o + (size_t)h * dv, (long long)p.H * dv, dv / 8);
    rows_in(sm.K, (const bf16 *)p.k + (size_t)hk * DK, p.k_stride, DK / 8);
    rows_in(sm.Q, (const bf16 *)p.q + (size_t)hk * DK, p.q_stride, DK / 8);
    sm100::cp_async_commit();
    if (tid < 3 * C) sm.gates[0][tid] = w.gates[idx * 3 * C + tid];
    if (tid < C) {
        sm.G[tid] = w.G[idx * C + tid];
        float past = 0.f, into = 0.f, db = 0.f;  // the slices' parts, in order
        for (int g = 0; g < nvf; ++g) {
            past += w.past[(idx * nvf + g) * C + tid];
            into += w.into[(idx * nvf + g) * C + tid];
            db += w.db[(idx * nvf + g) * C + tid];
        }
        sm.past[tid] = past;
        sm.into[tid] = into;
        sm.db[tid] = db;
    }
    const float *Sig = w.Sig + idx * dv * DK, *Dm = w.D + idx * dv * DK, *Um = w.U + idx * dv * C, *Rm = w.dR + idx * dv * C;
    const uint32_t aSD = sm100::smem_u32(sm.SD), aK = sm100::smem_u32(sm.K), aQ = sm100::smem_u32(sm.Q), aO = sm100::smem_u32(sm.dO);
    constexpr uint32_t kPlane = 128 * 64 * 2;
    const int i0 = 16 * mt + lane / 4, j0 = 2 * (lane & 3);  // this lane's rows i0, i0 + 8; its columns 8 t + j0, + 1
    // fragment of a fp32 [dv][64 tokens] matrix as the A operand (rows: this warp's tokens), NT terms
    auto frag = [&](auto &a, const float *m, int ks) {
        constexpr int NT = sizeof(a) / sizeof(a[0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float *x = m + (size_t)(16 * ks + j0 + (e >> 1) * 8) * C + i0 + (e & 1) * 8;
            uint32_t t[NT];
            split(x[0], x[C], t);
#pragma unroll
            for (int n = 0; n < NT; ++n) a[n][e] = t[n];
        }
    };
    float acc[2 * NF][4];  // dQ's or dK's rows of this warp
#pragma unroll
    for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
    float all = 0.f;
#pragma unroll
    for (int slab = 0; slab < (NF + 3) / 4; ++slab) {
        constexpr int kLast = DK % 64 ? DK % 64 : 64;
        const int cols = slab + 1 < (NF + 3) / 4 ? 64 : kLast;
        for (int i = tid; i < dv * (cols / 4); i += 256) {
            const int n = i / (cols / 4), col = i % (cols / 4) * 4;
            const float4 s = *reinterpret_cast<const float4 *>(Sig + (size_t)n * DK + 64 * slab + col);
            const float4 d = *reinterpret_cast<const float4 *>(Dm + (size_t)n * DK + 64 * slab + col);
            all += (s.x * d.x + s.y * d.y) + (s.z * d.z + s.w * d.w);
            uint32_t a[3], b[3], e[2], f[2];
            split(s.x, s.y, a);
            split(s.z, s.w, b);
            split(d.x, d.y, e);
            split(d.z, d.w, f);
            char *at = (char *)sm.SD + sw_byte(0, n, col) + (col & 4) * 2;
#pragma unroll
            for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2 *>(at + x * kPlane) = make_uint2(a[x], b[x]);
#pragma unroll
            for (int x = 0; x < 2; ++x) *reinterpret_cast<uint2 *>(at + (3 + x) * kPlane) = make_uint2(e[x], f[x]);
        }
        sm100::cp_async_wait_all();
        __syncthreads();
        if (role == 0) {
            float hi[8][4], lo[8][4];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) hi[t][e] = lo[t][e] = 0.f;
            for (int ks = 0; ks < nvf; ++ks) {
                uint32_t a[4];
                ldsm4(a, aO + sw_byte(C, 16 * mt + (lane & 15), 16 * ks + (lane >> 4) * 8));
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (16 * g >= cols) continue;
                    uint32_t b[3][4];
#pragma unroll
                    for (int x = 0; x < 3; ++x) ldsm4_t(b[x], aSD + x * kPlane + bt_lane(0, 16 * g, lane) + ks * 2048);
#pragma unroll
                    for (int x = 2; x >= 0; --x)
#pragma unroll
                        for (int t = 0; t < 2; ++t) mma::mma(x ? lo[2 * g + t] : hi[2 * g + t], a, b[x][2 * t], b[x][2 * t + 1]);
                }
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (8 * slab + t >= 2 * NF) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[(8 * slab + t) % (2 * NF)][e] = sm.gates[0][i0 + (e >> 1) * 8] * (hi[t][e] + lo[t][e]);
            }
        } else {
            float x0[8][4], x1[8][4];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x0[t][e] = x1[t][e] = 0.f;
            for (int ks = 0; ks < nvf; ++ks) {
                uint32_t r[2][4], u[2][4];
                frag(r, Rm, ks);
                frag(u, Um, ks);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (16 * g >= cols) continue;
                    uint32_t b[2][4], d[2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        ldsm4_t(b[x], aSD + x * kPlane + bt_lane(0, 16 * g, lane) + ks * 2048);
                        ldsm4_t(d[x], aSD + (3 + x) * kPlane + bt_lane(0, 16 * g, lane) + ks * 2048);
                    }
#pragma unroll
                    for (int x = 2; x >= 0; --x)  // terms (0, 1), (1, 0), (0, 0)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            mma::mma(x0[2 * g + t], r[x == 1], b[x == 2][2 * t], b[x == 2][2 * t + 1]);
                            mma::mma(x1[2 * g + t], u[x == 1], d[x == 2][2 * t], d[x == 2][2 * t + 1]);
                        }
                }
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (8 * slab + t >= 2 * NF) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + (e >> 1) * 8;
                    acc[(8 * slab + t) % (2 * NF)][e] = fmaf(-sm.gates[2][i] * sm.gates[0][i], x0[t][e], sm.gates[1][i] * x1[t][e]);
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) sm.red[warp] = all;
    // a pair of a row of K or Q
    auto pair = [&](const bf16 *tile, int row, int col) {
        return *reinterpret_cast<const uint32_t *>((const char *)tile + sw_byte(C, row, col) + (col & 7) * 2);
    };
    auto quad = [](float x) {
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        return x + __shfl_xor_sync(0xffffffffu, x, 2);
    };
    if (role == 0) {  // q . dq so far: the terms that come from before the chunk
        float x[2] = {};
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t q = pair(sm.Q, i0 + 8 * half, 8 * t + j0);
                x[half] += low_of(q) * acc[t][2 * half] + high_of(q) * acc[t][2 * half + 1];
            }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float y = quad(x[half]);
            if ((lane & 3) == 0) sm.into[i0 + 8 * half] += y;
        }
    }
    // dP, dA
    for (int i = tid; i < dv * (C / 4); i += 256) {
        const int n = i / (C / 4), col = i % (C / 4) * 4;
        const float4 u = *reinterpret_cast<const float4 *>(Um + (size_t)n * C + col);
        uint32_t a[3], b[3];
        split(u.x, u.y, a);
        split(u.z, u.w, b);
        char *at = (char *)sm.U + sw_byte(0, n, col) + (col & 4) * 2;
#pragma unroll
        for (int x = 0; x < 3; ++x) *reinterpret_cast<uint2 *>(at + x * kPlane) = make_uint2(a[x], b[x]);
    }
    __syncthreads();
    uint32_t op[4][2][4];  // dP's or dA's rows as an A operand, two terms
    {
        float hi[8][4], lo[8][4], kk[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) hi[t][e] = lo[t][e] = kk[t][e] = 0.f;
        for (int ks = 0; ks < nvf; ++ks) {
            uint32_t a[3][4];
            if (role == 0) ldsm4(a[0], aO + sw_byte(C, 16 * mt + (lane & 15), 16 * ks + (lane >> 4) * 8));
            else frag(a, Rm, ks);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (g > mt) continue;
                uint32_t b[3][4];
#pragma unroll
                for (int x = 0; x < 3; ++x) ldsm4_t(b[x], aSD + x * kPlane + bt_lane(0, 16 * g, lane) + ks * 2048);
#pragma unroll
                for (int x = 2; x >= 0; --x)
#pragma unroll
                    for (int t = 0; t < 2; ++t) mma::mma(x ? lo[2 * g + t] : hi[2 * g + t], a[0], b[x][2 * t], b[x][2 * t + 1]);
                if (role) {
#pragma unroll
                    for (int x = 0; x < 3; ++x)  // terms (1, 0), (1, 1), (2, 0)
#pragma unroll
                        for (int t = 0; t < 2; ++t) mma::mma(lo[2 * g + t], a[1 + (x == 2)], b[x == 1][2 * t], b[x == 1][2 * t + 1]);
                }
            }
        }
        const uint32_t left = role ? aK : aQ;
#pragma unroll
        for (int ks = 0; ks < NF; ++ks) {
            uint32_t a[4];
            ldsm4(a, left + sw_byte(C, 16 * mt + (lane & 15), 16 * ks + (lane >> 4) * 8));
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (g > mt) continue;
                uint32_t b[4];
                ldsm4(b, aK + b_lane(16 * g, 16 * g + 8, ks & 3, lane) + (ks >> 2) * C * 128);
                mma::mma(kk[2 * g], a, b[0], b[1]);
                mma::mma(kk[2 * g + 1], a, b[2], b[3]);
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half, j = 8 * t + j0;
                const float be = role ? sm.gates[2][i] : 1.f;
                float x[2], m[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool in = role ? j + e < i : j + e <= i;
                    const float gam = in ? expf((float)(sm.G[i] - sm.G[j + e])) : 0.f;
                    x[e] = gam * (hi[t][2 * half + e] + lo[t][2 * half + e]);
                    if (role) x[e] = -x[e];
                    m[e] = be * x[e] * kk[t][2 * half + e];
                }
                uint32_t s[2];
                split(x[0], x[1], s);
#pragma unroll
                for (int n = 0; n < 2; ++n) op[t / 2][n][half + 2 * (t & 1)] = s[n];
                split(be * x[0], be * x[1], s);
#pragma unroll
                for (int n = 0; n < 2; ++n) *reinterpret_cast<uint32_t *>(&sm.PA[2 * role + n][i][j]) = s[n];
                hi[t][2 * half] = m[0];
                hi[t][2 * half + 1] = m[1];
            }
        }
        auto put_m = [&](bool add) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &m = sm.M[i0 + (e >> 1) * 8][8 * t + j0 + (e & 1)];
                    m = add ? m + hi[t][e] : hi[t][e];
                }
        };
        if (role == 0) put_m(false);
        __syncthreads();
        if (role) put_m(true);
    }
    // rows x K: dQ's or dK's part inside the chunk
#pragma unroll
    for (int g = 0; g < NF; ++g) {
        float x[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
            if (kb > mt) continue;
            uint32_t b[4];
            ldsm4_t(b, aK + bt_lane(C, 16 * g, lane) + kb * 2048);
#pragma unroll
            for (int n = 1; n >= 0; --n)
#pragma unroll
                for (int t = 0; t < 2; ++t) mma::mma(x[t], op[kb][n], b[2 * t], b[2 * t + 1]);
        }
        float db[2] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half;
                const float be = role ? sm.gates[2][i] : 1.f;
                if (role) {
                    const uint32_t k = pair(sm.K, i, 16 * g + 8 * t + j0);
                    db[half] += low_of(k) * x[t][2 * half] + high_of(k) * x[t][2 * half + 1];
                }
                acc[2 * g + t][2 * half] = fmaf(be, x[t][2 * half], acc[2 * g + t][2 * half]);
                acc[2 * g + t][2 * half + 1] = fmaf(be, x[t][2 * half + 1], acc[2 * g + t][2 * half + 1]);
            }
        if (role)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float y = quad(db[half]);
                if ((lane & 3) == 0) sm.db[i0 + 8 * half] += y;
            }
    }
    auto store = [&](bf16 *dst, float *dst32) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = i0 + 8 * half;
            if (i >= ch.rows) continue;
            const size_t at = ((size_t)(ch.first + i) * p.H + h) * DK + j0;
#pragma unroll
            for (int t = 0; t < 2 * NF; ++t) {
                if (dst32) *reinterpret_cast<float2 *>(dst32 + at + 8 * t) = make_float2(acc[t][2 * half], acc[t][2 * half + 1]);
                else *reinterpret_cast<uint32_t *>(dst + at + 8 * t) = pack(acc[t][2 * half], acc[t][2 * half + 1]);
            }
        }
    };
    __syncthreads();  // U has been read (dP, dA: before the last barrier), PA is complete; M too
    if (role == 0) {
        store((bf16 *)p.dq, w.dqh);
        // rows j of [dP; beta dA]^T [Q; K]
        float x[2 * NF][4];
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
        const uint32_t aPA = sm100::smem_u32(sm.PA) + at_lane(PC, lane) + 32 * mt;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
            if (kb < mt) continue;
            uint32_t a[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) ldsm4_t(a[n], aPA + n * C * PC * 2 + kb * 16 * PC * 2);
#pragma unroll
            for (int g = 0; g < NF; ++g) {
                uint32_t q[4], k[4];
                ldsm4_t(q, aQ + bt_lane(C, 16 * g, lane) + kb * 2048);
                ldsm4_t(k, aK + bt_lane(C, 16 * g, lane) + kb * 2048);
#pragma unroll
                for (int n = 1; n >= 0; --n)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        mma::mma(x[2 * g + t], a[n], q[2 * t], q[2 * t + 1]);
                        mma::mma(x[2 * g + t], a[2 + n], k[2 * t], k[2 * t + 1]);
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][e] = x[t][e];
    } else if (warp < 6) {
        const int j = tid - 128;  // column sums of M over the rows from each row on
        for (int i = C - 2; i >= 0; --i) sm.M[i][j] += sm.M[i + 1][j];
    }
    __syncthreads();  // PA has been read: kT lies there
    if (role == 0) {
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                *reinterpret_cast<float2 *>(&sm.kT[i0 + 8 * half][8 * t + j0]) = make_float2(acc[t][2 * half], acc[t][2 * half + 1]);
    }
    __syncthreads();
    if (role) {
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 x = *reinterpret_cast<const float2 *>(&sm.kT[i0 + 8 * half][8 * t + j0]);
                acc[t][2 * half] += x.x;
                acc[t][2 * half + 1] += x.y;
            }
        store((bf16 *)p.dk_out, w.dkh);
    } else if (tid < ch.rows) {
        float g = 0.f;
        for (int i = 0; i < 8; ++i) g += sm.red[i];
        g *= sm.gates[0][C - 1];
        for (int j = 0; j < tid; ++j) g += sm.M[tid][j] + sm.past[j];
        for (int i = tid; i < C; ++i) g += sm.into[i];
        const size_t at = (size_t)(ch.first + tid) * p.H + h;
        p.dalpha[at] = g / fmaxf(p.alpha[at], expf(kSeqBwdLogFloor));
        p.dbeta[at] = sm.db[tid];
    }
}

template <int NF> cudaError_t prep(const SeqProblem &p, const ChunkWork &w, float floor_log, cudaStream_t s) {
    const unsigned blocks = (unsigned)(seq_max_chunks(p) * p.H);
    if (blocks) k_prep<NF><<<blocks, 128, 0, s>>>(p, w, floor_log);
    return cudaGetLastError();
}

template <typename K, int NF, bool BWD> cudaError_t chain(K kernel, int threads, const SeqProblem &p, const ChunkWork &w, const ChainMaps &m, cudaStream_t s) {
    const int bytes = (int)sizeof(ChainSmem<NF, BWD>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e) return e;
    kernel<<<(unsigned)((long long)p.n_seqs * p.H * (p.dv / NV)), threads, bytes, s>>>(p, w, m);
    return cudaGetLastError();
}

bool make_maps(ChainMaps &m, const SeqProblem &p, const void *v, long long v_stride) {
    return seq_row_map(&m.q, p.q, p.n_tokens, p.q_stride, p.Hk, p.dk, 64) &&
           seq_row_map(&m.k, p.k, p.n_tokens, p.k_stride, p.Hk, p.dk, 64) &&
           seq_row_map(&m.v, v, p.n_tokens, v_stride, p.H, p.dv, NV);
}

template <int NF> cudaError_t fwd(const SeqProblem &p, const ChunkWork &w, cudaStream_t s) {
    ChainMaps m;
    if (!make_maps(m, p, p.v, p.v_stride)) return cudaErrorInvalidValue;
    cudaError_t e = prep<NF>(p, w, kLogAlphaFloor, s);
    return e ? e : chain<decltype(&k_chunk_fwd<NF, false>), NF, false>(k_chunk_fwd<NF, false>, chain_threads(true), p, w, m, s);
}

template <int NF> cudaError_t bwd(const SeqProblem &p, const ChunkWork &w, cudaStream_t s) {
    ChainMaps m, mo;
    if (!make_maps(m, p, p.v, p.v_stride) || !make_maps(mo, p, p.d_o, (long long)p.H * p.dv)) return cudaErrorInvalidValue;
    cudaError_t e = prep<NF>(p, w, kSeqBwdLogFloor, s);
    if (!e) e = chain<decltype(&k_chunk_fwd<NF, true>), NF, false>(k_chunk_fwd<NF, true>, chain_threads(false), p, w, m, s);
    if (!e) e = chain<decltype(&k_chunk_bwd<NF>), NF, true>(k_chunk_bwd<NF>, chain_threads(false), p, w, mo, s);
    const int bytes = (int)sizeof(GradSmem<NF>) + 1024;
    if (!e) e = cudaFuncSetAttribute(k_chunk_grads<NF>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e) return e;
    k_chunk_grads<NF><<<(unsigned)(seq_max_chunks(p) * p.H), 256, bytes, s>>>(p, w);
    return cudaGetLastError();
}

ChunkWork carve(const SeqProblem &p, void *base, bool bwd, size_t *total) {
    const size_t n = (size_t)seq_max_chunks(p) * p.H, rows = (size_t)p.n_tokens * p.H;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *x = (char *)base + at;
        at += align256(bytes);
        return x;
    };
    const size_t frag = n * kUnits * 32 * sizeof(uint2);  // a term of T or P
    ChunkWork w = {};
    w.T = (uint2 *)take(3 * frag);
    w.gates = (float *)take(n * 3 * C * 4);
    w.err = (int *)take(sizeof(int));
    if (!bwd) {
        w.P = (uint2 *)take(2 * frag);
    } else {
        w.Tt = (uint2 *)take(3 * frag);
        w.Pt = (uint2 *)take(3 * frag);
        w.G = (double *)take(n * C * 8);
        w.Sig = (float *)take(n * p.dk * p.dv * 4);
        w.D = (float *)take(n * p.dk * p.dv * 4);
        w.U = (float *)take(n * C * p.dv * 4);
        w.X = (float *)take(n * C * p.dv * 4);
        w.dR = (float *)take(n * C * p.dv * 4);
        w.past = (float *)take(n * (p.dv / NV) * C * 4);
        w.into = (float *)take(n * (p.dv / NV) * C * 4);
        w.db = (float *)take(n * (p.dv / NV) * C * 4);
        w.dqh = p.H > p.Hk ? (float *)take(rows * p.dk * 4) : nullptr;
        w.dkh = p.H > p.Hk ? (float *)take(rows * p.dk * 4) : nullptr;
    }
    if (total) *total = at;
    return w;
}

}  // namespace

size_t seq_chunk_workspace(const SeqProblem &p, bool bwd) {
    size_t n;
    carve(p, nullptr, bwd, &n);
    return n;
}

cudaError_t launch_seq_chunk(const SeqProblem &p, void *ws, cudaStream_t s) {
    const ChunkWork w = carve(p, ws, false, nullptr);
    switch (p.dk / 16) {
        case 1: return fwd<1>(p, w, s);
        case 2: return fwd<2>(p, w, s);
        case 3: return fwd<3>(p, w, s);
        case 4: return fwd<4>(p, w, s);
        case 5: return fwd<5>(p, w, s);
        case 6: return fwd<6>(p, w, s);
        case 7: return fwd<7>(p, w, s);
        default: return fwd<8>(p, w, s);
    }
}

cudaError_t launch_seq_bwd_chunk(const SeqProblem &p, void *ws, cudaStream_t s) {
    const ChunkWork w = carve(p, ws, true, nullptr);
    cudaError_t e = launch_seq_zero_rows(p, w.dqh, w.dkh, s);
    if (!e && p.n_seqs) {
        switch (p.dk / 16) {
            case 1: e = bwd<1>(p, w, s); break;
            case 2: e = bwd<2>(p, w, s); break;
            case 3: e = bwd<3>(p, w, s); break;
            case 4: e = bwd<4>(p, w, s); break;
            case 5: e = bwd<5>(p, w, s); break;
            case 6: e = bwd<6>(p, w, s); break;
            case 7: e = bwd<7>(p, w, s); break;
            default: e = bwd<8>(p, w, s);
        }
    }
    return e ? e : launch_seq_share(p, w.dqh, w.dkh, s);
}

}  // namespace gdn
