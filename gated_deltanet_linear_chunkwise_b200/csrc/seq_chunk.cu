// seq_chunk.cu -- the chunked gated delta rule over packed sequences on the tensor cores (bf16 q, k, v).
//
// Notation and formulas as in seq_simt.cu; chunks of 64 tokens.
//
// k_prep         every (chunk, head) by itself: T, P and the decays; one block more: the sequences' order and verdicts.
// k_chunk_fwd    a block walks the chunks of one sequence and head with 16 columns of the state
//                (d_v columns are independent), S = Sig^T's 16 rows in registers:
//                  X^T = S [K;Q]^T,  Y = V - e^G X_K,  U^T = (beta Y)^T T^T,
//                  O^T = e^G X_Q^T + U^T P^T,  S <- e^{G_L} S + (e^{G_L-G} U)^T K
// k_chunk_bwd    the same walk backwards with 16 rows of D^T:
//                  dU^T = e^{G_L-G} D^T K^T + dO^T P,  dR^T = dU^T T,
//                  D^T <- e^{G_L} D^T + (e^G dO)^T Q - (beta e^G dR)^T K
// k_walk_fwd, k_walk_bwd   the same with a warp for each 16 columns, where there are many chains.
// k_chunk_grads  every (chunk, head) by itself: dQ, dK and the gates' gradients.
//
// gdn_packed runs the first and a forward walk, gdn_bwd all of them (its forward walk keeps what the others read).
//
// Precision.  The state leaves in fp32 and has to be as exact as a fp32 recurrence, so its products are split ones
// (seq_mma.cuh); what only reaches a bf16 output (Q S, P U) takes two terms, whose 2^-17 vanish in its 2^-9.  With two
// terms everywhere the state would be 3.7e-6 off (2-norm, a 64-bit model of the walk, 2048 tokens, d = 112), with three 2e-7.
//
// Why warp-level products and not tcgen05.  One sequence of 20 heads has 140 slices of 16 columns, one for nearly every SM, and its
// 64-token step is as short as it gets.  A tcgen05 product has 128 rows of K and Q against N = 16 there and is bound by its A
// operand's shared memory reads (128 x 16 x 2 bytes at 128 B/clk: 32 clk an instruction, as long as the 16 warp products
// that it replaces); with all terms of S side by side (N = 48) it would be three times faster, but T's terms have to come as
// full 64 x 64 operands then (76 KB a step and slice instead of 60), which is more than L2 gives 140 blocks at that rate, and
// each of the step's three dependent products pays a round trip through tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>

#include "seq_gates.cuh"
#include "seq_mma.cuh"

namespace gdn {

bool seq_row_map(CUtensorMap *m, const void *x, long long rows, long long row_stride, int heads, int d, int cols);
bool seq_matrix_map(CUtensorMap *m, const float *x, long long rows, int cols, int box_rows);  // both gdn_tc.cu

namespace {

using namespace mma;
using sm100::cp_async16;

constexpr int C = kSeqChunk;
constexpr int NV = 16;       // rows of S (columns of d_v) that a block holds
constexpr int kPlane = NV * 128;  // bytes of a term's 16 rows of 64 columns, swizzled

// T and P lie in the order of the B operand's fragments, a term behind the other: unit (t, b) is the n-tile of 8
// tokens from 8t against the 16 tokens from 16b, a lane's two words of it.  Below the diagonal b <= t / 2 (20
// units), above it (the transposes) b >= t / 2.  P reaches O only and has two terms; T and the transposes have three.
__host__ __device__ constexpr int low_unit(int t) { return (t / 2) * (t / 2 + 1) + (t & 1) * (t / 2 + 1); }
__host__ __device__ constexpr int up_unit(int t) { return 20 - low_unit(8 - t) ; }
constexpr int kUnits = 20;

struct ChunkWork {
    uint2 *T, *P, *Tt, *Pt;  // [chunk x H][terms][20][32]; P or the transposes may be null
    float *gates;            // [chunk x H][3][64]: e^G, e^{G_L - G}, beta
    float4 *gam;             // [chunk x H][20][32]: e^{G_i - G_j} (0 above the diagonal) in the order of a product's result, or null
    // gdn_bwd: the chains' matrices, fp32
    float *Sig, *D;          // [chunk x H][dv][dk]: the state entering the chunk; the gradient of the one leaving it
    float *U, *dR, *X, *Z;   // [chunk x H][dv][64]; X = e^G K Sig, Z = e^{G_L-G} K D
    float *dqh, *dkh;        // as in SeqWork
    int *err;                // a bounded wait that gave up (k_prep clears it)
    int *order;              // [n_seqs]: the sequences, the longest first (up to kSorted); -1 - s of one that starts inside an earlier one
    unsigned char *good;     // [n_seqs]: its rows are in order, by themselves and among the others
    SeqChunk *chunks;        // gdn_bwd: [chunks], what seq_chunk finds
    uint64_t wait_ns;        // limit of the bounded waits
    int drop;                // debug: the first block's K (1) or T (2) is never fetched, so its wait gives up
};

// The chains' blocks start with the longest sequences: a long one that starts last runs alone.  A sequence's place is the
// number of longer ones, ties by index.  One block counts them, so with more than 512 sequences they stay in their order:
// counting n^2 / 128 steps then takes longer than it saves.  Measured (us, longest first / as they are, lengths 1 to 600, many of
// them short; 20 heads, d = 112, and 4 heads, d = 64): 32 sequences 157 / 169 and 41 / 48, 128 677 / 695 and 84 / 99, 256
// 1384 / 1425 and 131 / 157, 512 2492 / 2522 and 290 / 307, 1024 4935 / 4934 and 621 / 587, 2048 10252 / 10093 and 1373 / 1140.
constexpr int kSorted = 512;
__device__ __forceinline__ void order_sequences(const SeqProblem &p, int *order, unsigned char *good, int *len) {  // len: room for kSorted
    const bool sort = p.cu && p.n_seqs <= kSorted;
    bool odd = false;
    if (p.cu)
        for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) {
            const SeqRange r = seq_rows(p, s);
            if (sort) len[s] = (int)r.len;
            odd |= r.bad != 0;
        }
    odd = __syncthreads_or(odd);  // else every range is in order
    if (odd) seq_each_in_order<128>(p, p.n_seqs, [&](int s, const SeqRange &r, bool late) { good[s] = !late && !r.bad; });
    __syncthreads();
    for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) {
        int place = s;
        if (sort) {
            place = 0;
            for (int j = 0; j < p.n_seqs; ++j) place += len[j] > len[s] || (len[j] == len[s] && j < s);
        }
        if (!odd) good[s] = 1;
        order[place] = odd && !good[s] && !seq_rows(p, s).bad ? -1 - s : s;
    }
}

// A sequence's rows and slot with all bits but that of a start inside an earlier one; called by a whole block.
__device__ __forceinline__ SeqRange seq_place(const SeqProblem &p, int s, const unsigned char *good) {
    SeqRange r = seq_rows(p, s);
    if (p.slots) {
        const int slot = p.slots[s];
        r.bad |= seq_slot_bits(p, s, slot, [&](int i) { return good[i] != 0; });
        r.slot = r.bad || slot < 0 ? -1 : slot;
    }
    return r;
}

// dS_in's columns of a sequence that starts inside an earlier one (NULL in a forward call), by a whole block.
__device__ __forceinline__ void no_state(const SeqProblem &p, int s, int h, int c0, int cols) {
    if (!p.dS_in) return;
    float *to = p.dS_in + (((size_t)s * p.H + h) * p.dv + c0) * p.dk;
    for (int i = threadIdx.x; i < cols * p.dk; i += blockDim.x) to[i] = 0.f;
}

template <int NF>
__global__ void __launch_bounds__(128) k_prep(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                              const float floor_log) {
    constexpr int DK = 16 * NF, kTile = (DK + 63) / 64 * C * 64;
    // K and Q, and in their place, once they have been multiplied, A and its inverse
    constexpr int kRows = 2 * kTile * (int)sizeof(bf16), PA = C + 4, kMat = C * PA * (int)sizeof(float);
    __shared__ __align__(16) unsigned char room[kRows > kMat ? kRows : kMat];
    bf16 *const sK = reinterpret_cast<bf16 *>(room), *const sQ = sK + kTile;
    float(*const sA)[PA] = reinterpret_cast<float(*)[PA]>(room);
    __shared__ double sG[C];
    __shared__ float sB[C];
    const long long c = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk), tid = threadIdx.x, lane = tid & 31, warp = warp_number();
    if (blockIdx.x == gridDim.x - 1) {  // one block more than chunks
        if (tid == 0) *w.err = 0;
        order_sequences(p, w.order, w.good, reinterpret_cast<int *>(room));
        return;
    }
    const SeqChunk ch = seq_chunk(p, c);
    if (w.chunks && h == 0 && tid == 0) w.chunks[c] = ch;
    if (ch.rows == 0 || (p.min_len > 0 && seq_rows(p, ch.seq).len < p.min_len)) return;
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
            g[e] = i < ch.rows ? seq_log_gate(p.alpha[at], floor_log) : 0.0;
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
        float gam[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + (e >> 1) * 8, j = 8 * t + j0 + (e & 1);
            if (t / 2 > warp) {
                sA[i][j] = 0.f;
                continue;
            }
            gam[e] = j <= i ? expf((float)(sG[i] - sG[j])) : 0.f;
            qk[t][e] *= gam[e];
            sA[i][j] = j < i ? sB[i] * gam[e] * kk[t][e] : 0.f;
        }
        if (w.gam && t / 2 <= warp) w.gam[(idx * kUnits + warp * (warp + 1) + t) * 32 + lane] = make_float4(gam[0], gam[1], gam[2], gam[3]);
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
    // T21 = -T22 (A21 T11), blocks of 16 then of 32, four rows a thread
    auto four = [&](int row, int col) { return *reinterpret_cast<const float4 *>(&sA[row][col]); };
    __syncthreads();
    {
        const int pair = tid >> 6, e = tid & 63, o = 32 * pair, r = o + 16 + e / 16 * 4, col = o + e % 16;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {  // A21 T11, then T22 times that
            float m[4] = {};
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                const int from = o + 16 * pass + k;
                const float b[4] = {sA[from][col], sA[from + 1][col], sA[from + 2][col], sA[from + 3][col]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 a = four(r + i, from);
                    m[i] = fmaf(a.x, b[0], fmaf(a.y, b[1], fmaf(a.z, b[2], fmaf(a.w, b[3], m[i]))));
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) sA[r + i][col] = pass ? -m[i] : m[i];
            __syncthreads();
        }
    }
    {
        const int r = 32 + tid / 16 * 4, col = tid % 16 * 2;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            float m[4][2] = {};
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                const int from = 32 * pass + k;
                float2 b[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) b[x] = *reinterpret_cast<const float2 *>(&sA[from + x][col]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 a = four(r + i, from);
                    m[i][0] = fmaf(a.x, b[0].x, fmaf(a.y, b[1].x, fmaf(a.z, b[2].x, fmaf(a.w, b[3].x, m[i][0]))));
                    m[i][1] = fmaf(a.x, b[0].y, fmaf(a.y, b[1].y, fmaf(a.z, b[2].y, fmaf(a.w, b[3].y, m[i][1]))));
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float2 *>(&sA[r + i][col]) = pass ? make_float2(-m[i][0], -m[i][1]) : make_float2(m[i][0], m[i][1]);
            __syncthreads();
        }
    }
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

// Shared memory of a chain block, 1024-byte aligned.  Only K, which is read from a step's first product to its
// last, has two buffers; the others are fetched again as soon as they have been read.
template <int NF, bool BWD> struct ChainSmem {
    static constexpr int kSlabs = (NF + 3) / 4, kTile = kSlabs * C * 64;
    static constexpr int kTermsP = BWD ? 3 : 2;
    bf16 K[2][kTile], Q[kTile];      // as the tensor maps leave them
    bf16 S[kSlabs][3][NV][64];       // the state's terms, lines in the same swizzle, as all of the following
    bf16 U[3][NV][64];               // e^{G_L-G} U; backwards e^G dO
    bf16 R[3][NV][64];               // beta Y; backwards dU, then -beta e^G dR
    bf16 W[2][NV][64];               // U, for O
    uint2 T[3][kUnits][32], P[kTermsP][kUnits][32];
    bf16 V[C][NV];                   // v, or do
    float gates[2][3][C];
    uint64_t bar[5];                 // K and gates (two), Q and V, T, P
};
enum { kBarK = 0, kBarV = 2, kBarT = 3, kBarP = 4 };
// Four warps carry the state from chunk to chunk, four more (where O is wanted) compute it beside them, one fetches.
// Bound by its latency: 3900 clocks a step of 64 tokens at d = 112, of which 1300 are the products' and 1700 shared memory's (every warp
// reads all of S's terms); one sequence of 8209 tokens, 20 heads: 344 us with k_prep.
constexpr int chain_threads(bool with_o) { return with_o ? 288 : 160; }

struct ChainMaps {
    CUtensorMap q, k, v;  // v: v, or do
};

// One thread's fetches, a handful of copies a chunk.  (As 16-byte copies by the threads they were 900 address lookups a
// chunk in ldmatrix's way, and loads of T and P to registers made every ldmatrix wait for them: 6400 clocks a step against
// 3900.  A copy a row, 193 of them, takes 4000 clocks to issue.)
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
        if (w.drop != 1 || blockIdx.x) tile(sm.K[b], &maps.k, bar, row);
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
        if (w.drop != 2 || blockIdx.x) sm100::bulk_copy_g2s(sm.T, src, sizeof(sm.T), &sm.bar[kBarT]);
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
__device__ __forceinline__ void chain_init(uint64_t (&bar)[5]) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < 5; ++i) sm100::mbar_init(&bar[i], 1);
        sm100::fence_barrier_init();
    }
    __syncthreads();
}
// A block that gave up leaves no copy in flight: the last copy of every barrier is waited for once more.  k_turn, p_turn: the
// last steps whose K and P were fetched (-1: no P).
template <int NF, bool BWD>
__device__ __forceinline__ void chain_leave(ChainSmem<NF, BWD> &sm, const SeqProblem &p, long long turn, long long k_turn, long long p_turn, int *err) {
    const uint32_t now = (uint32_t)turn & 1;
    sm100::mbar_wait(&sm.bar[kBarK + (k_turn & 1)], (uint32_t)(k_turn >> 1) & 1, err, sm100::kWaitLimitNs, true);
    sm100::mbar_wait(&sm.bar[kBarV], now, err, sm100::kWaitLimitNs, true);
    sm100::mbar_wait(&sm.bar[kBarT], now, err, sm100::kWaitLimitNs, true);
    if (p_turn >= 0) sm100::mbar_wait(&sm.bar[kBarP], (uint32_t)p_turn & 1, err, sm100::kWaitLimitNs, true);
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
    const uint32_t at = planes + lane / 4 * 128 + 4 * (lane & 3), x0 = ((2 * warp) ^ (lane / 4)) << 4;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (warp + 4 * m >= NF) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[3];
            split(st.x[m][i / 2][2 * (i & 1)], st.x[m][i / 2][2 * (i & 1) + 1], t);
#pragma unroll
            for (int e = 0; e < 3; ++e) sts(at + (x0 ^ (i / 2 * 16)) + (3 * m + e) * kPlane + (i & 1) * 1024, t[e]);
        }
    }
}
// The address of a lane's pairs of tokens (tile t, rows n and n + 8) in planes of 64 tokens.
__device__ __forceinline__ uint32_t pair_addr(uint32_t planes, int t, int lane) {
    return planes + lane / 4 * 128 + ((t ^ (lane / 4)) << 4) + 4 * (lane & 3);
}
template <int N> __device__ __forceinline__ void put_pair(uint32_t at, int half, float x, float y) {
    uint32_t t[N];
    split(x, y, t);
#pragma unroll
    for (int e = 0; e < N; ++e) sts(at + e * kPlane + half * 1024, t[e]);
}
// st = decay st + sum over the planes pl: (plane's 3 terms [16][64 tokens]) x (rows [64 tokens][dk]).
// Here and below the next step's fragments are loaded before a step's products: left to the compiler, each
// step waited for its own loads (840 clocks for 48 products a warp).
template <int NF, int SETS>
__device__ __forceinline__ void update_state(StateRows<NF> &st, float decay, const uint32_t (&planes)[SETS], const uint32_t (&rows)[SETS],
                                             int warp, int lane) {
    float hi[2][2][4], lo[2][2][4];
    uint32_t a[2][3][4], b[2][2][4];
    const uint32_t b0 = bt_lane(C, 16 * warp, lane), b1 = bt_lane(C, 16 * (warp + 4), lane);
    uint32_t al[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) al[x] = a_lane(x, lane);
    auto load = [&](int i) {
        const int s = i / 4, kb = i % 4;
#pragma unroll
        for (int e = 0; e < 3; ++e) ldsm4(a[i & 1][e], planes[s] + al[kb] + e * kPlane);
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
    uint32_t a[2][TERMS][4], b[2][4], al[4], bl[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) al[x] = planes + a_lane(x, lane), bl[x] = rows + b_lane(8 * t0, 8 * t1, x, lane);
    auto load = [&](int ks) {
#pragma unroll
        for (int e = 0; e < TERMS; ++e) ldsm4(a[ks & 1][e], al[ks & 3] + (3 * (ks >> 2) + e) * kPlane);
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
// LOW: T as it is; else its transpose.  TRANS: one plane, held [64 tokens][16].
template <bool LOW, int AT, int BT, bool TRANS = false>
__device__ __forceinline__ void times_triangle(float (&hi)[2][4], float (&lo)[2][2][4], uint32_t planes, uint32_t tri, int t0, int t1,
                                               int lane) {
    const int n0 = LOW ? t0 / 2 + 1 : 4 - t0 / 2, n1 = LOW ? t1 / 2 + 1 : 4 - t1 / 2;  // n0 <= 2, n1 >= 3
    uint32_t a[2][AT][4];
    uint2 f0[2][BT], f1[2][BT];
    const uint32_t src0 = tri_addr<LOW>(tri, t0, lane), src1 = tri_addr<LOW>(tri, t1, lane);
    auto load = [&](int m) {
#pragma unroll
        for (int e = 0; e < AT; ++e) {
            const int x = LOW ? m : 3 - m;
            if (TRANS) ldsm4_t(a[m & 1][e], planes + at_lane(NV, lane) + x * 16 * NV * 2);
            else ldsm4(a[m & 1][e], planes + a_lane(x, lane) + e * kPlane);
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
    constexpr int DK = 16 * NF, kSlabs = (NF + 3) / 4;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<ChainSmem<NF, false> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const uint32_t aS = sm100::smem_u32(sm.S), aU = sm100::smem_u32(sm.U), aR = sm100::smem_u32(sm.R), aT = sm100::smem_u32(sm.T),
                   aP = sm100::smem_u32(sm.P);
    const int groups = p.dv / NV, next = w.order[blockIdx.x / (p.H * groups)], h = blockIdx.x / groups % p.H, c0 = blockIdx.x % groups * NV;
    const int hk = h / (p.H / p.Hk), lane = threadIdx.x & 31, warp = warp_number();
    if (next < 0) {
        seq_report(p, GDN_SEQ_BAD_ROWS, h == 0 && c0 == 0 && threadIdx.x == 0);
        return no_state(p, -1 - next, h, c0, NV);
    }
    const int s = next;
    const SeqRange r = seq_place(p, s, w.good);
    seq_report(p, r.bad, h == 0 && c0 == 0 && threadIdx.x == 0);
    if (r.slot < 0 || r.len < p.min_len) return;
    const long long n_chunks = seq_chunks_of(r.len), base = seq_chunk_base(p, s, r.first);
    const size_t soff = (((size_t)r.slot * p.H + h) * p.dv + c0) * DK;
    const ChainFetch<NF, false> fetch = {sm, maps, w, hk, h, c0};
    constexpr int kFetchWarp = SAVE ? 4 : 8;
    const bool fetcher = threadIdx.x == 32 * kFetchWarp;
    auto index = [&](long long c) { return (size_t)(base + c) * p.H + h; };
    auto first_row = [&](long long c) { return (int)(r.first + c * C); };
    chain_init(sm.bar);
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
        ok = ok && sm100::mbar_wait(&sm.bar[kBarK + b], (uint32_t)(c >> 1) & 1, w.err, w.wait_ns) && sm100::mbar_wait(&sm.bar[kBarV], parity, w.err, w.wait_ns);
        // behind this barrier the state's terms are there and the last step's buffers have been read
        if (!__syncthreads_and(ok)) return chain_leave(sm, p, c, c, SAVE ? -1 : c - 1, w.err);
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
        const long long k_turn = c + 1 < n_chunks ? c + 1 : c;
        if (warp == kFetchWarp) {  // it keeps the barriers' count
            if (!__syncthreads_and(true)) return chain_leave(sm, p, c, k_turn, SAVE ? -1 : c, w.err);
            if (fetcher && c + 1 < n_chunks) fetch.v(first_row(c + 1), !SAVE);
            __syncthreads();
            if (fetcher && c + 1 < n_chunks) fetch.t(w.T + index(c + 1) * 3 * kUnits * 32);
            continue;
        }
        if (warp >= 4) {  // O^T = e^G S Q^T + U^T P^T
            float qh[2][4], ql[2][4], oh[2][4], ol[2][2][4];
            state_times<NF, 2>(qh, ql, aS, sm100::smem_u32(sm.Q), t0, t1, lane);
            ok = sm100::mbar_wait(&sm.bar[kBarP], parity, w.err, w.wait_ns);
            if (!__syncthreads_and(ok)) return chain_leave(sm, p, c, k_turn, c, w.err);
            __syncthreads();
            times_triangle<true, 2, 2>(oh, ol, sm100::smem_u32(sm.W), aP, t0, t1, lane);
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
            st.each(warp, lane, [&](int n, int k, float &x, float &y) {
                *reinterpret_cast<float2 *>(w.Sig + (idx * p.dv + c0 + n) * DK + k) = make_float2(x, y);
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
        ok = sm100::mbar_wait(&sm.bar[kBarT], parity, w.err, w.wait_ns);
        if (!__syncthreads_and(ok)) return chain_leave(sm, p, c, k_turn, SAVE ? -1 : c, w.err);
        // U^T = (beta Y)^T T^T
        float uh[2][4], ul[2][2][4];
        times_triangle<true, 3, 3>(uh, ul, aR, aT, t0, t1, lane);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 el = *reinterpret_cast<const float2 *>(&sm.gates[b][1][tok]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = lane / 4 + 8 * half, i = 2 * half;
                const float x = uh[t][i] + (ul[t][0][i] + ul[t][1][i]), y = uh[t][i + 1] + (ul[t][0][i + 1] + ul[t][1][i + 1]);
                put_pair<3>(pair_addr(aU, t ? t1 : t0, lane), half, el.x * x, el.y * y);
                if (SAVE) *reinterpret_cast<float2 *>(w.U + (idx * p.dv + c0 + n) * C + tok) = make_float2(x, y);
                else put_pair<2>(pair_addr(sm100::smem_u32(sm.W), t ? t1 : t0, lane), half, x, y);
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
}

template <int NF>
__global__ void __launch_bounds__(chain_threads(false), 1) k_chunk_bwd(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                                                const __grid_constant__ ChainMaps maps) {
    constexpr int DK = 16 * NF, kSlabs = (NF + 3) / 4;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<ChainSmem<NF, true> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const uint32_t aS = sm100::smem_u32(sm.S), aU = sm100::smem_u32(sm.U), aR = sm100::smem_u32(sm.R), aT = sm100::smem_u32(sm.T),
                   aP = sm100::smem_u32(sm.P);
    const int groups = p.dv / NV, next = w.order[blockIdx.x / (p.H * groups)], h = blockIdx.x / groups % p.H, c0 = blockIdx.x % groups * NV;
    const int hk = h / (p.H / p.Hk), lane = threadIdx.x & 31, warp = warp_number();
    if (next < 0) return;  // the forward walk has written its dS_in
    const int s = next;
    const SeqRange r = seq_rows(p, s);
    const size_t soff = (((size_t)s * p.H + h) * p.dv + c0) * DK;
    const long long n_chunks = seq_chunks_of(r.len), base = seq_chunk_base(p, s, r.first);  // 0 of a bad range
    const ChainFetch<NF, true> fetch = {sm, maps, w, hk, h, c0};
    const bool fetcher = threadIdx.x == 128;
    auto index = [&](long long c) { return (size_t)(base + c) * p.H + h; };
    auto first_row = [&](long long c) { return (int)(r.first + c * C); };
    chain_init(sm.bar);
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
        ok = ok && sm100::mbar_wait(&sm.bar[kBarK + b], (uint32_t)(turn >> 1) & 1, w.err, w.wait_ns) &&
             sm100::mbar_wait(&sm.bar[kBarV], parity, w.err, w.wait_ns) && sm100::mbar_wait(&sm.bar[kBarP], parity, w.err, w.wait_ns);
        if (!__syncthreads_and(ok)) return chain_leave(sm, p, turn, turn, turn, w.err);
        if (fetcher && c > 0) fetch.k(b ^ 1, first_row(c - 1), index(c - 1));
        if (rows < C) {
            zero_tail(sm.K[b], kSlabs, 8, rows);
            zero_tail(sm.Q, kSlabs, 8, rows);
            zero_tail(&sm.V[0][0], 1, NV / 8, rows);
            __syncthreads();
        }
        const long long k_turn = c > 0 ? turn + 1 : turn;
        if (warp == 4) {
            if (!__syncthreads_and(true)) return chain_leave(sm, p, turn, k_turn, turn, w.err);
            if (fetcher && c > 0) fetch.v(first_row(c - 1), false);
            __syncthreads();
            if (fetcher && c > 0) fetch.t(w.Tt + index(c - 1) * 3 * kUnits * 32);
            __syncthreads();
            __syncthreads();
            if (fetcher && c > 0) fetch.p(w.Pt + index(c - 1) * 3 * kUnits * 32, first_row(c - 1), true);
            continue;
        }
        st.each(warp, lane, [&](int n, int k, float &x, float &y) {
            *reinterpret_cast<float2 *>(w.D + (idx * p.dv + c0 + n) * DK + k) = make_float2(x, y);
        });
        // D^T K^T, and dO^T P
        float zh[2][4], zl[2][4], ph[2][4], pl[2][2][4];
        state_times<NF, 3>(zh, zl, aS, sm100::smem_u32(sm.K[b]), t0, t1, lane);
        times_triangle<false, 1, 3, true>(ph, pl, sm100::smem_u32(sm.V), aP, t0, t1, lane);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 el = *reinterpret_cast<const float2 *>(&sm.gates[b][1][tok]);
            const float2 eg = *reinterpret_cast<const float2 *>(&sm.gates[b][0][tok]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int n = lane / 4 + 8 * half, i = 2 * half;
                const float zx = el.x * (zh[t][i] + zl[t][i]), zy = el.y * (zh[t][i + 1] + zl[t][i + 1]);
                *reinterpret_cast<float2 *>(w.Z + (idx * p.dv + c0 + n) * C + tok) = make_float2(zx, zy);
                put_pair<3>(pair_addr(aR, t ? t1 : t0, lane), half, zx + (ph[t][i] + (pl[t][0][i] + pl[t][1][i])),
                            zy + (ph[t][i + 1] + (pl[t][0][i + 1] + pl[t][1][i + 1])));  // dU
                put_pair<3>(pair_addr(aU, t ? t1 : t0, lane), half, eg.x * __bfloat162float(sm.V[tok][n]),
                            eg.y * __bfloat162float(sm.V[tok + 1][n]));
            }
        }
        ok = sm100::mbar_wait(&sm.bar[kBarT], parity, w.err, w.wait_ns);
        if (!__syncthreads_and(ok)) return chain_leave(sm, p, turn, k_turn, turn, w.err);
        // dR^T = dU^T T
        float rh[2][4], rl[2][2][4];
        times_triangle<false, 3, 3>(rh, rl, aR, aT, t0, t1, lane);
        __syncthreads();  // dU has been read: -beta e^G dR takes its place
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 8 * (t ? t1 : t0) + 2 * (lane & 3);
            const float2 eg = *reinterpret_cast<const float2 *>(&sm.gates[b][0][tok]);
            const float2 be = *reinterpret_cast<const float2 *>(&sm.gates[b][2][tok]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = 2 * half;
                float x = rh[t][i] + (rl[t][0][i] + rl[t][1][i]), y = rh[t][i + 1] + (rl[t][0][i + 1] + rl[t][1][i + 1]);
                *reinterpret_cast<float2 *>(w.dR + (idx * p.dv + c0 + lane / 4 + 8 * half) * C + tok) = make_float2(x, y);
                x *= be.x;
                y *= be.y;
                put_pair<3>(pair_addr(aR, t ? t1 : t0, lane), half, -eg.x * x, -eg.y * y);
                // dV: as with O, pairs of columns
                const bool odd = lane & 4;
                const float other = __shfl_xor_sync(0xffffffffu, odd ? x : y, 4);
                const int at = tok + odd, n = (lane / 4 & ~1) + 8 * half;
                if (at < rows)
                    *reinterpret_cast<uint32_t *>((bf16 *)p.dv_out + ((row + at) * p.H + h) * p.dv + c0 + n) =
                        odd ? pack(other, y) : pack(x, other);
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
}

// ---------------------------------------------------------------- a warp a slice
// The same walks with a warp for each 16 columns and no exchange between warps: a product's result lies in a lane as
// the next product's A operand does (rows n, pairs along k), so S, beta Y, U, dU and dR stay in registers from
// product to product and shared memory holds only what all slices read: K, Q, T, P and v (a step and slice takes a quarter of
// the shared memory reads of k_chunk_fwd).  16384 tokens in 24 sequences, 20 heads, d = 112: 297 us (97 GFLOP executed in 628 products
// a step and slice, 56 % of the warp products' rate of 1024 multiply-adds a clock and SM), against 492 us.  A block has up to four
// slices of one sequence and head; one of its threads fetches.
constexpr int kSlices = 4;
// eight warps an SM, two blocks, leave a thread its 255 registers (d_k = 112 and 128 spill 8 to 88 bytes)
constexpr int kWalkThreads = 32 * kSlices;

template <int NF, bool BWD> struct WalkSmem {  // 1024-byte aligned
    static constexpr int kSlabs = (NF + 3) / 4, kTile = kSlabs * C * 64, kTermsP = BWD ? 3 : 2;
    bf16 K[2][kTile], Q[kTile];
    bf16 V[C * 64];  // the block's 64 columns of v, or do
    uint2 T[3][kUnits][32], P[kTermsP][kUnits][32];
    float gates[2][3][C];
    uint64_t bar[5];
};

template <int NF, bool BWD> struct WalkFetch {
    WalkSmem<NF, BWD> &sm;
    const ChainMaps &maps;  // v, or do, in boxes of 64 columns
    const ChunkWork &w;
    int hk, h, c0;
    static constexpr uint32_t kTileBytes = WalkSmem<NF, BWD>::kTile * 2;
    __device__ __forceinline__ void tile(bf16 *dst, const CUtensorMap *map, uint64_t *bar, int row) const {
#pragma unroll
        for (int c = 0; c < 16 * NF; c += 64) sm100::tma_load_3d(dst + c * C, map, bar, c, hk, row);
    }
    __device__ __forceinline__ void k(int b, int row, size_t idx) const {  // and the gates
        uint64_t *bar = &sm.bar[kBarK + b];
        sm100::mbar_arrive_expect_tx(bar, kTileBytes + 3 * C * 4);
        if (w.drop != 1 || blockIdx.x) tile(sm.K[b], &maps.k, bar, row);
        sm100::bulk_copy_g2s(&sm.gates[b][0][0], w.gates + idx * 3 * C, 3 * C * 4, bar);
    }
    __device__ __forceinline__ void t(const uint2 *src) const {
        sm100::mbar_arrive_expect_tx(&sm.bar[kBarT], sizeof(sm.T));
        if (w.drop != 2 || blockIdx.x) sm100::bulk_copy_g2s(sm.T, src, sizeof(sm.T), &sm.bar[kBarT]);
    }
    // forwards (not SAVE): Q and P, read at a step's end.  Backwards Q alone.
    __device__ __forceinline__ void qp(const uint2 *src, int row) const {
        sm100::mbar_arrive_expect_tx(&sm.bar[kBarP], kTileBytes + (BWD ? 0 : sizeof(sm.P)));
        tile(sm.Q, &maps.q, &sm.bar[kBarP], row);
        if (!BWD) sm100::bulk_copy_g2s(sm.P, src, sizeof(sm.P), &sm.bar[kBarP]);
    }
    // v; backwards do and P
    __device__ __forceinline__ void v(const uint2 *src, int row) const {
        uint64_t *bar = &sm.bar[kBarV];
        sm100::mbar_arrive_expect_tx(bar, C * 128 + (BWD ? sizeof(sm.P) : 0));
        sm100::tma_load_3d(sm.V, &maps.v, bar, c0, h, row);
        if (BWD) sm100::bulk_copy_g2s(sm.P, src, sizeof(sm.P), bar);
    }
};

// Two tiles of a result (16 columns along k) as an A operand's terms.
template <int N> __device__ __forceinline__ void as_operand(uint32_t (&a)[N][4], const float (&x)[4], const float (&y)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float *s = (e & 2) ? y : x;
        uint32_t t[N];
        split(s[2 * (e & 1)], s[2 * (e & 1) + 1], t);
#pragma unroll
        for (int n = 0; n < N; ++n) a[n][e] = t[n];
    }
}

// hi (+ lo) = S rows^T, all eight token tiles; TERMS terms of S.  MERGE: one sum (what only reaches a bf16 output).
template <int NF, int TERMS, bool MERGE>
__device__ __forceinline__ void walk_state_times(float (&hi)[8][4], float (&lo)[MERGE ? 1 : 8][4], const float (&S)[2 * NF][4], uint32_t rows,
                                                 const uint32_t (&bl)[4]) {
#pragma unroll
    for (int ks = 0; ks < NF; ++ks) {
        uint32_t a[TERMS][4];
        as_operand<TERMS>(a, S[2 * ks], S[2 * ks + 1]);
#pragma unroll
        for (int t = 0; t < 8; t += 4) {
            uint32_t b[2][4];
            ldsm4(b[0], rows + bl[ks & 3] + (ks >> 2) * C * 128 + t * 1024);
            ldsm4(b[1], rows + bl[ks & 3] + (ks >> 2) * C * 128 + t * 1024 + 2048);
#pragma unroll
            for (int n = TERMS - 1; n >= 0; --n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float(&d)[4] = MERGE || n == 0 ? hi[t + i] : lo[MERGE ? 0 : t + i];
                    const bool first = ks == 0 && (MERGE ? n == TERMS - 1 : n == 0 || n == TERMS - 1);
                    mma::mma(d, a[n], b[i / 2][2 * (i & 1)], b[i / 2][2 * (i & 1) + 1], first);
                }
        }
    }
}

// hi, lo += a T for the 16-token block kb of the rows: the units of the tiles that hold it.  MERGE as above.
template <bool LOW, int AT, int BT, bool MERGE>
__device__ __forceinline__ void walk_triangle(float (&hi)[8][4], float (&lo)[MERGE ? 1 : 8][4], const uint32_t (&a)[AT][4], uint32_t tri, int kb) {
#pragma unroll
    for (int t2 = 0; t2 < 8; t2 += 2) {
        if (LOW ? t2 / 2 < kb : t2 / 2 > kb) continue;
        uint2 f[2][BT];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < BT; ++e) f[i][e] = lds2(tri + (e * kUnits + (LOW ? low_unit(t2 + i) + kb : up_unit(t2 + i) + kb - t2 / 2)) * 256);
#pragma unroll
        for (int k = (AT > BT ? AT : BT) - 1; k >= 0; --k)
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                const int y = k - x;
                if (y < 0 || y >= BT) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) mma::mma(MERGE || k == 0 ? hi[t2 + i] : lo[MERGE ? 0 : t2 + i], a[x], f[i][y].x, f[i][y].y);
            }
    }
}

// S += a rows, a: four 16-token blocks' terms, rows [64 tokens][dk].
template <int NF>
__device__ __forceinline__ void walk_update(float (&S)[2 * NF][4], const uint32_t (&a)[4][3][4], uint32_t rows, int lane) {
#pragma unroll
    for (int g = 0; g < NF; ++g) {
        float hi[2][4], lo[2][4];
        const uint32_t at = rows + bt_lane(C, 16 * g, lane);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
            uint32_t b[4];
            ldsm4_t(b, at + kb * 2048);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(lo[t], a[kb][2], b[2 * t], b[2 * t + 1], kb == 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(hi[t], a[kb][0], b[2 * t], b[2 * t + 1], kb == 0);
#pragma unroll
            for (int t = 0; t < 2; ++t) mma::mma(lo[t], a[kb][1], b[2 * t], b[2 * t + 1]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[2 * g + t][e] += hi[t][e] + lo[t][e];
    }
}

// A warp's columns of v or do [64 tokens][64]: x[t][half] is a pair of tokens of tile t, row n or n + 8.
__device__ __forceinline__ void walk_columns(uint32_t (&x)[8][2], uint32_t tile, int slice, int lane) {
    // blocks (tile t, n 0-7), (t, n 8-15), (t + 1, n 0-7), (t + 1, n 8-15)
    const uint32_t at = tile + ((lane >> 4) * 8 + (lane & 7)) * 128 + (((2 * slice + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
#pragma unroll
    for (int t = 0; t < 8; t += 2) {
        uint32_t r[4];
        ldsm4_t(r, at + t * 1024);
        x[t][0] = r[0];
        x[t][1] = r[1];
        x[t + 1][0] = r[2];
        x[t + 1][1] = r[3];
    }
}

// bf16 rows of [tokens][H][dv] from x[t]: lanes of neighbouring rows swap, so that each writes a pair of columns.
__device__ __forceinline__ void walk_store(bf16 *dst, long long row_elems, const float (&x)[8][4], int rows, int lane) {
    const bool odd = lane & 4;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float mine = odd ? x[t][2 * half + 1] : x[t][2 * half];
            const float other = __shfl_xor_sync(0xffffffffu, odd ? x[t][2 * half] : x[t][2 * half + 1], 4);
            const int i = 8 * t + 2 * (lane & 3) + odd, n = (lane / 4 & ~1) + 8 * half;
            if (i < rows) *reinterpret_cast<uint32_t *>(dst + i * row_elems + n) = odd ? pack(other, mine) : pack(mine, other);
        }
}

// Which slice a thread's warp walks.
struct WalkPlace {
    int s, h, hk, c0, slice, slices;  // c0: the block's first column; slices: how many the block has
    bool late;
};
__device__ __forceinline__ WalkPlace walk_place(const SeqProblem &p, const int *order) {
    const int groups = (p.dv + 16 * kSlices - 1) / (16 * kSlices);
    WalkPlace x;
    const int next = order[blockIdx.x / (p.H * groups)];
    x.late = next < 0;
    x.s = x.late ? -1 - next : next;
    x.h = blockIdx.x / groups % p.H;
    x.hk = x.h / (p.H / p.Hk);
    x.c0 = blockIdx.x % groups * 16 * kSlices;
    x.slice = warp_number();
    x.slices = min(kSlices, (p.dv - x.c0) / 16);
    return x;
}
template <typename Smem> __device__ __forceinline__ void walk_leave(Smem &sm, const SeqProblem &p, const int (&last)[5], int *err) {
    for (int i = 0; i < 5; ++i)  // the last fetch of each barrier, if it had one
        if (last[i] >= 0) sm100::mbar_wait(&sm.bar[i], last[i] & 1, err, sm100::kWaitLimitNs, true);
    if (p.status && threadIdx.x == 0) atomicOr(p.status, GDN_SEQ_TIMEOUT);
}

template <int NF, bool SAVE>
__global__ void __launch_bounds__(kWalkThreads, 2) k_walk_fwd(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                                              const __grid_constant__ ChainMaps maps) {
    constexpr int DK = 16 * NF, kSlabs = (NF + 3) / 4;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<WalkSmem<NF, false> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const WalkPlace at = walk_place(p, w.order);
    const int lane = threadIdx.x & 31, n0 = lane / 4, j0 = 2 * (lane & 3), col = at.c0 + 16 * at.slice;
    if (at.late) {
        seq_report(p, GDN_SEQ_BAD_ROWS, at.h == 0 && at.c0 == 0 && threadIdx.x == 0);
        return no_state(p, at.s, at.h, at.c0, 16 * at.slices);
    }
    const SeqRange r = seq_place(p, at.s, w.good);
    seq_report(p, r.bad, at.h == 0 && at.c0 == 0 && threadIdx.x == 0);
    if (r.slot < 0 || r.len < p.min_len) return;
    const long long n_chunks = seq_chunks_of(r.len), base = seq_chunk_base(p, at.s, r.first);
    const WalkFetch<NF, false> fetch = {sm, maps, w, at.hk, at.h, at.c0};
    const bool fetcher = threadIdx.x == 0, walks = at.slice < at.slices;
    auto index = [&](long long c) { return (size_t)(base + c) * p.H + at.h; };
    auto first_row = [&](long long c) { return (int)(r.first + c * C); };
    chain_init(sm.bar);
    if (fetcher && n_chunks > 0) {
        fetch.k(0, first_row(0), index(0));
        fetch.v(nullptr, first_row(0));
        fetch.t(w.T + index(0) * 3 * kUnits * 32);
        if (!SAVE) fetch.qp(w.P + index(0) * 2 * kUnits * 32, first_row(0));
    }
    float S[2 * NF][4] = {};
    float *const s_out = p.S_out + (((size_t)r.slot * p.H + at.h) * p.dv + col + n0) * DK + j0;
    if (walks && !seq_starts_zero(p, at.s)) {
        const float *s_in = p.S_in + (((size_t)r.slot * p.H + at.h) * p.dv + col + n0) * DK + j0;
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 x = *reinterpret_cast<const float2 *>(s_in + half * 8 * DK + 8 * t);
                S[t][2 * half] = x.x;
                S[t][2 * half + 1] = x.y;
            }
    }
    uint32_t bl[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) bl[x] = b_lane(0, 8, x, lane);
    const uint32_t aT = sm100::smem_u32(sm.T) + lane * 8, aP = sm100::smem_u32(sm.P) + lane * 8;
    bool ok = true;
#pragma unroll 1
    for (long long c = 0; c < n_chunks; ++c) {
        const int b = (int)(c & 1);
        const uint32_t parity = (uint32_t)c & 1;
        const size_t idx = index(c);
        const long long row = r.first + c * C;
        const int rows = (int)min((long long)C, r.len - c * C);
        ok = ok && sm100::mbar_wait(&sm.bar[kBarK + b], (uint32_t)(c >> 1) & 1, w.err, w.wait_ns) && sm100::mbar_wait(&sm.bar[kBarV], parity, w.err, w.wait_ns) &&
             sm100::mbar_wait(&sm.bar[kBarT], parity, w.err, w.wait_ns) && (SAVE || sm100::mbar_wait(&sm.bar[kBarP], parity, w.err, w.wait_ns));
        if (!__syncthreads_and(ok)) {
            const int last[5] = {(int)((c - (c & 1)) >> 1), c ? (int)((c - !(c & 1)) >> 1) : -1, (int)c, (int)c, SAVE ? -1 : (int)c};
            return walk_leave(sm, p, last, w.err);
        }
        if (fetcher && c + 1 < n_chunks) fetch.k(b ^ 1, first_row(c + 1), index(c + 1));
        if (rows < C) {
            zero_tail(sm.K[b], kSlabs, 8, rows);
            if (!SAVE) zero_tail(sm.Q, kSlabs, 8, rows);
            zero_tail(sm.V, 1, 8, rows);
            __syncthreads();
        }
        if (!walks) {  // it keeps the barriers' count
            __syncthreads();
            __syncthreads();
            continue;
        }
        const uint32_t aK = sm100::smem_u32(sm.K[b]);
        const float *eg = sm.gates[b][0] + j0, *el = sm.gates[b][1] + j0, *be = sm.gates[b][2] + j0;
        if (SAVE) {
#pragma unroll
            for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    *reinterpret_cast<float2 *>(w.Sig + (idx * p.dv + col + n0 + 8 * half) * DK + 8 * t + j0) =
                        make_float2(S[t][2 * half], S[t][2 * half + 1]);
        }
        float R[8][4];
        {
            float lo[8][4];
            uint32_t v[8][2];
            walk_state_times<NF, 3, false>(R, lo, S, aK, bl);
            walk_columns(v, sm100::smem_u32(sm.V), at.slice, lane);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 g = *reinterpret_cast<const float2 *>(eg + 8 * t), h = *reinterpret_cast<const float2 *>(be + 8 * t);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float x = g.x * (R[t][2 * half] + lo[t][2 * half]), y = g.y * (R[t][2 * half + 1] + lo[t][2 * half + 1]);
                    if (SAVE) *reinterpret_cast<float2 *>(w.X + (idx * p.dv + col + n0 + 8 * half) * C + 8 * t + j0) = make_float2(x, y);
                    R[t][2 * half] = h.x * (low_of(v[t][half]) - x);
                    R[t][2 * half + 1] = h.y * (high_of(v[t][half]) - y);
                }
            }
        }
        float U[8][4];
        {
            float lo[8][4];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) U[t][e] = lo[t][e] = 0.f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t a[3][4];
                as_operand<3>(a, R[2 * kb], R[2 * kb + 1]);
                walk_triangle<true, 3, 3, false>(U, lo, a, aT, kb);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) U[t][e] += lo[t][e];
        }
        __syncthreads();  // v and T have been read
        if (fetcher && c + 1 < n_chunks) {
            fetch.v(nullptr, first_row(c + 1));
            fetch.t(w.T + index(c + 1) * 3 * kUnits * 32);
        }
        if (SAVE) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    *reinterpret_cast<float2 *>(w.U + (idx * p.dv + col + n0 + 8 * half) * C + 8 * t + j0) =
                        make_float2(U[t][2 * half], U[t][2 * half + 1]);
        } else {
            float O[8][4], none[1][4];
            walk_state_times<NF, 2, true>(O, none, S, sm100::smem_u32(sm.Q), bl);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 g = *reinterpret_cast<const float2 *>(eg + 8 * t);
#pragma unroll
                for (int e = 0; e < 4; ++e) O[t][e] *= e & 1 ? g.y : g.x;
            }
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t a[2][4];
                as_operand<2>(a, U[2 * kb], U[2 * kb + 1]);
                walk_triangle<true, 2, 2, true>(O, none, a, aP, kb);
            }
            walk_store((bf16 *)p.o + (row * p.H + at.h) * p.dv + col, (long long)p.H * p.dv, O, rows, lane);
        }
        __syncthreads();  // Q and P have been read
        if (!SAVE && fetcher && c + 1 < n_chunks) fetch.qp(w.P + index(c + 1) * 2 * kUnits * 32, first_row(c + 1));
        uint32_t a[4][3][4];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float2 g = *reinterpret_cast<const float2 *>(el + 8 * t);
#pragma unroll
            for (int e = 0; e < 4; ++e) U[t][e] *= e & 1 ? g.y : g.x;
        }
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) as_operand<3>(a[kb], U[2 * kb], U[2 * kb + 1]);
        const float decay = sm.gates[b][0][C - 1];
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[t][e] *= decay;
        walk_update<NF>(S, a, aK, lane);
    }
    if (!SAVE && p.S_out && walks) {
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                *reinterpret_cast<float2 *>(s_out + half * 8 * DK + 8 * t) = make_float2(S[t][2 * half], S[t][2 * half + 1]);
    }
}

template <int NF>
__global__ void __launch_bounds__(kWalkThreads, 2) k_walk_bwd(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                                              const __grid_constant__ ChainMaps maps) {
    constexpr int DK = 16 * NF, kSlabs = (NF + 3) / 4;
    extern __shared__ unsigned char raw[];
    auto &sm = *reinterpret_cast<WalkSmem<NF, true> *>(raw + (-sm100::smem_u32(raw) & 1023));
    const WalkPlace at = walk_place(p, w.order);
    const int lane = threadIdx.x & 31, n0 = lane / 4, j0 = 2 * (lane & 3), col = at.c0 + 16 * at.slice;
    if (at.late) return;  // the forward walk has written its dS_in
    const SeqRange r = seq_rows(p, at.s);
    const long long n_chunks = seq_chunks_of(r.len), base = seq_chunk_base(p, at.s, r.first);  // 0 of a bad range
    const WalkFetch<NF, true> fetch = {sm, maps, w, at.hk, at.h, at.c0};
    const bool fetcher = threadIdx.x == 0, walks = at.slice < at.slices;
    auto index = [&](long long c) { return (size_t)(base + c) * p.H + at.h; };
    auto first_row = [&](long long c) { return (int)(r.first + c * C); };
    chain_init(sm.bar);
    if (fetcher && n_chunks > 0) {
        const long long c = n_chunks - 1;
        fetch.k(0, first_row(c), index(c));
        fetch.v(w.Pt + index(c) * 3 * kUnits * 32, first_row(c));
        fetch.t(w.Tt + index(c) * 3 * kUnits * 32);
        fetch.qp(nullptr, first_row(c));
    }
    float D[2 * NF][4] = {};
    const size_t soff = (((size_t)at.s * p.H + at.h) * p.dv + col + n0) * DK + j0;
    if (walks && r.slot >= 0 && p.dS_out) {
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float2 x = *reinterpret_cast<const float2 *>(p.dS_out + soff + half * 8 * DK + 8 * t);
                D[t][2 * half] = x.x;
                D[t][2 * half + 1] = x.y;
            }
    }
    uint32_t bl[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) bl[x] = b_lane(0, 8, x, lane);
    const uint32_t aT = sm100::smem_u32(sm.T) + lane * 8, aP = sm100::smem_u32(sm.P) + lane * 8;
    bool ok = true;
#pragma unroll 1
    for (long long turn = 0; turn < n_chunks; ++turn) {
        const long long c = n_chunks - 1 - turn;
        const int b = (int)(turn & 1);
        const uint32_t parity = (uint32_t)turn & 1;
        const size_t idx = index(c);
        const long long row = r.first + c * C;
        const int rows = (int)min((long long)C, r.len - c * C);
        ok = ok && sm100::mbar_wait(&sm.bar[kBarK + b], (uint32_t)(turn >> 1) & 1, w.err, w.wait_ns) && sm100::mbar_wait(&sm.bar[kBarV], parity, w.err, w.wait_ns) &&
             sm100::mbar_wait(&sm.bar[kBarT], parity, w.err, w.wait_ns) && sm100::mbar_wait(&sm.bar[kBarP], parity, w.err, w.wait_ns);
        if (!__syncthreads_and(ok)) {
            const int i = (int)turn, last[5] = {(i - (i & 1)) >> 1, i ? (i - !(i & 1)) >> 1 : -1, i, i, i};
            return walk_leave(sm, p, last, w.err);
        }
        if (fetcher && c > 0) fetch.k(b ^ 1, first_row(c - 1), index(c - 1));
        if (rows < C) {
            zero_tail(sm.K[b], kSlabs, 8, rows);
            zero_tail(sm.Q, kSlabs, 8, rows);
            zero_tail(sm.V, 1, 8, rows);
            __syncthreads();
        }
        if (!walks) {
            __syncthreads();
            __syncthreads();
            continue;
        }
        const uint32_t aK = sm100::smem_u32(sm.K[b]), aO = sm100::smem_u32(sm.V);
        const float *eg = sm.gates[b][0] + j0, *el = sm.gates[b][1] + j0, *be = sm.gates[b][2] + j0;
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                *reinterpret_cast<float2 *>(w.D + (idx * p.dv + col + n0 + 8 * half) * DK + 8 * t + j0) =
                    make_float2(D[t][2 * half], D[t][2 * half + 1]);
        float X[8][4];  // dU, then dR
        {
            float Z[8][4], lo[8][4];
            walk_state_times<NF, 3, false>(Z, lo, D, aK, bl);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 l = *reinterpret_cast<const float2 *>(el + 8 * t);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    Z[t][2 * half] = l.x * (Z[t][2 * half] + lo[t][2 * half]);
                    Z[t][2 * half + 1] = l.y * (Z[t][2 * half + 1] + lo[t][2 * half + 1]);
                    *reinterpret_cast<float2 *>(w.Z + (idx * p.dv + col + n0 + 8 * half) * C + 8 * t + j0) =
                        make_float2(Z[t][2 * half], Z[t][2 * half + 1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) X[t][e] = lo[t][e] = 0.f;
            }
            const uint32_t o_at = aO + ((lane >> 4) * 8 + (lane & 7)) * 128 + (((2 * at.slice + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t a[1][4];
                ldsm4_t(a[0], o_at + kb * 2048);
                walk_triangle<false, 1, 3, false>(X, lo, a, aP, kb);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) Z[t][e] += X[t][e] + lo[t][e], X[t][e] = lo[t][e] = 0.f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                uint32_t a[3][4];
                as_operand<3>(a, Z[2 * kb], Z[2 * kb + 1]);
                walk_triangle<false, 3, 3, false>(X, lo, a, aT, kb);
            }
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) X[t][e] += lo[t][e];
        }
        __syncthreads();  // T has been read
        if (fetcher && c > 0) fetch.t(w.Tt + index(c - 1) * 3 * kUnits * 32);
        uint32_t a[4][3][4];
        {  // (e^G dO)^T Q
            uint32_t v[8][2];
            walk_columns(v, aO, at.slice, lane);
            float x[8][4];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float2 g = *reinterpret_cast<const float2 *>(eg + 8 * t);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    x[t][2 * half] = g.x * low_of(v[t][half]);
                    x[t][2 * half + 1] = g.y * high_of(v[t][half]);
                }
            }
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) as_operand<3>(a[kb], x[2 * kb], x[2 * kb + 1]);
            const float decay = sm.gates[b][0][C - 1];
#pragma unroll
            for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) D[t][e] *= decay;
            walk_update<NF>(D, a, sm100::smem_u32(sm.Q), lane);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float2 h = *reinterpret_cast<const float2 *>(be + 8 * t);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                *reinterpret_cast<float2 *>(w.dR + (idx * p.dv + col + n0 + 8 * half) * C + 8 * t + j0) =
                    make_float2(X[t][2 * half], X[t][2 * half + 1]);
                X[t][2 * half] *= h.x;
                X[t][2 * half + 1] *= h.y;
            }
        }
        __syncthreads();  // do, P and Q have been read
        if (fetcher && c > 0) {
            fetch.v(w.Pt + index(c - 1) * 3 * kUnits * 32, first_row(c - 1));
            fetch.qp(nullptr, first_row(c - 1));
        }
        walk_store((bf16 *)p.dv_out + (row * p.H + at.h) * p.dv + col, (long long)p.H * p.dv, X, rows, lane);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float2 g = *reinterpret_cast<const float2 *>(eg + 8 * t);
#pragma unroll
            for (int e = 0; e < 4; ++e) X[t][e] *= e & 1 ? -g.y : -g.x;
        }
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) as_operand<3>(a[kb], X[2 * kb], X[2 * kb + 1]);
        walk_update<NF>(D, a, aK, lane);
    }
    if (p.dS_in && walks) {
#pragma unroll
        for (int t = 0; t < 2 * NF; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                *reinterpret_cast<float2 *>(p.dS_in + soff + half * 8 * DK + 8 * t) = make_float2(D[t][2 * half], D[t][2 * half + 1]);
    }
}

// The gradients of a chunk and head from what the chains left: 8 warps, warp w has the 16 tokens from 16 (w % 4).
// Warps 0-3 (role 0) make dQ, warps 4-7 dK, first the parts inside the chunk, then those through the states:
//   dQ = dP K + e^G dO Sig^T,  dK = (beta dA) K + [dP; beta dA]^T [Q; K] - beta e^G dR Sig^T + e^{G_L-G} U D^T
// Products that reach the gates' fp32 gradients are at fp32 accuracy (dP, dA, dO Sig^T: every term); those that only
// reach the bf16 dQ and dK take two terms of each operand.
// The fp32 matrices come by the copy engine (as the threads' loads they took most of the kernel's time), 64 columns a
// line, and a warp turns a line of 256 bytes into its first two terms in place.
struct GradMaps {
    CUtensorMap q, k, v, o, Sig, D;
};
// Shared memory, sizes from dv: K, Q, dO rows | U, dR | U's and dR's third terms, dP and beta dA (before them Z), M (before
// it v's rows), X where there is room; in the place of the third terms to M, when they have been read, 64 columns of Sig, of D
// and Sig's third terms.
template <int NF> struct GradLayout {
    static constexpr int kSlabs = (NF + 3) / 4, kTile = kSlabs * C * 128, kT = C * (16 * NF + 4) * 4, kPA = kT > 32768 ? kT : 32768;
    int plane, K, Q, O, UR, last, PA, M, X, total;  // X: 0 where it would not fit
    __host__ __device__ explicit GradLayout(int dv) {
        plane = dv * 128;
        K = 0;
        Q = K + kTile;
        O = Q + kTile;
        UR = O + 2 * C * 128;
        last = UR + 4 * plane;
        PA = last + 2 * plane;
        M = PA + kPA;
        X = M + C * (C + 4) * 4;  // 5 planes of Sig and D fit between `last` and X: 3 planes are at most 48 KB
        total = X + 2 * plane;
        if (total > 222 * 1024) {
            total = X;
            X = 0;
        }
    }
};

template <int NF>
__global__ void __launch_bounds__(256, 1) k_chunk_grads(const __grid_constant__ SeqProblem p, const __grid_constant__ ChunkWork w,
                                                        const __grid_constant__ GradMaps maps) {
    constexpr int DK = 16 * NF, kSlabs = (NF + 3) / 4, PM = C + 4;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(16) float gates[3][C];  // read in pairs
    __shared__ float into[C], past[C], db[C], sums[4][C], dg[C], red[8];
    __shared__ uint64_t bar[4];
    const long long c = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk), tid = threadIdx.x, lane = tid & 31, warp = warp_number();
    const int mt = warp & 3, role = warp >> 2, dv = p.dv, nvf = dv / 16;
    const SeqChunk ch = w.chunks[c];
    if (ch.rows == 0) return;
    const size_t idx = (size_t)c * p.H + h;
    const GradLayout<NF> at(dv);
    unsigned char *const sm = raw + (-sm100::smem_u32(raw) & 1023);
    const uint32_t base = sm100::smem_u32(sm), plane = at.plane;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) sm100::mbar_init(&bar[i], 1);
        sm100::fence_barrier_init();
    }
    __syncthreads();
    const float *Um = w.U + idx * dv * C, *Rm = w.dR + idx * dv * C, *Xm = w.X + idx * dv * C, *Zm = w.Z + idx * dv * C;
    if (tid == 32) {  // into L2 for later
        sm100::bulk_prefetch_l2(w.Sig + idx * dv * DK, dv * DK * 4);
        sm100::bulk_prefetch_l2(w.D + idx * dv * DK, dv * DK * 4);
        sm100::bulk_prefetch_l2(w.gam + idx * kUnits * 32, kUnits * 32 * 16);
    }
    if (tid == 0) {
        sm100::mbar_arrive_expect_tx(&bar[0], 2 * at.kTile + (dv + 63) / 64 * 2 * C * 128 + (at.X ? 8 : 6) * plane);
        sm100::bulk_copy_g2s(sm + at.UR, Um, 2 * plane, &bar[0]);
        sm100::bulk_copy_g2s(sm + at.UR + 2 * plane, Rm, 2 * plane, &bar[0]);
        sm100::bulk_copy_g2s(sm + at.PA, Zm, 2 * plane, &bar[0]);
        if (at.X) sm100::bulk_copy_g2s(sm + at.X, Xm, 2 * plane, &bar[0]);
        for (int x = 0; x < kSlabs; ++x) {
            sm100::tma_load_3d(sm + at.K + x * C * 128, &maps.k, &bar[0], 64 * x, hk, (int)ch.first);
            sm100::tma_load_3d(sm + at.Q + x * C * 128, &maps.q, &bar[0], 64 * x, hk, (int)ch.first);
        }
        for (int x = 0; x < (dv + 63) / 64; ++x) sm100::tma_load_3d(sm + at.O + x * C * 128, &maps.o, &bar[0], 64 * x, h, (int)ch.first);
        for (int x = 0; x < (dv + 63) / 64; ++x) sm100::tma_load_3d(sm + at.M + x * C * 128, &maps.v, &bar[0], 64 * x, h, (int)ch.first);
    }
    if (tid < 3 * C) gates[0][tid] = w.gates[idx * 3 * C + tid];
    const int i0 = 16 * mt + lane / 4, j0 = 2 * (lane & 3);  // this lane's rows i0, i0 + 8; its columns 8 t + j0, + 1
    if (!__syncthreads_and(sm100::mbar_wait(&bar[0], 0, w.err, w.wait_ns))) {
        sm100::mbar_wait(&bar[0], 0, w.err, sm100::kWaitLimitNs, true);
        if (p.status && tid == 0) atomicOr(p.status, GDN_SEQ_TIMEOUT);
        return;
    }
    if (ch.rows < C) {
        zero_tail((bf16 *)(sm + at.K), kSlabs, 8, ch.rows);
        zero_tail((bf16 *)(sm + at.Q), kSlabs, 8, ch.rows);
        zero_tail((bf16 *)(sm + at.O), (dv + 63) / 64, 8, ch.rows);
        zero_tail((bf16 *)(sm + at.M), (dv + 63) / 64, 8, ch.rows);
        __syncthreads();
    }
    // A warp's line n (64 columns, fp32) becomes its first two terms, and a third one of `third`'s lines where that is given.
    auto line_terms = [&](uint32_t line, int n, float2 x, uint32_t third) {
        uint32_t a[3];
        split(x.x, x.y, a);
        const uint32_t piece = ((lane >> 2 ^ (n & 7)) << 4) + (lane & 3) * 4;
        sts(line + piece, a[0]);
        sts(line + 128 + piece, a[1]);
        if (third) sts(third + piece, a[2]);
    };
    {  // U and dR, and the sums over dv: past = U . Z, into = -beta dR . X (k's part), db = dR . (V - X).  A pair of tokens a lane
        const float2 be = *reinterpret_cast<const float2 *>(&gates[2][2 * lane]);
        const float *Xs = at.X ? reinterpret_cast<const float *>(sm + at.X) : Xm;
        float s[3][2] = {};
#pragma unroll 2
        for (int n = warp; n < dv; n += 8) {
            const int from = n * C + 2 * lane;
            const float2 u = *reinterpret_cast<const float2 *>(sm + at.UR + from * 4), r = *reinterpret_cast<const float2 *>(sm + at.UR + 2 * plane + from * 4),
                         z = *reinterpret_cast<const float2 *>(sm + at.PA + from * 4), x = *reinterpret_cast<const float2 *>(Xs + from);
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                v[e] = __bfloat162float(*reinterpret_cast<const bf16 *>(sm + at.M + sw_byte(C, 2 * lane + e, n) + (n & 7) * 2));
            __syncwarp();
            line_terms(base + at.UR + n * 256, n, u, base + at.last + n * 128);
            line_terms(base + at.UR + 2 * plane + n * 256, n, r, base + at.last + plane + n * 128);
            s[0][0] = fmaf(u.x, z.x, s[0][0]);
            s[0][1] = fmaf(u.y, z.y, s[0][1]);
            s[1][0] = fmaf(-be.x * r.x, x.x, s[1][0]);
            s[1][1] = fmaf(-be.y * r.y, x.y, s[1][1]);
            s[2][0] = fmaf(r.x, v[0] - x.x, s[2][0]);
            s[2][1] = fmaf(r.y, v[1] - x.y, s[2][1]);
        }
        sm100::fence_proxy_async_smem();
        __syncthreads();  // the terms are there; X, Z and v have been read
        float *sum = reinterpret_cast<float *>(sm + at.PA);  // [8][3][64]
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<float2 *>(sum + (warp * 3 + i) * C + 2 * lane) = make_float2(s[i][0], s[i][1]);
        if (tid == 0 && at.X) {  // X has been read: the first columns of Sig take its place
            sm100::mbar_arrive_expect_tx(&bar[1], 2 * plane);
            sm100::tma_load_2d(sm + at.X, &maps.Sig, &bar[1], 0, (int)(idx * dv));
        }
        __syncthreads();
        if (tid < 3 * C) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x += sum[i * 3 * C + tid];
            (tid < C ? past : tid < 2 * C ? into : db)[tid % C] = x;
        }
        __syncthreads();
    }
    const uint32_t aK = base + at.K, aQ = base + at.Q, aO = base + at.O;
    // lane parts: an A operand from token rows; from [dv][64 tokens] lines; two n-tiles of a B operand from 64-column lines
    const uint32_t rows_at = (16 * mt + (lane & 15)) * 128;
    auto row_a = [&](uint32_t tile, int ks) {
        return tile + rows_at + (ks >> 2) * C * 128 + (((2 * (ks & 3) + (lane >> 4)) ^ (lane & 7)) << 4);
    };
    // lines of 128 bytes (a third term, dP and beta dA) and of 256 (two terms): a line's part, and the 16 bytes in it
    const uint32_t row_l = (lane >> 4) * 8 + (lane & 7), piece_a = ((2 * mt + ((lane >> 3) & 1)) ^ (lane & 7)) << 4;
    const uint32_t a128 = row_l * 128 + piece_a, a256 = row_l * 256 + piece_a;
    const uint32_t row_b = ((lane >> 3) & 1) * 8 + (lane & 7);
    uint32_t b128[4], b256[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const uint32_t piece = ((2 * g + (lane >> 4)) ^ (lane & 7)) << 4;
        b128[g] = row_b * 128 + piece;
        b256[g] = row_b * 256 + piece;
    }
    auto pair = [&](int tile, int row, int col) {  // of a row of K or Q
        return *reinterpret_cast<const uint32_t *>(sm + tile + sw_byte(C, row, col) + (col & 7) * 2);
    };
    auto quad = [](float x) {
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        return x + __shfl_xor_sync(0xffffffffu, x, 2);
    };
    float acc[2 * NF][4];  // dQ's or dK's rows of this warp
    // ---- inside the chunk
    {
        uint32_t op[4][2][4];  // dP's or dA's rows as an A operand, two terms
        float hi[8][4], lo[8][4], kk[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) hi[t][e] = lo[t][e] = kk[t][e] = 0.f;
        const uint32_t u01 = base + at.UR, u2 = base + at.last;
#pragma unroll 1
        for (int ks = 0; ks < nvf; ++ks) {
            uint32_t a[3][4];
            if (role == 0) {
                ldsm4(a[0], row_a(aO, ks));
            } else {
                ldsm4_t(a[0], u01 + 2 * plane + a256 + ks * 4096);
                ldsm4_t(a[1], u01 + 2 * plane + a256 + ks * 4096 + 128);
                ldsm4_t(a[2], u2 + plane + a128 + ks * 2048);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (g > mt) break;
                uint32_t b[3][4];
                ldsm4_t(b[0], u01 + b256[g] + ks * 4096);
                ldsm4_t(b[1], u01 + b256[g] + ks * 4096 + 128);
                ldsm4_t(b[2], u2 + b128[g] + ks * 2048);
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
        float4 gam[8];  // on their way under the products that follow
#pragma unroll
        for (int t = 0; t < 8; ++t)
            gam[t] = t / 2 <= mt ? w.gam[(idx * kUnits + mt * (mt + 1) + t) * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t left = role ? aK : aQ;
#pragma unroll 1
        for (int ks = 0; ks < NF; ++ks) {
            uint32_t a[4];
            ldsm4(a, row_a(left, ks));
            const uint32_t k = aK + b_lane(0, 8, ks & 3, lane) + (ks >> 2) * C * 128;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (g > mt) break;
                uint32_t b[4];
                ldsm4(b, k + g * 2048);
                mma::mma(kk[2 * g], a, b[0], b[1]);
                mma::mma(kk[2 * g + 1], a, b[2], b[3]);
            }
        }
        float *M = reinterpret_cast<float *>(sm + at.M);
        const uint32_t aPA = base + at.PA + role * 2 * C * 128;
        const float be0 = role ? gates[2][i0] : 1.f, be1 = role ? gates[2][i0 + 8] : 1.f;
        float part[2] = {};  // rowsum(dA o K K^T) reaches dbeta: from the fp32 values, before they become terms
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float gm[4] = {gam[t].x, gam[t].y, gam[t].z, gam[t].w};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half, j = 8 * t + j0;
                const float be = half ? be1 : be0;
                float x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = gm[2 * half + e] * (hi[t][2 * half + e] + lo[t][2 * half + e]);
                    if (role) x[e] = j + e < i ? -x[e] : 0.f;
                }
                if (role) part[half] += x[0] * kk[t][2 * half] + x[1] * kk[t][2 * half + 1];
                uint32_t s[2];
                split(x[0], x[1], s);
#pragma unroll
                for (int n = 0; n < 2; ++n) op[t / 2][n][half + 2 * (t & 1)] = s[n];
                hi[t][2 * half] = be * x[0] * kk[t][2 * half];
                hi[t][2 * half + 1] = be * x[1] * kk[t][2 * half + 1];
                if (role == 0)  // role 1 adds its own behind the barrier
                    *reinterpret_cast<float2 *>(&M[i * PM + j]) = make_float2(hi[t][2 * half], hi[t][2 * half + 1]);
                if (role) split(be * x[0], be * x[1], s);
#pragma unroll
                for (int n = 0; n < 2; ++n) sts(aPA + n * C * 128 + sw_byte(0, i, 8 * t) + j0 * 2, s[n]);
            }
        }
        __syncthreads();
        if (role) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float2 &m = *reinterpret_cast<float2 *>(&M[(i0 + 8 * half) * PM + 8 * t + j0]);
                    m = make_float2(m.x + hi[t][2 * half], m.y + hi[t][2 * half + 1]);
                }
        }
        // rows x K
#pragma unroll
        for (int g = 0; g < NF; ++g) {
            float x[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
            const uint32_t k = aK + bt_lane(C, 16 * g, lane);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                if (kb > mt) break;
                uint32_t b[4];
                ldsm4_t(b, k + kb * 2048);
#pragma unroll
                for (int n = 1; n >= 0; --n)
#pragma unroll
                    for (int t = 0; t < 2; ++t) mma::mma(x[t], op[kb][n], b[2 * t], b[2 * t + 1]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float be = half ? be1 : be0;
                    acc[2 * g + t][2 * half] = be * x[t][2 * half];
                    acc[2 * g + t][2 * half + 1] = be * x[t][2 * half + 1];
                }
        }
        if (role)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float y = quad(part[half]);
                if ((lane & 3) == 0) db[i0 + 8 * half] += y;
            }
    }
    // rows j of [dP; beta dA]^T [Q; K]: half of the columns by each role, handed over through shared memory
    float *const kT = reinterpret_cast<float *>(sm + at.PA);
    {
        constexpr int kMine = (NF + 1) / 2;  // groups of 16 columns: role 0 the first ones, role 1 the others
        float x[2 * kMine][4];
#pragma unroll
        for (int t = 0; t < 2 * kMine; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = 0.f;
        const uint32_t pa = base + at.PA + a128;
#pragma unroll 1
        for (int kb = mt; kb < 4; ++kb) {
            uint32_t a[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) ldsm4_t(a[n], pa + n * C * 128 + kb * 2048);
#pragma unroll
            for (int y = 0; y < kMine; ++y) {
                const int g = role ? kMine + y : y;
                if (g >= NF) break;
                uint32_t q[4], k[4];
                ldsm4_t(q, aQ + bt_lane(C, 16 * g, lane) + kb * 2048);
                ldsm4_t(k, aK + bt_lane(C, 16 * g, lane) + kb * 2048);
#pragma unroll
                for (int n = 1; n >= 0; --n)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        mma::mma(x[2 * y + t], a[n], q[2 * t], q[2 * t + 1]);
                        mma::mma(x[2 * y + t], a[2 + n], k[2 * t], k[2 * t + 1]);
                    }
            }
        }
        // sums of M's columns over the rows from each row on: a quarter of the rows a thread, then the quarters below
        float *M = reinterpret_cast<float *>(sm + at.M);
        __syncthreads();  // M is complete, PA has been read
        {
            const int j = tid & 63, q = tid >> 6;
            float s = 0.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) {
                s += M[(16 * q + i) * PM + j];
                M[(16 * q + i) * PM + j] = s;
            }
            sums[q][j] = s;
        }
        if (role == 0) {
#pragma unroll
            for (int t = 0; t < 2 * kMine; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    *reinterpret_cast<float2 *>(kT + (i0 + 8 * half) * (DK + 4) + 8 * t + j0) = make_float2(x[t][2 * half], x[t][2 * half + 1]);
        } else {
#pragma unroll
            for (int t = 2 * kMine; t < 2 * NF; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] += x[t - 2 * kMine][e];
        }
        __syncthreads();
        if (role) {
#pragma unroll
            for (int t = 0; t < 2 * kMine && t < 2 * NF; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float2 y = *reinterpret_cast<const float2 *>(kT + (i0 + 8 * half) * (DK + 4) + 8 * t + j0);
                    acc[t][2 * half] += y.x;
                    acc[t][2 * half + 1] += y.y;
                }
        }
        {  // row i of the sums: the columns before it, four threads a row
            const int i = tid >> 2;
            float s = 0.f;
            for (int j = tid & 3; j < i; j += 4) {
                s += M[i * PM + j];
                for (int q = i / 16 + 1; q < 4; ++q) s += sums[q][j];
            }
            s = quad(s);
            if ((tid & 3) == 0) dg[i] = s;
        }
        sm100::fence_proxy_async_smem();
        __syncthreads();  // all that the state's columns take the place of has been read
    }
    // ---- through the states
    float part[2] = {}, all = 0.f;
#pragma unroll
    for (int slab = 0; slab < kSlabs; ++slab) {
        constexpr int kLast = NF % 4 ? NF % 4 : 4;
        constexpr int kFull = 4;
        const int groups = slab + 1 < kSlabs ? kFull : kLast;  // of 16 columns
        // Places: Sig in X's and behind `last` + 2 planes in turn, D in `last` and then X's, so that the second columns come
        // under the first ones' products; without X's place both wait for them.
        const uint32_t where_s = !at.X ? at.last : slab ? at.last + 2 * plane : at.X, where_d = !at.X ? at.last + 2 * plane : slab ? at.X : at.last;
        if (tid == 0) {
            if (!at.X) {
                sm100::mbar_arrive_expect_tx(&bar[1], 4 * plane);
                sm100::tma_load_2d(sm + where_s, &maps.Sig, &bar[1], 64 * slab, (int)(idx * dv));
                sm100::tma_load_2d(sm + where_d, &maps.D, &bar[1], 64 * slab, (int)(idx * dv));
            } else {
                sm100::mbar_arrive_expect_tx(&bar[2], 2 * plane);
                sm100::tma_load_2d(sm + where_d, &maps.D, &bar[2], 64 * slab, (int)(idx * dv));
                if (slab + 1 < kSlabs) {
                    sm100::mbar_arrive_expect_tx(&bar[3], 2 * plane);
                    sm100::tma_load_2d(sm + at.last + 2 * plane, &maps.Sig, &bar[3], 64, (int)(idx * dv));
                }
            }
        }
        uint64_t *const bar_s = at.X && slab ? &bar[3] : &bar[1];
        const uint32_t parity_s = at.X ? 0 : slab;
        bool ok = sm100::mbar_wait(bar_s, parity_s, w.err, w.wait_ns);
        const uint32_t s0 = base + where_s, d0 = base + where_d, s2 = base + at.last + 4 * plane, u01 = base + at.UR;
        // their terms, a warp a line, and <D, Sig> (columns behind d_k are zeros)
        float2 mine[16];  // this lane's columns of the warp's lines of Sig
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = warp + 8 * i;
            if (n >= dv) break;
            mine[i] = *reinterpret_cast<const float2 *>(sm + where_s + n * 256 + lane * 8);
            __syncwarp();
            line_terms(s0 + n * 256, n, mine[i], s2 + n * 128);
        }
        if (at.X) ok = sm100::mbar_wait(&bar[2], slab, w.err, w.wait_ns) && ok;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = warp + 8 * i;
            if (n >= dv) break;
            const float2 d = *reinterpret_cast<const float2 *>(sm + where_d + n * 256 + lane * 8);
            __syncwarp();
            all = fmaf(mine[i].x, d.x, fmaf(mine[i].y, d.y, all));
            line_terms(d0 + n * 256, n, d, 0);
        }
        if (!__syncthreads_and(ok)) {  // what is on its way lands before the block's shared memory goes
            sm100::mbar_wait(bar_s, parity_s, w.err, sm100::kWaitLimitNs, true);
            if (at.X) sm100::mbar_wait(&bar[2], slab, w.err, sm100::kWaitLimitNs, true);
            if (at.X && kSlabs > 1) sm100::mbar_wait(&bar[3], 0, w.err, sm100::kWaitLimitNs, true);
            if (p.status && tid == 0) atomicOr(p.status, GDN_SEQ_TIMEOUT);
            return;
        }
        float x[8][4], y[8][4];  // role 0: leading and small products; role 1: dR Sig^T and U D^T
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = y[t][e] = 0.f;
        if (role == 0) {
#pragma unroll 1
            for (int ks = 0; ks < nvf; ++ks) {
                uint32_t a[4];
                ldsm4(a, row_a(aO, ks));
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g >= groups) break;
                    uint32_t b[3][4];
#pragma unroll
                    for (int n = 0; n < 3; ++n) ldsm4_t(b[n], n < 2 ? s0 + b256[g] + ks * 4096 + n * 128 : s2 + b128[g] + ks * 2048);
#pragma unroll
                    for (int n = 2; n >= 0; --n)
#pragma unroll
                        for (int t = 0; t < 2; ++t) mma::mma(n ? y[2 * g + t] : x[2 * g + t], a, b[n][2 * t], b[n][2 * t + 1]);
                }
            }
        } else {
#pragma unroll 1
            for (int ks = 0; ks < nvf; ++ks) {
                uint32_t r[2][4], u[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    ldsm4_t(u[n], u01 + a256 + ks * 4096 + n * 128);
                    ldsm4_t(r[n], u01 + 2 * plane + a256 + ks * 4096 + n * 128);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g >= groups) break;
                    uint32_t b[2][4], d[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        ldsm4_t(b[n], s0 + b256[g] + ks * 4096 + n * 128);
                        ldsm4_t(d[n], d0 + b256[g] + ks * 4096 + n * 128);
                    }
#pragma unroll
                    for (int n = 2; n >= 0; --n)  // terms (0, 1), (1, 0), (0, 0)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            mma::mma(x[2 * g + t], r[n == 1], b[n == 2][2 * t], b[n == 2][2 * t + 1]);
                            mma::mma(y[2 * g + t], u[n == 1], d[n == 2][2 * t], d[n == 2][2 * t + 1]);
                        }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            if (t >= 2 * groups) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = i0 + 8 * half;
                float *to = acc[(8 * slab + t) % (2 * NF)] + 2 * half;
                if (role == 0) {
                    const float eg = gates[0][i], z0 = eg * (x[t][2 * half] + y[t][2 * half]), z1 = eg * (x[t][2 * half + 1] + y[t][2 * half + 1]);
                    const uint32_t q = pair(at.Q, i, 64 * slab + 8 * t + j0);
                    part[half] += low_of(q) * z0 + high_of(q) * z1;
                    to[0] += z0;
                    to[1] += z1;
                } else {
                    const float s = -gates[2][i] * gates[0][i], el = gates[1][i];
#pragma unroll
                    for (int e = 0; e < 2; ++e) to[e] += fmaf(s, x[t][2 * half + e], el * y[t][2 * half + e]);
                }
            }
        }
        sm100::fence_proxy_async_smem();
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) red[warp] = all;
    if (role == 0)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float x = quad(part[half]);
            if ((lane & 3) == 0) into[i0 + 8 * half] += x;
        }
    {
        bf16 *const dst = role ? (bf16 *)p.dk_out : (bf16 *)p.dq;
        float *const dst32 = role ? w.dkh : w.dqh;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = i0 + 8 * half;
            if (i >= ch.rows) continue;
            const size_t to = ((size_t)(ch.first + i) * p.H + h) * DK + j0;
#pragma unroll
            for (int t = 0; t < 2 * NF; ++t) {
                if (dst32) *reinterpret_cast<float2 *>(dst32 + to + 8 * t) = make_float2(acc[t][2 * half], acc[t][2 * half + 1]);
                else *reinterpret_cast<uint32_t *>(dst + to + 8 * t) = pack(acc[t][2 * half], acc[t][2 * half + 1]);
            }
        }
    }
    __syncthreads();
    if (warp < 2) {  // token tid: the terms from before the chunk to it or later ones, those from earlier ones past its end
        float in = into[tid], out = tid ? past[tid - 1] : 0.f, g = 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_down_sync(0xffffffffu, in, o), y = __shfl_up_sync(0xffffffffu, out, o);
            in += lane + o < 32 ? x : 0.f;
            out += lane >= o ? y : 0.f;
        }
        if (warp == 0) {
            float later = into[32 + lane];
#pragma unroll
            for (int o = 16; o; o >>= 1) later += __shfl_xor_sync(0xffffffffu, later, o);
            in += later;
        } else {
            float before = lane < 31 ? past[lane] : 0.f;  // past[31] is in `out` already
#pragma unroll
            for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
            out += before;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) g += red[i];
        if (tid < ch.rows) {
            const size_t to = (size_t)(ch.first + tid) * p.H + h;
            p.dalpha[to] = (fmaf(g, gates[0][C - 1], dg[tid]) + (in + out)) / fmaxf(p.alpha[to], expf(kSeqBwdLogFloor));
            p.dbeta[to] = db[tid];
        }
    }
}

template <int NF> cudaError_t prep(const SeqProblem &p, const ChunkWork &w, float floor_log, cudaStream_t s) {
    k_prep<NF><<<(unsigned)(seq_max_chunks(p) * p.H) + 1, 128, 0, s>>>(p, w, floor_log);
    return cudaGetLastError();
}

template <typename K, int NF, bool BWD> cudaError_t chain(K kernel, int threads, const SeqProblem &p, const ChunkWork &w, const ChainMaps &m, cudaStream_t s) {
    const int bytes = (int)sizeof(ChainSmem<NF, BWD>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e) return e;
    kernel<<<(unsigned)((long long)p.n_seqs * p.H * (p.dv / NV)), threads, bytes, s>>>(p, w, m);
    return cudaGetLastError();
}

bool make_maps(ChainMaps &m, const SeqProblem &p, const void *v, long long v_stride, int v_cols) {
    return seq_row_map(&m.q, p.q, p.n_tokens, p.q_stride, p.Hk, p.dk, 64) &&
           seq_row_map(&m.k, p.k, p.n_tokens, p.k_stride, p.Hk, p.dk, 64) &&
           seq_row_map(&m.v, v, p.n_tokens, v_stride, p.H, p.dv, v_cols);
}

// A warp a slice, or four warps on each?  With few slices a step's length counts, and four warps halve it; with many
// the SMs are full either way and a warp a slice moves less through shared memory.  Measured on 8192 tokens in equal
// sequences, their gradients on 4096 (us, a warp / four warps): 20 heads, d = 112: 280 slices 387 / 339 and 678 / 651, 560
// 315 / 339 and 615 / 655, 840 242 / 354 and 532 / 675, 1400 232 / 357 and 557 / 736.  8 heads, d = 128: 256 213 / 171 and
// 393 / 364, 576 123 / 170 and 301 / 380.  16 heads, d = 64: 256 163 / 172 and 301 / 319, 576 104 / 173 and 259 / 345.
bool walk(const SeqProblem &p) { return (long long)p.n_seqs * p.H * (p.dv / NV) >= 3ll * seq_num_sms(); }
unsigned walk_blocks(const SeqProblem &p) {
    return (unsigned)((long long)p.n_seqs * p.H * ((p.dv + 16 * kSlices - 1) / (16 * kSlices)));
}

template <int NF, bool SAVE> cudaError_t walk_fwd(const SeqProblem &p, const ChunkWork &w, const ChainMaps &m, cudaStream_t s) {
    const int bytes = (int)sizeof(WalkSmem<NF, false>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_walk_fwd<NF, SAVE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e) return e;
    k_walk_fwd<NF, SAVE><<<walk_blocks(p), kWalkThreads, bytes, s>>>(p, w, m);
    return cudaGetLastError();
}

template <int NF> cudaError_t fwd(SeqProblem p, const ChunkWork &w, long long short_len, cudaStream_t s) {
    ChainMaps m;
    const bool walks = walk(p);
    if (!make_maps(m, p, p.v, p.v_stride, walks ? 64 : NV)) return cudaErrorInvalidValue;
    p.min_len = short_len + 1;
    cudaError_t e = prep<NF>(p, w, kLogAlphaFloor, s);
    if (e == cudaSuccess && short_len >= 0) {
        SeqProblem few = p;
        few.max_len = short_len;
        few.good = w.good;
        e = launch_seq_recurrent(few, false, s);
    }
    if (e) return e;
    if (walks) return walk_fwd<NF, false>(p, w, m, s);
    return chain<decltype(&k_chunk_fwd<NF, false>), NF, false>(k_chunk_fwd<NF, false>, chain_threads(true), p, w, m, s);
}

template <int NF> cudaError_t bwd(const SeqProblem &p, const ChunkWork &w, cudaStream_t s) {
    const int cols = walk(p) ? 64 : NV;
    ChainMaps m, mo;
    if (!make_maps(m, p, p.v, p.v_stride, cols) || !make_maps(mo, p, p.d_o, (long long)p.H * p.dv, cols)) return cudaErrorInvalidValue;
    cudaError_t e = prep<NF>(p, w, kSeqBwdLogFloor, s);
    if (walk(p)) {
        if (!e) e = walk_fwd<NF, true>(p, w, m, s);
        const int bytes = (int)sizeof(WalkSmem<NF, true>) + 1024;
        if (!e) e = cudaFuncSetAttribute(k_walk_bwd<NF>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e) return e;
        k_walk_bwd<NF><<<walk_blocks(p), kWalkThreads, bytes, s>>>(p, w, mo);
        e = cudaGetLastError();
    } else {
        if (!e) e = chain<decltype(&k_chunk_fwd<NF, true>), NF, false>(k_chunk_fwd<NF, true>, chain_threads(false), p, w, m, s);
        if (!e) e = chain<decltype(&k_chunk_bwd<NF>), NF, true>(k_chunk_bwd<NF>, chain_threads(false), p, w, mo, s);
    }
    GradMaps g;
    g.q = m.q;
    g.k = m.k;
    if (!seq_row_map(&g.v, p.v, p.n_tokens, p.v_stride, p.H, p.dv, 64) ||
        !seq_row_map(&g.o, p.d_o, p.n_tokens, (long long)p.H * p.dv, p.H, p.dv, 64) ||
        !seq_matrix_map(&g.Sig, w.Sig, seq_max_chunks(p) * p.H * p.dv, p.dk, p.dv) ||
        !seq_matrix_map(&g.D, w.D, seq_max_chunks(p) * p.H * p.dv, p.dk, p.dv))
        return cudaErrorInvalidValue;
    const int bytes = GradLayout<NF>(p.dv).total + 1024;
    if (!e) e = cudaFuncSetAttribute(k_chunk_grads<NF>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e) return e;
    k_chunk_grads<NF><<<(unsigned)(seq_max_chunks(p) * p.H), 256, bytes, s>>>(p, w, g);
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
    w.wait_ns = wait_limit_ns();
    w.drop = debug_drop_signal();
    w.T = (uint2 *)take(3 * frag);
    w.gates = (float *)take(n * 3 * C * 4);
    w.err = (int *)take(sizeof(int));
    w.order = (int *)take((size_t)p.n_seqs * sizeof(int));
    w.good = (unsigned char *)take((size_t)p.n_seqs);
    if (!bwd) {
        w.P = (uint2 *)take(2 * frag);
    } else {
        w.chunks = (SeqChunk *)take(seq_max_chunks(p) * sizeof(SeqChunk));
        w.Tt = (uint2 *)take(3 * frag);
        w.Pt = (uint2 *)take(3 * frag);
        w.gam = (float4 *)take(n * kUnits * 32 * sizeof(float4));
        w.Sig = (float *)take(n * p.dk * p.dv * 4);
        w.D = (float *)take(n * p.dk * p.dv * 4);
        w.U = (float *)take(n * C * p.dv * 4);
        w.dR = (float *)take(n * C * p.dv * 4);
        w.X = (float *)take(n * C * p.dv * 4);
        w.Z = (float *)take(n * C * p.dv * 4);
        w.dqh = p.H > p.Hk ? (float *)take(rows * p.dk * 4) : nullptr;
        w.dkh = p.H > p.Hk ? (float *)take(rows * p.dk * 4) : nullptr;
    }
    if (total) *total = at;
    return w;
}

}  // namespace

int seq_num_sms() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

size_t seq_chunk_workspace(const SeqProblem &p, bool bwd) {
    size_t n;
    carve(p, nullptr, bwd, &n);
    return n;
}

cudaError_t launch_seq_chunk(const SeqProblem &p, long long short_len, void *ws, cudaStream_t s) {
    const ChunkWork w = carve(p, ws, false, nullptr);
    switch (p.dk / 16) {
        case 1: return fwd<1>(p, w, short_len, s);
        case 2: return fwd<2>(p, w, short_len, s);
        case 3: return fwd<3>(p, w, short_len, s);
        case 4: return fwd<4>(p, w, short_len, s);
        case 5: return fwd<5>(p, w, short_len, s);
        case 6: return fwd<6>(p, w, short_len, s);
        case 7: return fwd<7>(p, w, short_len, s);
        default: return fwd<8>(p, w, short_len, s);
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
