// seq_recurrent.cu -- the token-wise rule walked token by token, the state in registers.
//
//   S <- alpha S;  u = beta (v - S k);  S <- S + u k^T;  o = S q
//
// Row r of S (one of the d_v) meets only k, q and its own v_r, so rows are independent: four
// lanes hold a row, a quarter of its 16-byte pieces each, and two shuffles finish each of the
// two dot products.  Everything is fp32.
//
// k_few: one or a few tokens (gdn_decode).  The state is read and written once and dominates
// (2 x 4 d_k d_v bytes a head against 2 (2 d_k + 2 d_v)): the bound is HBM.
// k_many: sequences of tokens (gdn_packed, where the chunked form does not serve), with the
// tokens' rows staged in shared memory a block ahead.  A long sequence is bound by the chain of a token's two dot products
// (996 tokens, d_k = 64: 132 us, 260 clocks a token), many short ones by the fp32 pipe: 4 d_k d_v instructions' lanes a token
// and head.
#include <cuda_bf16.h>
#include <type_traits>

#include "seq_internal.h"

namespace gdn {
namespace {

__device__ __forceinline__ float4 ld4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x;
}

__device__ __forceinline__ float4 floats(float4 x) { return x; }
__device__ __forceinline__ float4 floats(uint2 r) {  // four bf16
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
}

// One token on a lane's piece of a row; k and q are this lane's pieces of the token's rows (as they lie in memory:
// widened where they are used, they take half the registers).  Returns o's value, summed over the row's lanes.
template <int NF, typename Piece>
__device__ __forceinline__ float token_step(float4 (&S)[NF], const Piece (&k)[NF], const Piece (&q)[NF], float alpha, float beta, float v) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const float4 x = floats(k[j]);
        S[j].x *= alpha; S[j].y *= alpha; S[j].z *= alpha; S[j].w *= alpha;
        a.x = fmaf(S[j].x, x.x, a.x); a.y = fmaf(S[j].y, x.y, a.y);
        a.z = fmaf(S[j].z, x.z, a.z); a.w = fmaf(S[j].w, x.w, a.w);
    }
    const float u = beta * (v - quad_sum((a.x + a.y) + (a.z + a.w)));
    a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const float4 x = floats(k[j]), y = floats(q[j]);
        S[j].x = fmaf(u, x.x, S[j].x); S[j].y = fmaf(u, x.y, S[j].y);
        S[j].z = fmaf(u, x.z, S[j].z); S[j].w = fmaf(u, x.w, S[j].w);
        a.x = fmaf(S[j].x, y.x, a.x); a.y = fmaf(S[j].y, y.y, a.y);
        a.z = fmaf(S[j].z, y.z, a.z); a.w = fmaf(S[j].w, y.w, a.w);
    }
    return quad_sum((a.x + a.y) + (a.z + a.w));
}

constexpr int kFewThreads = 64;  // 16 rows: d_v is a multiple of 16, so a block stays in one head

// A lane's pieces of a token's k and q rows as they lie in memory, and its row's v and gates.
template <typename T, int NF> struct Token {
    using Piece = typename std::conditional<sizeof(T) == 2, uint2, float4>::type;
    Piece k[NF], q[NF];
    float v, alpha, beta;
    __device__ __forceinline__ void load(const SeqProblem &p, long long tok, int h, int hk, int r, int part) {
        const T *kp = (const T *)p.k + tok * p.k_stride + (size_t)hk * p.dk + part * 4;
        const T *qp = (const T *)p.q + tok * p.q_stride + (size_t)hk * p.dk + part * 4;
#pragma unroll
        for (int j = 0; j < NF; ++j) k[j] = *reinterpret_cast<const Piece *>(kp + 16 * j);
#pragma unroll
        for (int j = 0; j < NF; ++j) q[j] = *reinterpret_cast<const Piece *>(qp + 16 * j);
        v = to_f(((const T *)p.v)[tok * p.v_stride + (size_t)h * p.dv + r]);
        alpha = seq_alpha(p.alpha[tok * p.H + h]);
        beta = p.beta[tok * p.H + h];
    }
};
// The state is read once and written once: it goes through L2 as a stream.
template <int NF> __device__ __forceinline__ void load_state(float4 (&S)[NF], const float *from) {
#pragma unroll
    for (int j = 0; j < NF; ++j) S[j] = __ldcs(reinterpret_cast<const float4 *>(from + 16 * j));
}
template <int NF> __device__ __forceinline__ void store_state(float *to, const float4 (&S)[NF]) {
#pragma unroll
    for (int j = 0; j < NF; ++j) __stcs(reinterpret_cast<float4 *>(to + 16 * j), S[j]);
}

// HEAD: a block has all rows of a head, 16 at a time, and loads the next 16 while it works on these; else it has 16.
template <typename T, int NF, bool HEAD>
__global__ void __launch_bounds__(kFewThreads) k_few(const __grid_constant__ SeqProblem p) {
    const int per_head = HEAD ? 1 : p.dv / 16, per_seq = p.H * per_head;
    const int s = blockIdx.x / per_seq, rb = blockIdx.x % per_seq;
    const int h = rb / per_head, hk = h / (p.H / p.Hk), part = threadIdx.x & 3;
    int r = rb % per_head * 16 + threadIdx.x / 4;
    const int slot = p.slots ? p.slots[s] : s;
    // The first token's loads wait for nothing, and the state's only for an index in range: both are on their way
    // while the slots are compared.
    Token<T, NF> now;
    if (p.seq_len > 0) now.load(p, (long long)s * p.seq_len, h, hk, r, part);
    const bool inside = slot >= 0 && (!p.slots || slot < p.n_slots);
    float4 S[NF], next[NF];
    size_t soff = (((size_t)(inside ? slot : 0) * p.H + h) * p.dv + r) * p.dk + part * 4;
    if (inside) load_state(S, p.S_in + soff);
    const int bad = seq_slot_bits(p, s, slot, [](int) { return true; });
    seq_report(p, bad, rb == 0 && threadIdx.x == 0);
    const SeqRange range = seq_rows(p, s);
    if (bad || slot < 0) return;
    const int last = HEAD ? p.dv - 16 : 0;
    for (int r0 = 0;; r0 += 16) {
        const size_t ahead = soff + (size_t)16 * p.dk;
        if (HEAD && r0 < last) load_state(next, p.S_in + ahead);
        float v_next = 0.f;
        if (HEAD && r0 < last && range.len > 0) v_next = to_f(((const T *)p.v)[range.first * p.v_stride + (size_t)h * p.dv + r + 16]);
        for (long long t = 0; t < range.len; ++t) {
            if (t) now.load(p, range.first + t, h, hk, r, part);
            const float o = token_step<NF>(S, now.k, now.q, now.alpha, now.beta, now.v);
            if (part == 0) put((T *)p.o + ((range.first + t) * p.H + h) * p.dv + r, o);
        }
        store_state(p.S_out + soff, S);
        if (r0 >= last) break;
        r += 16;
        soff = ahead;
        if (range.len > 1) now.load(p, range.first, h, hk, r, part);
        now.v = v_next;
#pragma unroll
        for (int j = 0; j < NF; ++j) S[j] = next[j];
    }
}

// 16 tokens' k and q rows (fp32), v values of the block's 16 rows and gates, one stage.
constexpr int kTok = 16;
constexpr int kManyThreads = 64;

// BLOCKS an SM.  Left to itself the compiler takes the registers it likes (four blocks an SM at d_k = 128), which is best for a few
// long chains; with many blocks six of them hide more, although d_k = 128 spills then (80 bytes).  Measured (us, free / six):
// 5 fp32 sequences of up to 996 tokens, 6 heads: d = 64 132 / 136, 96 174 / 180, 112 197 / 218, 128 208 / 275; 40 prompts of 20
// tokens, 20 heads: 64 36 / 31, 96 75 / 65, 112 97 / 83, 128 117 / 107.
template <typename T, int NF, int BLOCKS>
__global__ void __launch_bounds__(kManyThreads, BLOCKS) k_many(const __grid_constant__ SeqProblem p) {
    constexpr int DK = 16 * NF;
    __shared__ __align__(16) float sk[2][kTok][DK], sq[2][kTok][DK];
    __shared__ float sv[2][kTok][16], sg[2][kTok][2];
    const int per_seq = p.H * (p.dv / 16);
    const int s = blockIdx.x / per_seq, rb = blockIdx.x % per_seq;
    const int h = rb / (p.dv / 16), r0 = (rb % (p.dv / 16)) * 16, hk = h / (p.H / p.Hk);
    const int lr = threadIdx.x / 4, part = threadIdx.x & 3;
    const SeqRange range = seq_rows(p, s);
    if (range.len > p.max_len) return;  // another kernel's, which looks at the others for it
    const int slot = p.slots ? p.slots[s] : s;
    // The state's and the first tokens' loads wait for nothing but an index in range: both are on their way while the other
    // sequences are looked at.
    const bool inside = !range.bad && slot >= 0 && (!p.slots || slot < p.n_slots);
    const size_t soff = (((size_t)(inside ? slot : 0) * p.H + h) * p.dv + r0 + lr) * DK + part * 4;
    float4 S[NF];
    const bool zero = !inside || seq_starts_zero(p, s);
#pragma unroll
    for (int j = 0; j < NF; ++j) S[j] = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : ld4(p.S_in + soff + 16 * j);

    // a thread's share of a stage: NF 16-byte (fp32) / 8-byte (bf16) pieces of k and of q, 4 of v
    constexpr int PIECES = kTok * DK / 4 / kManyThreads;  // = NF
    float4 nk[PIECES], nq[PIECES];
    float nv[4], ng = 0.f;
    auto fetch = [&](long long t0) {
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int i = j * kManyThreads + threadIdx.x, tt = i / (DK / 4), c = (i % (DK / 4)) * 4;
            const bool on = t0 + tt < range.len;
            const long long tok = range.first + t0 + tt;
            nk[j] = on ? ld4((const T *)p.k + tok * p.k_stride + (size_t)hk * DK + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            nq[j] = on ? ld4((const T *)p.q + tok * p.q_stride + (size_t)hk * DK + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = j * kManyThreads + threadIdx.x, tt = i / 16;
            nv[j] = t0 + tt < range.len
                        ? to_f(((const T *)p.v)[(range.first + t0 + tt) * p.v_stride + (size_t)h * p.dv + r0 + i % 16])
                        : 0.f;
        }
        if (threadIdx.x < 2 * kTok && t0 + threadIdx.x / 2 < range.len)
            ng = ((threadIdx.x & 1) ? p.beta : p.alpha)[(range.first + t0 + threadIdx.x / 2) * p.H + h];
    };
    auto stash = [&](int b) {
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int i = j * kManyThreads + threadIdx.x, tt = i / (DK / 4), c = (i % (DK / 4)) * 4;
            *reinterpret_cast<float4 *>(&sk[b][tt][c]) = nk[j];
            *reinterpret_cast<float4 *>(&sq[b][tt][c]) = nq[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = j * kManyThreads + threadIdx.x;
            sv[b][i / 16][i % 16] = nv[j];
        }
        if (threadIdx.x < 2 * kTok) sg[b][threadIdx.x / 2][threadIdx.x & 1] = threadIdx.x & 1 ? ng : seq_alpha(ng);
    };
    T *out = (T *)p.o + (range.first * p.H + h) * p.dv + r0 + lr;
    const size_t out_step = (size_t)p.H * p.dv;
    if (inside && range.len > 0) fetch(0);
    int bad;
    if (p.good) {
        if (!p.good[s]) return;
        bad = seq_slot_bits(p, s, slot, [&](int i) { return p.good[i] != 0; });
    } else {
        bad = seq_refused<kManyThreads>(p, s, slot);
        seq_report(p, bad, rb == 0 && threadIdx.x == 0);
    }
    if (bad || slot < 0) return;
    if (range.len > 0) stash(0);
    __syncthreads();
    int b = 0;
    for (long long t0 = 0; t0 < range.len; t0 += kTok, b ^= 1) {
        const bool more = t0 + kTok < range.len;
        if (more) fetch(t0 + kTok);
        const int n = (int)min((long long)kTok, range.len - t0);
        const float *ks = &sk[b][0][part * 4], *qs = &sq[b][0][part * 4];
        auto token = [&](int t) {
            float4 k[NF], q[NF];
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                k[j] = ld4(ks + t * DK + 16 * j);
                q[j] = ld4(qs + t * DK + 16 * j);
            }
            return token_step<NF>(S, k, q, sg[b][t][0], sg[b][t][1], sv[b][t][lr]);
        };
        // Four tokens' outputs are kept and then stored, a token a lane of a row's four
        int t = 0;
        for (; t + 4 <= n; t += 4) {
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = token(t + i);
            put(out + part * out_step, part & 2 ? (part & 1 ? o[3] : o[2]) : (part & 1 ? o[1] : o[0]));
            out += 4 * out_step;
        }
        for (; t < n; ++t) {
            const float o = token(t);
            if (part == 0) put(out, o);
            out += out_step;
        }
        if (more) stash(b ^ 1);
        __syncthreads();
    }
    if (p.S_out) {
#pragma unroll
        for (int j = 0; j < NF; ++j) *reinterpret_cast<float4 *>(p.S_out + soff + 16 * j) = S[j];
    }
}

template <typename T, int NF> cudaError_t launch(const SeqProblem &p, bool few, cudaStream_t s) {
    const long long heads = (long long)p.n_seqs * p.H, blocks = heads * (p.dv / 16);
    // A block a head once there are 24 for every SM.  Below that the blocks are too few; above it the fewer looks at the slots
    // count.  Measured with states that come from HBM (us, a head / 16 rows a block; heads 1280, 1920, 3200, 5120): d = 112 27.5 /
    // 25.0, 39.4 / 35.5, 58.9 / 58.6, 90.7 / 90.3; 128 33.9 / 29.8, 48.7 / 44.1, 72.1 / 70.3, 110.7 / 110.7; 64 10.0 / 10.4, 14.8 /
    // 14.2, 21.8 / 22.0, 31.6 / 33.6; 32 5.1 / 4.7, 5.8 / 6.2, 8.5 / 9.0, 12.0 / 13.2.  With new inputs too at every call, 256
    // sequences of 20 heads, d = 112: 92.4 / 97.4 (5.6 TB/s; an in-place product of the same bytes takes 78).
    if (few && heads >= 24ll * seq_num_sms()) k_few<T, NF, true><<<(unsigned)heads, kFewThreads, 0, s>>>(p);
    else if (few) k_few<T, NF, false><<<(unsigned)blocks, kFewThreads, 0, s>>>(p);
    else if (blocks > 4ll * seq_num_sms()) k_many<T, NF, 6><<<(unsigned)blocks, kManyThreads, 0, s>>>(p);
    else k_many<T, NF, 1><<<(unsigned)blocks, kManyThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_t(const SeqProblem &p, bool few, cudaStream_t s) {
    switch (p.dk / 16) {
        case 1: return launch<T, 1>(p, few, s);
        case 2: return launch<T, 2>(p, few, s);
        case 3: return launch<T, 3>(p, few, s);
        case 4: return launch<T, 4>(p, few, s);
        case 5: return launch<T, 5>(p, few, s);
        case 6: return launch<T, 6>(p, few, s);
        case 7: return launch<T, 7>(p, few, s);
        default: return launch<T, 8>(p, few, s);
    }
}

}  // namespace

cudaError_t launch_seq_recurrent(const SeqProblem &p, bool few, cudaStream_t s) {
    return p.dtype == GDN_DTYPE_BF16 ? launch_t<__nv_bfloat16>(p, few, s) : launch_t<float>(p, few, s);
}

}  // namespace gdn
