// seq_internal.h -- the gated delta rule over packed sequences: what its
// entry points (seq_api.cu) and kernels (seq_*.cu) share.
#pragma once

#include "gdn_internal.h"

namespace gdn {

constexpr int kSeqChunk = 64;  // tokens of a chunk in the chunked kernels

struct SeqProblem {
    int dtype;
    const void *q, *k, *v;
    const float *alpha, *beta;
    long long q_stride, k_stride, v_stride;  // elements between token rows
    void *o;
    const float *S_in;
    float *S_out;
    const int *cu, *slots;
    const unsigned char *fresh;
    int n_seqs, n_slots;
    long long seq_len, n_tokens;
    int H, Hk, dk, dv;
    const void *d_o;
    const float *dS_out;
    void *dq, *dk_out, *dv_out;
    float *dalpha, *dbeta, *dS_in;
    int *status;
    long long min_len, max_len;  // gdn_packed: a kernel leaves sequences of other lengths to another one
    const unsigned char *good;   // k_many beside a walk: the verdicts that k_prep has left (the walk reports the bits), or null
};

// Rows and state entry of a sequence.  slot < 0: the sequence is skipped.
struct SeqRange {
    long long first;
    long long len;
    int slot;
    int bad;  // GDN_SEQ_* bits
};

// Rows of sequence s by itself, 0 of them where they are no ordered range inside the tensors.
__device__ __forceinline__ SeqRange seq_rows(const SeqProblem &p, int s) {
    SeqRange r;
    r.bad = 0;
    r.slot = s;
    if (p.cu) {
        const long long a = p.cu[s], b = p.cu[s + 1];
        const bool ok = a >= 0 && b >= a && b <= p.n_tokens;
        r.first = ok ? a : 0;
        r.len = ok ? b - a : 0;
        if (!ok) {
            r.bad = GDN_SEQ_BAD_ROWS;
            r.slot = -1;
        }
    } else {
        r.first = (long long)s * p.seq_len;
        r.len = p.seq_len;
    }
    return r;
}

// Does sequence j, an ordered range by itself, reach behind row `first`?
__device__ __forceinline__ bool seq_reaches(const SeqProblem &p, int j, long long first) {
    const SeqRange r = seq_rows(p, j);
    return r.len > 0 && r.first + r.len > first;
}

// Does an earlier sequence reach behind the first row of s?  Such a sequence is skipped, so that no two share rows or a
// chunk's index.  Called by a whole block.
__device__ __forceinline__ bool seq_late_odd(const SeqProblem &p, int s) {
    const SeqRange r = seq_rows(p, s);
    bool late = false;
    for (int j = threadIdx.x; j < s; j += blockDim.x) late |= seq_reaches(p, j, r.first);
    return __syncthreads_or(late && r.len > 0);
}
// A thread's share of: is one of the ranges before s no ordered one?  Where none is, all of them are in order, and s, if it
// is by itself, is too.  (Every block of a batch looks: with thousands of short sequences the loads count, four a thread.)
__device__ __forceinline__ bool seq_odd_before(const SeqProblem &p, int s) {
    bool odd = s > 0 && p.cu[0] < 0;
    int from = 0;
    if (((size_t)p.cu & 15) == 0) {
        from = s & ~3;
        for (int j = 4 * threadIdx.x; j < from; j += 4 * blockDim.x) {
            const int4 x = *reinterpret_cast<const int4 *>(p.cu + j);
            odd |= x.x > x.y || x.y > x.z || x.z > x.w || x.w > p.cu[j + 4];
        }
    }
    for (int j = from + threadIdx.x; j < s; j += blockDim.x) odd |= p.cu[j] > p.cu[j + 1];
    return odd;
}
__device__ __forceinline__ bool seq_late(const SeqProblem &p, int s) {
    return p.cu && __syncthreads_or(seq_odd_before(p, s)) && seq_late_odd(p, s);
}
__device__ constexpr SeqRange kSeqLate = {0, 0, -1, GDN_SEQ_BAD_ROWS};
__device__ __forceinline__ SeqRange seq_rows_in_order(const SeqProblem &p, int s) { return seq_late(p, s) ? kSeqLate : seq_rows(p, s); }

// The slot's bits of a sequence; called by a whole block (it votes on an earlier sequence of the same slot whose rows are
// good, so that of two writers of one state only the first runs).
template <typename Good> __device__ __forceinline__ int seq_slot_bits(const SeqProblem &p, int s, int slot, Good good) {
    if (!p.slots) return 0;
    bool same = false;
    if (slot >= 0)
        for (int i = threadIdx.x; i < s; i += blockDim.x) same |= p.slots[i] == slot && good(i);
    return (__syncthreads_or(same) ? GDN_SEQ_SAME_SLOT : 0) | (slot >= p.n_slots ? GDN_SEQ_BAD_SLOT : 0);
}

// f(i, range, late) for the sequences before n, a thread each: the running maximum of the ends says where an earlier one
// reaches behind a sequence's first row.  Called by a whole block of THREADS.
template <int THREADS, typename F> __device__ __forceinline__ void seq_each_in_order(const SeqProblem &p, int n, F f) {
    __shared__ int ends[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    int reached = 0;  // by the sequences before these THREADS
    for (int i0 = 0; i0 < n; i0 += THREADS) {
        const int i = i0 + threadIdx.x;
        SeqRange r = {0, 0, -1, 0};
        if (i < n) r = seq_rows(p, i);
        int end = r.len > 0 ? (int)(r.first + r.len) : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end = max(end, x);
        }
        __syncthreads();
        if (lane == 31) ends[warp] = end;
        __syncthreads();
        int before = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) before = 0;
        before = max(before, reached);
        for (int k = 0; k < THREADS / 32; ++k) {
            if (k < warp) before = max(before, ends[k]);
            reached = max(reached, ends[k]);
        }
        if (i < n) f(i, r, r.len > 0 && r.first < before);
    }
}

// All bits of a sequence (any of them: it is skipped), where nothing is known of the others; called by a whole block of
// THREADS.  What is rarely true is looked into behind one vote.  (The bits alone: a range put together on several paths
// cost k_many 340 bytes of spills.)
template <int THREADS> __device__ __forceinline__ int seq_refused(const SeqProblem &p, int s, int slot) {
    int bad = seq_rows(p, s).bad;
    bool odd = p.cu && seq_odd_before(p, s);
    if (p.slots)
        for (int i = threadIdx.x; i < s; i += blockDim.x) odd |= p.slots[i] == slot;
    if (__syncthreads_or(odd)) {
        bool rows = false, same = false;
        seq_each_in_order<THREADS>(p, s + 1, [&](int i, const SeqRange &r, bool late) {
            if (i == s) rows = late;
            else same |= p.slots && p.slots[i] == slot && !r.bad && !late;
        });
        if (__syncthreads_or(rows)) bad |= GDN_SEQ_BAD_ROWS;
        if (__syncthreads_or(same) && slot >= 0) bad |= GDN_SEQ_SAME_SLOT;
    }
    return p.slots && slot >= p.n_slots ? bad | GDN_SEQ_BAD_SLOT : bad;
}

// One block of a launch reports a sequence's bits.
__device__ __forceinline__ void seq_report(const SeqProblem &p, int bad, bool reporter) {
    if (bad && p.status && reporter) atomicOr(p.status, bad);
}

__device__ __forceinline__ bool seq_starts_zero(const SeqProblem &p, int s) {
    return !p.S_in || (p.fresh && p.fresh[s]);
}

// Chunks.  Chunk i of sequence s has the index seq_chunk_base(s) + i, unique without a table where the sequences lie in
// the order of their rows: ceil(len / 64) <= floor(end / 64) - floor(first / 64) + 1.
__host__ __device__ __forceinline__ long long seq_chunks_of(long long len) {
    return (len + kSeqChunk - 1) / kSeqChunk;
}
__device__ __forceinline__ long long seq_chunk_base(const SeqProblem &p, int s, long long first) {
    return p.cu ? first / kSeqChunk + s : s * seq_chunks_of(p.seq_len);
}
__host__ inline long long seq_max_chunks(const SeqProblem &p) {
    return p.cu ? p.n_tokens / kSeqChunk + p.n_seqs : p.n_seqs * seq_chunks_of(p.seq_len);
}

// The chunk that has index c: its first row and how many rows it has (0: no chunk has it).
struct SeqChunk {
    long long first;
    int rows;
    int seq;
};
// Of the sequences that by themselves have a chunk c only the first can be in order (the others' bases lie behind its
// end).  Called by a whole block, where a range is wrong.
__device__ __forceinline__ SeqChunk seq_chunk_odd(const SeqProblem &p, long long c) {
    __shared__ int least;
    if (threadIdx.x == 0) least = p.n_seqs;
    __syncthreads();
    for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) {
        const SeqRange r = seq_rows(p, s);
        const long long t = (c - seq_chunk_base(p, s, r.first)) * kSeqChunk;
        if (t >= 0 && t < r.len) atomicMin(&least, s);
    }
    __syncthreads();
    const int s = least;
    if (s == p.n_seqs) return {0, 0, -1};
    const SeqRange r = seq_rows_in_order(p, s);
    if (r.len == 0) return {0, 0, -1};
    const long long t = (c - seq_chunk_base(p, s, r.first)) * kSeqChunk;
    return {r.first + t, (int)min((long long)kSeqChunk, r.len - t), s};
}
// Called by a whole block.  Where every range is in order by itself, all of them are, and the one that has c is it.
__device__ __forceinline__ SeqChunk seq_chunk(const SeqProblem &p, long long c) {
    __shared__ SeqChunk found;
    __shared__ int odd;
    if (!p.cu) {
        const long long n = seq_chunks_of(p.seq_len);
        const int s = (int)(c / n);
        const long long t = (c % n) * kSeqChunk;
        return {s * p.seq_len + t, (int)min((long long)kSeqChunk, p.seq_len - t), s};
    }
    if (threadIdx.x == 0) {
        found = {0, 0, -1};
        odd = 0;
    }
    __syncthreads();
    for (int s = threadIdx.x; s < p.n_seqs; s += blockDim.x) {
        const SeqRange r = seq_rows(p, s);
        const long long t = (c - seq_chunk_base(p, s, r.first)) * kSeqChunk;
        if (t >= 0 && t < r.len) found = {r.first + t, (int)min((long long)kSeqChunk, r.len - t), s};
        if (r.bad) odd = 1;
    }
    __syncthreads();
    return odd ? seq_chunk_odd(p, c) : found;
}

// What the chunk kernels keep of each (chunk, head), index chunk * H + head (fp32):
struct SeqWork {
    float *T, *P;      // [64][64]: (I + A)^-1 and tril(Q K^T o decay)
    float *eg, *el;    // [64]: e^{G_i}, e^{G_last - G_i}
    float *Sig, *D;    // [dv][dk]: the state entering the chunk; the gradient of the one leaving it
    float *U, *Y, *dR; // [64][dv]
    float *dqh, *dkh;  // [n_tokens][H][dk]: the gradients before heads are summed (shared heads only)
};
size_t seq_bwd_workspace(const SeqProblem &p, void *base, SeqWork *w);

constexpr float kSeqBwdLogFloor = -60.f;  // log alpha in gdn_bwd; see gdn.h

// alpha as the token-by-token kernels multiply by it: one that is negative, which the kernels in log space cannot hold, is
// not a number in either, so that a gate gone wrong shows the same in all of them.
__device__ __forceinline__ float seq_alpha(float a) { return a >= 0.f ? a : __int_as_float(0x7fffffff); }

// gdn_bwd on the CUDA cores (seq_simt.cu).
cudaError_t launch_seq_bwd_simt(const SeqProblem &p, void *ws, cudaStream_t s);
// Zeros in the gradients of rows that no sequence covers; with cu_seqlens only.
// (also in dqh / dkh, where they are given).
cudaError_t launch_seq_zero_rows(const SeqProblem &p, float *dqh, float *dkh, cudaStream_t s);
// dq, dk from the heads' dqh, dkh.
cudaError_t launch_seq_share(const SeqProblem &p, const float *dqh, const float *dkh, cudaStream_t s);

// gdn_packed and gdn_bwd in chunks on the tensor cores, bf16 q, k, v (seq_chunk.cu).
size_t seq_chunk_workspace(const SeqProblem &p, bool bwd);
// Sequences of up to short_len go token by token.
cudaError_t launch_seq_chunk(const SeqProblem &p, long long short_len, void *ws, cudaStream_t s);
cudaError_t launch_seq_bwd_chunk(const SeqProblem &p, void *ws, cudaStream_t s);

int seq_num_sms();  // of the current device

// The recurrent form (seq_recurrent.cu).  `few`: one or a few tokens of each sequence.
cudaError_t launch_seq_recurrent(const SeqProblem &p, bool few, cudaStream_t s);

}  // namespace gdn
