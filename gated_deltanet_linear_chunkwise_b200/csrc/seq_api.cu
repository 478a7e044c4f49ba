// seq_api.cu -- gdn_decode, gdn_packed, gdn_bwd: argument checks, workspace, dispatch.
//
// As in gdn_api.cu, everything the host can see is checked before anything is enqueued, and no
// C++ exception crosses the ABI.  What only the GPU can see (slots, cu_seqlens) the kernels check.
#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "seq_internal.h"

namespace {

enum Which { kDecode, kPacked, kBwd };

// In a batch of short prompts the ones up to short_len() go token by token and the others in chunks, two launches beside one
// another's sequences: a chunk step and its block's start take as long as some tokens of the state's size, and as 24 where the
// token loop's blocks are on the SMs together.  Where the average is kMixed or more, few can be short, and the chunks take
// them all.  Measured (us, token by token / in chunks), 64 prompts of one length and 8 of 100 tokens: 20 heads, d = 64: 8 tokens
// 56 / 91, 24 85 / 93; 16 heads, d = 80: 8 66 / 114, 24 102 / 115; 20 heads, d = 96: 8 101 / 159, 16 137 / 160, 20 166 / 160; 20
// heads, d = 112: 8 135 / 174, 16 173 / 174, 20 202 / 174; 16 heads, d = 128: 8 127 / 155, 12 149 / 156, 16 168 / 155.  256 prompts
// alone: d = 96: 16 401 / 480, 20 488 / 481; 112: 16 507 / 523, 20 605 / 526; 128: 12 430 / 473, 16 493 / 472.  9 of together 72
// tokens, 4 heads, d = 96: 12 / 24.  Averages (20 heads, d = 112; both / chunks alone): 32 83 / 102, 43 149 / 165, 64 82.2 / 82.9,
// 128 120 / 104, 256 197 / 182.
constexpr long long kMixed = 48;
long long short_len(const gdn::SeqProblem &p) {
    if ((long long)p.n_seqs * p.H * (p.dv / 16) <= 6ll * gdn::seq_num_sms()) return 24;
    return std::min(24, 25 - p.dk * p.dv / 1200);  // through the even points: 18 at d = 96, 15 at 112, 12 at 128
}
constexpr long long kEqual = 24;  // see chunked()

int fail(int status, const char *fmt, ...) {
    char text[400];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    gdn::set_error_text(text);
    return status;
}

struct Span {
    const char *name;
    const void *ptr;
    size_t bytes;
};

bool meet(const Span &a, const Span &b) {
    if (!a.ptr || !b.ptr || !a.bytes || !b.bytes) return false;
    const char *x = (const char *)a.ptr, *y = (const char *)b.ptr;
    return x < y + b.bytes && y < x + a.bytes;
}

int check_sizes(const gdn_seq_args &a) {
    if (a.dtype != GDN_DTYPE_BF16 && a.dtype != GDN_DTYPE_F32)
        return fail(GDN_ERR_INVALID_ARG, "dtype %d is neither GDN_DTYPE_BF16 nor GDN_DTYPE_F32", a.dtype);
    if (a.n_seqs < 0 || a.n_slots < 0 || a.seq_len < 0 || a.n_tokens < 0 || a.H < 0 || a.Hk < 0)
        return fail(GDN_ERR_INVALID_ARG, "negative size: n_seqs=%d n_slots=%d seq_len=%lld n_tokens=%lld H=%d Hk=%d",
                    a.n_seqs, a.n_slots, a.seq_len, a.n_tokens, a.H, a.Hk);
    for (int d : {a.d_k, a.d_v})
        if (d < 16 || d > 128 || d % 16)
            return fail(GDN_ERR_UNSUPPORTED, "head dims d_k=%d d_v=%d: each must be a multiple of 16 in [16, 128]", a.d_k, a.d_v);
    if (a.H > 0 && (a.Hk < 1 || a.H % a.Hk))
        return fail(GDN_ERR_SHAPE, "H (%d) is not a multiple of Hk (%d)", a.H, a.Hk);
    if (a.n_tokens >= 2147483648ll)
        return fail(GDN_ERR_SHAPE, "n_tokens (%lld) exceeds 2^31 - 1", a.n_tokens);
    // seq_len <= n_tokens keeps the product inside 2^62
    if (!a.cu_seqlens && (a.n_seqs ? a.seq_len > a.n_tokens || a.seq_len * a.n_seqs != a.n_tokens : a.n_tokens != 0))
        return fail(GDN_ERR_SHAPE, "n_tokens (%lld) is not n_seqs (%d) x seq_len (%lld)", a.n_tokens, a.n_seqs, a.seq_len);
    // one block for 16 rows of a state, one for a chunk of a head: both counts stay in a grid
    const long double blocks = (long double)a.n_seqs * a.H * (a.d_v / 16);
    const long double chunks = ((long double)a.n_tokens / gdn::kSeqChunk + a.n_seqs + 1) * a.H + 1;
    if (blocks >= 2147483648.0L || chunks >= 2147483648.0L)
        return fail(GDN_ERR_SHAPE, "n_seqs x H x d_v / 16 or chunks x H exceeds 2^31");
    return GDN_OK;
}

int check(const gdn_seq_args &a, Which which, gdn::SeqProblem &p) {
    if (a.struct_size != (int)sizeof(gdn_seq_args))
        return fail(GDN_ERR_INVALID_ARG, "gdn_seq_args.struct_size = %d, this library expects %d", a.struct_size, (int)sizeof(gdn_seq_args));
    int st = check_sizes(a);
    if (st != GDN_OK) return st;
    const size_t es = a.dtype == GDN_DTYPE_BF16 ? 2 : 4;
    const long long wq = (long long)a.Hk * a.d_k, wv = (long long)a.H * a.d_v;
    const struct { const char *name; long long stride, width; } rows[] = {
        {"q_stride", a.q_stride, wq}, {"k_stride", a.k_stride, wq}, {"v_stride", a.v_stride, wv}};
    for (const auto &r : rows) {
        if (r.stride && (r.stride < r.width || r.stride > (1ll << 31)))
            return fail(GDN_ERR_INVALID_ARG, "%s (%lld) is smaller than a row (%lld) or above 2^31", r.name, r.stride, r.width);
        if (r.stride * es % 16) return fail(GDN_ERR_ALIGNMENT, "%s (%lld elements) is not a multiple of 16 bytes", r.name, r.stride);
    }
    const bool empty = a.n_tokens == 0 || a.H == 0;
    if (!empty && (!a.q || !a.k || !a.v || !a.alpha || !a.beta))
        return fail(GDN_ERR_INVALID_ARG, "q, k, v, alpha and beta are required (one is NULL)");
    if (which != kBwd) {
        if (!empty && !a.o) return fail(GDN_ERR_INVALID_ARG, "o is required (NULL)");
        if (a.d_o || a.dS_out || a.dq || a.dk || a.dv || a.dalpha || a.dbeta || a.dS_in)
            return fail(GDN_ERR_INVALID_ARG, "gradients are arguments of gdn_bwd");
        if (!a.slots && (a.S_in || a.S_out) && a.n_slots < a.n_seqs)
            return fail(GDN_ERR_SHAPE, "n_slots (%d) states for n_seqs (%d) sequences without slots", a.n_slots, a.n_seqs);
    } else {
        if (!empty && (!a.d_o || !a.dq || !a.dk || !a.dv || !a.dalpha || !a.dbeta))
            return fail(GDN_ERR_INVALID_ARG, "d_o, dq, dk, dv, dalpha and dbeta are required (one is NULL)");
        if (a.o || a.S_out || a.slots || a.fresh)
            return fail(GDN_ERR_INVALID_ARG, "gdn_bwd takes no o, S_out, slots or fresh");
    }
    if (which == kDecode) {
        if (a.n_seqs && a.H && (!a.S_in || a.S_in != a.S_out)) return fail(GDN_ERR_INVALID_ARG, "gdn_decode updates its states in place: S_in and S_out must be the same, not NULL");
        if (a.fresh || a.cu_seqlens) return fail(GDN_ERR_INVALID_ARG, "gdn_decode takes no fresh or cu_seqlens");
    }
    const size_t n = (size_t)a.n_tokens, ng = n * a.H * 4;
    const size_t ns = (size_t)(which == kBwd ? a.n_seqs : a.n_slots) * a.H * a.d_k * a.d_v * 4;
    const size_t nds = (size_t)a.n_seqs * a.H * a.d_k * a.d_v * 4;
    auto extent = [&](long long stride, long long width) {
        return n ? ((n - 1) * (size_t)(stride ? stride : width) + (size_t)width) * es : (size_t)0;
    };
    const Span in[] = {{"q", a.q, extent(a.q_stride, wq)}, {"k", a.k, extent(a.k_stride, wq)}, {"v", a.v, extent(a.v_stride, wv)},
                       {"alpha", a.alpha, ng}, {"beta", a.beta, ng}, {"S_in", a.S_in, ns}, {"d_o", a.d_o, n * wv * es},
                       {"dS_out", a.dS_out, nds}, {"cu_seqlens", a.cu_seqlens, ((size_t)a.n_seqs + 1) * 4},
                       {"slots", a.slots, (size_t)a.n_seqs * 4}, {"fresh", a.fresh, (size_t)a.n_seqs}};
    const Span out[] = {{"o", a.o, n * wv * es}, {"S_out", a.S_out, ns}, {"dq", a.dq, n * wq * es}, {"dk", a.dk, n * wq * es},
                        {"dv", a.dv, n * wv * es}, {"dalpha", a.dalpha, ng}, {"dbeta", a.dbeta, ng}, {"dS_in", a.dS_in, nds},
                        {"workspace", a.workspace, a.workspace_bytes}, {"status_dev", a.status_dev, 4}};
    auto aligned = [&](const Span &x, size_t to) { return ((uintptr_t)x.ptr & (to - 1)) == 0; };
    for (int i = 0; i < 11; ++i)
        if (!aligned(in[i], i < 8 ? 16 : i < 10 ? 4 : 1))
            return fail(GDN_ERR_ALIGNMENT, "%s = %p is not %d-byte aligned", in[i].name, in[i].ptr, i < 8 ? 16 : 4);
    for (int i = 0; i < 10; ++i)
        if (!aligned(out[i], i < 8 ? 16 : i == 8 ? 256 : 4))
            return fail(GDN_ERR_ALIGNMENT, "%s = %p is not %d-byte aligned", out[i].name, out[i].ptr, i < 8 ? 16 : i == 8 ? 256 : 4);
    for (int i = 0; i < 10; ++i) {
        for (const Span &x : in)
            if (meet(out[i], x) && !(i == 1 && x.ptr == a.S_in && a.S_in == a.S_out))
                return fail(GDN_ERR_INVALID_ARG, "%s overlaps input %s", out[i].name, x.name);
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
    }
    p.dtype = a.dtype;
    p.q = a.q; p.k = a.k; p.v = a.v; p.alpha = a.alpha; p.beta = a.beta;
    p.q_stride = a.q_stride ? a.q_stride : wq;
    p.k_stride = a.k_stride ? a.k_stride : wq;
    p.v_stride = a.v_stride ? a.v_stride : wv;
    p.o = a.o; p.S_in = a.S_in; p.S_out = a.S_out;
    p.cu = a.cu_seqlens; p.slots = a.slots; p.fresh = a.fresh;
    p.n_seqs = a.n_seqs; p.n_slots = a.n_slots; p.seq_len = a.cu_seqlens ? 0 : a.seq_len; p.n_tokens = a.n_tokens;
    p.H = a.H; p.Hk = a.Hk; p.dk = a.d_k; p.dv = a.d_v;
    p.d_o = a.d_o; p.dS_out = a.dS_out; p.dq = a.dq; p.dk_out = a.dk; p.dv_out = a.dv;
    p.dalpha = a.dalpha; p.dbeta = a.dbeta; p.dS_in = a.dS_in;
    p.status = a.status_dev;
    p.min_len = 0;
    p.max_len = a.n_tokens;
    p.good = nullptr;
    return GDN_OK;
}

// Which form serves a gdn_packed or gdn_bwd call.  The tensor cores take bf16 operands.  Few tokens for the states that
// they pass through go token by token: about 0.25 us a token of the longest sequence, against 16 us and 2 us a sequence
// of 140 slices (16 columns of a head's state) in chunks.  The longest sequence is not known on the host, so the rule
// takes all tokens for one's (of equal sequences it leaves the token loop too early, by a factor of two and more).  Measured
// on equal sequences (us, token by token / chunks): 20 heads, d = 112: 1 of 32 tokens 10 / 17, of 64 18 / 16; 16 of together 128
// 19 / 44, 256 30 / 44, 512 51 / 45; 40 of 200 34 / 90, 400 50 / 91, 800 83 / 91.  8 heads, d = 128: 1 of 32 11 / 17, of 64 21 / 17;
// 16 of 128 13 / 28, 512 33 / 28; 40 of 400 26 / 49, 800 45 / 48.
// Without cu_seqlens every length is known: up to kEqual tokens go token by token (16 x 16 tokens 30 / 44 and 19 / 28, 40 x 20
// 83 / 91 and 45 / 48, 16 x 32 51 / 45 and 33 / 28).
bool chunked(const gdn::SeqProblem &p, Which which) {
    if (p.dtype != GDN_DTYPE_BF16 || p.n_tokens == 0) return false;
    if (which == kPacked && !p.cu) return p.seq_len > kEqual;
    return which == kBwd || p.n_tokens >= 50 + (long long)p.n_seqs * p.H * (p.dv / 16) / 20;
}

size_t workspace_for(const gdn::SeqProblem &p, Which which) {
    if (which == kDecode) return 0;
    if (chunked(p, which)) return gdn::seq_chunk_workspace(p, which == kBwd);
    return which == kBwd ? gdn::seq_bwd_workspace(p, nullptr, nullptr) : 0;
}

int run(const gdn_seq_args *a, Which which) noexcept {
    try {
        static const char *const names[] = {"gdn_decode", "gdn_packed", "gdn_bwd"};
        gdn::NvtxRange range(names[which]);
        gdn::set_error_text("");
        if (!a) return fail(GDN_ERR_INVALID_ARG, "%s: args is NULL", names[which]);
        gdn::SeqProblem p;
        int st = check(*a, which, p);
        if (st != GDN_OK) return st;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(a->stream);
        auto cuda = [&](cudaError_t e, const char *what) {
            return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
        };
        if (p.status && (st = cuda(cudaMemsetAsync(p.status, 0, sizeof(int), s), "status word"))) return st;
        if (p.H == 0 || (p.n_seqs == 0 && p.n_tokens == 0)) return GDN_OK;
        const size_t need = workspace_for(p, which);
        void *ws = a->workspace;
        const bool owned = need && !ws;
        if (ws && a->workspace_bytes < need)
            return fail(GDN_ERR_NO_MEMORY, "workspace_bytes = %zu < %zu required", a->workspace_bytes, need);
        if (owned) {
            cudaError_t e = gdn::pool_scratch(&ws, need, s);
            if (e != cudaSuccess || !ws) {
                cudaGetLastError();
                return fail(GDN_ERR_NO_MEMORY, "device scratch allocation (%zu bytes) failed: %s", need, cudaGetErrorString(e));
            }
        }
        cudaError_t e = cudaSuccess;
        if (which == kBwd) e = chunked(p, which) ? gdn::launch_seq_bwd_chunk(p, ws, s) : gdn::launch_seq_bwd_simt(p, ws, s);
        else if (p.n_seqs && which == kPacked && chunked(p, which)) {
            const bool mixed = p.cu && p.n_tokens < kMixed * p.n_seqs;
            e = gdn::launch_seq_chunk(p, mixed ? short_len(p) : -1, ws, s);
        }
        else if (p.n_seqs) e = gdn::launch_seq_recurrent(p, which == kDecode, s);
        if (owned) {
            cudaError_t e2 = cudaFreeAsync(ws, s);
            if (e == cudaSuccess) e = e2;
        }
        return cuda(e, "kernel launch");
    } catch (...) {
        gdn::set_error_text("internal error (exception caught at the ABI boundary)");
        return GDN_ERR_CUDA;
    }
}

}  // namespace

extern "C" {

int gdn_decode(const gdn_seq_args *a) { return run(a, kDecode); }
int gdn_packed(const gdn_seq_args *a) { return run(a, kPacked); }
int gdn_bwd(const gdn_seq_args *a) { return run(a, kBwd); }

size_t gdn_seq_workspace_bytes(const gdn_seq_args *a, int bwd) {
    if (!a || check_sizes(*a) != GDN_OK || a->H == 0) return 0;
    gdn::SeqProblem p;
    memset(&p, 0, sizeof(p));
    p.dtype = a->dtype;
    p.cu = a->cu_seqlens;
    p.n_seqs = a->n_seqs; p.seq_len = a->seq_len; p.n_tokens = a->n_tokens;
    p.H = a->H; p.Hk = a->Hk; p.dk = a->d_k; p.dv = a->d_v;
    return workspace_for(p, bwd ? kBwd : kPacked);
}

}  // extern "C"
