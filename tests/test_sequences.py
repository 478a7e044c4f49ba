"""gdn_decode, gdn_packed, gdn_bwd and gated_delta_rule against the token loop in 64 bits.

Tolerances.  A result is a sum of N = d_k + T rounded fp32 terms (the dot products of a token, the
tokens that the state holds); roundings of 2^-24 with both signs add up like a walk, so sqrt(N)
2^-24 of the largest value, and 8 standard deviations of it are allowed: TOL32 = 8 sqrt(N) 2^-24.  A gradient
passes through four such sums one behind another (state, U, dU, dR), whose walks add: x 4.  A bf16
result is rounded once more: 2^-8 of its own value.
"""
import ctypes
import math

import pytest
import torch

import gated_deltanet_linear_chunkwise_b200 as g
from gated_deltanet_linear_chunkwise_b200 import binding

F64 = torch.float64


# ---------------------------------------------------------------- the definition, in 64 bits
def token_loop(q, k, v, alpha, beta, S, lens, first):
    """o rows and final states of sequences (first row, length) in fp64; differentiable."""
    N, H = alpha.shape
    rep = H // q.shape[1]
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    rows, states = {}, []
    for s, (a, n) in enumerate(zip(first, lens)):
        St = S[s]
        for t in range(a, a + n):
            St = alpha[t, :, None, None] * St
            u = beta[t, :, None] * (v[t] - (St * k[t, :, None, :]).sum(-1))
            St = St + u[..., None] * k[t, :, None, :]
            rows[t] = (St * q[t, :, None, :]).sum(-1)
        states.append(St)
    return rows, states


def draw(N, H, Hk, dk, dv, dtype, seed, gates="slow"):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v = unit(n(N, Hk, dk)).to(dt), unit(n(N, Hk, dk)).to(dt), n(N, H, dv).to(dt)
    alpha = torch.exp(-torch.nn.functional.softplus(n(N, H) + (2.0 if gates == "lit" else -4.0)))
    return q, k, v, alpha, torch.sigmoid(n(N, H))


def tol32(dk, T, passes=1):
    return 8 * passes * math.sqrt(dk + T) * 2.0 ** -24


def close(x, ref, tol, what=""):
    """|x - ref| <= tol max|ref| (+ half a bf16 step of the value)."""
    x, ref = x.detach().cpu(), ref.detach().cpu().to(F64)
    assert x.shape == ref.shape, (what, x.shape, ref.shape)
    if not ref.numel():
        return
    assert torch.isfinite(x.double()).all(), what
    allowed = tol * float(ref.abs().max()) + (2.0 ** -8 * ref.abs() if x.dtype == torch.bfloat16 else 0.0)
    off = ((x.to(F64) - ref).abs() - allowed).max()
    assert off <= 0, (what, float((x.to(F64) - ref).abs().max()), float(ref.abs().max()), tol)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ---------------------------------------------------------------- refusals (CPU)
FAKE = 1 << 40


def seq_args(which, **kw):
    a = binding.GdnSeqArgs()
    a.struct_size = ctypes.sizeof(binding.GdnSeqArgs)
    a.q, a.k, a.v, a.alpha, a.beta = (FAKE + (i << 24) for i in range(5))
    a.n_seqs, a.seq_len, a.n_tokens, a.n_slots = 2, 3, 6, 2
    a.H, a.Hk, a.d_k, a.d_v = 4, 2, 64, 64
    if which == "gdn_bwd":
        a.d_o, a.dq, a.dk, a.dv, a.dalpha, a.dbeta = (FAKE + (i << 24) for i in range(5, 11))
    else:
        a.o = FAKE + (11 << 24)
        if which == "gdn_decode":
            a.S_in = a.S_out = FAKE + (12 << 24)
    for name, value in kw.items():
        setattr(a, name, value)
    return a


ALL = ("gdn_decode", "gdn_packed", "gdn_bwd")


@pytest.mark.parametrize("kw,status,text,which", [
    (dict(struct_size=8), 1, "struct_size", ALL),
    (dict(dtype=2), 1, "dtype", ALL),
    (dict(n_seqs=-1), 1, "negative", ALL),
    (dict(d_k=72), 3, "d_k", ALL), (dict(d_v=144), 3, "d_v", ALL), (dict(d_k=0), 3, "d_k", ALL),
    (dict(Hk=3), 2, "multiple of Hk", ALL), (dict(Hk=0), 2, "multiple of Hk", ALL),
    (dict(n_tokens=7), 2, "n_tokens", ALL),
    (dict(n_tokens=1 << 31, seq_len=1 << 30), 2, "2^31", ALL),
    (dict(n_seqs=1 << 30, n_tokens=3 << 30, n_slots=1 << 30), 2, "2^31", ALL),
    (dict(n_seqs=1 << 20, n_tokens=3 << 20, n_slots=1 << 20, H=1 << 10, Hk=1 << 10), 2, "2^31", ALL),
    (dict(q_stride=64), 1, "q_stride", ALL), (dict(v_stride=260), 4, "v_stride", ALL),
    (dict(q=None), 1, "required", ALL), (dict(alpha=None), 1, "required", ALL),
    (dict(k=FAKE + 8), 4, "k =", ALL),
    (dict(status_dev=FAKE + (13 << 24) + 2), 4, "status_dev", ALL),
    (dict(status_dev=FAKE), 1, "status_dev overlaps input q", ALL),
    (dict(o=None), 1, "o is required", ALL[:2]),
    (dict(o=FAKE + (2 << 24)), 1, "o overlaps input v", ALL[:2]),
    (dict(dq=FAKE + (20 << 24)), 1, "gdn_bwd", ALL[:2]),
    (dict(n_slots=1, S_in=FAKE + (12 << 24), S_out=FAKE + (12 << 24)), 2, "n_slots", ALL[:2]),
    (dict(slots=FAKE + (14 << 24) + 2), 4, "slots", ALL[:2]),
    (dict(S_in=FAKE + (12 << 24) + 64, S_out=FAKE + (12 << 24)), 1, "", ALL[:2]),   # partly over one another
    (dict(S_out=None), 1, "in place", ALL[:1]), (dict(S_in=None), 1, "in place", ALL[:1]),
    (dict(fresh=FAKE + (14 << 24)), 1, "fresh", ALL[:1]), (dict(cu_seqlens=FAKE + (14 << 24)), 1, "cu_seqlens", ALL[:1]),
    (dict(d_o=None), 1, "required", ALL[2:]), (dict(dbeta=None), 1, "required", ALL[2:]),
    (dict(slots=FAKE + (14 << 24)), 1, "no o, S_out, slots", ALL[2:]),
    (dict(dq=FAKE + (5 << 24)), 1, "dq overlaps input d_o", ALL[2:]),
    (dict(dv=FAKE + (6 << 24)), 1, "dv overlaps dq", ALL[2:]),
    (dict(workspace=FAKE + (1 << 32), workspace_bytes=256), 5, "workspace_bytes", ALL[2:]),
    (dict(workspace=FAKE + (1 << 32) + 16, workspace_bytes=1 << 30), 4, "workspace", ALL[2:]),
])
def test_refusals(kw, status, text, which):
    for name in which:
        rc = getattr(g.load_library(), name)(ctypes.byref(seq_args(name, **kw)))
        assert rc == status and text in g.last_error(), (name, rc, g.last_error())


def test_null_args_and_empty_calls():
    lib = g.load_library()
    for name in ALL:
        assert getattr(lib, name)(None) == 1 and name in g.last_error()
        for kw in (dict(n_seqs=0, n_tokens=0, seq_len=0), dict(H=0, Hk=0)):  # nothing to do, nothing launched
            assert getattr(lib, name)(ctypes.byref(seq_args(name, **kw))) == 0, g.last_error()


def test_struct_layout():
    assert ctypes.sizeof(binding.GdnSeqArgs) == 256  # LP64 layout of gdn_seq_args


def test_workspace_sizes():
    w = g.seq_workspace_bytes
    assert w(640, 4, 4, 64, 64, n_seqs=5, bwd=True) > w(320, 4, 4, 64, 64, n_seqs=5, bwd=True) > 0
    assert w(640, 4, 2, 64, 64, n_seqs=5, bwd=True) > w(640, 4, 4, 64, 64, n_seqs=5, bwd=True)  # the heads' own gradients
    assert w(640, 4, 3, 64, 64, n_seqs=5, bwd=True) == 0 and w(640, 4, 4, 60, 64, n_seqs=5, bwd=True) == 0


@pytest.mark.parametrize("call", [
    lambda x, a, S: g.gdn_decode(x, x, x, a, a, S),
    lambda x, a, S: g.gdn_packed(x, x, x, a, a),
    lambda x, a, S: g.gdn_bwd(x, x, x, a, a, x),
    lambda x, a, S: g.gdn_decode(x, x, None, a, a, S),
    lambda x, a, S: g.gdn_packed(x[0], x[0], x[0], a[0], a[0]),              # 3-D without cu_seqlens
    lambda x, a, S: g.gdn_packed(x, x, x, a, a, torch.zeros(2, dtype=torch.int32)),  # 4-D with them
])
def test_binding_refuses_on_cpu(call):
    with pytest.raises(g.GdnError):
        call(torch.zeros(2, 3, 2, 16), torch.zeros(2, 3, 2), torch.zeros(2, 2, 16, 16))


# ---------------------------------------------------------------- decode
DECODE = [
    # B, n, H, Hk, dk, dv, dtype, gates
    (1, 1, 2, 2, 16, 16, "bf16", "slow"),
    (3, 1, 20, 20, 112, 112, "bf16", "slow"),
    (5, 3, 6, 2, 128, 48, "bf16", "lit"),
    (2, 8, 4, 1, 32, 128, "fp32", "slow"),
    (70, 1, 3, 3, 96, 80, "fp32", "lit"),
    (1, 33, 1, 1, 64, 112, "bf16", "slow"),
    (75, 2, 20, 10, 32, 48, "bf16", "slow"),  # a block a head
    (1, 0, 2, 2, 32, 32, "bf16", "slow"),     # no token: the states stay
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,n,H,Hk,dk,dv,dtype,gates", DECODE)
def test_decode(B, n, H, Hk, dk, dv, dtype, gates):
    q, k, v, alpha, beta = draw(B * n, H, Hk, dk, dv, dtype, 7 + B, gates)
    pool = torch.randn(B + 3, H, dv, dk, generator=torch.Generator().manual_seed(1))
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(2))[:B].int()
    rows, states = token_loop(q.double(), k.double(), v.double(), alpha.double(), beta.double(),
                              pool.double()[slots.long()], [n] * B, [n * i for i in range(B)])
    want = pool.double()
    want[slots.long()] = torch.stack(states)
    S = pool.cuda()
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    args = [t.cuda().reshape(B, n, *t.shape[1:]) for t in (q, k, v, alpha, beta)]
    o, S2 = g.gdn_decode(*args, S, slots.cuda(), status=status)
    assert S2 is S and int(status) == 0
    if n:
        close(o.reshape(B * n, H, dv), torch.stack([rows[t] for t in range(B * n)]), tol32(dk, n), "o")
    close(S, want, tol32(dk, n), "S")
    if n == 1:  # the n dimension left out; no slots: state b is sequence b's
        S3 = pool[slots.long()].cuda()
        o3, _ = g.gdn_decode(*[t[:, 0] for t in args], S3)
        assert torch.equal(o3, o[:, 0]) and torch.equal(S3, S[slots.long().cuda()])


@pytest.mark.gpu
def test_decode_padding_and_bad_slots():
    B, H, dk, dv = 8, 2, 48, 32
    q, k, v, alpha, beta = cuda(*draw(B, H, H, dk, dv, "bf16", 3))
    pool = torch.randn(6, H, dv, dk).cuda()
    slots = torch.tensor([2, -1, 0, 2, 6, 1 << 30, 5, -7], dtype=torch.int32, device="cuda")
    S, o = pool.clone(), torch.full((B, H, dv), 5.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.gdn_decode(q, k, v, alpha, beta, S, slots, o=o, status=status)
    assert int(status) == binding.GDN_SEQ_BAD_SLOT | binding.GDN_SEQ_SAME_SLOT
    ran = [0, 2, 6]
    S1 = pool[slots[ran].long()].clone()
    o1, _ = g.gdn_decode(q[ran], k[ran], v[ran], alpha[ran], beta[ran], S1)
    assert torch.equal(o[ran], o1) and torch.equal(S[slots[ran].long()], S1)
    left = [1, 3, 4, 5, 7]
    assert (o[left] == 5).all()
    untouched = [i for i in range(6) if i not in (2, 0, 5)]
    assert torch.equal(S[untouched], pool[untouched])


def fused(q, k, v):
    """q, k, v as slices of the rows of one fused projection."""
    lead = q.shape[:-2]
    w = [t.shape[-1] * t.shape[-2] for t in (q, k, v)]
    row = torch.randn(*lead, sum(w) + 16, device=q.device).to(q.dtype)
    out, at = [], 8
    for t, n in zip((q, k, v), w):
        row[..., at:at + n] = t.reshape(*lead, n)
        out.append(row[..., at:at + n].unflatten(-1, t.shape[-2:]))
        at += n
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_rows(dtype):
    B, n, H, Hk, dk, dv = 3, 70, 4, 2, 48, 80
    q, k, v, alpha, beta = [t.cuda().reshape(B, n, *t.shape[1:]) for t in draw(B * n, H, Hk, dk, dv, dtype, 5)]
    fq, fk, fv = fused(q, k, v)
    assert not fq.is_contiguous()
    S = torch.randn(B, H, dv, dk).cuda()
    S1, S2 = S.clone(), S.clone()
    assert torch.equal(g.gdn_decode(q, k, v, alpha, beta, S1)[0], g.gdn_decode(fq, fk, fv, alpha, beta, S2)[0])
    assert torch.equal(S1, S2)
    a, b = (g.gdn_packed(*x, alpha, beta, None, S, return_state=True) for x in ((q, k, v), (fq, fk, fv)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    do = torch.randn_like(v)
    for x, y in zip(g.gdn_bwd(q, k, v, alpha, beta, do, None, S), g.gdn_bwd(fq, fk, fv, alpha, beta, do, None, S)):
        assert torch.equal(x, y)
    with pytest.raises(g.GdnError, match="heads of a token"):
        g.gdn_decode(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, alpha, beta, S1)
    with pytest.raises(g.GdnError, match="equally far"):
        wide = torch.zeros(B, n + 1, Hk, dk, device="cuda", dtype=q.dtype)
        g.gdn_packed(wide[:, :n], k, v, alpha, beta)


# ---------------------------------------------------------------- packed
PACKED = [
    # lens, first row, rows behind, H, Hk, dk, dv, dtype, gates
    ([1], 0, 0, 1, 1, 16, 16, "bf16", "slow"),
    ([64], 0, 0, 2, 2, 112, 112, "bf16", "slow"),
    ([65, 1, 0, 63, 64, 130], 0, 0, 4, 2, 64, 48, "bf16", "slow"),
    ([200], 3, 5, 2, 1, 128, 128, "bf16", "lit"),
    ([0, 0, 17, 300, 0], 1, 70, 3, 3, 80, 96, "bf16", "slow"),
    ([129, 7, 256], 0, 0, 2, 2, 32, 64, "fp32", "slow"),
    ([33, 150], 2, 2, 4, 1, 128, 112, "fp32", "lit"),
    ([5] * 40, 0, 0, 2, 2, 48, 32, "bf16", "slow"),
    ([3, 0, 9, 20], 1, 1, 4, 2, 112, 48, "bf16", "lit"),   # few tokens: token by token
    # chains enough for a warp a slice of 16 columns (900 and more of them): blocks of four slices and of three
    ([17] * 64, 0, 0, 4, 2, 48, 64, "bf16", "slow"),
    ([64, 65, 1, 0, 130] * 13, 2, 3, 2, 1, 32, 112, "bf16", "slow"),
    ([2, 40] * 32, 0, 0, 2, 2, 112, 112, "bf16", "lit"),
]


def packed_case(lens, first, behind, H, Hk, dk, dv, dtype, gates, seed=11):
    N = first + sum(lens) + behind
    tensors = draw(N, H, Hk, dk, dv, dtype, seed, gates)
    starts = [first + sum(lens[:i]) for i in range(len(lens))]
    cu = torch.tensor(starts + [first + sum(lens)], dtype=torch.int32)
    return tensors, starts, cu


@pytest.mark.gpu
@pytest.mark.parametrize("lens,first,behind,H,Hk,dk,dv,dtype,gates", PACKED)
@pytest.mark.parametrize("with_state", [False, True])
def test_packed(lens, first, behind, H, Hk, dk, dv, dtype, gates, with_state):
    (q, k, v, alpha, beta), starts, cu = packed_case(lens, first, behind, H, Hk, dk, dv, dtype, gates)
    n, T = len(lens), max(lens)
    alpha[first] = 0.0  # a full reset
    alpha[-1 - behind] = 1.0
    pool = torch.randn(n + 2, H, dv, dk, generator=torch.Generator().manual_seed(4))
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(5))[:n].int()
    fresh = torch.arange(n) % 3 == 1
    S0 = torch.zeros(n, H, dv, dk, dtype=F64)
    if with_state:
        S0 = pool.double()[slots.long()] * ~fresh[:, None, None, None]
    rows, states = token_loop(*(t.double() for t in (q, k, v, alpha, beta)), S0, lens, starts)
    dq, dk_, dv_, da, db = cuda(q, k, v, alpha, beta)
    o = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    if with_state:
        S = pool.cuda()
        g.gdn_packed(dq, dk_, dv_, da, db, cu.cuda(), S, S_out=S, slots=slots.cuda(), fresh=fresh.cuda(), o=o, status=status)
        want = pool.double()
        want[slots.long()] = torch.stack(states)
    else:
        _, S = g.gdn_packed(dq, dk_, dv_, da, db, cu.cuda(), return_state=True, o=o, status=status)
        want = torch.stack(states)
    assert int(status) == 0
    close(S, want, tol32(dk, T), "S")
    covered = sorted(rows)
    close(o[covered], torch.stack([rows[t] for t in covered]), tol32(dk, T), "o")
    rest = [t for t in range(v.shape[0]) if t not in rows]
    assert (o[rest] == 7).all()


@pytest.mark.gpu
def test_packed_bad_ranges_and_slots():
    H, dk, dv = 2, 64, 64
    q, k, v, alpha, beta = cuda(*draw(200, H, H, dk, dv, "bf16", 9))
    cu = torch.tensor([0, 70, 900, 60, 100, -5, 200], dtype=torch.int32, device="cuda")
    # good: [0, 70); out of range: [70, 900), [900, 60), [100, -5), [-5, 200); shares rows with the first: none
    cu[3] = 80  # [900, 80) stays bad, [80, 100) is good
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    _, S = g.gdn_packed(q, k, v, alpha, beta, cu, return_state=True, o=o, status=status)
    assert int(status) == binding.GDN_SEQ_BAD_ROWS
    for s, (a, b) in {0: (0, 70), 3: (80, 100)}.items():  # alone a sequence may take another kernel: two TOL32 and a bf16 step
        o1, S1 = g.gdn_packed(*(t[None, a:b] for t in (q, k, v, alpha, beta)), return_state=True)
        close(o[a:b], o1[0], 2 * tol32(dk, 70) + 2.0 ** -8)
        close(S[s], S1[0], 2 * tol32(dk, 70))
    assert (o[70:80] == 7).all() and (o[100:] == 7).all()
    # gradients: zeros where no good sequence is
    do = torch.randn_like(v)
    got = g.gdn_bwd(q, k, v, alpha, beta, do, cu, status=status, need_dS_in=True)
    assert int(status) == binding.GDN_SEQ_BAD_ROWS
    for s, (a, b) in {0: (0, 70), 3: (80, 100)}.items():
        one = g.gdn_bwd(*(t[None, a:b] for t in (q, k, v, alpha, beta)), do[None, a:b].contiguous(), need_dS_in=True)
        for x, y in zip(got[:5], one):
            assert torch.equal(x[a:b], y[0])
        assert torch.equal(got[5][s], one[5][0])
    for x in got[:5]:
        assert not x[70:80].any() and not x[100:].any()
    assert not got[5][[1, 2, 4, 5]].any()
    # two sequences of one slot: the first runs
    cu = torch.tensor([0, 70, 100, 200], dtype=torch.int32, device="cuda")
    pool = torch.randn(3, H, dv, dk).cuda()
    S, o = pool.clone(), torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    g.gdn_packed(q, k, v, alpha, beta, cu, S, S_out=S, slots=torch.tensor([1, 1, 3], dtype=torch.int32).cuda(), o=o, status=status)
    assert int(status) == binding.GDN_SEQ_SAME_SLOT | binding.GDN_SEQ_BAD_SLOT
    o1, S1 = g.gdn_packed(*(t[None, :70] for t in (q, k, v, alpha, beta)), None, pool[1:2], return_state=True)
    assert torch.equal(o[:70], o1[0]) and torch.equal(S[1], S1[0]) and (o[70:] == 7).all()
    assert torch.equal(S[[0, 2]], pool[[0, 2]])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 75])
def test_neighbours_do_not_mix(n):
    """What is not finite in one sequence stays there: chunks end inside the tiles that hold the next one's rows."""
    H, dk, dv, L = 2, 64, 112, 70
    q, k, v, alpha, beta = cuda(*draw(n * L, H, H, dk, dv, "bf16", 71))
    do = torch.randn_like(v)
    cu = torch.arange(0, n * L + 1, L, dtype=torch.int32, device="cuda")
    clean = [*g.gdn_packed(q, k, v, alpha, beta, cu, return_state=True), *g.gdn_bwd(q, k, v, alpha, beta, do, cu, need_dS_in=True)]
    for t in (q, k, v, do):
        t[L:2 * L] = float("nan")
        t[2 * L - 1] = float("inf")
    dirty = [*g.gdn_packed(q, k, v, alpha, beta, cu, return_state=True), *g.gdn_bwd(q, k, v, alpha, beta, do, cu, need_dS_in=True)]
    for x, y in zip(clean, dirty):
        one = L if x.shape[0] == n * L else 1
        assert torch.equal(x[:one], y[:one]) and torch.equal(x[2 * one:], y[2 * one:])
        assert not torch.isfinite(y[one:2 * one].double()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompt_then_tokens(dtype):
    """A prompt in two pieces and then token by token leaves what one pass leaves."""
    H, Hk, dk, dv, T = 4, 2, 112, 96, 150
    q, k, v, alpha, beta = cuda(*draw(T, H, Hk, dk, dv, dtype, 21))
    whole_o, whole_S = g.gdn_packed(*(t[None] for t in (q, k, v, alpha, beta)), return_state=True)
    S = torch.randn(3, H, dv, dk).cuda()
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([True], device="cuda")
    outs = []
    for a, b in ((0, 77), (77, 140)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        outs.append(g.gdn_packed(*(t[a:b] for t in (q, k, v, alpha, beta)), cu, S, S_out=S, slots=slot,
                                 fresh=fresh if a == 0 else None)[0])
    for t in range(140, T):
        outs.append(g.gdn_decode(*(x[t:t + 1] for x in (q, k, v, alpha, beta)), S, slot)[0])
    # two fp32 evaluations, each TOL32 from the exact one
    close(torch.cat(outs), whole_o[0].double(), 2 * tol32(dk, T) + (2.0 ** -8 if dtype == "bf16" else 0), "o")
    close(S[2], whole_S[0].double(), 2 * tol32(dk, T), "S")


@pytest.mark.gpu
def test_packed_is_the_frames_pass():
    """Whole frames: what gdn_fwd computes in fp32."""
    B, T, H, d = 2, 256, 3, 64
    q, k, v, alpha, beta = [t.cuda().reshape(B, T, *t.shape[1:]) for t in draw(B * T, H, H, d, d, "fp32", 2)]
    o, S = g.gdn_packed(q, k, v, alpha, beta, return_state=True)
    o1, S1 = g.gdn_fwd(q, k, v, alpha, beta, 64, return_state=True)
    close(o, o1.double(), 1e-5, "o")  # gdn_fwd's own bar in fp32
    close(S, S1.double(), 1e-5, "S")


# ---------------------------------------------------------------- gradients
def exact_grads(tensors, starts, lens, S_in, do, dS_out):
    """The token loop's gradients, by differentiating it in 64 bits."""
    leaves = [t.double().requires_grad_(True) for t in tensors] + [S_in.double().requires_grad_(True)]
    rows, states = token_loop(*leaves, lens, starts)
    loss = (torch.stack(states) * dS_out.double()).sum()
    for t, o in rows.items():
        loss = loss + (o * do[t].double()).sum()
    loss.backward()
    return [torch.zeros_like(x) if x.grad is None else x.grad for x in leaves]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,first,behind,H,Hk,dk,dv,dtype,gates", PACKED)
def test_gradients(lens, first, behind, H, Hk, dk, dv, dtype, gates):
    tensors, starts, cu = packed_case(lens, first, behind, H, Hk, dk, dv, dtype, gates, seed=13)
    n, T = len(lens), max(lens)
    gen = torch.Generator().manual_seed(6)
    do = torch.randn(tensors[2].shape, generator=gen).to(tensors[2].dtype)
    S_in, dS_out = torch.randn(n, H, dv, dk, generator=gen), torch.randn(n, H, dv, dk, generator=gen)
    want = exact_grads(tensors, starts, lens, S_in, do, dS_out)
    got = g.gdn_bwd(*cuda(*tensors), do.cuda(), cu.cuda(), S_in.cuda(), dS_out=dS_out.cuda())
    for name, x, y in zip(("dq", "dk", "dv", "dalpha", "dbeta", "dS_in"), got, want):
        close(x, y, tol32(dk, T, 4), name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_of_resets(dtype):
    """alpha = 0 and tiny alphas: the outputs are affine in each alpha, and its gradient is not lost."""
    T, H, dk, dv = 140, 2, 32, 48
    tensors = draw(T, H, H, dk, dv, dtype, 31)
    alpha = tensors[3]
    alpha[[5, 64, 65, 127]] = 0.0
    alpha[20], alpha[100] = 1e-30, 1e-12
    do = torch.randn(T, H, dv, generator=torch.Generator().manual_seed(8)).to(tensors[2].dtype)
    S = torch.randn(1, H, dv, dk, generator=torch.Generator().manual_seed(9))
    want = exact_grads(tensors, [0], [T], S, do, S)
    got = g.gdn_bwd(*(t.cuda()[None] for t in tensors), do.cuda()[None], None, S.cuda(), dS_out=S.cuda())
    for name, x, y in zip(("dq", "dk", "dv", "dalpha", "dbeta"), got, want):
        close(x[0], y, tol32(dk, T, 4), name)
    # the reset tokens' own entries, against their own size
    at = [5, 20, 64, 65, 100, 127]
    close(got[3][0, at], want[3][at], tol32(dk, T, 4), "dalpha at resets")


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of the fp64 loop at a few entries.  Step h: the loss is a polynomial of the entry whose third
    derivative is of its own order, so the error is h^2 + 2^-52 / h of it: 1e-9 at h = 1e-5."""
    lens, starts, H, Hk, dk, dv = [70, 3], [0, 70], 2, 1, 16, 16
    tensors, _, cu = packed_case(lens, 0, 0, H, Hk, dk, dv, "fp32", "slow", seed=17)
    gen = torch.Generator().manual_seed(3)
    S_in, dS_out = torch.randn(2, H, dv, dk, generator=gen), torch.randn(2, H, dv, dk, generator=gen)
    do = torch.randn(tensors[2].shape, generator=gen)

    def loss(leaves):
        rows, states = token_loop(*leaves, lens, starts)
        return float((torch.stack(states) * dS_out.double()).sum() + sum((rows[t] * do[t].double()).sum() for t in rows))

    got = g.gdn_bwd(*cuda(*tensors), do.cuda(), cu.cuda(), S_in.cuda(), dS_out=dS_out.cuda())
    base = [t.double() for t in tensors] + [S_in.double()]
    for i, x in enumerate(got):
        for at in torch.randint(base[i].numel(), (4,), generator=gen).tolist():
            d = []
            for sign in (1, -1):
                leaves = [t.clone() for t in base]
                leaves[i].view(-1)[at] += sign * 1e-5
                d.append(loss(leaves))
            diff = (d[0] - d[1]) / 2e-5
            assert abs(float(x.reshape(-1)[at]) - diff) <= tol32(dk, 70, 4) * float(x.abs().max()) + 1e-7, (i, at)


@pytest.mark.gpu
def test_gradients_leave_out_what_is_not_asked():
    q, k, v, alpha, beta = cuda(*(t[None] for t in draw(100, 2, 2, 64, 64, "bf16", 3)))
    do = torch.randn_like(v)
    zero = torch.zeros(1, 2, 64, 64, device="cuda")
    full = g.gdn_bwd(q, k, v, alpha, beta, do, None, zero, dS_out=zero)
    short = g.gdn_bwd(q, k, v, alpha, beta, do)
    assert short[5] is None
    for x, y in zip(short[:5], full):
        assert torch.equal(x, y)
    assert torch.equal(g.gdn_bwd(q, k, v, alpha, beta, do, need_dS_in=True)[5], full[5])


# ---------------------------------------------------------------- the differentiable function
@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_autograd(packed):
    B, T, H, Hk, dk, dv = 2, 90, 4, 2, 48, 64
    tensors = draw(B * T, H, Hk, dk, dv, "fp32", 41)
    S_in = torch.randn(B, H, dv, dk, generator=torch.Generator().manual_seed(1))
    lens, starts = [T] * B, [0, T]
    leaves = [t.double().requires_grad_(True) for t in tensors] + [S_in.double().requires_grad_(True)]
    rows, states = token_loop(*leaves, lens, starts)
    o_ref, S_ref = torch.stack([rows[t] for t in range(B * T)]), torch.stack(states)
    ((o_ref ** 2).sum() + (S_ref ** 3).sum()).backward()
    shape = (lambda t: t) if packed else (lambda t: t.reshape(B, T, *t.shape[1:]))
    mine = [shape(t).cuda().requires_grad_(True) for t in tensors] + [S_in.cuda().requires_grad_(True)]
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda") if packed else None
    o, S = g.gated_delta_rule(*mine, cu)
    ((o ** 2).sum() + (S ** 3).sum()).backward()
    # the loss's own gradients carry the forward's error: one more pass
    for name, x, y in zip(("q", "k", "v", "alpha", "beta", "S_in"), mine, leaves):
        close(x.grad.reshape(y.grad.shape), y.grad, tol32(dk, T, 5 * 3), name)
    # one output only, and inputs that need none
    q = mine[0].detach().clone().requires_grad_(True)
    o, S = g.gated_delta_rule(q, *(t.detach() for t in mine[1:]), cu)
    S.sum().backward()
    assert torch.equal(q.grad, torch.zeros_like(q))  # the final state does not read q


@pytest.mark.gpu
def test_streams_and_graphs():
    B, n, H, d = 4, 100, 4, 64
    q, k, v, alpha, beta = [t.cuda().reshape(B, n, *t.shape[1:]) for t in draw(B * n, H, H, d, d, "bf16", 51)]
    do, S0 = torch.randn_like(v), torch.randn(B, H, d, d, device="cuda")

    def everything(stream=None):
        S = S0.clone()
        kw = {"stream": stream}
        o, S1 = g.gdn_packed(q, k, v, alpha, beta, None, S, return_state=True, **kw)
        o2, _ = g.gdn_decode(q[:, :2].contiguous(), k[:, :2].contiguous(), v[:, :2].contiguous(), alpha[:, :2].contiguous(), beta[:, :2].contiguous(), S1, **kw)
        return [o, S1, o2, *g.gdn_bwd(q, k, v, alpha, beta, do, None, S, **kw)]

    want = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = everything()
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    side.wait_stream(torch.cuda.current_stream())
    S = S0.clone()
    side.wait_stream(torch.cuda.current_stream())
    o, S1 = g.gdn_packed(q, k, v, alpha, beta, None, S, return_state=True, stream=side)  # the stream as an argument
    grads = g.gdn_bwd(q, k, v, alpha, beta, do, None, S, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])
    for x, y in zip(grads, want[3:]):
        assert torch.equal(x, y)
    graphs, results = [], []
    for _ in range(2):  # two graphs: each keeps scratch of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(everything())
        graphs.append(graph)
    for _ in range(3):
        for r in results:
            for x in r:
                x.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for r in results:
            for x, y in zip(r, want):
                assert torch.equal(x, y)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls that run beside one another share no scratch."""
    H, d, n = 4, 64, 300
    sets = []
    for seed in (1, 2):
        q, k, v, alpha, beta = [t.cuda()[None] for t in draw(n, H, H, d, d, "bf16", seed)]
        do = torch.randn_like(v)
        sets.append((q, k, v, alpha, beta, do))
    run = lambda s: [*g.gdn_packed(*s[:5], return_state=True), *g.gdn_bwd(*s)[:5]]  # noqa: E731
    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(run(s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.gpu
def test_same_bits_again():
    q, k, v, alpha, beta = cuda(*draw(700, 4, 2, 112, 112, "bf16", 61))
    cu = torch.tensor([0, 300, 301, 700], dtype=torch.int32, device="cuda")
    do = torch.randn_like(v)
    one, two = ([*g.gdn_packed(q, k, v, alpha, beta, cu, return_state=True), *g.gdn_bwd(q, k, v, alpha, beta, do, cu, need_dS_in=True)] for _ in range(2))
    for x, y in zip(one, two):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [2, 75])  # four warps a slice, and one
def test_a_wait_that_gives_up(seqs, monkeypatch):
    """The first block's keys are never fetched: its wait runs out, the status says so, and the next call is right."""
    H, L, d, dv = 4, 70, 64, 48
    q, k, v, alpha, beta = [t.cuda().reshape(seqs, L, *t.shape[1:]) for t in draw(seqs * L, H, H, d, dv, "bf16", 81)]
    do = torch.randn_like(v)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both():
        return [*g.gdn_packed(q, k, v, alpha, beta, return_state=True, status=status), *g.gdn_bwd(q, k, v, alpha, beta, do)]

    want = both()
    assert int(status) == 0
    monkeypatch.setenv("GDN_DEBUG_DROP_SIGNAL", "1")
    monkeypatch.setenv("GDN_DEBUG_WAIT_LIMIT_US", "1000")
    g.gdn_packed(q, k, v, alpha, beta, status=status)
    assert int(status) == binding.GDN_SEQ_TIMEOUT
    g.gdn_bwd(q, k, v, alpha, beta, do, status=status)
    assert int(status) == binding.GDN_SEQ_TIMEOUT
    monkeypatch.undo()
    for x, y in zip(both()[:7], want):
        assert torch.equal(x, y)
    assert int(status) == 0
