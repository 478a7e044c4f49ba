"""The sequence operators at the edges of what their callers may pass.  Tolerances as in test_sequences.py."""
import random

import pytest
import torch

import gated_deltanet_linear_chunkwise_b200 as g
from gated_deltanet_linear_chunkwise_b200 import binding
from test_sequences import F64, close, cuda, draw, exact_grads, packed_case, tol32, token_loop


# ---------------------------------------------------------------- rows of q, k and v
def rows_apart(t, lead):
    return binding._tokens("q", t, t.dtype, t.device, lead, t.shape[-2], t.shape[-1])


@pytest.mark.parametrize("t,lead", [
    (torch.zeros(1, 2, 64).expand(5, 2, 64), (5,)),                       # one token for all
    (torch.zeros(1, 1, 2, 64).expand(5, 7, 2, 64), (5, 7)),
    (torch.zeros(1, 1, 2, 64).expand(1, 7, 2, 64), (1, 7)),
    (torch.zeros(1, 1, 2, 64).expand(5, 1, 2, 64), (5, 1)),
    (torch.zeros(1, 1, 64).expand(5, 1, 64), (5,)),                       # one head
    (torch.zeros(6 * 64 + 64).as_strided((5, 2, 64), (64, 64, 1)), (5,)),  # a row starts inside the one before
])
def test_rows_over_one_another_are_refused(t, lead):
    with pytest.raises(g.GdnError, match="over one another"):
        rows_apart(t, lead)


@pytest.mark.parametrize("t,lead,step", [
    (torch.zeros(5, 1, 384)[..., :128].view(5, 1, 2, 64), (5, 1), 384),              # a step behind one projection
    (torch.zeros(5, 384)[:, :128].unflatten(-1, (2, 64)).unsqueeze(1), (5, 1), 384),
    (torch.zeros(5, 9, 384)[:, 3:4, 128:256].unflatten(-1, (2, 64)), (5, 1), 9 * 384),  # one token of each of five rows
    (torch.zeros(5, 9, 384)[:1, :, 128:256].unflatten(-1, (2, 64)), (1, 9), 384),
    (torch.zeros(5, 9, 384)[..., :64].unflatten(-1, (1, 64)), (5, 9), 384),
    (torch.zeros(5, 9, 2, 64), (5, 9), 128),
])
def test_rows_apart(t, lead, step):
    assert rows_apart(t, lead) == step


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_token_slices_of_a_projection(dtype):
    """[B, 1, ...] slices of a fused projection are the same call as their copies."""
    B, H, Hk, dk, dv = 5, 4, 2, 48, 80
    q, k, v, alpha, beta = [t.reshape(B, 1, *t.shape[1:]) for t in cuda(*draw(B, H, Hk, dk, dv, dtype, 15))]
    at = [Hk * dk, 2 * Hk * dk]
    row = torch.cat([t.flatten(2) for t in (q, k, v)], -1)
    slices = [row[..., :at[0]].unflatten(-1, (Hk, dk)), row[..., at[0]:at[1]].unflatten(-1, (Hk, dk)), row[..., at[1]:].unflatten(-1, (H, dv))]
    assert not slices[0].is_contiguous()
    S = torch.randn(B, H, dv, dk).cuda()
    do = torch.randn_like(v)

    def everything(q, k, v):
        Sd = S.clone()
        o, _ = g.gdn_decode(q, k, v, alpha, beta, Sd)
        return [o, Sd, *g.gdn_packed(q, k, v, alpha, beta, None, S, return_state=True), *g.gdn_bwd(q, k, v, alpha, beta, do, None, S)]

    for x, y in zip(everything(*slices), everything(q, k, v)):
        assert torch.equal(x, y)


# ---------------------------------------------------------------- sequences out of order
def in_order(cu, N):
    """The sequences that run: ordered ranges inside the tensors, none of which an earlier one reaches into."""
    ok = [0 <= a <= b <= N for a, b in zip(cu, cu[1:])]
    ends = [b if o and b > a else 0 for o, a, b in zip(ok, cu, cu[1:])]
    return [o and (a == b or a >= max(ends[:s], default=0)) for s, (o, a, b) in enumerate(zip(ok, cu, cu[1:]))]


def shuffled(n, N, seed):
    rng = random.Random(seed)
    cu = sorted(rng.randint(0, N) for _ in range(n + 1))
    for _ in range(n // 20):
        i, j = rng.randint(0, n), rng.randint(0, n)
        cu[i], cu[j] = cu[j], cu[i]
    return cu


OUT_OF_ORDER = [
    [100, 200, 0, 64],          # two ranges that would share a chunk's index
    [0, 150, 100, 200],         # two that share rows
    [50, 50, 0, 30, 200],       # an empty one reaches nowhere
    [0, 64, 10, 10, 64, 199],   # an empty one inside another
    [130, 140, 0, 130, 140, 200],
    shuffled(300, 2000, 3),     # chains enough for a warp a slice; more sequences than a block has threads
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cu", OUT_OF_ORDER, ids=lambda c: str(len(c) - 1))
def test_sequences_out_of_order(cu, dtype):
    N, H, Hk, dk, dv = max(cu), 4, 2, 32, 64
    n = len(cu) - 1
    good = in_order(cu, N)
    assert not all(good) and any(good)
    tensors = draw(N, H, Hk, dk, dv, dtype, 19)
    gen = torch.Generator().manual_seed(5)
    do = torch.randn(tensors[2].shape, generator=gen).to(tensors[2].dtype)
    S, dS = torch.randn(n, H, dv, dk, generator=gen), torch.randn(n, H, dv, dk, generator=gen)
    run = [s for s in range(n) if good[s]]
    lens, starts = [cu[s + 1] - cu[s] for s in run], [cu[s] for s in run]
    rows, states = token_loop(*(t.double() for t in tensors), S[run].double(), lens, starts)
    tol, T = tol32(dk, max(lens)), max(lens)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S_out = torch.full(tensors[2].shape, 7.0, dtype=tensors[2].dtype, device="cuda"), torch.full(S.shape, 7.0, device="cuda")
    at = torch.tensor(cu, dtype=torch.int32, device="cuda")
    g.gdn_packed(*cuda(*tensors), at, S.cuda(), S_out=S_out, o=o, status=status)
    assert int(status) == binding.GDN_SEQ_BAD_ROWS
    covered, skipped = sorted(rows), [s for s in range(n) if not good[s]]
    close(o[covered], torch.stack([rows[t] for t in covered]), tol, "o")
    close(S_out[run], torch.stack(states), tol, "S")
    left = [t for t in range(N) if t not in rows]
    assert (o[left] == 7).all() and (S_out[skipped] == 7).all()
    status.zero_()
    got = g.gdn_bwd(*cuda(*tensors), do.cuda(), at, S.cuda(), dS_out=dS.cuda(), status=status)
    assert int(status) == binding.GDN_SEQ_BAD_ROWS
    want = exact_grads(tensors, starts, lens, S[run], do, dS[run])
    for name, x, y in zip(("dq", "dk", "dv", "dalpha", "dbeta"), got, want):
        close(x, y, tol32(dk, T, 4), name)
        assert not x[left].any()
    close(got[5][run], want[5], tol32(dk, T, 4), "dS_in")
    assert not got[5][skipped].any()


# ---------------------------------------------------------------- waits that give up in the middle of a step
@pytest.mark.gpu
@pytest.mark.parametrize("seqs", [2, 75])  # four warps a slice, and one
def test_a_wait_inside_a_step_gives_up(seqs, monkeypatch):
    """The first block's T is never fetched: its warps leave together, the status says so, and the next call is right."""
    H, L, d, dv = 4, 150, 64, 48
    q, k, v, alpha, beta = [t.cuda().reshape(seqs, L, *t.shape[1:]) for t in draw(seqs * L, H, H, d, dv, "bf16", 83)]
    do = torch.randn_like(v)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both():
        return [*g.gdn_packed(q, k, v, alpha, beta, return_state=True, status=status), *g.gdn_bwd(q, k, v, alpha, beta, do)]

    want = both()
    assert int(status) == 0
    monkeypatch.setenv("GDN_DEBUG_DROP_SIGNAL", "2")
    monkeypatch.setenv("GDN_DEBUG_WAIT_LIMIT_US", "1000")
    g.gdn_packed(q, k, v, alpha, beta, status=status)
    assert int(status) == binding.GDN_SEQ_TIMEOUT
    g.gdn_bwd(q, k, v, alpha, beta, do, status=status)
    assert int(status) == binding.GDN_SEQ_TIMEOUT
    monkeypatch.undo()
    for x, y in zip(both()[:7], want):
        assert torch.equal(x, y)
    assert int(status) == 0


# ---------------------------------------------------------------- gates that are no numbers
@pytest.mark.gpu
@pytest.mark.parametrize("gate,value", [("alpha", float("nan")), ("alpha", -0.5), ("alpha", float("inf")), ("beta", float("nan"))])
@pytest.mark.parametrize("n,L,dtype", [(3, 150, "bf16"), (75, 40, "bf16"), (20, 5, "bf16"), (3, 150, "fp32")],
                         ids=["four warps a slice", "a warp a slice", "token by token", "fp32"])
def test_a_bad_gate_shows(gate, value, n, L, dtype):
    """One head's gate of one token of the second sequence: not finite from there on, and nowhere else."""
    H, dk, dv, t = 2, 64, 112, L + L // 2
    q, k, v, alpha, beta = cuda(*draw(n * L, H, H, dk, dv, dtype, 73))
    do, S0 = torch.randn_like(v), torch.randn(n, H, dv, dk, device="cuda")
    cu = torch.arange(0, n * L + 1, L, dtype=torch.int32, device="cuda")

    def everything():
        Sd = S0.clone()  # and the token alone, as a decode step
        step = [x.unflatten(0, (n, L))[:, L // 2].contiguous() for x in (q, k, v, alpha, beta)]
        return [*g.gdn_packed(q, k, v, alpha, beta, cu, S0, return_state=True), *g.gdn_decode(*step, Sd),
                *g.gdn_bwd(q, k, v, alpha, beta, do, cu, S0)]

    clean = everything()
    {"alpha": alpha, "beta": beta}[gate][t, 1] = value
    dirty = everything()
    for x, y in zip(clean, dirty):
        one = L if x.shape[0] == n * L else 1
        assert torch.equal(x[:one], y[:one]) and torch.equal(x[2 * one:], y[2 * one:])
        assert torch.equal(x[one:2 * one, 0], y[one:2 * one, 0])  # the other head
    o, S, o1, S1, dq, dk_, dv_, da, db, dS = dirty
    for x in (o[t:2 * L, 1], S[1, 1], o1[1, 1], S1[1, 1], dq[t:2 * L, 1], dv_[L:t, 1], da[t, 1], dS[1, 1]):
        assert not torch.isfinite(x.double()).any()


# ---------------------------------------------------------------- slots of sequences that are skipped
@pytest.mark.gpu
@pytest.mark.parametrize("more", [0, 80])  # four warps a slice (bf16), and one
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_skipped_sequence_blocks_no_slot(more, dtype):
    """Of the sequences of one slot the first whose rows are good runs."""
    H, Hk, dk, dv = 4, 2, 32, 64
    cu, slots = [0, 64, 30, 64, 130, 160, 200], [0, 2, 3, 3, 2, 0]  # good, wrong, inside the first, good, good, a slot in use
    cu, slots = cu + [200 + 30 * (i + 1) for i in range(more)], slots + [6 + i for i in range(more)]
    N, n = cu[-1], len(slots)
    run = [0, 3, 4, *range(6, n)]
    tensors = draw(N, H, Hk, dk, dv, dtype, 91)
    pool = torch.randn(6 + more, H, dv, dk, generator=torch.Generator().manual_seed(2))
    at = [slots[s] for s in run]
    rows, states = token_loop(*(t.double() for t in tensors), pool.double()[at], [cu[s + 1] - cu[s] for s in run], [cu[s] for s in run])
    want = pool.double()
    want[at] = torch.stack(states)
    S, o = pool.cuda(), torch.full(tensors[2].shape, 7.0, dtype=tensors[2].dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g.gdn_packed(*cuda(*tensors), ints(cu), S, S_out=S, slots=ints(slots), o=o, status=status)
    assert int(status) == binding.GDN_SEQ_BAD_ROWS | binding.GDN_SEQ_SAME_SLOT
    close(S, want, tol32(dk, 66), "S")
    covered = sorted(rows)
    close(o[covered], torch.stack([rows[t] for t in covered]), tol32(dk, 66), "o")
    assert (o[[t for t in range(N) if t not in rows]] == 7).all()


# ---------------------------------------------------------------- what no sequence covers, in a graph of gradients
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd_of_rows_that_no_sequence_covers(dtype):
    """Rows behind the last sequence and of a wrong range are zeros and stay out of every gradient, whatever the memory held."""
    N, H, Hk, dk, dv = 210, 4, 2, 48, 64
    cu = torch.tensor([0, 70, 400, 80, 200], dtype=torch.int32, device="cuda")  # [70, 400) and [400, 80) are wrong
    covered = [*range(70), *range(80, 200)]
    left = [t for t in range(N) if t not in covered]
    tensors = draw(N, H, Hk, dk, dv, dtype, 95)
    S_in = torch.randn(4, H, dv, dk, generator=torch.Generator().manual_seed(1))
    mine = [t.cuda().requires_grad_(True) for t in (*tensors, S_in)]
    for shape, t in ((tensors[2].shape, tensors[2].dtype), (S_in.shape, torch.float32)):
        held = [torch.full(shape, float("nan"), dtype=t, device="cuda") for _ in range(4)]
        del held  # the allocator hands it out again
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = g.gated_delta_rule(*mine, cu, status=status)
    assert int(status) == binding.GDN_SEQ_BAD_ROWS
    assert not o[left].any() and not S[[1, 2]].any()
    status.zero_()
    ((o.float() ** 2).sum() + S.sum()).backward()
    assert int(status) == binding.GDN_SEQ_BAD_ROWS
    do = 2 * o.detach()
    want = exact_grads(tensors, [0, 80], [70, 120], S_in[[0, 3]], do.cpu(), torch.ones(2, H, dv, dk))
    for name, x, y in zip(("q", "k", "v", "alpha", "beta"), mine, want):
        close(x.grad, y, tol32(dk, 120, 4), name)
        assert not x.grad[left].any()
    close(mine[5].grad[[0, 3]], want[5], tol32(dk, 120, 4), "S_in")
    assert not mine[5].grad[[1, 2]].any()
    _, S = g.gdn_packed(*(t.detach() for t in mine[:5]), cu, return_state=True)
    assert not S[[1, 2]].any()


# ---------------------------------------------------------------- the gates' gradients of bf16 calls
@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 40])  # four warps a slice, and one
def test_gate_gradients_are_fp32(n):
    """dalpha and dbeta leave in fp32 and are sums of fp32 accuracy: five sums lie one behind another (state, U, dU, dR, the row
    sums), each within a half step, 2^-24, of the result's 2-norm.  Operands of two bf16 terms (2^-17 each) are not."""
    H, Hk, d, L = 4, 2, 112, 140
    tensors = draw(n * L, H, Hk, d, d, "bf16", 97)
    do = torch.randn(tensors[2].shape, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    cu = torch.arange(0, n * L + 1, L, dtype=torch.int32)
    got = g.gdn_bwd(*cuda(*tensors), do.cuda(), cu.cuda())
    some = min(n, 3)  # the sequences do not meet
    want = exact_grads([t[:some * L] for t in tensors], [s * L for s in range(some)], [L] * some, torch.zeros(some, H, d, d), do, torch.zeros(some, H, d, d))
    for name, x, y in (("dalpha", got[3], want[3]), ("dbeta", got[4], want[4])):
        off = (x[:some * L].cpu().to(F64) - y).norm() / y.norm()
        assert off <= 5 * 2.0 ** -24, (name, float(off))


# ---------------------------------------------------------------- states that a graph has saved
@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["decode", "packed", "packed o", "frames", "maps"])
def test_a_saved_state_that_is_overwritten_raises(entry):
    """The backward pass recomputes from S_in: one that a later call has written does not go unnoticed."""
    B, T, H, d = 2, 64, 2, 64
    q, k, v, alpha, beta = [t.cuda().reshape(B, T, *t.shape[1:]) for t in draw(B * T, H, H, d, d, "fp32", 99)]
    S, w = torch.randn(B, H, d, d, device="cuda"), v.clone()
    leaf = q.clone().requires_grad_(True)
    for spoil in (False, True):
        o, _ = g.gated_delta_rule(leaf, k, w, alpha, beta, S)
        if spoil and entry == "decode":
            g.gdn_decode(*(x[:, 0].contiguous() for x in (q, k, v, alpha, beta)), S)
        elif spoil and entry == "packed":
            g.gdn_packed(q, k, v, alpha, beta, None, S, S_out=S)
        elif spoil and entry == "packed o":
            g.gdn_packed(q, k, v, alpha, beta, o=w)
        elif spoil and entry == "frames":
            g.gdn_step(q, k, v, alpha, beta, T, S, S_out=S)
        elif spoil:
            binding.apply_maps(S, torch.zeros(1, B, H, 2 * d, d, device="cuda"))
        if not spoil:
            o.sum().backward()
            continue
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            o.sum().backward()


# ---------------------------------------------------------------- decode of many heads
@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv,n,dtype", [(128, 128, 1, "bf16"), (128, 48, 3, "fp32"), (112, 112, 1, "fp32"), (16, 16, 2, "bf16"), (80, 96, 2, "bf16")])
def test_decode_of_many_heads(dk, dv, n, dtype):
    """A block a head (24 of them an SM) gives what 16 rows a block give, and both the definition's."""
    B, H, Hk = 190, 20, 5
    q, k, v, alpha, beta = [t.reshape(B, n, *t.shape[1:]) for t in cuda(*draw(B * n, H, Hk, dk, dv, dtype, 27))]
    S = torch.randn(B + 2, H, dv, dk, generator=torch.Generator().manual_seed(3)).cuda()
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(4))[:B].int().cuda()
    slots[[7, 100]] = torch.tensor([-1, 10 * B], dtype=torch.int32, device="cuda")
    whole, parts = S.clone(), S.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _ = g.gdn_decode(q, k, v, alpha, beta, whole, slots, o=torch.zeros_like(v), status=status)
    assert int(status) == binding.GDN_SEQ_BAD_SLOT
    for a in range(0, B, 19):
        some = slice(a, a + 19)
        o1, _ = g.gdn_decode(*(t[some] for t in (q, k, v, alpha, beta)), parts, slots[some], o=torch.zeros_like(v[some]))
        assert torch.equal(o[some], o1)
    assert torch.equal(whole, parts)
    at = [0, 50, 189]
    rows, states = token_loop(*(t[at].flatten(0, 1).cpu().double() for t in (q, k, v, alpha, beta)), S[slots[at].long()].cpu().double(),
                              [n] * 3, [n * i for i in range(3)])
    close(o[at].flatten(0, 1), torch.stack([rows[t] for t in range(3 * n)]), tol32(dk, n), "o")
    close(whole[slots[at].long()], torch.stack(states), tol32(dk, n), "S")


# ---------------------------------------------------------------- sizes and paths that the cases above leave out
@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_autograd_bf16(packed):
    B, T, H, Hk, dk, dv = 2, 90, 4, 2, 48, 64
    tensors = draw(B * T, H, Hk, dk, dv, "bf16", 43)
    gen = torch.Generator().manual_seed(1)
    S_in, wS = torch.randn(B, H, dv, dk, generator=gen), torch.randn(B, H, dv, dk, generator=gen)
    w = torch.randn(B * T, H, dv, generator=gen).to(torch.bfloat16)
    shape = (lambda t: t) if packed else (lambda t: t.reshape(B, T, *t.shape[1:]))
    mine = [shape(t).cuda().requires_grad_(True) for t in tensors] + [S_in.cuda().requires_grad_(True)]
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda") if packed else None
    o, S = g.gated_delta_rule(*mine, cu)
    torch.autograd.backward([o, S], [shape(w).cuda(), wS.cuda()])
    rows, states = token_loop(*(t.double() for t in tensors), S_in.double(), [T] * B, [0, T])
    close(o.reshape(B * T, H, dv), torch.stack([rows[t] for t in range(B * T)]), tol32(dk, T), "o")
    close(S, torch.stack(states), tol32(dk, T), "S")
    want = exact_grads(tensors, [0, T], [T] * B, S_in, w, wS)
    for name, x, y in zip(("q", "k", "v", "alpha", "beta", "S_in"), mine, want):
        assert x.grad.dtype == x.dtype
        close(x.grad.reshape(y.shape), y, tol32(dk, T, 4), name)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk,dk,dv", [(2, 1, 128, 128), (4, 4, 128, 80), (4, 2, 96, 112)])
def test_walks_of_large_states(H, Hk, dk, dv):
    """Chains enough for a warp a slice, with the largest states."""
    lens = [70, 130, 64] + [33] * 35
    tensors, starts, cu = packed_case(lens, 0, 0, H, Hk, dk, dv, "bf16", "slow", seed=45)
    n, some, N = len(lens), 3, sum(lens[:3])  # the sequences do not meet: three are looked at
    gen = torch.Generator().manual_seed(6)
    do = torch.randn(tensors[2].shape, generator=gen).to(torch.bfloat16)
    S_in, dS_out = torch.randn(n, H, dv, dk, generator=gen), torch.randn(n, H, dv, dk, generator=gen)
    first = [t[:N] for t in tensors]
    rows, states = token_loop(*(t.double() for t in first), S_in[:some].double(), lens[:some], starts[:some])
    o, S = g.gdn_packed(*cuda(*tensors), cu.cuda(), S_in.cuda(), return_state=True)
    close(o[:N], torch.stack([rows[t] for t in range(N)]), tol32(dk, 130), "o")
    close(S[:some], torch.stack(states), tol32(dk, 130), "S")
    want = exact_grads(first, starts[:some], lens[:some], S_in[:some], do[:N], dS_out[:some])
    got = g.gdn_bwd(*cuda(*tensors), do.cuda(), cu.cuda(), S_in.cuda(), dS_out=dS_out.cuda())
    for name, x, y in zip(("dq", "dk", "dv", "dalpha", "dbeta", "dS_in"), got, want):
        close(x[:some if name == "dS_in" else N], y, tol32(dk, 130, 4), name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_long_sequence(dtype):
    T, H, dk, dv = 2500, 1, 48, 32
    tensors = draw(T, H, H, dk, dv, dtype, 47)
    gen = torch.Generator().manual_seed(7)
    do = torch.randn(tensors[2].shape, generator=gen).to(tensors[2].dtype)
    S_in, dS = torch.randn(1, H, dv, dk, generator=gen), torch.randn(1, H, dv, dk, generator=gen)
    rows, states = token_loop(*(t.double() for t in tensors), S_in.double(), [T], [0])
    one = [t.cuda()[None] for t in tensors]
    o, S = g.gdn_packed(*one, None, S_in.cuda(), return_state=True)
    close(o[0], torch.stack([rows[t] for t in range(T)]), tol32(dk, T), "o")
    close(S, torch.stack(states), tol32(dk, T), "S")
    want = exact_grads(tensors, [0], [T], S_in, do, dS)
    got = g.gdn_bwd(*one, do.cuda()[None], None, S_in.cuda(), dS_out=dS.cuda())
    for name, x, y in zip(("dq", "dk", "dv", "dalpha", "dbeta", "dS_in"), got, want):
        close(x if name == "dS_in" else x[0], y, tol32(dk, T, 4), name)


@pytest.mark.gpu
def test_one_captured_call_serves_other_sequences():
    """A graph replayed with other lengths, slots and gates in the same tensors: nothing of the first ones is kept."""
    N, n, H, d = 400, 6, 4, 64
    sets = [draw(N, H, 2, d, d, "bf16", seed) for seed in (101, 102)]
    cus = [[0, 100, 100, 164, 300, 310, 400], [0, 3, 9, 50, 51, 390, 400]]
    slots = [[3, 1, 0, 7, 2, 4], [0, 1, 2, 3, 4, 5]]
    pool = torch.randn(8, H, d, d, generator=torch.Generator().manual_seed(1)).cuda()
    do = torch.randn(N, H, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def everything(x, cu, sl, S):
        o, _ = g.gdn_packed(*x, cu, S, S_out=S, slots=sl)
        return [o, S, *g.gdn_bwd(*x, do, cu, need_dS_in=True)]

    want = [[t.clone() for t in everything(cuda(*s), ints(c), ints(sl), pool.clone())] for s, c, sl in zip(sets, cus, slots)]
    x, cu, sl, S = cuda(*sets[0]), ints(cus[0]), ints(slots[0]), pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(x, cu, sl, S)
    for i in (1, 0, 1):
        for a, b in zip(x, sets[i]):
            a.copy_(b)
        cu.copy_(ints(cus[i]))
        sl.copy_(ints(slots[i]))
        S.copy_(pool)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("more", [20, 100])
def test_one_slot_of_a_short_and_a_long_sequence(more):
    """In a batch of short prompts they go through different kernels, which have to agree on which one runs."""
    H, Hk, dk, dv = 4, 2, 48, 64
    lens = [5, 40, 70, 6, 0, 33, 12] + [20] * more
    slots = [0, 0, 1, 1, 2, 2, -1] + [3 + i for i in range(more)]  # the second of each slot is skipped, an empty one runs too
    N, n = sum(lens), len(lens)
    starts = [sum(lens[:i]) for i in range(n)]
    run = [0, 2, 4, *range(7, n)]
    tensors = draw(N, H, Hk, dk, dv, "bf16", 93)
    pool = torch.randn(3 + more, H, dv, dk, generator=torch.Generator().manual_seed(2))
    fresh = torch.arange(n) % 5 == 2
    at = [slots[s] for s in run]
    S0 = pool.double()[at] * ~fresh[run][:, None, None, None]
    rows, states = token_loop(*(t.double() for t in tensors), S0, [lens[s] for s in run], [starts[s] for s in run])
    want = pool.double()
    want[at] = torch.stack(states)
    S, o = pool.cuda(), torch.full(tensors[2].shape, 7.0, dtype=tensors[2].dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g.gdn_packed(*cuda(*tensors), ints(starts + [N]), S, S_out=S, slots=ints(slots), fresh=fresh.cuda(), o=o, status=status)
    assert int(status) == binding.GDN_SEQ_SAME_SLOT
    close(S, want, tol32(dk, 70), "S")
    covered = sorted(rows)
    close(o[covered], torch.stack([rows[t] for t in covered]), tol32(dk, 70), "o")
    assert (o[[t for t in range(N) if t not in rows]] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_thousands_of_wrong_sequences(dtype):
    """Many entries of one slot and a range that is wrong: looked through once a block, not once an entry."""
    n, H, d = 3000, 2, 32
    q, k, v, alpha, beta = cuda(*draw(64 + n, H, H, d, d, dtype, 103))
    cu = torch.cat([torch.tensor([0, 64, -1]), 64 + torch.arange(n - 1)]).int().cuda()  # good, two wrong ones, then a token each
    assert cu.numel() == n + 2
    slots = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    pool = torch.randn(2, H, d, d, device="cuda")
    S, status = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full(v.shape, 7.0, dtype=v.dtype, device="cuda")
    g.gdn_packed(q, k, v, alpha, beta, cu, S, S_out=S, slots=slots, o=o, status=status)  # warm
    assert int(status) == binding.GDN_SEQ_SAME_SLOT | binding.GDN_SEQ_BAD_ROWS
    assert (o[64:] == 7).all() and not (o[:64] == 7).all(dim=-1).any() and torch.equal(S[1], pool[1])
    o1, S1 = g.gdn_packed(*(t[None, :64] for t in (q, k, v, alpha, beta)), None, pool[:1], return_state=True)
    close(S[:1], S1.double(), 2 * tol32(d, 64), "S")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    g.gdn_packed(q, k, v, alpha, beta, cu, S, S_out=S, slots=slots, o=o)
    end.record()
    end.synchronize()
    assert start.elapsed_time(end) < 100  # ms: 3000 x 4 blocks that each look at 3000 entries; by pairs it would be seconds
