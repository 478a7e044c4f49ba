"""Cases of the gated delta rule over packed sequences: serving and training.

Three operators, all of the token-wise rule (per sequence and head, S is d_v x d_k)

    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,    o_t = S_t q_t

* ``decode``: one or a few new tokens for each of a batch of sequences whose states live in a
  pool; each sequence names its slot, and the states are updated in place.
* ``packed``: whole prompts of different lengths packed behind one another, from the pool's
  states and back into them.
* ``bwd``: the gradients of the rule over packed or equal sequences (q, k, v, alpha, beta and the
  entering state) from the gradients of the outputs and of the final state.

q and k may have fewer heads than v (``hk`` divides ``h``): head j reads q/k head j // (h / hk).
"""
import random

import torch

own = False

C = 64  # tokens of a chunk in the plain chunked form


def listed():
    return [
        # the next token of one stream: launch latency
        {"name": "decode one stream", "op": "decode", "b": 1, "n": 1, "h": 20, "hk": 20, "dk": 112, "dv": 112, "pool": 8, "dtype": "bf16", "gates": "slow"},
        # a full serving batch
        {"name": "decode batch", "op": "decode", "b": 256, "n": 1, "h": 20, "hk": 20, "dk": 112, "dv": 112, "pool": 288, "dtype": "bf16", "gates": "slow"},
        # a few drafted tokens of each stream checked at once, q/k heads shared by two value heads
        {"name": "decode draft tokens", "op": "decode", "b": 27, "n": 5, "h": 16, "hk": 8, "dk": 128, "dv": 128, "pool": 32, "dtype": "bf16", "gates": "lit"},
        # short prompts, most under one chunk
        {"name": "packed short prompts", "op": "packed", "seqs": 37, "tokens": 1201, "h": 20, "hk": 20, "dk": 112, "dv": 112, "dtype": "bf16", "gates": "slow"},
        # an ordinary prefill batch
        {"name": "packed prompts", "op": "packed", "seqs": 24, "tokens": 16384, "h": 20, "hk": 20, "dk": 112, "dv": 112, "dtype": "bf16", "gates": "slow"},
        # one long prompt of odd length: few chains, many steps
        {"name": "packed one long", "op": "packed", "seqs": 1, "tokens": 8209, "h": 20, "hk": 20, "dk": 112, "dv": 112, "dtype": "bf16", "gates": "slow"},
        # full precision, small heads
        {"name": "packed fp32", "op": "packed", "seqs": 5, "tokens": 1500, "h": 6, "hk": 3, "dk": 64, "dv": 80, "dtype": "fp32", "gates": "slow"},
        # a small model in full precision (four 64-token frames of two heads)
        {"name": "bwd small fp32", "op": "bwd", "seqs": 2, "tokens": 512, "h": 2, "hk": 2, "dk": 64, "dv": 64, "dtype": "fp32", "gates": "slow", "equal": True, "state": False},
        # documents packed into one training row, strong decay
        {"name": "bwd documents", "op": "bwd", "seqs": 9, "tokens": 8192, "h": 20, "hk": 20, "dk": 112, "dv": 112, "dtype": "bf16", "gates": "lit", "equal": False, "state": False},
        # shared q/k heads, a carried state with its gradient
        {"name": "bwd shared heads", "op": "bwd", "seqs": 2, "tokens": 3520, "h": 16, "hk": 4, "dk": 64, "dv": 128, "dtype": "bf16", "gates": "slow", "equal": True, "state": True},
        # a short clip: 21 frames of 880 tokens in one sequence
        {"name": "bwd clip", "op": "bwd", "seqs": 1, "tokens": 18480, "h": 20, "hk": 20, "dk": 112, "dv": 112, "dtype": "bf16", "gates": "slow", "equal": True, "state": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["decode", "packed", "bwd"])
    hk = rng.choice([1, 2, 4, 8, 10, 20])
    h = hk * rng.choice([1, 1, 1, 2, 4])
    h, hk = (h, hk) if h <= 20 else (20, 20)
    case = {"op": op, "h": h, "hk": hk, "dk": 16 * rng.randint(2, 8), "dv": 16 * rng.randint(2, 8),
            "dtype": rng.choice(["bf16", "bf16", "bf16", "fp32"]), "gates": rng.choice(["slow", "slow", "lit"])}
    if op == "decode":
        case["b"] = _log_int(rng, 1, 256)
        case["n"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        case["pool"] = case["b"] + rng.randint(0, 16)
    else:
        case["tokens"] = _log_int(rng, 40, 16384 if op == "packed" else 6000)
        case["seqs"] = min(case["tokens"], _log_int(rng, 1, 40))
        if op == "bwd":
            case["equal"] = rng.random() < 0.4
            case["state"] = rng.random() < 0.5
            if case["equal"]:
                case["tokens"] -= case["tokens"] % case["seqs"]
    return case


def _lengths(case):
    """The lengths of a packed case's sequences: a fixed ragged split of its tokens."""
    n, total = case["seqs"], case["tokens"]
    if case.get("equal"):
        return [total // n] * n
    r = random.Random(1000003 * total + n)
    w = [r.random() ** 2 + 0.02 for _ in range(n)]
    got = [max(1, int(x / sum(w) * total)) for x in w]
    i = 0
    while sum(got) != total:  # the rounding goes to the sequences in turn
        step = 1 if sum(got) < total else -1
        if got[i % n] + step >= 1:
            got[i % n] += step
        i += 1
    return got


def work(case):
    """Each input read once, each output written once; operations of the token recurrence."""
    h, hk, dk, dv = case["h"], case["hk"], case["dk"], case["dv"]
    es = 2 if case["dtype"] == "bf16" else 4
    seqs = case["b"] if case["op"] == "decode" else case["seqs"]
    tokens = case["b"] * case["n"] if case["op"] == "decode" else case["tokens"]
    row = es * (2 * hk * dk + h * dv) + 8 * h        # q, k, v and the two gates of a token
    state = 4 * seqs * h * dk * dv
    if case["op"] != "bwd":                          # o out; the state in and out
        return {"bytes": tokens * (row + es * h * dv) + 2 * state, "flops": 6 * tokens * h * dk * dv}
    # the inputs and do in, one gradient out for each input; S_in and dS_out in, dS_in out.
    # Operations of the adjoint recurrence: the states again (S k and the update, 4), do q^T and
    # S^T do (4), dS k, dS^T u and (alpha S)^T dr (6), the update of dS and <dS, S> (4).
    return {"bytes": tokens * (2 * row + es * h * dv) + (3 * state if case["state"] else 0),
            "flops": 18 * tokens * h * dk * dv}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _draw_rows(case, g, lead):
    """q, k, v, alpha, beta of `lead` token rows: unit q/k, normal v, beta a sigmoid, alpha the
    exponential of a negated softplus (weak decay "slow", strong decay "lit")."""
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    q = unit(n(*lead, case["hk"], case["dk"])).to(dt)
    k = unit(n(*lead, case["hk"], case["dk"])).to(dt)
    v = n(*lead, case["h"], case["dv"]).to(dt)
    beta = torch.sigmoid(n(*lead, case["h"]))
    alpha = torch.exp(-torch.nn.functional.softplus(n(*lead, case["h"]) + (2.0 if case["gates"] == "lit" else -4.0)))
    return q, k, v, alpha, beta


def prepare(case, seed):
    g = _gen(seed)
    h, dk, dv = case["h"], case["dk"], case["dv"]
    s = {"case": dict(case)}
    if case["op"] == "decode":
        s["q"], s["k"], s["v"], s["alpha"], s["beta"] = _draw_rows(case, g, (case["b"], case["n"]))
        s["S"] = 0.1 * torch.randn(case["pool"], h, dv, dk, device="cuda", generator=g)
        s["slots"] = torch.randperm(case["pool"], device="cuda", generator=g)[: case["b"]].to(torch.int32)
        return s
    lens = _lengths(case)
    s["lens"] = lens
    if case.get("equal"):  # [B, T, heads, d], as a training batch holds it
        s["cu"] = None
        lead = (case["seqs"], lens[0])
    else:
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        lead = (case["tokens"],)
    s["q"], s["k"], s["v"], s["alpha"], s["beta"] = _draw_rows(case, g, lead)
    if case["op"] == "packed":  # a pool with more slots than sequences
        s["S"] = 0.1 * torch.randn(case["seqs"] + 3, h, dv, dk, device="cuda", generator=g)
        s["slots"] = torch.randperm(case["seqs"] + 3, device="cuda", generator=g)[: case["seqs"]].to(torch.int32)
        return s
    s["do"] = torch.randn(*lead, h, dv, device="cuda", generator=g).to(s["v"].dtype)
    s["S_in"] = s["dS_out"] = None
    if case["state"]:
        s["S_in"] = 0.1 * torch.randn(case["seqs"], h, dv, dk, device="cuda", generator=g)
        s["dS_out"] = torch.randn(case["seqs"], h, dv, dk, device="cuda", generator=g)
    return s


def run(s):
    if own:
        import gated_deltanet_linear_chunkwise_b200 as gdn

        if s["case"]["op"] == "decode":
            o, S = gdn.gdn_decode(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["S"], s["slots"])
            return [o, S]
        if s["case"]["op"] == "packed":
            o, S = gdn.gdn_packed(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["cu"], s["S"], S_out=s["S"], slots=s["slots"])
            return [o, S]
        return list(gdn.gdn_bwd(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["do"], s["cu"], s["S_in"], dS_out=s["dS_out"]))
    return {"decode": _plain_decode, "packed": _plain_packed, "bwd": _plain_bwd}[s["case"]["op"]](s)


# ---------------------------------------------------------------- the plain forms
def _heads(x, h):
    """[..., hk, d] with each head repeated to h heads, in 32 bits."""
    return x.float().repeat_interleave(h // x.shape[-2], dim=-2)


def _plain_decode(s):
    """The recurrence as it is written, token by token, on the batch's states."""
    h = s["case"]["h"]
    slots = s["slots"].long()
    q, k, v = _heads(s["q"], h), _heads(s["k"], h), s["v"].float()
    S = s["S"][slots]
    out = []
    for t in range(s["case"]["n"]):
        S = S * s["alpha"][:, t, :, None, None]
        u = s["beta"][:, t, :, None] * (v[:, t] - (S @ k[:, t, :, :, None]).squeeze(-1))
        S = S + u[..., :, None] * k[:, t, :, None, :]
        out.append((S @ q[:, t, :, :, None]).squeeze(-1))
    s["S"][slots] = S
    return [torch.stack(out, 1).to(s["v"].dtype), s["S"]]


def _grid(s):
    """Where the padded chunks' tokens come from: rows [B, n, C] of the packed tensors, and which are real."""
    lens, dev = s["lens"], s["q"].device
    n = -(-max(lens) // C)
    t = torch.arange(n * C, device=dev)
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(len(lens) + 1, device=dev) * lens[0]
    real = t[None] < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(real, cu[:-1, None] + t[None], 0)
    return at.reshape(len(lens), n, C), real.reshape(len(lens), n, C)


def _chunks(x, at, real, fill=0.0):
    """[rows, h, ...] -> [B, n, h, C, ...] in 32 bits; padding holds `fill`."""
    x = x.float()[at]
    x = torch.where(real.reshape(*real.shape, *([1] * (x.dim() - 3))), x, fill)
    return x.transpose(2, 3)


def _rows(x, at, real, like):
    """The reverse of _chunks: [B, n, h, C, ...] back to the packed rows, rounded to like's type."""
    x = x.transpose(2, 3)
    n = like.numel() // x[0, 0, 0].numel()
    buf = torch.empty((n + 1, *x.shape[3:]), dtype=x.dtype, device=x.device)
    buf[torch.where(real, at, n)] = x  # padding goes to a row behind the last one
    return buf[:n].reshape(like.shape).to(like.dtype)


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular C x C blocks, by halves: T21 = -T22 A21 T11."""
    T = torch.eye(C, device=A.device).expand(A.shape).clone()
    w = 1
    while w < C:
        a = A.reshape(*A.shape[:-2], C // (2 * w), 2 * w, C // (2 * w), 2 * w).diagonal(dim1=-4, dim2=-2)
        t = T.reshape(*A.shape[:-2], C // (2 * w), 2 * w, C // (2 * w), 2 * w).diagonal(dim1=-4, dim2=-2)
        a21, t11, t22 = (x.movedim(-1, -3) for x in (a[..., w:, :w, :], t[..., :w, :w, :], t[..., w:, w:, :]))
        t[..., w:, :w, :] = -(t22 @ (a21 @ t11)).movedim(-3, -1)
        w *= 2
    return T


def _chunk_terms(s):
    """All that a chunk's tokens give before any state is known."""
    h = s["case"]["h"]
    at, real = _grid(s)
    flat = lambda x, tail: x.reshape(-1, *x.shape[x.dim() - tail:])  # noqa: E731
    c = {"at": at, "real": real}
    c["q"], c["k"], c["v"] = (_chunks(flat(x, 2), at, real) for x in (_heads(s["q"], h), _heads(s["k"], h), s["v"]))
    alpha = _chunks(flat(s["alpha"], 1), at, real, 1.0)
    c["alpha"], c["beta"] = alpha, _chunks(flat(s["beta"], 1), at, real)
    G = alpha.double().log().cumsum(-1)  # decays are differences of long sums
    low = torch.ones(C, C, dtype=torch.bool, device=G.device).tril()
    c["decay"] = torch.where(low, (G[..., :, None] - G[..., None, :]), -torch.inf).exp().float()  # e^{G_i - G_j}, j <= i
    c["eg"], c["el"], c["gl"] = G.exp().float(), (G[..., -1:] - G).exp().float(), G[..., -1].exp().float()
    c["qk"], c["kk"] = c["q"] @ c["k"].mT, c["k"] @ c["k"].mT
    c["P"] = c["qk"] * c["decay"]
    c["A0"] = (c["kk"] * c["decay"]).tril(-1)
    c["T"] = _unit_lower_inverse(c["beta"][..., None] * c["A0"])
    return c


def _chunk_scan(c, S, out):
    """From chunk to chunk: the states entering each chunk [B, h, d_k, d_v], Y = V - e^G K S and U."""
    Sig, Ys, Us = [], [], []
    kl = c["k"] * c["el"][..., None]
    for i in range(c["k"].shape[1]):
        Y = c["v"][:, i] - c["eg"][:, i, ..., None] * (c["k"][:, i] @ S)
        U = c["T"][:, i] @ (c["beta"][:, i, ..., None] * Y)
        if out is not None:
            out.append(c["eg"][:, i, ..., None] * (c["q"][:, i] @ S) + c["P"][:, i] @ U)
        else:
            Sig.append(S), Ys.append(Y), Us.append(U)
        S = c["gl"][:, i, :, None, None] * S + kl[:, i].mT @ U
    return S, Sig, Ys, Us


def _plain_packed(s):
    c = _chunk_terms(s)
    slots = s["slots"].long()
    out = []
    S, _, _, _ = _chunk_scan(c, s["S"][slots].mT, out)
    s["S"][slots] = S.mT
    return [_rows(torch.stack(out, 1), c["at"], c["real"], s["v"]), s["S"]]


def _plain_bwd(s):
    """The chunked form's adjoint.  Gate gradients: every product of the form carries a decay over a
    range of tokens, and a token's log-gate gets the terms whose range holds it."""
    case = s["case"]
    B, h, hk, dk, dv = len(s["lens"]), case["h"], case["hk"], case["dk"], case["dv"]
    c = _chunk_terms(s)
    do = _chunks(s["do"].reshape(-1, h, dv), c["at"], c["real"])
    S0 = s["S_in"].mT if s["S_in"] is not None else torch.zeros(B, h, dk, dv, device=do.device)
    _, Sig, Ys, Us = _chunk_scan(c, S0, None)
    Sig, Y, U = torch.stack(Sig, 1), torch.stack(Ys, 1), torch.stack(Us, 1)
    D = s["dS_out"].mT if s["dS_out"] is not None else torch.zeros(B, h, dk, dv, device=do.device)
    qg, kg, kl = c["q"] * c["eg"][..., None], c["k"] * (c["beta"] * c["eg"])[..., None], c["k"] * c["el"][..., None]
    dU0 = c["P"].mT @ do
    Ds, dRs = [], []
    for i in reversed(range(c["k"].shape[1])):
        Ds.append(D)
        dR = c["T"][:, i].mT @ (dU0[:, i] + kl[:, i] @ D)
        dRs.append(dR)
        D = c["gl"][:, i, :, None, None] * D + qg[:, i].mT @ do[:, i] - kg[:, i].mT @ dR
    D1, dR = torch.stack(Ds[::-1], 1), torch.stack(dRs[::-1], 1)
    dP = (do @ U.mT) * c["decay"]
    dA = -(dR @ U.mT) * c["decay"].tril(-1)
    dAb = dA * c["beta"][..., None]
    dv_ = c["beta"][..., None] * dR
    dbeta = (dR * Y).sum(-1) + (dA * c["kk"]).sum(-1)
    dq_in = c["eg"][..., None] * (do @ Sig.mT)
    dk_in = -(c["beta"] * c["eg"])[..., None] * (dR @ Sig.mT)
    dk_out = c["el"][..., None] * (U @ D1.mT)
    dq = dq_in + dP @ c["k"]
    dk_ = dk_in + dk_out + dP.mT @ c["q"] + dAb @ c["k"] + dAb.mT @ c["k"]
    M = dP * c["qk"] + dAb * c["kk"]
    into = (c["q"] * dq_in).sum(-1) + (c["k"] * dk_in).sum(-1)   # from before the chunk to token i
    past = (c["k"] * dk_out).sum(-1)                             # from token j to the chunk's end
    below = M.flip(-2).cumsum(-2).flip(-2)                       # sums over rows i >= t
    dg = below.tril(-1).sum(-1) + into.flip(-1).cumsum(-1).flip(-1) + past.cumsum(-1) - past
    dg = dg + (c["gl"] * (D1 * Sig).sum((-1, -2)))[..., None]
    dalpha = dg / c["alpha"]
    share = lambda x: x.reshape(*x.shape[:2], hk, h // hk, *x.shape[3:]).sum(3)  # noqa: E731
    dq, dk_ = share(dq), share(dk_)
    got = [_rows(x, c["at"], c["real"], y) for x, y in ((dq, s["q"]), (dk_, s["k"]), (dv_, s["v"]), (dalpha, s["alpha"]), (dbeta, s["beta"]))]
    return got + ([D.mT.contiguous()] if s["S_in"] is not None else [None])


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """The token recurrence, and its adjoint token by token, in 64 bits."""
    s = prepare(case, seed)
    h = case["h"]
    if case["op"] == "decode":
        lens, cu = [case["n"]] * case["b"], None
    else:
        lens, cu = s["lens"], s["cu"]
    B, T = len(lens), max(lens)
    start = cu[:-1].long() if cu is not None else torch.arange(B, device="cuda") * T
    length = torch.tensor(lens, device="cuda")

    def tokens(x, *row):  # time first: [T, B, *row]; steps past a sequence's end hold zeros
        x = x.reshape(-1, *row)
        t = torch.arange(T, device="cuda")[:, None]
        on = t < length[None]
        got = x[torch.where(on, start[None] + t, 0)].double()
        return got * on.reshape(T, B, *([1] * (got.dim() - 2)))

    rep = lambda x: x.repeat_interleave(h // case["hk"], dim=2)  # noqa: E731
    q, k, v = rep(tokens(s["q"], case["hk"], case["dk"])), rep(tokens(s["k"], case["hk"], case["dk"])), tokens(s["v"], h, case["dv"])
    beta = tokens(s["beta"], h)
    on = torch.arange(T, device="cuda")[:, None] < length[None]
    alpha = torch.where(on[..., None], tokens(s["alpha"], h), 1.0)

    def step(S, t):
        S = alpha[t, :, :, None, None] * S
        r = v[t] - (S * k[t, :, :, None, :]).sum(-1)
        return S + (beta[t, :, :, None] * r)[..., None] * k[t, :, :, None, :], r

    def packed(x, like):  # [T, B, ...] back to the operator's layout
        out = torch.empty(like.reshape(sum(lens), *x.shape[2:]).shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            out[int(start[b]): int(start[b]) + lens[b]] = x[: lens[b], b]
        return out.reshape(like.shape)

    if case["op"] != "bwd":
        slots = s["slots"].long()
        S, out = s["S"].double()[slots], []
        for t in range(T):
            S, _ = step(S, t)
            out.append((S * q[t, :, :, None, :]).sum(-1))
        pool = s["S"].double()
        pool[slots] = S
        return [packed(torch.stack(out), s["v"]), pool]

    do = tokens(s["do"], h, case["dv"])
    S = s["S_in"].double() if s["S_in"] is not None else torch.zeros(B, h, case["dv"], case["dk"], dtype=torch.float64, device="cuda")
    D = s["dS_out"].double() if s["dS_out"] is not None else torch.zeros_like(S)
    W, kept = 128, []
    for t in range(T):  # the state before every W-th token
        if t % W == 0:
            kept.append(S)
        S, _ = step(S, t)
    dq, dk, dv, da, db = (torch.zeros_like(x) for x in (q, k, v, alpha, beta))
    for first in reversed(range(0, T, W)):
        S, before, after, rs = kept.pop(), [], [], []
        for t in range(first, min(first + W, T)):
            before.append(S)
            S, r = step(S, t)
            after.append(S), rs.append(r)
        for t in reversed(range(first, min(first + W, T))):
            S0, S1, r = before.pop(), after.pop(), rs.pop()
            dq[t] = (S1 * do[t, :, :, :, None]).sum(-2)
            D = D + do[t, :, :, :, None] * q[t, :, :, None, :]
            du = (D * k[t, :, :, None, :]).sum(-1)
            u = beta[t, :, :, None] * r
            db[t] = (du * r).sum(-1)
            dr = beta[t, :, :, None] * du
            dv[t] = dr
            aS = alpha[t, :, :, None, None] * S0
            dk[t] = (D * u[..., None]).sum(-2) - (aS * dr[..., None]).sum(-2)
            D = D - dr[..., None] * k[t, :, :, None, :]
            da[t] = (D * S0).sum((-1, -2))
            D = alpha[t, :, :, None, None] * D
    share = lambda x: x.reshape(T, B, case["hk"], h // case["hk"], -1).sum(3)  # noqa: E731
    got = [packed(x, y) for x, y in ((share(dq), s["q"]), (share(dk), s["k"]), (dv, s["v"]), (da, s["alpha"]), (db, s["beta"]))]
    return got + [D if s["S_in"] is not None else None]
