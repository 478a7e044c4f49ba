"""The sequence operators at the edges of what their callers may pass.  Tolerances as in test_sequences.py."""
import pytest
import torch

import gated_deltanet_linear_chunkwise_b200 as g
from gated_deltanet_linear_chunkwise_b200 import binding
from test_sequences import cuda, draw


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
