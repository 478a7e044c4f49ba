"""The sequence operators at the edges of what their callers may pass.  Tolerances as in test_sequences.py."""
import pytest
import torch

import gated_deltanet_linear_chunkwise_b200 as g
from gated_deltanet_linear_chunkwise_b200 import binding


# ---------------------------------------------------------------- rows of q, k and v
def rows_apart(t, lead):
    return binding._tokens("q", t, t.dtype, t.device, lead, t.shape[-2], t.shape[-1])


@pytest.mark.parametrize("t,lead", [
    (torch.zeros(1, 2, 64).expand(5, 2, 64), (5,)),                       # one token for all
    (torch.zeros(1, 1, 2, 64).expand(5, 7, 2, 64), (5, 7)),
    (torch.zeros(1, 1, 2, 64).expand(1, 7, 2, 64), (1, 7)),
    (torch.zeros(1, 1, 64).expand(5, 1, 64), (5,)),                       # one head
    (torch.zeros(6 * 64 + 64).as_strided((5, 2, 64), (64, 64, 1)), (5,)),  # a row starts inside the one before
])
def test_rows_over_one_another_are_refused(t, lead):
    with pytest.raises(g.GdnError, match="over one another"):
        rows_apart(t, lead)
