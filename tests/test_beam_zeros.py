"""Logits of either zero are equal: the lower row and then the lower token wins, as among all equals."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa
from tests.test_beam import BF16, F16, F32, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("K", [1, 2, 3, 8])
@pytest.mark.parametrize("V", [4, 100, 9001, 70_000])
def test_either_zero(dtype, K, V):
    g = torch.Generator(device="cuda").manual_seed(V + K)
    st = ssa.BeamState(3, K)
    st.scores.zero_()
    # only zeros, and zeros above the rest of the row
    zero = torch.where(torch.rand((3 * K, V), generator=g, device="cuda") < 0.5, -0.0, 0.0).to(dtype)
    check(zero, st, exact=True)
    x = torch.full((3 * K, V), -1.0, dtype=dtype, device="cuda")
    some = torch.rand((3 * K, V), generator=g, device="cuda") < 0.3
    some[:, 1:3] = True
    x = torch.where(some, zero, x)
    x[:, 1], x[:, 2] = -0.0, 0.0
    check(x, st, exact=True)
