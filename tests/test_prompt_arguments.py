"""Arguments of ssa_prompt_attention beside its tensors, on the CPU: what the kernel would write past, or on
another device, is refused."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa
from tests.test_prompt import _call_cpu

SIZE = ssa.ssa_prompt_workspace_size()


@pytest.mark.parametrize("kw,match", [
    (dict(status=torch.zeros((1,), dtype=torch.int64)), "status"),
    (dict(status=torch.zeros((1,))), "status"),
    (dict(status=torch.zeros((0,), dtype=torch.int32)), "status"),
    (dict(ws=torch.zeros((2 * SIZE,), dtype=torch.uint8)[::2]), "ws"),
    (dict(ws=torch.zeros((SIZE - 1,), dtype=torch.uint8)), "ws"),
    (dict(status=torch.zeros((1,), dtype=torch.int32)), "current CUDA device"),
])
def test_refusals(kw, match):
    with pytest.raises(ValueError, match=match):
        _call_cpu(**kw)
