"""One workspace of ssa_beam_select, zeroed once, for batches of changing size."""
import pytest
import torch

import sparse_attention_decode_indexer_gb300 as ssa
from tests.test_beam import BF16, copy_of, make, select

NAMES = ("scores", "finished", "history", "hist_len")


@pytest.mark.gpu
def test_batches_of_other_sizes():
    """Each call in the shared workspace gives what it gives in one of its own."""
    ws = torch.zeros((ssa.ssa_beam_workspace_size(200, 8),), dtype=torch.uint8, device="cuda")
    for i, (G, K, V, max_len) in enumerate([(64, 4, 20000, 4000), (100, 4, 20000, 4000), (3, 8, 90000, 0), (200, 1, 5000, 50),
                                            (1, 1, 300000, 9000), (128, 8, 1000, 700), (65, 2, 30000, 2000), (200, 8, 9000, 0)]):
        eos = 5 if i % 2 else -1
        x, st = make(G, K, V, BF16, seed=i, max_len=max_len, eos=eos)
        a, b = copy_of(st), copy_of(st)
        lens = torch.arange(G * K, dtype=torch.int32, device="cuda")
        own, shared = select(x, st, eos, out=a, lens=lens), select(x, st, eos, out=b, lens=lens, ws=ws)
        assert all(torch.equal(p, q) for p, q in zip(own, shared))
        for name in NAMES:
            p, q = getattr(a, name), getattr(b, name)
            assert p is None or torch.equal(p, q)


def test_a_larger_batch_needs_no_smaller_workspace():
    """What holds a batch holds every smaller one."""
    size = ssa.ssa_beam_workspace_size
    for G, K in ((1, 1), (64, 1), (3, 32), (1000, 4), (65535, 32)):
        for g in {1, (G + 1) // 2, G}:
            for k in {1, (K + 1) // 2, K}:
                assert size(g, k) <= size(G, K)
