"""Runner steps by graph replay with rope, whose queries may be strided views: views of one buffer that start
at the same address are different queries."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_views_of_one_buffer_have_graphs_of_their_own():
    import sparse_attention_decode_indexer_gb300 as ssa
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    P, Hq, Hkv, L, B, n = 16, 4, 2, 2, 2, 4
    lay = ssa.Layout(P, Hq, Hkv, 128, False, L, B * n, B * n, B, n, 2, kv_format="int8_page_head")
    kw = dict(host_tier=False, identity=True, block_table=torch.arange(B * n).view(B, n),
              seq_lens=torch.tensor([n * P, n * P - 7]), rope=ssa.RopePlan(128))
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((L, B * n * P, Hkv, 128), generator=g).bfloat16().cuda() for _ in range(2))
    at = torch.arange(n * P, device="cuda").repeat(B)
    runs = [DecodeRunner(lay, graphs=graphs, **kw) for graphs in (True, False)]
    for run in runs:
        run.store(0, L, k, v, torch.arange(B * n * P, device="cuda"), positions=at)
    buf = torch.empty((L, B, 3 * Hq, 128), dtype=torch.bfloat16, device="cuda")
    views = [buf[:, :, :Hq], buf.view(-1)[:L * B * Hq * 128].view(L, B, Hq, 128), buf[:, :, :2 * Hq:2]]
    for step in range(3):
        for q in views:
            assert q.data_ptr() == buf.data_ptr() and q.shape == views[0].shape
            buf.copy_(torch.randn(buf.shape, generator=g).bfloat16())
            a, b = (run.step(q) for run in runs)
            assert torch.equal(a, b)
