"""The miss fetch inside the attention, and the preload, over pages of every size: the same outputs and pool
bytes as a copy before the attention."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_fetch_and_preload_equal_the_copy(fmt, P):
    from sparse_attention_decode_indexer_gb300 import Layout
    from sparse_attention_decode_indexer_gb300.runner import DecodeRunner
    Hq, Hkv, L, B, nmax, k = 8, 2, 2, 3, 20, 6
    S = B * (2 * k + 8)                          # as few slots as the calls allow
    lay = Layout(P, Hq, Hkv, 128, True, L, B * nmax + 1, S, B, nmax, k, kv_format=fmt)
    rng = np.random.default_rng(P)
    bt = rng.permutation(B * nmax).astype(np.int32).reshape(B, nmax)
    bt[2, :7] = bt[0, :7]                        # two requests share pages, and so misses
    kw = dict(host_tier=True, identity=False, block_table=bt,
              seq_lens=np.array([nmax * P, nmax * P - 5, 9 * P + 1], np.int32))
    runs = [DecodeRunner(lay, **kw), DecodeRunner(lay, fetch_in_attention=True, **kw),
            DecodeRunner(lay, preload_width=2 * k, **kw)]
    g = torch.Generator().manual_seed(P)
    x = torch.randn((2, L, B * nmax * P, Hkv, 128), generator=g)
    x = (x * torch.exp2(torch.randn((2, L, B * nmax, 1, Hkv, 1), generator=g)).expand(
        -1, -1, -1, P, -1, 1).reshape(2, L, B * nmax * P, Hkv, 1)).bfloat16().cuda()
    for run in runs:
        run.store(0, L, x[0], x[1], torch.arange(B * nmax * P, device="cuda"))
    missed = [0, 0, 0]
    for step in range(8):
        q = torch.randn((L, B, Hq, 128), generator=g).bfloat16().cuda()
        outs = [run.step(q) for run in runs]
        torch.cuda.synchronize()
        assert all(int(run.status.item()) == 0 for run in runs)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        for i, run in enumerate(runs):
            missed[i] += int(run.n_miss.sum())
            c = run.cache
            for l in range(L):
                own = c.page_of[l].cpu().long()
                at = torch.nonzero(own >= 0)[:, 0]
                for n in ("k_pool", "v_pool", "k_scale", "v_scale"):
                    mir = getattr(c, n.replace("_pool", "") + "_mirror")
                    assert torch.equal(getattr(c, n)[l].cpu()[at], mir[l][own[at]]), (i, n)
    assert missed[0] == missed[1] > 0 and missed[2] > 0
