"""Attention over pages of 16 and 32 tokens, whose stages several lanes of the producer fill."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("P", [16, 32])
def test_the_same_bits_every_time(fmt, P):
    """Stages filled over several windows of the selection (holes leave 1 to 4 pages to a window's part of a
    stage), many CTAs, 100 runs: a stage that is handed on before its last page gives other bits."""
    import sparse_attention_decode_indexer_gb300 as ssa
    L, B, Hkv, Hq, nmax, k = 2, 20, 4, 8, 90, 70
    rng = np.random.default_rng(P)
    Lp = 300
    lay = ssa.Layout(P, Hq, Hkv, 128, True, L, Lp, Lp, B, nmax, k, kv_format=fmt)
    c = ssa.KVCache(lay, False)
    ssa.ssa_lru_init(c, True)
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((2, L, Lp * P, Hkv, 128)).astype(np.float32)).bfloat16().cuda()
    ssa.ssa_store_kv_mirror(c, 0, L, x[0], x[1], torch.arange(Lp * P, device="cuda"), status)
    sel = np.full((L, B, lay.max_sel), -1, np.int32)
    phys = np.full_like(sel, -1)
    for l in range(L):
        for b in range(B):
            at = np.sort(rng.permutation(lay.max_sel)[:k + 1])           # padding between the entries
            sel[l, b, at] = np.sort(rng.permutation(nmax)[:k + 1])
            phys[l, b, at] = rng.permutation(Lp)[:k + 1]
    dev = lambda t: torch.from_numpy(np.ascontiguousarray(t.astype(np.int32))).cuda()  # noqa: E731
    args = dev(sel), dev(phys), dev(rng.integers(nmax * P // 2, nmax * P + 1, B)), 128 ** -0.5
    q = torch.from_numpy(rng.standard_normal((L, B, Hq, 128)).astype(np.float32)).bfloat16().cuda()
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    outs = torch.empty((100, L, B, Hq, 128), dtype=torch.bfloat16, device="cuda")
    for out in outs:
        ssa.ssa_sparse_paged_decode(c, 0, L, q, *args, out, status, ws)
    assert int(status.item()) == 0
    assert bool((outs == outs[0]).all()) and bool(outs[0].isfinite().all())
