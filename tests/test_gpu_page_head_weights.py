"""Attention weights of the page_head formats beside attention sinks: tokens that take nearly all the weight and
have no V, in a page of large V scale, while what the output is made of lies 12 to 24 octaves below them
in pages of small V scale."""
import numpy as np
import pytest
import torch

from tests.page_head_ref import RefPages, attend, sm_scale, values

pytestmark = pytest.mark.gpu
D = 128


def _small_weights(fmt, ref, ids, h, live):
    """What attend()'s bound leaves out: a weight enters PV as f16, p * v_scale / r * 2^7 with r a power of
    two at most 16 v_scale and p relative to at most the row's largest, and below 2^-14 f16 has steps of
    2^-24: half a step is at most 2^-25 * 2^-7 * 16 = 2^-28 of the largest weight, so of their sum."""
    V = np.abs(values(fmt, ref.v[ids, h]).astype(np.float64)) * ref.vs[ids, h, None, None].astype(np.float64)
    return 2.0 ** -28 * (1 + 2.0 ** -7) * V[live].sum(0)


@pytest.mark.parametrize("fmt", ["int8_page_head", "e4m3_page_head"])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("down", [1, 8, 20])
def test_weights_beside_a_sink_without_v(fmt, P, down):
    import sparse_attention_decode_indexer_gb300 as ssa
    n, H, B = 32, 8, 40                          # whole (request, head) units for most CTAs
    gaps = np.array([12.0, 14.0, 16.0, 20.0, 24.0])          # octaves, one per query head of the group
    G = len(gaps)
    lay = ssa.Layout(P, H * G, H, D, True, 1, n, n, B, n, n, kv_format=fmt)
    c = ssa.KVCache(lay, False)
    ssa.ssa_lru_init(c, True)
    rng = np.random.default_rng([P, down])
    k = rng.standard_normal((n * P, H, D)) * 0.05
    v = rng.standard_normal((n * P, H, D)) * 2.0 ** -down
    k[..., 0] = 0
    # the first page: a sink in each block of 16 tokens, no V but for one token without weight
    k[:P:16] = 0
    k[:P:16, :, 0] = 8
    v[:P] = 0
    k[1, :, 0] = -8
    v[1] = rng.standard_normal((H, D))
    k, v = (torch.from_numpy(x.astype(np.float32)).bfloat16() for x in (k, v))
    status = torch.zeros((1,), dtype=torch.int32, device="cuda")
    ssa.ssa_store_kv_mirror(c, 0, 1, k[None].cuda(), v[None].cuda(), torch.arange(n * P, device="cuda"), status)
    ref = RefPages(fmt, n, H, P)
    ref.store(k.float().numpy(), v.float().numpy(), np.arange(n * P))
    q = rng.standard_normal((1, B, H, G, D))
    q[..., 0] = gaps / (8 * sm_scale() * np.log2(np.e))
    q = torch.from_numpy(q.astype(np.float32)).bfloat16().view(1, B, H * G, D)
    sel = torch.full((1, B, lay.max_sel), -1, dtype=torch.int32, device="cuda")
    sel[..., :n] = torch.arange(n)
    lens = torch.full((B,), n * P - 5, dtype=torch.int32, device="cuda")
    ws = torch.zeros((ssa.ssa_workspace_size(lay),), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, B, H * G, D), dtype=torch.bfloat16, device="cuda")
    ssa.ssa_sparse_paged_decode(c, 0, 1, q.cuda(), sel, sel, lens, sm_scale(), out, status, ws)
    assert int(status.item()) == 0
    out, qn, ids = out.float().cpu().numpy(), q.float().numpy(), np.arange(n)
    live = np.arange(n * P).reshape(n, P) < n * P - 5
    for b in (0, 1, 19, B - 1):
        for h in range(H):
            want, bound = attend(fmt, ref.k[:, h], ref.v[:, h], ref.ks[:, h], ref.vs[:, h],
                                 qn[0, b, h * G:(h + 1) * G], sm_scale(), live)
            off = np.abs(out[0, b, h * G:(h + 1) * G] - want) / (bound + _small_weights(fmt, ref, ids, h, live))
            assert off.max() <= 1, (b, h, off.max(-1))
